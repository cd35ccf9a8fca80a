"""The oracle's angles at far positions against decimal arithmetic."""
from decimal import Decimal, getcontext

import numpy as np

from oracle import block_oracle as B

# 2 pi to 60 digits (OEIS A019692)
TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194989")


def test_angles_of_far_positions():
    getcontext().prec = 60
    r = np.random.default_rng(1)
    freq = np.float32(np.concatenate([10000.0 ** -np.linspace(0, 1, 20), [-1.0, 3.1415926, -6.2831, 6.2831, 5.5]]))
    pos = np.concatenate([[0, 1, -1, 1000, 2 ** 31 - 1, -2 ** 31], r.integers(-2 ** 31, 2 ** 31, 40)])
    got = B._angles(pos[:, None], freq[None].astype(np.float64))
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            off = (Decimal(int(p)) * Decimal(float(f)) - Decimal(float(got[i, j]))) / TWO_PI
            off -= off.to_integral_value()
            # half a step of a 64-bit angle of up to 1024, or of pi and its factor
            assert abs(off * TWO_PI) <= 2.0 ** -43
