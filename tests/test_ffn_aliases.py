"""The gated block refuses outputs in its inputs' arrays: tiles would be overwritten that others still read.  Only
refused calls are made here (the pointers are never dereferenced)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def P():
    from orthogonal_reparameterized_gb300 import build
    build.build()
    import orthogonal_reparameterized_gb300.poetx as P
    P.lib()
    return P


ARG = 1
X, W, Z, DH, DX, DW, WS = (ctypes.c_void_p(1 << (20 + i)) for i in range(7))


@pytest.mark.parametrize("dt", ["BF16", "F32"])
@pytest.mark.parametrize("N", [1, 40, 300])
@pytest.mark.parametrize("h,z", [(X, None), (X, Z), (W, None), (Z, Z), (DX, X), (DX, W)])
def test_forward(P, N, dt, h, z):
    st = P.lib().poetx_ffn_fwd(getattr(P, dt), 0, X, N, 64, W, 64, h, z, WS, 1 << 30, None)
    assert st == ARG


@pytest.mark.parametrize("dt", ["BF16", "F32"])
@pytest.mark.parametrize("N", [1, 40, 100, 300])
@pytest.mark.parametrize("z", [Z, None])
@pytest.mark.parametrize("dx,dW", [(X, DW), (W, DW), (W, None), (DX, W), (DX, X), (None, W), (None, X), (DX, DX)])
def test_backward(P, N, dt, z, dx, dW):
    st = P.lib().poetx_ffn_bwd(getattr(P, dt), 0, X, N, 64, W, 64, z, DH, dx, dW, 0, WS, 1 << 30, None)
    assert st == ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kept", [True, False], ids=["kept", "mem"])
@pytest.mark.parametrize("N", [1, 5, 16, 40, 100, 300])
def test_dx_alone_may_be_x(P, N, kept, dt):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(N)
    T = torch.bfloat16 if dt == "bf16" else torch.float32
    t = lambda *s: torch.randn(*s, generator=g, device="cuda").to(T)
    x, W, dh, z = t(N, 264), t(2000, 264) / 16, t(N, 1000), t(N, 2000)
    z = z if kept else None
    dx = torch.empty_like(x)
    P.poetx_ffn_bwd(x, W, dh, z=z, dx=dx)
    P.poetx_ffn_bwd(x, W, dh, z=z, dx=x)
    torch.cuda.synchronize()
    assert torch.equal(x, dx) and dx.isfinite().all()
    with pytest.raises(P.PoetxError):
        P.poetx_ffn_bwd(x, W, dh, z=z, dx=x, dW=torch.empty_like(W))
