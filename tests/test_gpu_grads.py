"""The global gradient norm, clipping and the many-tensor optimizer step.

Tolerances: a norm is the root of sums of squares, each fp32 sum over at most a few hundred terms of one
sign (2^-24 each at most, half of that in the root), then 64 bits: 2^-18.  Clipped gradients: the
factor's two roundings and the product's (and bf16's).  The optimizer step without a factor is
poetx_adam_triu's, bit for bit."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, P, TOL_F32, dev, host  # noqa: F401
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu


def _grads(sizes, seed, scale=1.0):
    r = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.tensor(r.standard_normal(n) * scale * 10.0 ** (i % 3 - 1), dtype=torch.float32)
        out.append(t.bfloat16() if i % 2 else t)
    return out


def _norm(P, ts, **kw):
    n = torch.full((1,), float("nan"), device=DEV)
    P.poetx_grad_norm(ts, n, **kw)
    torch.cuda.synchronize()
    return n


SIZES = [[1], [7, 3], [0, 5, 0], [4096, 4097, 8191], [8192, 8193, 40000, 3], [1000003, 77, 500000],
         list(range(1, 700)), [5] * 48, [9] * 49, [3] * 512, [6] * 513]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm(P, sizes):
    ts = _grads(sizes, len(sizes))
    got, again = (_norm(P, [t.to(DEV) for t in ts]) for _ in range(2))
    ref = B.grad_norm([host(t) for t in ts])
    assert abs(float(got) - ref) <= 2.0 ** -18 * ref
    assert torch.equal(got, again)


def test_norms_in_one_array(P):
    """A norm per group of tensors, side by side."""
    ts = [t.to(DEV) for t in _grads([100, 5000, 77], 3)]
    norms = torch.zeros(5, device=DEV)
    for i, t in enumerate(ts):
        P.poetx_grad_norm([t], norms[i + 1:i + 2])
    ref = [B.grad_norm([host(t)]) for t in ts]
    assert np.abs(host(norms)[1:4] / ref - 1).max() <= 2.0 ** -18
    assert float(norms[0]) == 0 and float(norms[4]) == 0
    P.poetx_grad_clip(ts[:1], norms[1:2], 0.5 * ref[0])
    assert abs(float(_norm(P, ts[:1])) / (0.5 * ref[0]) - 1) <= 1e-5


def test_norm_of_nothing(P):
    assert float(_norm(P, [])) == 0
    assert float(_norm(P, [torch.empty(0, device=DEV)])) == 0
    assert float(_norm(P, [torch.zeros(1000, device=DEV)])) == 0


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e15, 1e30])
def test_norm_of_tiny_and_huge_values(P, scale):
    """Squares beyond fp32's range; a tiny value beside ordinary ones."""
    for n in (3, 5000):
        x = torch.tensor(np.random.default_rng(n).standard_normal(n) * scale, dtype=torch.float32)
        ref = B.grad_norm([host(x)])
        assert abs(float(_norm(P, [x.to(DEV)])) - ref) <= 2.0 ** -18 * ref
        y = torch.cat([x, torch.ones(64)])
        ref = B.grad_norm([host(y)])
        assert abs(float(_norm(P, [y.to(DEV)])) - ref) <= 2.0 ** -18 * ref


def test_norm_not_finite(P):
    inf = float("inf")
    for bad in (inf, -inf):
        x = torch.ones(5001, device=DEV)
        x[5000] = bad
        assert float(_norm(P, [x])) == inf
    x[17] = float("nan")
    assert np.isnan(float(_norm(P, [x])))
    y = torch.ones(5001, device=DEV)
    y[8] = float("nan")
    assert np.isnan(float(_norm(P, [torch.ones(9, device=DEV), y])))


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(P, sizes):
    ts = _grads(sizes, 3 * len(sizes))
    ds = [t.to(DEV) for t in ts]
    norm = _norm(P, ds)
    P.poetx_grad_clip(ds, norm, 2.0 * float(norm) + 1.0)  # nothing to clip
    for d, t in zip(ds, ts):
        assert torch.equal(d.cpu(), t)
    f = B.clip_factor(float(norm), 0.25)
    P.poetx_grad_clip(ds, norm, 0.25)
    for d, t in zip(ds, ts):
        # the factor as fp32 arithmetic has it (two roundings), the product's rounding, bf16's
        tol = 2.0 ** -22 + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0)
        ref = host(t) * f
        assert (np.abs(host(d) - ref) <= tol * np.abs(ref) + 1e-40).all()


def test_clip_by_norms_that_are_not_finite(P):
    x = torch.tensor([1.0, 2.0, float("inf"), -1.0], device=DEV)
    P.poetx_grad_clip([x], torch.tensor([float("inf")], device=DEV), 1.0)
    assert host(x)[[0, 1, 3]].tolist() == [0, 0, 0] and np.isnan(host(x)[2])
    y = torch.ones(3, device=DEV)
    P.poetx_grad_clip([y], torch.tensor([float("nan")], device=DEV), 1.0)
    assert torch.isnan(y).all()
    z = torch.ones(3, device=DEV)
    P.poetx_grad_clip([z], torch.tensor([5.0], device=DEV), float("inf"))
    assert (z == 1).all()
    P.poetx_grad_clip([z], torch.tensor([5.0], device=DEV), 0.0)
    assert not z.any()


def _state(sizes, seed):
    r = np.random.default_rng(seed)
    mk = lambda n, s: torch.tensor(r.standard_normal(n) * s, dtype=torch.float32)
    return {"q": [mk(n, 0.02) for n in sizes], "dq": [mk(n, 1e-2) for n in sizes],
            "m": [mk(n, 1e-3) for n in sizes], "v": [mk(n, 1e-3) ** 2 for n in sizes]}


HP = dict(step=3, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.mark.parametrize("sizes", [[1], [7, 0, 1001], [4096 * 3, 4095, 4097], [500000, 9],
                                   list(range(1, 600)), [5] * 48, [9] * 49, [3] * 512, [6] * 513],
                         ids=lambda s: f"{len(s)}x{max(s)}")
def test_adam_group(P, sizes):
    s = _state(sizes, len(sizes))
    a, b, c = ({k: [t.to(DEV) for t in ts] for k, ts in s.items()} for _ in range(3))
    for q, g, m, v in zip(a["q"], a["dq"], a["m"], a["v"]):
        P.poetx_adam_triu(q, g, m, v, **HP)
    P.poetx_adam_group(b["q"], b["dq"], b["m"], b["v"], **HP)
    norm = _norm(P, c["dq"])
    P.poetx_adam_group(c["q"], c["dq"], c["m"], c["v"], norm=norm, max_norm=2 * float(norm), **HP)
    for k in ("q", "m", "v", "dq"):
        for x, y, z in zip(a[k], b[k], c[k]):
            assert torch.equal(x, y) and torch.equal(x, z), k
    # clipped: the step of the scaled gradient
    d = {k: [t.to(DEV) for t in ts] for k, ts in s.items()}
    limit = 0.3 * float(norm)
    P.poetx_adam_group(d["q"], d["dq"], d["m"], d["v"], norm=norm, max_norm=limit, **HP)
    f = B.clip_factor(float(norm), limit)
    hp = {k: float(np.float32(v)) for k, v in HP.items() if k != "step"}
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        q0 = host(s["q"][i])
        q, m, v = O.adam_step(q0, host(s["dq"][i]) * f, host(s["m"][i]), host(s["v"][i]), 3, **hp)
        # the update is a difference of q, which is rounded to 2^-24 of 0.02 or so
        assert np.linalg.norm(host(d["q"][i]) - q) <= TOL_F32 * np.linalg.norm(q - q0) + \
            2.0 ** -24 * np.linalg.norm(q0)
        assert O.rel_fro(host(d["m"][i]), m) <= TOL_F32 and O.rel_fro(host(d["v"][i]), v) <= TOL_F32
        assert torch.equal(d["dq"][i].cpu(), s["dq"][i])


def test_norm_clip_and_step_in_a_graph_and_on_another_stream(P):
    s = _state([3000, 17, 100000], 9)
    a, b = ({k: [t.to(DEV) for t in ts] for k, ts in s.items()} for _ in range(2))

    def step(t, norm, stream=None):
        P.poetx_grad_norm(t["dq"], norm, stream=stream)
        P.poetx_adam_group(t["q"], t["dq"], t["m"], t["v"], norm=norm, max_norm=0.5, stream=stream, **HP)

    na, nb = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(a, na, st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, nb)
    graph.replay()  # (the capture itself ran nothing)
    torch.cuda.synchronize()
    assert torch.equal(na, nb) and float(na) > 0.5
    for k in ("q", "m", "v"):
        for x, y in zip(a[k], b[k]):
            assert torch.equal(x, y), k


def test_norm_beyond_32_bit_counts(P):
    n = (1 << 31) + 12345
    if torch.cuda.mem_get_info()[0] < 5 * n:
        pytest.skip("needs 10 GB")
    x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    x[0], x[-1], x[1 << 30] = 3.0, 4.0, 12.0
    norm = _norm(P, [x])
    assert float(norm) == 13.0
    P.poetx_grad_clip([x], norm, 6.5)
    assert float(x[-1]) == 2.0 and float(x[0]) == 1.5
