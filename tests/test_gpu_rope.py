"""Query and key norms with the rotation, forward and backward, against the fp64 definition.

Tolerances, elementwise against the largest element of the token's head (an output is a sum of two
products).  bf16: one rounding, 2^-8 of the value, and 2^-18 of the largest (sine and cosine to 2^-21,
norm and products in fp32).  fp32: some sixteen roundings of 2^-24, 2^-20.  dgamma: fp32 sums of values
of either sign, TOL_F32 of the norm of its terms' column sums."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, P, TOL_F32, dev, host  # noqa: F401
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(N, Hq, Hk, dh, rot, axes, dt, seed, far=1 << 20):
    r = np.random.default_rng(seed)
    t = lambda H, s: torch.tensor(r.standard_normal((N, H, dh)) * s + 0.1).to(DT[dt])
    c = {"q": t(Hq, 2.0), "k": t(Hk, 0.5), "dq": t(Hq, 1.0), "dk": t(Hk, 1.0)}
    c["gq"], c["gk"] = ((1 + 0.2 * r.standard_normal(dh)).astype(np.float32) for _ in range(2))
    c["pos"] = r.integers(-far, far, (axes, N)).astype(np.int32)
    c["freq"] = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    c["axis"] = r.integers(0, axes, rot // 2).astype(np.int32) if axes > 1 else None
    return c


def _opt(c, interleaved, norm, gamma, rot):
    kw = dict(rot_dim=rot, axis=None if c["axis"] is None else dev(c["axis"], torch.int32),
              interleaved=interleaved, norm=norm)
    if gamma:
        kw.update(gamma_q=dev(c["gq"], torch.float32), gamma_k=dev(c["gk"], torch.float32))
    return kw


def _near(got, ref, dt):
    if not ref.size:
        return True
    top = np.abs(ref).max(axis=-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * top if dt == "bf16" else 2.0 ** -20 * top
    return (np.abs(got - ref) <= tol).all()


def _check(P, c, dt, rot, interleaved=False, norm=True, gamma=True):
    N = c["q"].shape[0]
    dev_t = {k: c[k].to(DEV) for k in ("q", "k", "dq", "dk")}
    pos, freq = dev(c["pos"], torch.int32), dev(c["freq"], torch.float32)
    kw = _opt(c, interleaved, norm, gamma, rot)
    out = {k: torch.full_like(dev_t[k], float("nan")) for k in dev_t}
    dg = {k: torch.full((c["q"].shape[2],), float("nan"), device=DEV) for k in ("q", "k")}
    P.poetx_qk_rope_fwd(dev_t["q"], dev_t["k"], pos, freq, out["q"], out["k"], **kw)
    P.poetx_qk_rope_bwd(dev_t["q"], dev_t["k"], dev_t["dq"], dev_t["dk"], pos, freq, out["dq"],
                        out["dk"], dgamma_q=dg["q"], dgamma_k=dg["k"], **kw)
    torch.cuda.synchronize()
    o = dict(axis=c["axis"], interleaved=interleaved, norm=norm)
    for s in ("q", "k"):
        g = c["g" + s] if gamma and norm else None
        ref = B.qk_rope(host(c[s]), c["pos"], c["freq"], gamma=g, **o)
        assert _near(host(out[s]), ref, dt), s
        dx, dgamma = B.qk_rope_bwd(host(c[s]), host(c["d" + s]), c["pos"], c["freq"], gamma=g, **o)
        # the gradient of a normalised head is a difference of its terms, of the size of dy rstd
        dn = np.abs(dx).max(axis=-1, keepdims=True)
        if norm:
            rstd = 1 / np.sqrt((host(c[s]) ** 2).mean(-1, keepdims=True) + 1e-6)
            dn = np.maximum(dn, np.abs(host(c["d" + s])).max(axis=-1, keepdims=True) * rstd)
        tol = 2.0 ** -8 * np.abs(dx) + 2.0 ** -17 * dn if dt == "bf16" else 2.0 ** -19 * dn
        assert (np.abs(host(out["d" + s]) - dx) <= tol).all(), s
        if norm:
            n_terms = max(1, N * c[s].shape[1])
            size = np.sqrt(n_terms) * np.abs(host(c["d" + s])).max() if N else 1.0
            assert np.abs(host(dg[s]) - dgamma).max() <= TOL_F32 * size
    return out, dg


# N, query and key heads, head width, rotated width, axes
SHAPES = [(1, 32, 8, 128, 128, 1), (1, 1, 1, 8, 8, 1), (3, 5, 1, 16, 16, 2), (7, 4, 2, 72, 32, 1),
          (130, 28, 4, 128, 128, 3), (33, 6, 6, 80, 40, 2), (257, 3, 1, 96, 48, 1), (9, 2, 1, 256, 64, 3),
          (5, 3, 2, 512, 512, 1), (64, 7, 1, 24, 8, 1), (2500, 4, 1, 64, 64, 1), (40, 64, 8, 192, 128, 1),
          (6, 2, 2, 248, 200, 8)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hk,dh,rot,axes", SHAPES)
def test_rope(P, N, Hq, Hk, dh, rot, axes, interleaved, dt):
    c = _case(N, Hq, Hk, dh, rot, axes, dt, N + dh + rot)
    for norm, gamma in ((True, True), (True, False), (False, False)):
        _check(P, c, dt, rot, interleaved, norm, gamma)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rope_far_positions(P, dt):
    """Angles of the largest and smallest positions (a product in fp32 would be off by hundreds of
    radians)."""
    c = _case(64, 2, 1, 64, 64, 1, dt, 1, far=(1 << 31) - 1)
    c["pos"][0, :3] = (2 ** 31 - 1, -2 ** 31, 0)
    _check(P, c, dt, 64, norm=False, gamma=False)


def test_rope_strided_rows_and_in_place(P):
    """q and k side by side in one row with the values; outputs into the same places."""
    N, Hq, Hk, dh = 50, 8, 2, 64
    c = _case(N, Hq, Hk, dh, dh, 1, "bf16", 4)
    ref, _ = _check(P, c, "bf16", dh)
    row = torch.cat([c["q"].flatten(1), c["k"].flatten(1), c["k"].flatten(1)], 1).to(DEV)
    keep = row.clone()
    q, k = row[:, :Hq * dh].unflatten(1, (Hq, dh)), row[:, Hq * dh:(Hq + Hk) * dh].unflatten(1, (Hk, dh))
    pos, freq = dev(c["pos"], torch.int32), dev(c["freq"], torch.float32)
    kw = _opt(c, False, True, True, dh)
    P.poetx_qk_rope_fwd(q, k, pos[0], freq, q, k, **kw)
    assert torch.equal(q, ref["q"]) and torch.equal(k, ref["k"])
    assert torch.equal(row[:, (Hq + Hk) * dh:], keep[:, (Hq + Hk) * dh:])  # the values
    # backward: over the upstream gradients
    dq, dk = c["dq"].to(DEV), c["dk"].to(DEV)
    P.poetx_qk_rope_bwd(c["q"].to(DEV), c["k"].to(DEV), dq, dk, pos, freq, dq, dk, **kw)
    assert torch.equal(dq, ref["dq"]) and torch.equal(dk, ref["dk"])


def test_rope_one_side_and_options(P):
    N, dh = 200, 128
    c = _case(N, 4, 4, dh, dh, 1, "bf16", 5)
    ref, dg = _check(P, c, "bf16", dh)
    again, dg2 = _check(P, c, "bf16", dh)
    for k in ref:
        assert torch.equal(ref[k], again[k]), k
    for k in dg:
        assert torch.equal(dg[k], dg2[k]), k
    pos, freq = dev(c["pos"], torch.int32), dev(c["freq"], torch.float32)
    kw = _opt(c, False, True, True, dh)
    kw.pop("gamma_k")
    q, out = c["q"].to(DEV), torch.empty_like(ref["q"])
    P.poetx_qk_rope_fwd(q, None, pos, freq, out, None, **kw)
    assert torch.equal(out, ref["q"])
    acc = torch.full((dh,), 0.5, device=DEV)
    P.poetx_qk_rope_bwd(q, None, c["dq"].to(DEV), None, pos, freq, out, None, dgamma_q=acc,
                        accumulate=True, **kw)
    assert torch.equal(out, ref["dq"])
    # (a side alone has more CTAs: another order of the sums)
    assert (acc - 0.5 - dg["q"]).abs().max() <= TOL_F32 * float(dg["q"].abs().max() + 1) * 10
    # no tokens
    e = torch.empty(0, 4, dh, device=DEV).bfloat16()
    p0 = torch.empty(1, 0, dtype=torch.int32, device=DEV)
    P.poetx_qk_rope_fwd(e, e, p0, freq, e.clone(), e.clone(), **kw)
    P.poetx_qk_rope_bwd(e, None, e, None, p0, freq, e.clone(), None, dgamma_q=acc, **kw)
    assert not acc.any()


def test_rope_shared_gamma(P):
    """One gamma for queries and keys: its gradient is the sum of both sides'."""
    N, dh = 90, 96
    c = _case(N, 6, 2, dh, dh, 1, "f32", 8)
    c["gk"] = c["gq"]
    _, dg = _check(P, c, "f32", dh)
    pos, freq = dev(c["pos"], torch.int32), dev(c["freq"], torch.float32)
    t = {k: c[k].to(DEV) for k in ("q", "k", "dq", "dk")}
    for acc in (False, True):
        both = torch.full((dh,), 0.5, device=DEV)
        P.poetx_qk_rope_bwd(t["q"], t["k"], t["dq"], t["dk"], pos, freq, torch.empty_like(t["q"]),
                            torch.empty_like(t["k"]), dgamma_q=both, dgamma_k=both, accumulate=acc,
                            **_opt(c, False, True, True, dh))
        ref = dg["q"] + dg["k"] + (0.5 if acc else 0.0)
        assert (both - ref).abs().max() <= TOL_F32 * float(ref.abs().max() + 1) * 4


def test_rope_nan_stays_in_its_head_and_bad_axis_in_its_pair(P):
    N, dh = 20, 64
    c = _case(N, 3, 1, dh, 32, 2, "f32", 6)
    c["q"][4, 1, 60] = float("nan")
    c["q"][5, 2, 50] = float("inf")  # beyond the rotated part: no NaN from the rotation
    pos, freq = dev(c["pos"], torch.int32), dev(c["freq"], torch.float32)
    q, out = c["q"].to(DEV), torch.empty(N, 3, dh, device=DEV)
    kw = dict(rot_dim=32, axis=dev(c["axis"], torch.int32))
    P.poetx_qk_rope_fwd(q, None, pos, freq, out, None, norm=False, **kw)
    o = host(out)
    assert np.isnan(o).sum() == 1 and np.isnan(o[4, 1, 60]) and np.isinf(o).sum() == 1
    P.poetx_qk_rope_fwd(q, None, pos, freq, out, None, **kw)
    o = host(out)
    assert np.isnan(o[4, 1]).all() and np.isfinite(o[4, [0, 2]]).all()
    c["axis"][3] = 2  # there are two axes
    kw["axis"] = dev(c["axis"], torch.int32)
    P.poetx_qk_rope_fwd(c["k"].to(DEV), None, pos, freq, out[:, :1].contiguous(), None, norm=False, **kw)
    y = torch.empty(N, 1, dh, device=DEV)
    P.poetx_qk_rope_fwd(c["k"].to(DEV), None, pos, freq, y, None, norm=False, **kw)
    bad = np.isnan(host(y))
    assert bad[..., [3, 19]].all() and bad.sum() == 2 * N


def test_rope_on_another_stream_and_in_a_graph(P):
    N, dh = 300, 64
    c = _case(N, 4, 2, dh, dh, 1, "bf16", 7)
    ref, dg = _check(P, c, "bf16", dh)
    pos, freq = dev(c["pos"], torch.int32), dev(c["freq"], torch.float32)
    kw = _opt(c, False, True, True, dh)
    t = {k: c[k].to(DEV) for k in ("q", "k", "dq", "dk")}
    out = {k: torch.zeros_like(v) for k, v in t.items()}
    g = torch.zeros(dh, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.poetx_qk_rope_bwd(t["q"], t["k"], t["dq"], t["dk"], pos, freq, out["dq"], out["dk"], dgamma_k=g,
                        stream=s, **kw)
    s.synchronize()
    assert torch.equal(out["dq"], ref["dq"]) and torch.equal(g, dg["k"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.poetx_qk_rope_fwd(t["q"], t["k"], pos, freq, out["q"], out["k"], **kw)
        P.poetx_qk_rope_bwd(t["q"], t["k"], t["dq"], t["dk"], pos, freq, out["dq"], out["dk"],
                            dgamma_k=g, **kw)
    for v in (*out.values(), g):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in out:
        assert torch.equal(out[k], ref[k]), k
    assert torch.equal(g, dg["k"])


def test_rope_beyond_32_bit_offsets(P):
    N, H, dh = 270000, 64, 128
    if torch.cuda.mem_get_info()[0] < 6 * N * H * dh:
        pytest.skip("needs 14 GB")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.zeros(N, H, dh, dtype=torch.bfloat16, device=DEV)
    x[-5:] = torch.randn(5, H, dh, generator=g, device=DEV).bfloat16()
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    freq = 10000.0 ** (-torch.arange(dh // 2, device=DEV, dtype=torch.float32) / (dh // 2))
    y = torch.empty_like(x)
    P.poetx_qk_rope_fwd(x, None, pos, freq, y, None)
    ref = torch.empty_like(x[-5:])
    P.poetx_qk_rope_fwd(x[-5:].contiguous(), None, pos[-5:].contiguous(), freq, ref, None)
    assert torch.equal(y[-5:], ref) and not y[:-5].any()
    P.poetx_qk_rope_bwd(x, None, x, None, pos, freq, y, None)
    P.poetx_qk_rope_bwd(x[-5:].contiguous(), None, x[-5:].contiguous(), None, pos[-5:].contiguous(), freq,
                        ref, None)
    assert torch.equal(y[-5:], ref)
