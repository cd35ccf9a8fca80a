"""Refusals of the gated feed-forward block, the query and key rotation and the many-tensor entry
points: host-side checks, before any launch (run without a GPU; the pointers are never
dereferenced)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def P():
    from orthogonal_reparameterized_gb300 import build
    build.build()
    import orthogonal_reparameterized_gb300.poetx as P
    P.lib()
    return P


ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
OK = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
HALF = ctypes.c_void_p(4098)
NAN = float("nan")


def _glu(P, **kw):
    a = dict(dt=P.BF16, act=0, g=OK, u=OK, N=4, F=64, pitch=64, h=OK)
    a.update(kw)
    return P.lib().poetx_glu_fwd(*a.values(), None)


def _glu_bwd(P, **kw):
    a = dict(dt=P.BF16, act=0, g=OK, u=OK, dh=OK, N=4, F=64, pitch=64, dg=OK, du=OK, d_pitch=64)
    a.update(kw)
    return P.lib().poetx_glu_bwd(*a.values(), None)


def _fwd(P, **kw):
    a = dict(dt=P.F32, act=0, x=OK, N=4, D=64, W=OK, F=64, h=OK, z=None, ws=OK, ws_bytes=1 << 30)
    a.update(kw)
    return P.lib().poetx_ffn_fwd(*a.values(), None)


def _bwd(P, **kw):
    a = dict(dt=P.BF16, act=0, x=OK, N=4, D=64, W=OK, F=64, z=OK, dh=OK, dx=OK, dW=OK, accumulate=0,
             ws=OK, ws_bytes=1 << 30)
    a.update(kw)
    return P.lib().poetx_ffn_bwd(*a.values(), None)


GLU = [(dict(N=-1), ARG), (dict(act=2), ARG), (dict(act=-1), ARG), (dict(dt=2), DTYPE),
       (dict(F=0), SHAPE), (dict(F=60), SHAPE), (dict(F=2097160, pitch=2097160), SHAPE),
       (dict(pitch=56), SHAPE), (dict(pitch=68), SHAPE), (dict(g=ODD), ALIGN), (dict(u=ODD), ALIGN),
       (dict(g=None), ARG), (dict(u=None), ARG), (dict(N=0), 0)]


@pytest.mark.parametrize("kw,st", GLU + [(dict(h=None), ARG), (dict(h=ODD), ALIGN)])
def test_glu_refusals(P, kw, st):
    assert _glu(P, **kw) == st


@pytest.mark.parametrize("kw,st", GLU + [
    (dict(dh=None), ARG), (dict(dg=None), ARG), (dict(du=None), ARG), (dict(dh=ODD), ALIGN),
    (dict(dg=ODD), ALIGN), (dict(d_pitch=8), SHAPE), (dict(d_pitch=66), SHAPE)])
def test_glu_bwd_refusals(P, kw, st):
    assert _glu_bwd(P, **kw) == st


FFN = [(dict(N=-1), ARG), (dict(act=7), ARG), (dict(dt=2), DTYPE), (dict(D=60), SHAPE),
       (dict(D=0), SHAPE), (dict(D=131080), SHAPE), (dict(F=12), SHAPE), (dict(F=2097160), SHAPE),
       (dict(x=None), ARG), (dict(W=None), ARG), (dict(ws=None), ARG), (dict(ws_bytes=1024), WORKSPACE),
       (dict(x=ODD), ALIGN), (dict(W=ODD), ALIGN), (dict(z=ODD), ALIGN), (dict(ws=ODD), ALIGN)]


@pytest.mark.parametrize("kw,st", FFN + [(dict(h=None), ARG), (dict(h=ODD), ALIGN), (dict(N=0), 0)])
def test_ffn_fwd_refusals(P, kw, st):
    assert _fwd(P, **kw) == st


@pytest.mark.parametrize("kw,st", FFN + [
    (dict(dh=None), ARG), (dict(dx=None, dW=None), ARG), (dict(dh=ODD), ALIGN), (dict(dx=ODD), ALIGN),
    (dict(dW=ODD), ALIGN), (dict(N=0, dW=None), 0), (dict(N=0, accumulate=1), 0)])
def test_ffn_bwd_refusals(P, kw, st):
    assert _bwd(P, **kw) == st


def test_ffn_workspaces(P):
    f, b = P.poetx_ffn_fwd_workspace_bytes, P.poetx_ffn_bwd_workspace_bytes
    assert f(P.BF16, 4096, 4096, 14336) == 0
    assert f(P.F32, 100, 64, 200) >= 6 * 64 * (100 + 400)
    kept, mem = b(P.BF16, 4096, 2048, 8192), b(P.BF16, 4096, 2048, 8192, have_z=False)
    assert kept >= 4096 * 16384 * 2 and mem == kept  # dz alone: the projections are not kept
    assert b(P.F32, 100, 64, 200, have_z=False) >= b(P.F32, 100, 64, 200) + 100 * 400 * 4
    assert b(P.BF16, 64, 2048, 8192) >= 2 * 64 * 16384 * 2  # dz in two pieces
    for bad in ((P.I8, 4, 64, 64), (P.BF16, -1, 64, 64), (P.BF16, 4, 60, 64), (P.BF16, 4, 64, 60)):
        assert f(*bad) == b(*bad) == 0, bad
    assert b(P.BF16, 4, 64, 64, True, False, False) == 0


def _rope(P, bwd=False, side=None, **kw):
    d = dict(head_dim=64, rot_dim=64, interleaved=0, axes=1, norm=1, eps=1e-6, inv_freq=OK, axis=None)
    c = dict(dt=P.BF16, pos=OK, N=4, accumulate=0, ws=OK, ws_bytes=1 << 30, q=True, k=True)
    for k, v in kw.items():
        (d if k in d else c)[k] = v
    h = dict(heads=4, x=OK, x_pitch=256, gamma=OK, dy=OK, dy_pitch=256, y=OK, y_pitch=256, dgamma=OK)
    h.update(side or {})
    val = [v if isinstance(v, (int, float)) or v is None else v.value for v in d.values()]
    r = P.RopeDesc(*val)
    s = P.HeadsDesc(*[v if isinstance(v, int) or v is None else v.value for v in h.values()])
    q, k = (ctypes.byref(s) if c[n] else None for n in ("q", "k"))
    if bwd:
        return P.lib().poetx_qk_rope_bwd(ctypes.byref(r), c["dt"], c["pos"], c["N"], q, k,
                                         c["accumulate"], c["ws"], c["ws_bytes"], None)
    return P.lib().poetx_qk_rope_fwd(ctypes.byref(r), c["dt"], c["pos"], c["N"], q, k, None)


ROPE = [(dict(N=-1), ARG), (dict(dt=2), DTYPE), (dict(q=False, k=False), ARG), (dict(eps=-1.0), ARG),
        (dict(eps=NAN), ARG), (dict(head_dim=60), SHAPE), (dict(head_dim=0), SHAPE),
        (dict(rot_dim=0), SHAPE), (dict(rot_dim=72), SHAPE), (dict(rot_dim=20), SHAPE),
        (dict(head_dim=264, rot_dim=8), SHAPE), (dict(head_dim=528, rot_dim=16), SHAPE),
        (dict(head_dim=512, rot_dim=24), SHAPE), (dict(axes=0), SHAPE), (dict(axes=9), SHAPE),
        (dict(pos=None), ARG), (dict(inv_freq=None), ARG), (dict(pos=HALF), ALIGN),
        (dict(axis=HALF), ALIGN), (dict(inv_freq=HALF), ALIGN), (dict(side=dict(heads=-1)), ARG), (dict(side=dict(x_pitch=248)), SHAPE),
        (dict(side=dict(x_pitch=260)), SHAPE), (dict(side=dict(y_pitch=255)), SHAPE),
        (dict(side=dict(x=None)), ARG), (dict(side=dict(y=None)), ARG), (dict(side=dict(x=ODD)), ALIGN),
        (dict(side=dict(y=ODD)), ALIGN), (dict(side=dict(gamma=ODD)), ALIGN),
        (dict(side=dict(heads=0)), 0),
        (dict(side=dict(heads=1 << 25, x_pitch=1 << 31, y_pitch=1 << 31, dy_pitch=1 << 31)), SHAPE)]


@pytest.mark.parametrize("kw,st", ROPE + [(dict(N=0), 0)])
def test_rope_fwd_refusals(P, kw, st):
    assert _rope(P, **kw) == st


@pytest.mark.parametrize("kw,st", ROPE + [
    (dict(side=dict(dy=None)), ARG), (dict(side=dict(dy=ODD)), ALIGN), (dict(ws=None), ARG),
    (dict(ws_bytes=16), WORKSPACE), (dict(side=dict(dgamma=ODD)), ALIGN),
    (dict(side=dict(dy_pitch=0)), SHAPE), (dict(N=0, accumulate=1), 0)])
def test_rope_bwd_refusals(P, kw, st):
    assert _rope(P, True, **kw) == st


def _list(kind, *v):
    return (kind * len(v))(*v)


def test_many_tensor_refusals(P):
    lib = P.lib()
    vp, ll, ci = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int
    p, c, dt = _list(vp, 4096, 8192), _list(ll, 8, 5), _list(ci, P.F32, P.BF16)

    def norm(g=p, t=dt, n=c, k=2, out=OK, ws=OK, b=1 << 20):
        return lib.poetx_grad_norm(g, t, n, k, out, ws, b, None)

    assert norm(k=-1) == norm(g=None) == norm(t=None) == norm(n=None) == ARG
    assert norm(out=None) == norm(ws=None) == ARG
    assert norm(b=16) == WORKSPACE and norm(out=HALF) == norm(ws=ODD) == ALIGN
    assert norm(t=_list(ci, P.F32, P.I8)) == DTYPE
    assert norm(n=_list(ll, 8, -1)) == ARG and norm(n=_list(ll, 8, (1 << 33) + 1)) == SHAPE
    assert norm(g=_list(vp, 4096, 8200)) == ALIGN and norm(g=_list(vp, 4096, None)) == ARG

    def clip(g=p, t=dt, n=c, k=2, m=1.0, out=OK):
        return lib.poetx_grad_clip(g, t, n, k, m, out, None)

    assert clip(m=-1.0) == clip(m=NAN) == clip(out=None) == clip(g=None) == ARG
    assert clip(out=HALF) == clip(g=_list(vp, 4100, 4096)) == ALIGN
    assert clip(k=0) == 0 and clip(n=_list(ll, 0, 0)) == 0

    def adam(q=p, g=p, m=p, v=p, n=c, k=2, step=1, limit=1.0, out=OK):
        hp = P.AdamDesc(1e-3, 0.9, 0.999, 1e-8, 0.0, step)
        return lib.poetx_adam_group(q, g, m, v, n, k, ctypes.byref(hp), limit, out, None)

    assert adam(step=0) == adam(q=None) == adam(v=None) == adam(n=None) == adam(k=-1) == ARG
    assert adam(limit=-1.0) == ARG and adam(out=HALF) == ALIGN
    assert adam(m=_list(vp, 4096, 4100)) == ALIGN and adam(k=0) == 0
    assert lib.poetx_adam_group(p, p, p, p, c, 2, None, 1.0, None, None) == ARG
    assert P.poetx_grad_norm_workspace_bytes(-1) == 0
    assert P.poetx_grad_norm_workspace_bytes(1) > 0


def test_binding_checks(P):
    x, W = torch.zeros(4, 64), torch.zeros(128, 64)
    h, pos, f = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="W must be"):
        P.poetx_ffn_fwd(x, W[:127], h)
    with pytest.raises(ValueError, match="h must be"):
        P.poetx_ffn_fwd(x, W, h[:3])
    with pytest.raises(ValueError, match="z must be"):
        P.poetx_ffn_fwd(x, W, h, z=h)
    with pytest.raises(ValueError, match="CUDA"):
        P.poetx_ffn_fwd(x, W, h)
    with pytest.raises(ValueError, match="dh must be"):
        P.poetx_ffn_bwd(x, W, h[:, :8], dx=x)
    with pytest.raises(ValueError, match="u must be"):
        P.poetx_glu_fwd(h, h.bfloat16(), h)
    with pytest.raises(ValueError, match="du must be"):
        P.poetx_glu_bwd(h, h, h, h, h[:2])
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="pos must be"):
        P.poetx_qk_rope_fwd(q, None, pos.long(), f, q, None)
    with pytest.raises(ValueError, match="inv_freq"):
        P.poetx_qk_rope_fwd(q, None, pos, f[:31], q, None)
    with pytest.raises(ValueError, match="axis"):
        P.poetx_qk_rope_fwd(q, None, pos, f, q, None, axis=pos)
    with pytest.raises(ValueError, match="CUDA"):
        P.poetx_qk_rope_fwd(q, None, pos, f, q, None)
    n = torch.zeros(1)
    with pytest.raises(ValueError, match="norm must be"):
        P.poetx_grad_norm([x], torch.zeros(2))
    with pytest.raises(ValueError, match="per q"):
        P.poetx_adam_group([x], [x], [x], [], 1, 1e-3)
    with pytest.raises(ValueError, match="CUDA"):
        P.poetx_grad_norm([x], n)
