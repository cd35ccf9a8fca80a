"""The linear head's cross entropy and distillation against the fp64 definition.

Tolerances, relative Frobenius error.  loss and lse (fp32): logits of bf16 operands are exact
products summed in fp32 (the tensor core's adds are handed over every 512 of K: about 32 x 2^-24 of
a partial sum), so TOL_F32.  bf16 dx and dW: dz is rounded to bf16 for its products and the result
once more, two roundings of at most 2^-8 (RMS 1.7e-3 each), TOL_BF16_STEP.  fp32 heads: TOL_F32
throughout."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import DEV, P, TOL_BF16_STEP, TOL_F32, dev, host  # noqa: F401
from oracle import head_oracle as H

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _inputs(N, V, D, dt, seed):
    r = np.random.default_rng(seed)
    W = r.standard_normal((V, D)) / np.sqrt(D)
    t = r.integers(0, V, N)
    x = r.standard_normal((N, D)) + r.uniform(0, 12, (N, 1)) * W[t] / (W[t] ** 2).sum(1)[:, None]
    x, W = torch.tensor(x).to(DT[dt]), torch.tensor(W).to(DT[dt])
    dloss = (r.uniform(0.5, 1.5, N) / N).astype(np.float32)
    return x, W, t.astype(np.int32), dloss


def _ce(P, x, W, t, dloss, z_loss=0.0, dx=True, dW=True, acc=None, **kw):
    xd, Wd = x.to(DEV), W.to(DEV)
    N = x.shape[0]
    o = {k: torch.full((N,), float("nan"), device=DEV) for k in ("loss", "lse")}
    if dx:
        o["dx"] = torch.full_like(xd, float("nan"))
    if dW:
        o["dW"] = torch.full_like(Wd, float("nan") if acc is None else acc)
    P.poetx_head_ce(xd, Wd, dev(t, torch.int32), o["loss"], lse=o["lse"], z_loss=z_loss,
                    dloss=dev(dloss, torch.float32) if dx or dW else None, dx=o.get("dx"),
                    dW=o.get("dW"), accumulate=acc is not None, **kw)
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    return o


def _distill(P, x, W, idx, u, dloss, T=1.0, grads=True):
    xd, Wd = x.to(DEV), W.to(DEV)
    N = x.shape[0]
    o = {k: torch.full((N,), float("nan"), device=DEV) for k in ("loss", "lse")}
    if grads:
        o["dx"], o["dW"] = torch.full_like(xd, float("nan")), torch.full_like(Wd, float("nan"))
    P.poetx_head_distill(xd, Wd, dev(idx, torch.int32), dev(u, torch.float32), o["loss"],
                         lse=o["lse"], dloss=dev(dloss, torch.float32) if grads else None,
                         dx=o.get("dx"), dW=o.get("dW"), temperature=T)
    torch.cuda.synchronize()
    assert P.poetx_get_device_error() == 0
    return o


def _near(got, ref, dt):
    for k in got:
        tol = TOL_BF16_STEP if dt == "bf16" and k in ("dx", "dW") else TOL_F32
        assert O.rel_fro(host(got[k]), ref[k]) <= tol, k


# one row, one class, less than a tile, tile and group edges, odd vocabularies, K tails
SHAPES = [(1, 1, 8), (1, 2, 64), (3, 33, 72), (5, 127, 8), (127, 129, 128), (128, 256, 64),
          (129, 257, 200), (256, 128, 520), (300, 1000, 1024), (257, 5003, 136), (700, 3001, 264)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D", SHAPES)
def test_ce(P, N, V, D, dt):
    x, W, t, g = _inputs(N, V, D, dt, N + V + D)
    got = _ce(P, x, W, t, g)
    ref = H.head_ce(host(x), host(W), t, g)
    if V == 1:  # p = 1: nothing to learn
        assert np.abs(host(got["loss"])).max() <= 1e-5 * np.abs(ref["lse"]).max()
        assert np.abs(host(got["dx"])).max() <= 1e-5 * np.abs(g).max() * np.abs(host(W)).max()
        return
    _near(got, ref, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("z_loss", [0.0, 0.02])
def test_ce_ignored_rows(P, dt, z_loss):
    x, W, t, g = _inputs(301, 777, 96, dt, 5)
    t[::3] = -100
    t[1] = -1
    got = _ce(P, x, W, t, g, z_loss)
    _near(got, H.head_ce(host(x), host(W), t, g, z_loss), dt)
    assert not host(got["loss"])[t < 0].any() and not host(got["dx"])[t < 0].any()
    t[:] = -100  # nothing left
    got = _ce(P, x, W, t, g, z_loss)
    assert not host(got["loss"]).any() and not host(got["dx"]).any() and not host(got["dW"]).any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ce_parts_agree(P, dt):
    """Loss alone, dx alone, dW alone and all at once give the same bits, every time."""
    x, W, t, g = _inputs(290, 1100, 192, dt, 6)
    full = _ce(P, x, W, t, g)
    for dx, dW in ((True, True), (True, False), (False, True), (False, False)):
        got = _ce(P, x, W, t, g, dx=dx, dW=dW)
        for k in got:
            assert torch.equal(got[k], full[k]), (k, dx, dW)


# one row to a full 128, one tile to several per SM, tiles of 16 rows and of odd heights, K past one
# accumulator hand-over
@pytest.mark.parametrize("N,V,D", [(1, 5, 64), (1, 32000, 2048), (2, 1, 8), (16, 333, 200),
                                   (17, 2433, 1032), (31, 40001, 128), (33, 5003, 72),
                                   (64, 50257, 64), (65, 19457, 2056), (128, 3000, 1600)])
def test_ce_loss_of_few_rows(P, N, V, D):
    x, W, t, g = _inputs(N, V, D, "bf16", N + V + D)
    t[N // 2] = -1 if N > 2 else t[N // 2]
    got = _ce(P, x, W, t, g, dx=False, dW=False)
    ref = H.head_ce(host(x), host(W), t)
    if V == 1:
        assert np.abs(host(got["loss"])).max() <= 1e-5 * np.abs(ref["lse"]).max()
        return
    _near(got, ref, "bf16")


@pytest.mark.parametrize("N,V,D,ignored", [(1, 700, 512, 0), (16, 1440, 264, 0), (17, 333, 1344, 2),
                                           (56, 1440, 1344, 28), (100, 9001, 136, 7),
                                           (128, 2433, 520, 0)])
def test_gradients_of_few_rows(P, N, V, D, ignored):
    """Up to 128 rows the gradients are as exact as their type: dz carries 16 bits, so what is left
    is the output's rounding.  Its RMS for values spread over a binade is 2^-8 / sqrt(3) x 0.74 =
    1.66e-3 (1 / m^2 averages 0.54 over a log-uniform m); 2^-9 leaves 17 % for the spread of a few
    large entries and the 2^-11 of the stored exponentials."""
    x, W, t, g = _inputs(N, V, D, "bf16", N + V + D)
    t[:ignored] = -1
    ref = H.head_ce(host(x), host(W), t, g)
    got = _ce(P, x, W, t, g)
    for k in ("dx", "dW"):
        assert O.rel_fro(host(got[k]), ref[k]) <= 2.0 ** -9, k
    assert not host(got["dx"])[:ignored].any()
    for dx, dW in ((True, False), (False, True)):  # the same bits alone
        part = _ce(P, x, W, t, g, dx=dx, dW=dW)
        assert all(torch.equal(part[k], got[k]) for k in part)
    acc = _ce(P, x, W, t, g, acc=0.25)
    assert O.rel_fro(host(acc["dW"]), ref["dW"] + 0.25) <= TOL_BF16_STEP


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ce_accumulates_dW(P, dt):
    x, W, t, g = _inputs(150, 500, 128, dt, 7)
    ref = H.head_ce(host(x), host(W), t, g)
    got = _ce(P, x, W, t, g, acc=0.25)
    assert O.rel_fro(host(got["dW"]), ref["dW"] + 0.25) <= \
        (TOL_BF16_STEP if dt == "bf16" else TOL_F32)


def test_ce_far_logits(P):
    """Logits in the hundreds: probabilities of exactly 0 and 1 in fp32, no overflow."""
    x, W, t, g = _inputs(64, 600, 64, "bf16", 8)
    x = x * 40
    t[::2] = (t[::2] + 1) % 600
    _near(_ce(P, x, W, t, g), H.head_ce(host(x), host(W), t, g), "bf16")


def test_ce_infinite_weights(P):
    """A vocabulary entry whose logit is -inf gets probability 0 (also where a whole group of 128
    has it); a NaN stays in its row."""
    x, W, t, g = _inputs(40, 700, 64, "bf16", 9)
    x = x.abs() + 0.1
    W[128:256] = float("-inf")
    W[300] = float("-inf")
    t[(t >= 128) & (t < 256) | (t == 300)] = 5
    got = _ce(P, x, W, t, g, dx=False, dW=False)
    keep = np.ones(700, bool)
    keep[128:256] = keep[300] = False
    place = np.cumsum(keep) - 1
    ref = H.head_ce(host(x), host(W)[keep], place[t])
    _near(got, ref, "bf16")
    x, W, t, g = _inputs(40, 700, 64, "bf16", 10)
    x[7, 3] = float("nan")
    got = _ce(P, x, W, t, g, dW=False)
    bad = torch.isnan(got["loss"])
    assert bad[7] and bad.sum() == 1
    assert torch.isfinite(got["dx"][[r for r in range(40) if r != 7]]).all()


def test_ce_target_beyond_the_vocabulary(P):
    x, W, t, g = _inputs(20, 90, 64, "bf16", 11)
    t[4] = 90
    got = _ce(P, x, W, t, g)
    t[4] = -1
    ref = _ce(P, x, W, t, g)
    assert torch.isnan(got["loss"][4]) and not got["dx"][4].any()
    assert torch.equal(got["dW"], ref["dW"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,K,T", [(1, 40, 64, 1, 1.0), (5, 300, 72, 300, 2.0),
                                       (130, 1001, 128, 7, 4.0), (257, 3001, 200, 64, 2.0),
                                       (33, 5000, 64, 1024, 1.0)])
def test_distill(P, N, V, D, K, T, dt):
    x, W, t, g = _inputs(N, V, D, dt, N + V + K)
    r = np.random.default_rng(K)
    idx = np.stack([r.permutation(V)[:K] for _ in range(N)]).astype(np.int32)
    idx[:, 0] = t if K == 1 else idx[:, 0]
    u = r.uniform(0, 10, (N, K)).astype(np.float32)
    _near(_distill(P, x, W, idx, u, g, T), H.head_distill(host(x), host(W), idx, u, g, T), dt)
    a = _distill(P, x, W, idx, u, g, T, grads=False)
    if dt == "f32" or N > 128:
        b = _distill(P, x, W, idx, u, g, T)
        assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["lse"], b["lse"])
    else:  # few rows, loss alone: a product of its own
        _near(a, H.head_distill(host(x), host(W), idx, u, None, T), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_distill_absent_repeated_and_empty(P, dt):
    x, W, _, g = _inputs(60, 400, 64, dt, 12)
    r = np.random.default_rng(1)
    idx = np.stack([r.permutation(400)[:9] for _ in range(60)]).astype(np.int32)
    u = r.uniform(-3, 6, (60, 9)).astype(np.float32)
    idx[3] = -1                       # an empty row
    u[4] = -np.inf                    # one whose every weight is zero
    idx[5, 2:] = -7
    u[5, 2:] = np.nan                 # absent entries are not read
    u[6, 0] = -np.inf
    u[7, 1:] = np.finfo(np.float32).min
    idx[8, :] = 17                    # one entry, nine times
    idx[9, 4] = idx[9, 0]
    got = _distill(P, x, W, idx, u, g, 2.0)
    ref = H.head_distill(host(x), host(W), idx, u, g, 2.0)
    _near(got, ref, dt)
    for row in (3, 4):
        assert host(got["loss"])[row] == 0 and not host(got["dx"])[row].any()


def test_distill_of_one_entry_is_cross_entropy(P):
    x, W, t, g = _inputs(140, 900, 128, "bf16", 13)
    a = _ce(P, x, W, t, g)
    b = _distill(P, x, W, t[:, None], np.zeros((140, 1), np.float32), g)
    for k in a:
        assert O.rel_fro(host(b[k]), host(a[k])) <= TOL_F32, k


def _torch64(x, W, t, g):
    x, W, g = x.double(), W.double(), g.double()
    z = x @ W.T
    lse = torch.logsumexp(z, 1)
    rows = torch.arange(len(t), device=DEV)
    loss = lse - z[rows, t.long()]
    dz = torch.exp(z - lse[:, None])
    dz[rows, t.long()] -= 1
    dz *= g[:, None]
    return {"loss": loss, "lse": lse, "dx": dz @ W, "dW": dz.T @ x}


@pytest.mark.parametrize("N", [4500, 9500])
@pytest.mark.parametrize("acc", [None, 0.001])
def test_ce_in_pieces_of_rows(P, acc, N):
    """Many rows, and more than one piece holds (about 2 GB of 16-bit values): dW is the sum over the
    pieces, rounded once."""
    r = torch.Generator(device=DEV).manual_seed(3)
    V, D = 128001, 64
    W = (torch.randn(V, D, generator=r, device=DEV) / 8).bfloat16()
    x = torch.randn(N, D, generator=r, device=DEV).bfloat16()
    t = torch.randint(0, V, (N,), generator=r, device=DEV).int()
    g = torch.full((N,), 1.0 / N, device=DEV)
    assert P.poetx_head_workspace_bytes(P.BF16, N, D, V) > V * D * 4
    got = _ce(P, x, W, t.cpu().numpy(), g.cpu().numpy(), acc=acc)
    ref = _torch64(x, W, t, g)
    if acc:
        # the sum is of the size of acc here: its rounding is the error
        ref["dW"] = ref["dW"] + float(torch.tensor(acc).bfloat16())
    for k in ref:
        tol = TOL_BF16_STEP if k in ("dx", "dW") else TOL_F32
        err = ((got[k].double() - ref[k]).norm() / ref[k].norm()).item()
        assert err <= tol, (k, err)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ce_many_rows(P, dt):
    """More rows than a piece takes whatever its bytes: dW over three pieces."""
    x, W, t, g = _inputs(150001, 7, 8, dt, 20)
    t[::5] = -1
    _near(_ce(P, x, W, t, g), H.head_ce(host(x), host(W), t, g), dt)
    got = _ce(P, x, W, t, g, dx=False, dW=False)
    _near(got, H.head_ce(host(x), host(W), t), dt)


@pytest.mark.parametrize("N,V,D", [(3, 4194304, 8), (5, 300, 131072)])
def test_ce_at_the_limits(P, N, V, D):
    x, W, t, g = _inputs(N, V, D, "bf16", 21)
    ref = H.head_ce(host(x), host(W), t, g)
    _near(_ce(P, x, W, t, g), ref, "bf16")
    _near(_ce(P, x, W, t, g, dx=False, dW=False), ref, "bf16")


def test_ce_uneven_upstream_gradients(P):
    """Upstream gradients over ten decades, zeros and signs among them; and all zero."""
    x, W, t, g = _inputs(300, 700, 64, "bf16", 22)
    r = np.random.default_rng(5)
    g = (10.0 ** r.uniform(-10, 0, 300) * r.choice([-1, 1, 0], 300)).astype(np.float32)
    _near(_ce(P, x, W, t, g), H.head_ce(host(x), host(W), t, g), "bf16")
    got = _ce(P, x, W, t, np.zeros(300, np.float32))
    assert not host(got["dx"]).any() and not host(got["dW"]).any()


def test_head_on_another_stream(P):
    x, W, t, g = _inputs(300, 2000, 256, "bf16", 14)
    ref = _ce(P, x, W, t, g)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _ce(P, x, W, t, g, stream=s)
    s.synchronize()
    for k in ref:
        assert torch.equal(got[k], ref[k]), k


def test_head_empty_batch(P):
    W = torch.randn(50, 64, device=DEV).bfloat16()
    x, e = W[:0], torch.empty(0, device=DEV)
    dW = torch.ones_like(W)
    P.poetx_head_ce(x, W, e.int(), e, dloss=e, dx=torch.empty_like(x), dW=dW, accumulate=True)
    assert (dW == 1).all()
    P.poetx_head_ce(x, W, e.int(), e, dloss=e, dx=torch.empty_like(x), dW=dW)
    assert not dW.any()


def test_head_default_stream_scratch_is_per_thread(P):
    """Calls of two threads on the default stream, interleaved as they come: each thread has its own
    scratch."""
    import threading
    cases = [_inputs(200, 1500, 128, "bf16", 15), _inputs(90, 2500, 256, "bf16", 16)]
    refs = [_ce(P, *c) for c in cases]
    errors = []

    def work(i):
        try:
            for _ in range(20):
                got = _ce(P, *cases[i])
                for k in got:
                    if not torch.equal(got[k], refs[i][k]):
                        errors.append((i, k))
        except Exception as e:  # noqa: BLE001
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


def test_head_in_a_cuda_graph(P):
    """Captured and replayed on new inputs, with its scratch from the graph's pool."""
    x, W, t, g = _inputs(130, 1100, 128, "bf16", 17)
    x2, _, t2, _ = _inputs(130, 1100, 128, "bf16", 18)
    ref = _ce(P, x2, W, t2, g)
    xd, Wd, td, gd = x.to(DEV), W.to(DEV), dev(t, torch.int32), dev(g, torch.float32)
    out = {"loss": torch.empty(130, device=DEV), "lse": torch.empty(130, device=DEV),
           "dx": torch.empty_like(xd), "dW": torch.empty_like(Wd)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.poetx_head_ce(xd, Wd, td, out["loss"], lse=out["lse"], dloss=gd, dx=out["dx"],
                        dW=out["dW"])
    xd.copy_(x2)
    td.copy_(dev(t2, torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(out[k], ref[k]), k
