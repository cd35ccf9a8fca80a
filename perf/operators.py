"""Measured cases of the training head's operators: layer norm (forward, and backward with the
reduction of its parameters' gradients), the softmax cross entropy of a linear head over a large
vocabulary (loss alone, or loss and gradients), and distillation from a teacher's top logits
through the same head.

`own = False` computes the operators in their plain form (elementary torch operations in fp32);
`own = True` makes the calls of ``orthogonal_reparameterized_gb300.poetx``.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}


def _norm(name, direction, N, D, dtype=BF16):
    return {"name": name, "op": "norm_" + direction, "N": N, "D": D, "dtype": dtype}


def _ce(name, N, V, D, grads=True, dtype=BF16, ignored=0.0, z_loss=0.0):
    return {"name": name, "op": "ce", "N": N, "V": V, "D": D, "grads": grads, "dtype": dtype,
            "ignored": ignored, "z_loss": z_loss}


def _distill(name, N, V, D, K, grads=True, dtype=BF16, ignored=0.0, temperature=1.0):
    return {"name": name, "op": "distill", "N": N, "V": V, "D": D, "K": K, "grads": grads,
            "dtype": dtype, "ignored": ignored, "temperature": temperature}


def listed():
    return [
        # the norm before a linear for one token being served: latency
        _norm("norm_fwd_1x4096", "fwd", 1, 4096),
        # the norms of one training step of the benchmark's block (8192 tokens, 4096 wide)
        _norm("norm_fwd_8192x4096", "fwd", 8192, 4096),
        _norm("norm_bwd_8192x4096", "bwd", 8192, 4096),
        # an odd width in fp32, rows that are not 16-byte aligned
        _norm("norm_bwd_f32_1001x1443", "bwd", 1001, 1443, F32),
        # the score of one next token: every weight of the head is read for one row
        _ce("ce_loss_1x32000x2048", 1, 32000, 2048, grads=False),
        # a training step's head at the 2048-wide layer with a vocabulary of ordinary size
        _ce("ce_4096x32000x2048", 4096, 32000, 2048),
        # a ragged batch with an odd vocabulary: prompts ignored, z-loss on
        _ce("ce_1021x50257x1600", 1021, 50257, 1600, ignored=0.5, z_loss=1e-4),
        # the largest: the benchmark's 8192 tokens, 4096 wide, a vocabulary of 128 thousand
        _ce("ce_8192x128256x4096", 8192, 128256, 4096, ignored=0.1),
        # the fp32 head beside the fp32 layer
        _ce("ce_f32_512x8000x1024", 512, 8000, 1024, dtype=F32),
        # validation of a student: the loss of a few sequences' ends
        _distill("distill_loss_33x32000x1024_k8", 33, 32000, 1024, 8, grads=False),
        # a distillation step from 64 kept logits at a raised temperature, some entries absent
        _distill("distill_2047x32000x2048_k64", 2047, 32000, 2048, 64, ignored=0.1,
                 temperature=2.0),
        # a large distillation step
        _distill("distill_4096x128256x4096_k128", 4096, 128256, 4096, 128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ce", "ce", "distill", "distill"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    if op.startswith("norm"):
        D = _log_int(rng, 8, 8192)
        if rng.random() < 0.5:  # widths of models are mostly multiples of 8
            D = max(8, D // 8 * 8)
        return {"op": op, "N": _log_int(rng, 1, 8192), "D": D, "dtype": dtype}
    small = dtype == F32
    c = {"op": op,
         "N": _log_int(rng, 1, 512 if small else 8192),
         "V": _log_int(rng, 500, 8000 if small else 128256),
         "D": 8 * _log_int(rng, 8, 128 if small else 512),
         "grads": rng.random() < 0.75,
         "dtype": dtype,
         "ignored": rng.choice([0.0, 0.1, 0.5])}
    if op == "ce":
        c["z_loss"] = rng.choice([0.0, 1e-4])
    else:
        c["K"] = _log_int(rng, 1, 256)
        c["temperature"] = rng.choice([1.0, 2.0, 4.0])
    return c


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    N, D = case["N"], case["D"]
    s = dict(case)
    if case["op"].startswith("norm"):
        # rows of different scale with a mean of their own, as a residual stream has
        x = _randn(g, N, D) * (0.5 + _randn(g, N, 1).abs()) + 0.3 * _randn(g, N, 1) + 0.2
        s["x"] = x.to(dt)
        s["gamma"] = 1.0 + 0.1 * _randn(g, D)
        s["beta"] = 0.1 * _randn(g, D)
        s["eps"] = 1e-5
        if case["op"] == "norm_bwd":
            s["dy"] = (_randn(g, N, D) * 0.1).to(dt)
            xf = s["x"].float()  # what the forward pass kept
            s["mean"] = xf.mean(1)
            s["rstd"] = 1.0 / torch.sqrt(((xf - s["mean"][:, None]) ** 2).mean(1) + s["eps"])
        return s
    V = case["V"]
    # head weights of 1/sqrt(D) scale; normalised hidden states that point, by a part of their
    # own, at the row's target, so that its probability runs from 1/V to about a third
    W = _randn(g, V, D) * D ** -0.5
    x = _randn(g, N, D)
    kept = torch.rand(N, generator=g, device="cuda") >= case["ignored"]
    if case["op"] == "ce":
        target = torch.randint(0, V, (N,), generator=g, device="cuda")
    else:
        K = case["K"]
        gap = torch.randint(1, max(2, V // (K + 1)), (N, K), generator=g, device="cuda")
        index = (torch.randint(0, V, (N, 1), generator=g, device="cuda") + gap.cumsum(1)) % V
        target = index[:, 0]
        logit = 12.0 - 10.0 * torch.rand(N, K, generator=g, device="cuda")
        # some entries of a row are absent, and where `kept` says so the whole row
        absent = torch.rand(N, K, generator=g, device="cuda") < 0.5 * case["ignored"]
        index = torch.where(absent | ~kept[:, None], torch.full_like(index, -1), index)
        s["t_index"], s["t_logit"] = index.int(), logit
    Wt = W[target]
    pull = math.log(V) * torch.rand(N, 1, generator=g, device="cuda")
    x = x + pull * Wt / (Wt * Wt).sum(1, keepdim=True)
    s["x"], s["W"] = x.to(dt), W.to(dt)
    if case["op"] == "ce":
        s["target"] = torch.where(kept, target, torch.full_like(target, -100)).int()
    # the mean over the kept rows
    s["dloss"] = torch.full((N,), 1.0, device="cuda") / kept.sum().clamp(min=1)
    return s


# ---------------------------------------------------------------- plain forms (fp32)
def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.sum(1) / x.shape[1]
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).sum(1) / x.shape[1] + s["eps"])
    y = c * rstd[:, None] * s["gamma"] + s["beta"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    D = x.shape[1]
    rstd = s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    dgamma, dbeta = (dy * xhat).sum(0), dy.sum(0)
    wdy = dy * s["gamma"]
    a = wdy.sum(1, keepdim=True) / D
    b = (wdy * xhat).sum(1, keepdim=True) / D
    dx = (wdy - a - xhat * b) * rstd
    return {"dx": dx.to(s["x"].dtype), "dgamma": dgamma, "dbeta": dbeta}


def _plain_softmax(z):
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    return e / total, (top + torch.log(total))[:, 0]


def _plain_grads(s, out, dlogit, x, W):
    if s["grads"]:
        out["dx"] = (dlogit @ W).to(s["x"].dtype)
        out["dW"] = (dlogit.t() @ x).to(s["W"].dtype)
    return out


def _plain_ce(s):
    x, W = s["x"].float(), s["W"].float()
    z = x @ W.t()
    p, lse = _plain_softmax(z)
    valid = s["target"] >= 0
    t = s["target"].clamp(min=0).long()[:, None]
    zt = z.gather(1, t)[:, 0]
    loss = torch.where(valid, lse - zt + s["z_loss"] * lse * lse, torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse}
    if not s["grads"]:
        return out
    g = torch.where(valid, s["dloss"], torch.zeros_like(lse))
    dz = p * (1.0 + 2.0 * s["z_loss"] * lse)[:, None]
    dz = dz.scatter_add(1, t, torch.full_like(zt, -1.0)[:, None]) * g[:, None]
    return _plain_grads(s, out, dz, x, W)


def _plain_distill(s):
    x, W, T = s["x"].float(), s["W"].float(), s["temperature"]
    z = (x @ W.t()) / T
    p, lse = _plain_softmax(z)
    there = s["t_index"] >= 0
    some = there.any(1)
    idx = s["t_index"].clamp(min=0).long()
    u = torch.where(there, s["t_logit"] / T, torch.full_like(s["t_logit"], -math.inf))
    top = torch.where(some, u.max(1).values, torch.zeros_like(lse))[:, None]
    e = torch.exp(u - top)
    total = torch.where(some, e.sum(1), torch.ones_like(lse))[:, None]
    q = e / total
    logq = (torch.where(there, s["t_logit"] / T, torch.zeros_like(u)) - top) - torch.log(total)
    loss = T * T * (q * (logq - (z.gather(1, idx) - lse[:, None]))).sum(1)
    out = {"loss": loss, "lse": lse}
    if not s["grads"]:
        return out
    g = torch.where(some, s["dloss"] * T, torch.zeros_like(lse))
    return _plain_grads(s, out, p.scatter_add(1, idx, -q) * g[:, None], x, W)


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "ce": _plain_ce,
          "distill": _plain_distill}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import orthogonal_reparameterized_gb300.poetx as P
    x = s["x"]
    N = x.shape[0]
    f32 = dict(dtype=torch.float32, device=x.device)
    if s["op"] == "norm_fwd":
        y, mean, rstd = torch.empty_like(x), torch.empty(N, **f32), torch.empty(N, **f32)
        P.poetx_layernorm_fwd(x, y, gamma=s["gamma"], beta=s["beta"], mean=mean, rstd=rstd,
                              eps=s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if s["op"] == "norm_bwd":
        dx = torch.empty_like(x)
        dgamma, dbeta = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
        P.poetx_layernorm_bwd(x, s["dy"], s["mean"], s["rstd"], dx, gamma=s["gamma"],
                              dgamma=dgamma, dbeta=dbeta)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    out = {"loss": torch.empty(N, **f32), "lse": torch.empty(N, **f32)}
    kw = dict(lse=out["lse"])
    if s["grads"]:
        out["dx"], out["dW"] = torch.empty_like(x), torch.empty_like(s["W"])
        kw.update(dloss=s["dloss"], dx=out["dx"], dW=out["dW"])
    if s["op"] == "ce":
        P.poetx_head_ce(x, s["W"], s["target"], out["loss"], z_loss=s["z_loss"], **kw)
    else:
        P.poetx_head_distill(x, s["W"], s["t_index"], s["t_logit"], out["loss"],
                             temperature=s["temperature"], **kw)
    return out


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    N, D = case["N"], case["D"]
    esz = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "norm_fwd":  # x in, y out, the row statistics out, gamma and beta in
        return {"bytes": 2 * N * D * esz + 8 * N + 8 * D, "flops": 8 * N * D}
    if case["op"] == "norm_bwd":  # x and dy in, dx out, row statistics and gamma in, dgamma, dbeta
        return {"bytes": 3 * N * D * esz + 8 * N + 12 * D, "flops": 14 * N * D}
    V = case["V"]
    rows = 8 * N + (4 * N if case["op"] == "ce" else 8 * N * case["K"])
    if not case["grads"]:  # the logits' product
        return {"bytes": esz * (N * D + V * D) + rows, "flops": 2 * N * V * D}
    # the logits' product and the two of the gradients
    return {"bytes": 2 * esz * (N * D + V * D) + rows + 4 * N, "flops": 6 * N * V * D}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_norm(s):
    x, gamma = s["x"].double(), s["gamma"].double()
    mean = x.mean(dim=1, keepdim=True)
    sd = torch.sqrt(x.var(dim=1, unbiased=False, keepdim=True) + s["eps"])
    if s["op"] == "norm_fwd":
        return {"y": (x - mean) / sd * gamma + s["beta"].double(), "mean": mean[:, 0],
                "rstd": 1.0 / sd[:, 0]}
    dy = s["dy"].double()
    h = (x - mean) / sd
    # the Jacobian of the normalised row: (I - 1 1^T / D - h h^T / D) / sd
    u = dy * gamma
    dx = (u - u.mean(dim=1, keepdim=True) - h * (u * h).mean(dim=1, keepdim=True)) / sd
    return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", dy, h), "dbeta": dy.sum(dim=0)}


def _exact_head(s):
    x, W = s["x"].double(), s["W"].double()
    N, V = x.shape[0], W.shape[0]
    T = s.get("temperature", 1.0)
    z = torch.einsum("nd,vd->nv", x, W).div_(T)
    lse = torch.logsumexp(z, dim=1)
    if s["op"] == "ce":
        rows = (s["target"] >= 0).nonzero()[:, 0]
        q_rows, q_cols = rows, s["target"][rows].long()
        q = torch.ones(rows.numel(), dtype=torch.float64, device=x.device)
        entropy = torch.zeros(N, dtype=torch.float64, device=x.device)
    else:
        u = s["t_logit"].double() / T
        u = u.masked_fill(s["t_index"] < 0, -math.inf)
        q_rows, k = (s["t_index"] >= 0).nonzero(as_tuple=True)
        q_cols = s["t_index"][q_rows, k].long()
        logq = (u - torch.logsumexp(u, dim=1, keepdim=True))[q_rows, k]
        q = torch.exp(logq)
        entropy = torch.zeros(N, dtype=torch.float64, device=x.device).index_add_(0, q_rows,
                                                                               q * logq)
    some = torch.zeros(N, dtype=torch.bool, device=x.device)
    some[q_rows] = True
    cross = torch.zeros(N, dtype=torch.float64, device=x.device).index_add_(
        0, q_rows, q * (lse[q_rows] - z[q_rows, q_cols]))
    zl = s.get("z_loss", 0.0)
    loss = (entropy + cross) * T * T + torch.where(some, zl * lse ** 2, torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse}
    if s["grads"]:
        weight = s["dloss"].double() * some * T
        p = torch.exp(z.sub_(lse[:, None]))
        p *= (weight * (1.0 + 2.0 * zl * lse))[:, None]
        p.index_put_((q_rows, q_cols), -q * weight[q_rows], accumulate=True)
        out["dx"] = torch.einsum("nv,vd->nd", p, W)
        out["dW"] = torch.einsum("nv,nd->vd", p, x)
    return out


def exact(case, seed):
    if case["op"].startswith("norm"):
        return _exact_norm(prepare(case, seed))
    if work(case)["flops"] > 8e12:  # 64-bit products run at about a teraflop per second
        return None
    return _exact_head(prepare(case, seed))
