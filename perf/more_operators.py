"""Measured cases of what a transformer block's training step has between its linears and behind
them: the gated feed-forward block (both projections, activation and product; backward from kept or
recomputed projections), the gated product alone between two POET-X layers, the norms of queries
and keys with the rotation by positions on one or several axes, and the global norm of many
gradients with the optimizer step that clips by it.

`own = False` computes the operators in their plain form (elementary torch operations in fp32,
angles and sums over whole models in 64 bits); `own = True` makes the calls of
``orthogonal_reparameterized_gb300.poetx``.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_GELU_C, _GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def _ffn(name, op, N, D, F, dtype=BF16, act="silu", keep=False):
    """op: ffn_fwd (keep: the projections are stored for the backward), ffn_bwd (from stored
    projections), ffn_mem (backward that computes them again)."""
    return {"name": name, "op": op, "N": N, "D": D, "F": F, "dtype": dtype, "act": act,
            "keep": keep}


def _glu(name, op, N, F, dtype=BF16, act="silu"):
    return {"name": name, "op": op, "N": N, "F": F, "dtype": dtype, "act": act}


def _rope(name, op, N, Hq, Hk, dh, rot, axes=1, interleaved=False, norm=True, fused=False,
          dtype=BF16):
    """fused: queries, keys and values lie side by side in one row."""
    return {"name": name, "op": op, "N": N, "Hq": Hq, "Hk": Hk, "dh": dh, "rot": rot, "axes": axes,
            "interleaved": interleaved, "norm": norm, "fused": fused, "dtype": dtype}


def _many(name, op, blocks, width, inner, b, V=0):
    """op: update (global norm of every block's triangle gradients, then the clipped optimizer
    step), grad_norm (the norm alone, with the bf16 gradient of a [V, width] head among them).
    blocks: transformer blocks of seven POET-X linears; 0: a single linear width -> inner."""
    return {"name": name, "op": op, "blocks": blocks, "width": width, "inner": inner, "b": b,
            "V": V}


def listed():
    return [
        # one token being served: every weight of the block is read for one row
        _ffn("ffn_fwd_1x4096x14336", "ffn_fwd", 1, 4096, 14336),
        # a training step of the benchmark's block (8192 tokens, 4096 wide, 14336 inside): the largest
        _ffn("ffn_fwd_8192x4096x14336", "ffn_fwd", 8192, 4096, 14336, keep=True),
        # the backward at the 2048-wide layer's tokens, from the kept projections
        _ffn("ffn_bwd_4096x2048x8192", "ffn_bwd", 4096, 2048, 8192),
        # a ragged batch with odd widths, the projections computed again
        _ffn("ffn_mem_1021x1600x4264_gelu", "ffn_mem", 1021, 1600, 4264, act="gelu"),
        # the fp32 block beside the fp32 layer
        _ffn("ffn_bwd_f32_512x1024x2816", "ffn_bwd", 512, 1024, 2816, dtype=F32),
        # the product between the benchmark's gate, up and down layers, on the way back
        _glu("glu_bwd_8192x14336", "glu_bwd", 8192, 14336),
        # queries and keys of one token being served: latency
        _rope("rope_fwd_1x32x8x128", "rope_fwd", 1, 32, 8, 128, 128, fused=True),
        # a training step's queries and keys (8192 tokens of 32 and 8 heads)
        _rope("rope_fwd_8192x32x8x128", "rope_fwd", 8192, 32, 8, 128, 128),
        # the way back at a 5120-wide layer's 40 heads, positions in time, height and width
        _rope("rope_bwd_4096x40x40x128_3axes", "rope_bwd", 4096, 40, 40, 128, 128, axes=3),
        # the step behind the backward of the benchmark's seven linears
        _many("update_1x4096x14336_b256", "update", 1, 4096, 14336, 256),
        # the same behind a whole model of 32 such blocks (360 M stored parameters, 448 tensors)
        _many("update_32x4096x14336_b256", "update", 32, 4096, 14336, 256),
        # the norm over the triangles of 16 blocks and a trained bf16 head
        _many("grad_norm_16x2048x8192_v128256", "grad_norm", 16, 2048, 8192, 256, V=128256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_bwd", "ffn_mem", "glu_fwd", "glu_bwd", "rope_fwd", "rope_fwd",
                     "rope_bwd", "rope_bwd", "update", "grad_norm"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    act = rng.choice(["silu", "silu", "gelu"])
    if op.startswith("ffn"):
        small = dtype == F32
        N, D = _log_int(rng, 1, 512 if small else 8192), 8 * _log_int(rng, 8, 128 if small else 512)
        F = 8 * _log_int(rng, 8, 352 if small else 1792)
        N = max(1, N // {"ffn_fwd": 1, "ffn_bwd": 2, "ffn_mem": 3}[op])  # the same cost at most
        c = _ffn("", op, N, D, F, dtype, act, op == "ffn_fwd" and rng.random() < 0.5)
    elif op.startswith("glu"):
        c = _glu("", op, _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1792), dtype, act)
    elif op.startswith("rope"):
        dh = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128, 192, 256])
        rot = rng.choice([dh, dh, max(8, dh // 16 * 8)])
        Hk = _log_int(rng, 1, 16)
        c = _rope("", op, _log_int(rng, 1, 8192), Hk * rng.choice([1, 2, 4, 7]), Hk, dh, rot,
                  rng.choice([1, 1, 2, 3]), rng.random() < 0.3, rng.random() < 0.75,
                  rng.random() < 0.3, dtype)
    else:
        b = rng.choice([32, 64, 128, 256])
        width, inner = 8 * _log_int(rng, 32, 512), 8 * _log_int(rng, 32, 1792)
        V = 0 if op == "update" else _log_int(rng, 100, 128256)
        c = _many("", op, rng.choice([0, 1, 2, 4, 8, 16, 32]), width, inner, b, V)
    del c["name"]
    return c


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _triangle_shapes(case):
    """The packed triangles' shapes, [blocks of a side, b (b - 1) / 2], both sides of each linear."""
    w, i, b = case["width"], case["inner"], case["b"]
    linears = ([(w, w)] * 4 + [(w, i)] * 2 + [(i, w)]) * case["blocks"] or [(w, i)]
    return [(-(-side // b), b * (b - 1) // 2) for lin in linears for side in lin]


def _views(flat, shapes):
    """The tensors of one flat buffer, each from a 16-byte boundary on."""
    out, at = [], 0
    for n, k in shapes:
        out.append(flat[at:at + n * k].view(n, k))
        at += -(-n * k // 4) * 4
    return out


def _prepare_many(case, g, s):
    shapes = _triangle_shapes(case)
    total = sum(-(-n * k // 4) * 4 for n, k in shapes)

    def flat(scale):
        return _randn(g, total) * scale

    s["dq_flat"] = flat(3e-3)
    s["dq"] = _views(s["dq_flat"], shapes)
    if case["op"] == "grad_norm":
        s["grads"] = s["dq"] + [(_randn(g, case["V"], case["width"]) * 1e-3).bfloat16(),
                                _randn(g, case["width"]) * 1e-2]
        return s
    s["flat"] = {"q": flat(0.02), "m": flat(1e-3), "v": flat(1e-3) ** 2}
    for k in ("q", "m", "v"):
        s[k] = _views(s["flat"][k], shapes)
    # (the gradients' norm is 3e-3 sqrt(total): beyond 1 from some 110 thousand parameters on)
    hp = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
    # fp32 numbers, as the optimizer takes them (1 - 0.999 is another number otherwise)
    s["hp"] = {"step": 100, **{k: torch.tensor(v).item() for k, v in hp.items()}}
    s["max_norm"] = 1.0
    return s


def _prepare_rope(case, g, s):
    N, dh, dt = case["N"], case["dh"], _DT[case["dtype"]]

    def heads(scale):
        # projections, some heads larger than others
        shape = {"q": case["Hq"], "k": case["Hk"]}
        t = {n: (_randn(g, N, h, dh) * (0.5 + _randn(g, 1, h, 1).abs()) * scale).to(dt)
             for n, h in shape.items()}
        if case["fused"]:
            row = torch.cat([t["q"].flatten(1), t["k"].flatten(1), t["k"].flatten(1)], 1)
            cut = case["Hq"] * dh
            t = {"q": row[:, :cut].unflatten(1, (case["Hq"], dh)),
                 "k": row[:, cut:cut + case["Hk"] * dh].unflatten(1, (case["Hk"], dh))}
        return t

    t = heads(1.0)
    s["q"], s["k"] = t["q"], t["k"]
    if case["op"] == "rope_bwd":
        t = heads(0.01)
        s["dq"], s["dk"] = t["q"], t["k"]
    s["gamma_q"] = s["gamma_k"] = None
    if case["norm"]:
        s["gamma_q"], s["gamma_k"] = 1.0 + 0.1 * _randn(g, dh), 1.0 + 0.1 * _randn(g, dh)
    half = case["rot"] // 2
    s["inv_freq"] = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / half)
    # tokens of long documents; an image's rows and columns on the other axes
    first = torch.randint(0, 100000, (1,), generator=g, device="cuda")
    pos = [first + torch.arange(N, device="cuda")]
    for a in range(1, case["axes"]):
        pos.append(torch.randint(0, 1000, (N,), generator=g, device="cuda"))
    s["pos"] = torch.stack(pos).int()
    s["axis"] = None
    if case["axes"] > 1:  # each axis its section of the frequencies
        s["axis"] = (torch.arange(half, device="cuda") * case["axes"] // half).int()
    s["eps"] = 1e-6
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("update", "grad_norm"):
        return _prepare_many(case, g, s)
    if op.startswith("rope"):
        return _prepare_rope(case, g, s)
    dt = _DT[case["dtype"]]
    N, F = case["N"], case["F"]
    if op.startswith("glu"):
        s["g"], s["u"] = _randn(g, N, F).to(dt), _randn(g, N, F).to(dt)
    else:
        # normalised hidden states, weights that keep their scale; rows 0..F-1 gate, the rest up
        s["x"] = _randn(g, N, case["D"]).to(dt)
        s["W"] = (_randn(g, 2 * F, case["D"]) * case["D"] ** -0.5).to(dt)
        s["z"] = s["x"] @ s["W"].t() if op == "ffn_bwd" else None  # what the forward kept
    if not op.endswith("fwd"):
        # the gradient of a mean over the tokens, larger in some rows
        s["dh"] = (_randn(g, N, F) * (0.1 + _randn(g, N, 1).abs()) / N).to(dt)
    return s


# ---------------------------------------------------------------- plain forms (fp32)
def _gate(g, act):
    """(a(g), a'(g)) of the activation."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    # the tanh form of GELU: (1 + tanh(t / 2)) / 2 = sigmoid(t)
    sig = 1.0 / (1.0 + torch.exp(-2.0 * _GELU_C * (g + _GELU_A * g * g * g)))
    return g * sig, sig + g * sig * (1.0 - sig) * 2.0 * _GELU_C * (1.0 + 3.0 * _GELU_A * g * g)


def _plain_glu_fwd(s):
    return {"h": (_gate(s["g"].float(), s["act"])[0] * s["u"].float()).to(s["g"].dtype)}


def _plain_dz(g, u, dh, act):
    a, d = _gate(g, act)
    return dh * u * d, dh * a


def _plain_glu_bwd(s):
    dg, du = _plain_dz(s["g"].float(), s["u"].float(), s["dh"].float(), s["act"])
    return {"dg": dg.to(s["g"].dtype), "du": du.to(s["g"].dtype)}


def _plain_ffn_fwd(s):
    F, dt = s["F"], s["x"].dtype
    z = s["x"].float() @ s["W"].float().t()
    out = {"h": (_gate(z[:, :F], s["act"])[0] * z[:, F:]).to(dt)}
    if s["keep"]:
        out["z"] = z.to(dt)
    return out


def _plain_ffn_bwd(s):
    F, dt = s["F"], s["x"].dtype
    x, W = s["x"].float(), s["W"].float()
    z = x @ W.t() if s["z"] is None else s["z"].float()
    dz = torch.cat(_plain_dz(z[:, :F], z[:, F:], s["dh"].float(), s["act"]), 1)
    return {"dx": (dz @ W).to(dt), "dW": (dz.t() @ x).to(dt)}


def _cos_sin(s):
    """[N, 1, rot / 2] cosines and sines; the angles in 64 bits (positions of 100 thousand)."""
    half = s["rot"] // 2
    axis = torch.zeros(half, dtype=torch.long, device="cuda") if s["axis"] is None else \
        s["axis"].long()
    angle = s["pos"].double()[axis].t() * s["inv_freq"].double()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _halves(t, s):
    """The pairs' first and second elements, and the elements that are not rotated."""
    r = s["rot"]
    if s["interleaved"]:
        return t[..., 0:r:2], t[..., 1:r:2], t[..., r:]
    return t[..., :r // 2], t[..., r // 2:r], t[..., r:]


def _joined(a, b, rest, s):
    both = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _plain_rope_one(t, gamma, cos, sin, s):
    x = t.float()
    if s["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["dh"] + s["eps"]) * gamma
    a, b, rest = _halves(x, s)
    return _joined(a * cos - b * sin, a * sin + b * cos, rest, s).to(t.dtype)


def _plain_rope_fwd(s):
    cos, sin = _cos_sin(s)
    return {"q": _plain_rope_one(s["q"], s["gamma_q"], cos, sin, s),
            "k": _plain_rope_one(s["k"], s["gamma_k"], cos, sin, s)}


def _plain_rope_bwd_one(t, dy, gamma, cos, sin, s):
    a, b, rest = _halves(dy.float(), s)
    d = _joined(a * cos + b * sin, b * cos - a * sin, rest, s)
    if not s["norm"]:
        return d.to(t.dtype), None
    x = t.float()
    rstd = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / s["dh"] + s["eps"])
    h = x * rstd
    u = d * gamma
    dx = (u - h * (u * h).sum(-1, keepdim=True) / s["dh"]) * rstd
    return dx.to(t.dtype), (d * h).sum((0, 1))


def _plain_rope_bwd(s):
    cos, sin = _cos_sin(s)
    dq, dgq = _plain_rope_bwd_one(s["q"], s["dq"], s["gamma_q"], cos, sin, s)
    dk, dgk = _plain_rope_bwd_one(s["k"], s["dk"], s["gamma_k"], cos, sin, s)
    out = {"dq": dq, "dk": dk}
    if s["norm"]:
        out["dgamma_q"], out["dgamma_k"] = dgq, dgk
    return out


def _plain_norm(grads):
    """One fp32 norm; squares in fp32, their sum in 64 bits (hundreds of millions of terms)."""
    parts = [(t.float() * t.float()).sum(dtype=torch.float64) for t in grads]
    return torch.sqrt(torch.stack(parts).sum()).float().reshape(1)


def _plain_grad_norm(s):
    return {"norm": _plain_norm(s["grads"])}


def _plain_update(s):
    hp = s["hp"]
    norm = _plain_norm(s["dq"])
    clip = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    c1, c2 = 1.0 / (1.0 - hp["beta1"] ** hp["step"]), 1.0 / (1.0 - hp["beta2"] ** hp["step"])
    for q, g, m, v in zip(s["q"], s["dq"], s["m"], s["v"]):
        g = g * clip
        m.mul_(hp["beta1"]).add_(g * (1.0 - hp["beta1"]))
        v.mul_(hp["beta2"]).add_(g * g * (1.0 - hp["beta2"]))
        q.sub_(((m * c1) / (torch.sqrt(v * c2) + hp["eps"]) + q * hp["weight_decay"]) * hp["lr"])
    return {"norm": norm, **s["flat"]}


_PLAIN = {"ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd, "ffn_mem": _plain_ffn_bwd,
          "glu_fwd": _plain_glu_fwd, "glu_bwd": _plain_glu_bwd, "rope_fwd": _plain_rope_fwd,
          "rope_bwd": _plain_rope_bwd, "update": _plain_update, "grad_norm": _plain_grad_norm}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import orthogonal_reparameterized_gb300.poetx as P
    op = s["op"]
    act = {"silu": P.SILU, "gelu": P.GELU}.get(s.get("act"))
    if op == "ffn_fwd":
        x, F = s["x"], s["F"]
        out = {"h": torch.empty(x.shape[0], F, dtype=x.dtype, device=x.device)}
        if s["keep"]:
            out["z"] = torch.empty(x.shape[0], 2 * F, dtype=x.dtype, device=x.device)
        P.poetx_ffn_fwd(x, s["W"], out["h"], z=out.get("z"), act=act)
        return out
    if op in ("ffn_bwd", "ffn_mem"):
        out = {"dx": torch.empty_like(s["x"]), "dW": torch.empty_like(s["W"])}
        P.poetx_ffn_bwd(s["x"], s["W"], s["dh"], z=s["z"], dx=out["dx"], dW=out["dW"], act=act)
        return out
    if op == "glu_fwd":
        h = torch.empty_like(s["g"])
        P.poetx_glu_fwd(s["g"], s["u"], h, act=act)
        return {"h": h}
    if op == "glu_bwd":
        out = {"dg": torch.empty_like(s["g"]), "du": torch.empty_like(s["u"])}
        P.poetx_glu_bwd(s["g"], s["u"], s["dh"], out["dg"], out["du"], act=act)
        return out
    if op.startswith("rope"):
        kw = dict(rot_dim=s["rot"], axis=s["axis"], interleaved=s["interleaved"], norm=s["norm"],
                  gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], eps=s["eps"])
        new = dict(dtype=s["q"].dtype, device=s["q"].device)
        q, k = torch.empty(s["q"].shape, **new), torch.empty(s["k"].shape, **new)
        if op == "rope_fwd":
            P.poetx_qk_rope_fwd(s["q"], s["k"], s["pos"], s["inv_freq"], q, k, **kw)
            return {"q": q, "k": k}
        out = {"dq": q, "dk": k}
        if s["norm"]:
            out["dgamma_q"], out["dgamma_k"] = (torch.empty_like(s[n]) for n in ("gamma_q", "gamma_k"))
        P.poetx_qk_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["pos"], s["inv_freq"], q, k,
                            dgamma_q=out.get("dgamma_q"), dgamma_k=out.get("dgamma_k"), **kw)
        return out
    norm = torch.empty(1, dtype=torch.float32, device="cuda")
    if op == "grad_norm":
        P.poetx_grad_norm(s["grads"], norm)
        return {"norm": norm}
    P.poetx_grad_norm(s["dq"], norm)
    P.poetx_adam_group(s["q"], s["dq"], s["m"], s["v"], norm=norm, max_norm=s["max_norm"], **s["hp"])
    return {"norm": norm, **s["flat"]}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    op = case["op"]
    if op in ("update", "grad_norm"):
        n = sum(a * b for a, b in _triangle_shapes(case))
        if op == "grad_norm":  # every gradient read once
            return {"bytes": 4 * n + 2 * case["V"] * case["width"] + 4 * case["width"],
                    "flops": 2 * n + 2 * case["V"] * case["width"]}
        # the gradient, q, m and v in; q, m and v out.  (The norm needs every gradient before the
        # first update, a second reading of 4 n bytes, which is not counted.)
        return {"bytes": 28 * n, "flops": 18 * n}
    esz = 2 if case["dtype"] == BF16 else 4
    N = case["N"]
    if op.startswith("rope"):
        n = N * (case["Hq"] + case["Hk"]) * case["dh"]
        # q and k in and out; backward without the norm: the upstream gradients in and out, with it
        # q and k as well
        t = 3 if op == "rope_bwd" and case["norm"] else 2
        return {"bytes": t * n * esz + 4 * N * case["axes"], "flops": (12 if t == 3 else 8) * n}
    F = case["F"]
    if op.startswith("glu"):
        return {"bytes": (3 if op == "glu_fwd" else 5) * N * F * esz,
                "flops": (6 if op == "glu_fwd" else 14) * N * F}
    D = case["D"]
    if op == "ffn_fwd":  # x, W in; h and where kept z out
        return {"bytes": esz * (N * D + 2 * F * D + (3 if case["keep"] else 1) * N * F),
                "flops": 4 * N * D * F}
    # x, W, dh and where kept z in; dx and dW out; two products, and the projections' again
    return {"bytes": esz * (2 * N * D + 4 * F * D + (3 if op == "ffn_bwd" else 1) * N * F),
            "flops": (8 if op == "ffn_bwd" else 12) * N * D * F}


# ---------------------------------------------------------------- the definitions in 64 bits
def _act64(t, act):
    if act == "silu":
        return t * torch.special.expit(t)
    return 0.5 * t * (1.0 + torch.tanh(_GELU_C * (t + _GELU_A * t ** 3)))


def _exact_glu_grads(g, u, dh, act):
    """By automatic differentiation of the definition."""
    with torch.enable_grad():
        g, u = g.requires_grad_(True), u.requires_grad_(True)
        return torch.autograd.grad(_act64(g, act) * u, (g, u), dh)


def _exact_block(s):
    op, F = s["op"], s["F"]
    if op.startswith("glu"):
        g, u = s["g"].double(), s["u"].double()
        if op == "glu_fwd":
            return {"h": _act64(g, s["act"]) * u}
        dg, du = _exact_glu_grads(g, u, s["dh"].double(), s["act"])
        return {"dg": dg, "du": du}
    x, W = s["x"].double(), s["W"].double()
    z = torch.einsum("nd,fd->nf", x, W) if s["z"] is None else s["z"].double()
    if op == "ffn_fwd":
        out = {"h": _act64(z[:, :F], s["act"]) * z[:, F:]}
        if s["keep"]:
            out["z"] = z
        return out
    dz = torch.cat(_exact_glu_grads(z[:, :F].clone(), z[:, F:].clone(), s["dh"].double(),
                                    s["act"]), dim=1)
    return {"dx": torch.einsum("nf,fd->nd", dz, W), "dW": torch.einsum("nf,nd->fd", dz, x)}


def _exact_rope(s):
    half, r = s["rot"] // 2, s["rot"]
    first = torch.arange(half, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else half)
    axis = s["axis"].long() if s["axis"] is not None else torch.zeros_like(first)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"][axis].t().double() * s["inv_freq"].double())[:, None, :]

    def forward(t, gamma):
        x = t
        if s["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * gamma
        c = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = c.real, c.imag
        return y

    out = {}
    for n in ("q", "k"):
        t = s[n].double()
        gamma = None if s["gamma_" + n] is None else s["gamma_" + n].double()
        if s["op"] == "rope_fwd":
            out[n] = forward(t, gamma)
            continue
        with torch.enable_grad():
            t.requires_grad_(True)
            leaves = (t,) if gamma is None else (t, gamma.requires_grad_(True))
            grads = torch.autograd.grad(forward(t, gamma), leaves, s["d" + n].double())
        out["d" + n] = grads[0]
        if gamma is not None:
            out["dgamma_" + n] = grads[1]
    return out


def _exact_many(s):
    grads = s["grads"] if s["op"] == "grad_norm" else [s["dq_flat"].clone()]
    if s["op"] == "update":  # the gaps between the tensors are none of theirs
        used = torch.zeros_like(s["dq_flat"], dtype=torch.bool)
        for t in _views(used, [tuple(t.shape) for t in s["dq"]]):
            t.fill_(True)
        grads[0][~used] = 0.0
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in grads))
    out = {"norm": torch.tensor([norm], dtype=torch.float64)}
    if s["op"] == "grad_norm":
        return out
    hp = s["hp"]
    b1, b2 = hp["beta1"], hp["beta2"]
    g = grads[0].double() * min(1.0, s["max_norm"] / (norm + 1e-6))
    m = b1 * s["flat"]["m"].double() + (1 - b1) * g
    v = b2 * s["flat"]["v"].double() + (1 - b2) * g * g
    del g
    q = s["flat"]["q"].double()
    step = m / (1 - b1 ** hp["step"]) / ((v / (1 - b2 ** hp["step"])).sqrt() + hp["eps"])
    q = q - hp["lr"] * (step + hp["weight_decay"] * q)
    out.update({k: torch.where(used, t, s["flat"][k].double())
                for k, t in (("q", q), ("m", m), ("v", v))})
    return out


def exact(case, seed):
    if work(case)["flops"] > 8e12:  # 64-bit products run at about a teraflop per second
        return None
    s = prepare(case, seed)
    if case["op"] in ("update", "grad_norm"):
        return _exact_many(s)
    if case["op"].startswith("rope"):
        return _exact_rope(s)
    return _exact_block(s)
