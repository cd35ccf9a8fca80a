"""A transformer block's training step whose seven linears are POET-X layers: layer norm, queries and keys
normalised per head and rotated, causal attention (plain torch), the gated product between the gate, up and
down layers, a linear head with softmax cross entropy; then the global norm of all gradients, and updates
clipped by it.

    python examples/train_block.py [--steps 20] [--tokens 256] [--width 256] [--inner 512] [--vocab 1009]

The data is a fixed random map from token to next token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import orthogonal_reparameterized_gb300.poetx as P  # noqa: E402

DEV = "cuda"
B = 64          # block size of the factors
HEAD_DIM = 64


def _f32(*shape):
    return torch.empty(*shape, device=DEV)


class Norm:
    def __init__(self, N, D):
        self.gamma, self.dgamma = torch.ones(D, device=DEV), _f32(D)
        self.mean, self.rstd = _f32(N), _f32(N)

    def forward(self, x):
        self.x, y = x, torch.empty_like(x)
        P.poetx_layernorm_fwd(x, y, gamma=self.gamma, mean=self.mean, rstd=self.rstd)
        return y

    def backward(self, dy):
        dx = torch.empty_like(dy)
        P.poetx_layernorm_bwd(self.x, dy, self.mean, self.rstd, dx, gamma=self.gamma,
                              dgamma=self.dgamma)
        return dx


class Linears:
    """The block's seven POET-X layers as one group: q, k, v, o, gate, up, down."""

    def __init__(self, N, D, F, dtype, g):
        self.N, self.dtype = N, dtype
        code = P.BF16 if dtype == torch.bfloat16 else P.F32
        shapes = [(D, D)] * 4 + [(D, F)] * 2 + [(F, D)]
        self.q, self.keep, layers = [], [], []
        for m, n in shapes:
            W0 = (torch.randn(n, m, generator=g, device=DEV) / m ** 0.5).to(dtype)
            pm, pn = (torch.randperm(k, generator=g, device=DEV).int() for k in (m, n))
            Wp = torch.empty_like(W0)
            P.poetx_merge_perm(W0, pn, pm, Wp)
            q = [torch.zeros(k // B, B * (B - 1) // 2, device=DEV) for k in (m, n)]
            self.q += q
            self.keep += [Wp, pm, pn]
            layers.append(P.make_layer(m, n, B, code, code, P.FAST, pm, pn, Wp, *q))
        self.dq, self.m, self.v = ([torch.zeros_like(t) for t in self.q] for _ in range(3))
        self.G = P.make_group(layers)
        self.saved = P.workspace(P.poetx_group_saved_bytes(self.G, N), DEV)
        self.ws = P.workspace(P.poetx_group_workspace_bytes(self.G, N), DEV)
        self.x, self.shapes = [None] * 7, shapes

    def start(self):
        P.poetx_group_cnp_fwd(self.G, self.N, self.saved)

    def forward(self, i, x):
        self.x[i], y = x, torch.empty(self.N, self.shapes[i][1], dtype=self.dtype, device=DEV)
        P.poetx_group_layer_fwd(self.G, i, x, y, self.saved, self.ws)
        return y

    def backward(self, i, dy):
        dx = torch.empty(self.N, self.shapes[i][0], dtype=self.dtype, device=DEV)
        P.poetx_group_layer_bwd(self.G, i, self.x[i], dy, self.saved, dx, self.ws)
        return dx

    def finish(self):
        P.poetx_group_cnp_bwd(self.G, self.N, self.saved, self.dq[0::2], self.dq[1::2], self.ws)


def _attention(q, k, v):
    """Causal attention of [N, H, dh] tensors."""
    s = torch.einsum("ihd,jhd->hij", q.float(), k.float()) / q.shape[2] ** 0.5
    s = s.masked_fill(torch.ones(s.shape[1:], dtype=torch.bool, device=DEV).triu(1), float("-inf"))
    return torch.einsum("hij,jhd->ihd", s.softmax(-1), v.float()).to(v.dtype).contiguous()


class Model:
    def __init__(self, tokens, width, inner, vocab, seed, dtype=torch.bfloat16):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.N, self.D, self.F, self.heads = tokens, width, inner, width // HEAD_DIM
        self.table = torch.randn(vocab, width, generator=g, device=DEV)  # embeddings, not trained here
        self.norm1, self.norm2 = Norm(tokens, width), Norm(tokens, width)
        self.linears = Linears(tokens, width, inner, dtype, g)
        self.gq, self.gk = torch.ones(HEAD_DIM, device=DEV), torch.ones(HEAD_DIM, device=DEV)
        self.dgq, self.dgk = _f32(HEAD_DIM), _f32(HEAD_DIM)
        half = HEAD_DIM // 2
        self.pos = torch.arange(tokens, device=DEV, dtype=torch.int32)
        self.freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float32) / half)
        self.W = (torch.randn(vocab, width, generator=g, device=DEV) / width ** 0.5).to(dtype)
        self.dW, self.loss = torch.empty_like(self.W), _f32(tokens)
        self.dloss = torch.full((tokens,), 1.0 / tokens, device=DEV)  # the mean over the tokens
        self.token = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
        self.target = torch.randint(0, vocab, (vocab,), generator=g, device=DEV)[self.token].int()

    def step(self):
        """Mean loss, with every gradient in its place."""
        N, D, lin = self.N, self.D, self.linears
        split = (N, self.heads, HEAD_DIM)
        lin.start()
        x0 = self.table[self.token].to(self.W.dtype)
        h = self.norm1.forward(x0)
        q, k, v = (lin.forward(i, h).view(split) for i in range(3))
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        rope = dict(gamma_q=self.gq, gamma_k=self.gk)
        P.poetx_qk_rope_fwd(q, k, self.pos, self.freq, qr, kr, **rope)
        for t in (qr, kr, v):
            t.requires_grad_(True)
        a = _attention(qr, kr, v)
        x1 = x0 + lin.forward(3, a.detach().view(N, D))
        h2 = self.norm2.forward(x1)
        gate, up = lin.forward(4, h2), lin.forward(5, h2)
        f = torch.empty_like(gate)
        P.poetx_glu_fwd(gate, up, f)
        x2 = x1 + lin.forward(6, f)
        dx2 = torch.empty_like(x2)
        P.poetx_head_ce(x2, self.W, self.target, self.loss, dloss=self.dloss, dx=dx2, dW=self.dW)

        df = lin.backward(6, dx2)
        P.poetx_glu_bwd(gate, up, df, gate, up)  # over gate and up, which nothing needs any more
        dx1 = dx2 + self.norm2.backward(lin.backward(4, gate) + lin.backward(5, up))
        da = lin.backward(3, dx1).view(split)
        dqr, dkr, dv = torch.autograd.grad(a, (qr, kr, v), da)
        dqr, dkr = dqr.contiguous(), dkr.contiguous()
        P.poetx_qk_rope_bwd(q, k, dqr, dkr, self.pos, self.freq, dqr, dkr, dgamma_q=self.dgq,
                            dgamma_k=self.dgk, **rope)
        dh = sum(lin.backward(i, t.contiguous().view(N, D)) for i, t in enumerate((dqr, dkr, dv)))
        self.norm1.backward(dh)
        lin.finish()
        return self.loss.mean()

    def others(self):
        """What a plain gradient step updates, and its gradients."""
        return ([self.W, self.norm1.gamma, self.norm2.gamma, self.gq, self.gk],
                [self.dW, self.norm1.dgamma, self.norm2.dgamma, self.dgq, self.dgk])

    def update(self, step, norm, max_norm):
        lin, (params, grads) = self.linears, self.others()
        P.poetx_grad_norm(lin.dq + grads, norm)
        P.poetx_adam_group(lin.q, lin.dq, lin.m, lin.v, step, lr=2e-3, norm=norm, max_norm=max_norm)
        P.poetx_grad_clip(grads, norm, max_norm)
        for p, g in zip(params, grads):
            p -= (1.0 * g.float()).to(p.dtype)


def train(steps=20, tokens=256, width=256, inner=512, vocab=1009, max_norm=1.0, seed=0):
    """(mean losses, gradient norms) per step."""
    model = Model(tokens, width, inner, vocab, seed)
    norm, losses, norms = _f32(1), [], []
    for step in range(1, steps + 1):
        losses.append(model.step())
        model.update(step, norm, max_norm)
        norms.append(norm.clone())
    if P.poetx_get_device_error() != 0:
        raise RuntimeError("device error word set")
    return [float(v) for v in losses], [float(v) for v in norms]


def check(tokens=256, width=256, inner=512, vocab=1009, seed=0, far=0.02):
    """(slope of the loss along a direction of the triangles by the gradients, by a difference), in fp32
    (in bf16 a small step is lost in the rounding of the activations)."""
    model = Model(tokens, width, inner, vocab, seed, torch.float32)
    lin = model.linears
    model.step()
    # along the gradient itself, so that the difference stands out of the loss's rounding
    size = torch.stack([(g * g).sum() for g in lin.dq]).sum().sqrt()
    way = [g / size for g in lin.dq]
    slope = float(sum((g * w).sum() for g, w in zip(lin.dq, way)))
    ends = []
    for sign in (1.0, -1.0):
        for q, w in zip(lin.q, way):
            q.add_(w, alpha=sign * far)
        ends.append(float(model.step()))
        for q, w in zip(lin.q, way):
            q.sub_(w, alpha=sign * far)
    return slope, (ends[0] - ends[1]) / (2 * far)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=1009)
    a = ap.parse_args()
    losses, norms = train(a.steps, a.tokens, a.width, a.inner, a.vocab)
    print(f"loss: first {losses[0]:.4f}, last {losses[-1]:.4f} ({len(losses)} steps); "
          f"gradient norm {norms[0]:.3g} to {norms[-1]:.3g}")


if __name__ == "__main__":
    main()
