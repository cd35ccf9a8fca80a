"""A small language model's training step with the library's calls alone: layer norm -> POET-X
linear (with a residual) -> layer norm -> linear head with softmax cross entropy, and the way back;
then the same head learning from a teacher's top logits.

    python examples/train_head.py [--steps 30] [--tokens 512] [--width 512] [--vocab 4001]

The POET-X factors are updated by the library's Adam inside the layer's backward, the head and the
norms' parameters by plain gradient steps.  The data is a fixed random map from token to next token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import orthogonal_reparameterized_gb300.poetx as P  # noqa: E402

DEV = "cuda"


class Norm:
    """Layer norm with its parameters, its saved statistics and its gradients."""

    def __init__(self, N, D):
        f32 = dict(device=DEV, dtype=torch.float32)
        self.gamma, self.beta = torch.ones(D, **f32), torch.zeros(D, **f32)
        self.dgamma, self.dbeta = torch.empty(D, **f32), torch.empty(D, **f32)
        self.mean, self.rstd = torch.empty(N, **f32), torch.empty(N, **f32)

    def forward(self, x):
        self.x, y = x, torch.empty_like(x)
        P.poetx_layernorm_fwd(x, y, gamma=self.gamma, beta=self.beta, mean=self.mean,
                              rstd=self.rstd)
        return y

    def backward(self, dy):
        dx = torch.empty_like(dy)
        P.poetx_layernorm_bwd(self.x, dy, self.mean, self.rstd, dx, gamma=self.gamma,
                              dgamma=self.dgamma, dbeta=self.dbeta)
        return dx

    def step(self, lr):
        self.gamma -= lr * self.dgamma
        self.beta -= lr * self.dbeta


class PoetxLinear:
    """A square POET-X layer: frozen permuted weight, learned block-diagonal orthogonal factors."""

    def __init__(self, N, D, b, g):
        bf16 = dict(device=DEV, dtype=torch.bfloat16)
        W0 = (torch.randn(D, D, generator=g, device=DEV) / D ** 0.5).bfloat16()
        self.pm, self.pn = (torch.randperm(D, generator=g, device=DEV).int() for _ in range(2))
        self.Wp = torch.empty_like(W0)
        P.poetx_merge_perm(W0, self.pn, self.pm, self.Wp)
        shape = (D // b, b * (b - 1) // 2)
        self.q = [torch.zeros(shape, device=DEV) for _ in range(2)]
        self.dq, self.m, self.v = ([torch.zeros(shape, device=DEV) for _ in range(2)]
                                   for _ in range(3))
        self.layer = P.make_layer(D, D, b, P.BF16, P.BF16, P.FAST, self.pm, self.pn, self.Wp,
                                  self.q[0], self.q[1])
        self.saved = P.workspace(P.poetx_layer_saved_bytes(self.layer, N), DEV)
        self.ws = P.workspace(max(P.poetx_layer_workspace_bytes(self.layer, N, k) for k in (0, 1)),
                              DEV)
        self.y, self.dx = torch.empty(N, D, **bf16), torch.empty(N, D, **bf16)

    def forward(self, x):
        self.x = x
        P.poetx_layer_fwd(self.layer, x, self.y, self.saved, self.ws)
        return self.y

    def backward_step(self, dy, step, lr):
        P.poetx_layer_bwd_adam(self.layer, self.x, dy, self.saved, self.dx, self.dq[0], self.dq[1],
                               self.ws, self.m[0], self.v[0], self.m[1], self.v[1], step, lr=lr)
        return self.dx


def train(steps=30, tokens=512, width=512, vocab=4001, top=16, seed=0):
    """Mean losses per step: (cross entropy, distillation)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    N, D, V = tokens, width, vocab
    table = torch.randn(V, D, generator=g, device=DEV)  # embeddings, not trained here
    target_of = torch.randint(0, V, (V,), generator=g, device=DEV)
    norm1, norm2, linear = Norm(N, D), Norm(N, D), PoetxLinear(N, D, 64, g)
    W = (torch.randn(V, D, generator=g, device=DEV) / D ** 0.5).bfloat16()
    loss, dW = torch.empty(N, device=DEV), torch.empty_like(W)
    dloss = torch.full((N,), 1.0 / N, device=DEV)  # the mean over the tokens

    def hidden(token):
        x0 = table[token].bfloat16()
        return norm2.forward(x0 + linear.forward(norm1.forward(x0)))

    token = torch.randint(0, V, (N,), generator=g, device=DEV)  # one batch, learned by heart
    target = target_of[token].int()
    history = []
    for step in range(1, steps + 1):
        h = hidden(token)
        dh = torch.empty_like(h)
        P.poetx_head_ce(h, W, target, loss, dloss=dloss, dx=dh, dW=dW)
        history.append(loss.mean())
        dx1 = norm2.backward(dh)  # into the residual sum: the linear's output gradient as well
        norm1.backward(linear.backward_step(dx1, step, lr=2e-3))
        W -= (4.0 * dW.float()).bfloat16()
        for n in (norm1, norm2):
            n.step(0.05)

    # the trained head as the teacher of a new one: its `top` largest logits per token
    h = hidden(token)
    t_logit, t_index = (h.float() @ W.float().t()).topk(top, dim=1)
    t_logit, t_index = t_logit.contiguous(), t_index.int().contiguous()
    S = (torch.randn(V, D, generator=g, device=DEV) / D ** 0.5).bfloat16()
    taught = []
    for _ in range(steps):
        P.poetx_head_distill(h, S, t_index, t_logit, loss, dloss=dloss, dW=dW, temperature=2.0)
        taught.append(loss.mean())
        S -= (1.0 * dW.float()).bfloat16()
    if P.poetx_get_device_error() != 0:
        raise RuntimeError("device error word set")
    return [float(v) for v in history], [float(v) for v in taught]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=4001)
    a = ap.parse_args()
    ce, kd = train(a.steps, a.tokens, a.width, a.vocab)
    for name, v in (("cross entropy", ce), ("distillation", kd)):
        print(f"{name}: first {v[0]:.4f}, last {v[-1]:.4f} ({len(v)} steps)")


if __name__ == "__main__":
    main()
