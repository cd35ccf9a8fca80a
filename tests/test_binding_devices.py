"""The binding refuses a tensor on another device than the current one, whichever argument it is (its memory
would be read or written from a kernel of the current device).  No GPU: tensors and library are stand-ins."""
import inspect

import pytest
import torch

import orthogonal_reparameterized_gb300.poetx as P

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
N, D, F, V, H, DH = 4, 64, 32, 96, 2, 64


class Tensor:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096


class Library:
    """Every function succeeds; sizes are 1024."""

    def __getattr__(self, name):
        return lambda *a: 1024 if name.endswith("_bytes") else 0


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(P, "lib", lambda: Library())
    monkeypatch.setattr(P, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(P, "_scratch", lambda n, t, stream, handle: Tensor((n,), torch.uint8))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def _t(dtype, *shape):
    return (shape, dtype)


X, W2, NF = _t(BF, N, D), _t(BF, 2 * F, D), _t(BF, N, F)
Q, ROW, GAM = _t(BF, N, H, DH), _t(F32, N), _t(F32, DH)
ROPE = dict(pos=_t(I32, N), inv_freq=_t(F32, DH // 2), axis=_t(I32, DH // 2), gamma_q=GAM, gamma_k=GAM)
WS = _t(torch.uint8, 1024)
CALLS = {
    "poetx_layernorm_fwd": dict(x=X, y=X, gamma=_t(F32, D), beta=_t(F32, D), mean=ROW, rstd=ROW),
    "poetx_layernorm_bwd": dict(x=X, dy=X, mean=ROW, rstd=ROW, dx=X, gamma=_t(F32, D), dgamma=_t(F32, D),
                                dbeta=_t(F32, D), ws=WS),
    "poetx_head_ce": dict(x=X, W=_t(BF, V, D), target=_t(I32, N), loss=ROW, dloss=ROW, dx=X, dW=_t(BF, V, D),
                          lse=ROW, ws=WS),
    "poetx_head_distill": dict(x=X, W=_t(BF, V, D), t_index=_t(I32, N, 8), t_logit=_t(F32, N, 8), loss=ROW,
                               dloss=ROW, dx=X, dW=_t(BF, V, D), lse=ROW, ws=WS),
    "poetx_glu_fwd": dict(g=NF, u=NF, h=NF),
    "poetx_glu_bwd": dict(g=NF, u=NF, dh=NF, dg=NF, du=NF),
    "poetx_ffn_fwd": dict(x=X, W=W2, h=NF, z=_t(BF, N, 2 * F), ws=WS),
    "poetx_ffn_bwd": dict(x=X, W=W2, dh=NF, z=_t(BF, N, 2 * F), dx=X, dW=W2, ws=WS),
    "poetx_qk_rope_fwd": dict(q=Q, k=Q, q_out=Q, k_out=Q, **ROPE),
    "poetx_qk_rope_bwd": dict(q=Q, k=Q, dq=Q, dk=Q, dq_in=Q, dk_in=Q, dgamma_q=GAM, dgamma_k=GAM, ws=WS, **ROPE),
}


def _call(name, devices):
    P.__dict__[name](**{k: Tensor(*v, devices.get(k, 0)) for k, v in CALLS[name].items()})


@pytest.mark.parametrize("name", CALLS)
def test_every_argument_is_on_the_current_device(name):
    _call(name, {})  # as it should be
    for k in CALLS[name]:
        with pytest.raises(ValueError, match="current device"):
            _call(name, {k: 1})
        with pytest.raises(ValueError, match="CUDA device"):
            _call(name, {k: -1})


def test_all_tensor_arguments_are_tried():
    other = {"stream", "ws", "act", "accumulate", "eps", "rot_dim", "interleaved", "norm", "z_loss", "temperature"}
    for name, args in CALLS.items():
        assert set(inspect.signature(P.__dict__[name]).parameters) - other <= set(args), name


def test_lists_and_norms():
    """(The lists themselves: torch's own methods, which these stand-ins do not have.)"""
    for call in (lambda n: P.poetx_grad_norm([], n), lambda n: P.poetx_grad_clip([], n, 1.0)):
        call(Tensor((1,), F32))
        with pytest.raises(ValueError, match="current device"):
            call(Tensor((1,), F32, 1))
