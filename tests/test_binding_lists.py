"""Lists in which a written tensor occurs twice: refused before the library is called (two thread blocks would
read and write it at the same time).  No GPU: CPU tensors before a stand-in of the library."""
import pytest
import torch

import orthogonal_reparameterized_gb300.poetx as P


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(P, "lib", lambda: Library())
    monkeypatch.setattr(P, "_addr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(P, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(P, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(P, "_scratch", lambda n, t, stream, handle: torch.empty(16, dtype=torch.uint8))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)  # the CPU's number
    return made


def _lists(n=4):
    return {k: [torch.ones(5 + i) for i in range(n)] for k in ("q", "dq", "m", "v")}


NORM = torch.ones(1)


def test_clip(calls):
    g = _lists()["q"]
    P.poetx_grad_clip(g, NORM, 1.0)
    assert calls == ["poetx_grad_clip"]
    for twice in (g + [g[1]], [g[0], g[0].view(5)]):
        with pytest.raises(ValueError, match="twice"):
            P.poetx_grad_clip(twice, NORM, 1.0)
    assert len(calls) == 1


def test_norm_may_name_one_twice(calls):
    """It only reads."""
    g = _lists()["q"]
    P.poetx_grad_norm(g + g, NORM)
    assert "poetx_grad_norm" in calls


@pytest.mark.parametrize("which", ["q", "m", "v"])
def test_step(calls, which):
    s = _lists()
    P.poetx_adam_group(*s.values(), step=1, lr=1e-3)
    assert calls == ["poetx_adam_group"]
    s = {k: [torch.ones(5) for _ in range(4)] for k in s}
    s[which][3] = s[which][0]
    with pytest.raises(ValueError, match=f"among {which} twice"):
        P.poetx_adam_group(*s.values(), step=1, lr=1e-3)
    assert len(calls) == 1


def test_step_may_read_a_gradient_twice(calls):
    s = {k: [torch.ones(5) for _ in range(2)] for k in ("q", "dq", "m", "v")}
    s["dq"][1] = s["dq"][0]
    P.poetx_adam_group(*s.values(), step=1, lr=1e-3)
    assert calls == ["poetx_adam_group"]


def test_empty_tensors_are_not_the_same(calls):
    e = [torch.empty(0) for _ in range(3)] + [torch.ones(3)]
    P.poetx_grad_clip(e, NORM, 1.0)
    P.poetx_grad_clip([], NORM, 1.0)
    P.poetx_adam_group(e, e, e, e, step=1, lr=1e-3)
    assert len(calls) == 3
