"""The fp32 forward's workspace: room for the pieces of W only where the call splits W."""
import pytest
import torch

DEV = "cuda:0"


@pytest.fixture(scope="module")
def P():
    from orthogonal_reparameterized_gb300 import build
    build.build()
    import orthogonal_reparameterized_gb300.poetx as P
    P.lib()
    return P


def _pieces(count):
    return 3 * (-(-2 * count // 1024) * 1024)


# blocks that the CUDA cores take, and others; W's pieces of up to a megabyte are asked for beyond 32 rows
FEW = [(1, 4096, 14336), (32, 4096, 14336), (33, 1024, 2816), (64, 1024, 2816), (128, 256, 512), (32, 64, 64)]
MANY = [(33, 4096, 14336), (128, 1024, 2816), (2000, 256, 512), (97, 1600, 8), (512, 64, 64), (97, 1400, 8)]


@pytest.mark.parametrize("N,D,F", FEW)
def test_sizes_without_the_pieces_of_W(P, N, D, F):
    assert P.poetx_ffn_fwd_workspace_bytes(P.F32, N, D, F) == _pieces(N * D)


@pytest.mark.parametrize("N,D,F", MANY)
def test_sizes_with_the_pieces_of_W(P, N, D, F):
    assert P.poetx_ffn_fwd_workspace_bytes(P.F32, N, D, F) == _pieces(N * D) + _pieces(2 * F * D)


@pytest.mark.parametrize("D,F", [(1024, 2816), (256, 512), (8, 8), (1416, 64), (1424, 64), (4096, 8)])
def test_room_for_more_rows_is_room_for_fewer(P, D, F):
    sizes = [P.poetx_ffn_fwd_workspace_bytes(P.F32, N, D, F) for N in range(0, 3000, 7)]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("N,D,F", [(33, 1024, 2816), (64, 1024, 2816), (512, 64, 64), (128, 1024, 2816)])
def test_a_call_with_just_that_much(P, N, D, F):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(N, D, generator=g, device=DEV)
    W = torch.randn(2 * F, D, generator=g, device=DEV) * D ** -0.5
    n = P.poetx_ffn_fwd_workspace_bytes(P.F32, N, D, F)
    ws = torch.full((n + 1024,), 0x5a, dtype=torch.uint8, device=DEV)
    h, h2 = torch.empty(N, F, device=DEV), torch.empty(N, F, device=DEV)
    P.poetx_ffn_fwd(x, W, h, ws=ws[:n])
    P.poetx_ffn_fwd(x, W, h2)
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and (ws[n:] == 0x5a).all()
    z = x.double() @ W.double().t()
    ref = torch.nn.functional.silu(z[:, :F]) * z[:, F:]
    # as the product behind another has it: twice the fp32 products' 1e-5
    assert (h - ref).norm() <= 2e-5 * ref.norm()
    with pytest.raises(P.PoetxError):
        P.poetx_ffn_fwd(x, W, h, ws=ws[:n - 16])
