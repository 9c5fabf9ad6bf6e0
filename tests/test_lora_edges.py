"""Low-rank adapters at the borders of their tiles and blocks, on the GPU."""
import pytest
import torch

from test_lora import F32, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_in,n_out,rank", [(64, 96, 32), (64, 96, 33), (100, 40, 128), (31, 33, 16)])
def test_fp32_gradients_through_every_element_of_the_transposed_tiles(cuda_lib, n_in, n_out, rank):
    """Matrices in which one element alone is not zero, in each corner of 32 x 32 tiles and beside it: the gradient of x
    is then exactly that element's share, so a tile that loses or mixes an element shows."""
    spots = sorted({(r, c) for r in (0, 31, rank - 1) for c in (0, 30, 31, 32, n_in - 1) if r < rank and c < n_in})
    p = problem([3], n_in, n_out, rank, adapters=len(spots), dtype=F32, idx=[0])
    d_out, x = torch.ones(3, n_out, device="cuda"), p["x"].cuda()
    a, b = torch.zeros(len(spots), rank, n_in), torch.zeros(len(spots), n_out, rank)
    for l, (r, c) in enumerate(spots):
        a[l, r, c] = 2.0 + l
        b[l, (r + c) % n_out, r] = 0.5
    a, b = a.cuda(), b.cuda()
    for l, (r, c) in enumerate(spots):
        dx, _, _ = cuda_lib.kda_lora_bwd(d_out, x, a, b, torch.tensor([l], device="cuda"))
        want = torch.zeros_like(dx)
        want[:, c] = 0.5 * (2.0 + l)
        assert torch.equal(dx, want), (r, c)
