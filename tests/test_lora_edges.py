"""Low-rank adapters at the borders of their tiles and blocks, on the GPU."""
import pytest
import torch

from test_lora import BF16, F32, problem, run

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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n_in,n_out,rank", [(256, 320, 1), (256, 320, 16), (100, 200, 24), (33, 31, 60), (1000, 36, 64), (64, 136, 128)])
def test_more_rows_than_small_tiles_take_at_once(cuda_lib, dtype, n_in, n_out, rank):
    """Tiles have 16 rows up to two of them an SM (4,864 rows at 152 SMs) and 64 above: both in one ragged batch's sizes."""
    for lens in ([5, 0, 4000, 64, 1, 900, 300], [17, 64, 65, 130]):
        run(cuda_lib, problem(lens, n_in, n_out, rank, dtype=dtype, idx=([2, 1, 0, 2, 3, 1, 0])[:len(lens)], seed=rank))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [17, 64, 100])
def test_more_equal_requests_than_small_tiles_take_at_once(cuda_lib, dtype, rows):
    run(cuda_lib, problem([rows] * 320, 136, 72, 16, dtype=dtype, packed=False, seed=rows))
