"""The matrix product of scaled 8-bit matrices in the plans that it gives
large problems, on the GPU."""
import pytest
import torch

import fp8_testutil as ref
from test_fp8_path import _operands, _product

pytestmark = pytest.mark.gpu


def _integers(shape, seed):
    """Up to 4, times a power of two for each 128 x 128 block: sums are exact
    in fp32 whatever their order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-4, 5, shape, device="cuda", generator=g).float()
    e = torch.exp2(torch.randint(-1, 2, [ref.blocks(s) for s in shape], device="cuda", generator=g).float())
    return x * e.repeat_interleave(128, 0)[:shape[0]].repeat_interleave(128, 1)[:, :shape[1]]


def _exact(form, a, b):
    return _product(form, *(torch.from_numpy(ref.values(x)).cuda() for x in (a, b)))


@pytest.mark.parametrize("left,pitch", [(5, 2063), (8, 2072)])
@pytest.mark.parametrize("m", [2201, 2901, 3501])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_pairs_write_only_their_result(cuda_lib, form, m, left, pitch):
    """Into the middle of a wider buffer, from an odd column on and from one
    that TMA stores take: nothing around the result is touched."""
    n, k = 2047, 1736
    a, b = _operands(cuda_lib, form, m, n, k, 210, _integers)
    want = _exact(form, a, b)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((m + 6, pitch), 7.0, dtype=dtype, device="cuda")
        out = buf[3:3 + m, left:left + n]
        cuda_lib.kda_fp8_matmul(a, b, form, out=out)
        assert torch.equal(out, want.to(dtype))
        out.fill_(7.0)
        assert torch.all(buf == 7.0)
