"""The tiles of the 8-bit product against exact products on the GPU, whole outputs, bit for bit."""
import pytest
import torch

import expert_cache_host_amd as m
from expert_cache_host_amd import step

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def product(codes, scales, w, w_scales, dtype):
    """Sums in binary64 (exact below 2^53), two float32 products, one rounding to the type."""
    return ((codes.double() @ w.double().t()).float() * scales[:, None] * w_scales).to(dtype)


@pytest.mark.parametrize("T,rows,stride", [(1, 40, 5), (1, 20000, (1 << 40) + 8), (40, 1, 3), (300, 1, -(1 << 33))])
def test_one_row_has_no_stride(T, rows, stride):
    """The stride of an operand of one row is not looked at, whatever it is."""
    g = gen(T)
    cols = 300
    x = m.q8_rows(torch.randn(T, cols, generator=g, device="cuda"))
    w = torch.randint(-128, 128, (rows, 304), generator=g, device="cuda").to(torch.int8)
    ws = 1e-3 * (1 + torch.rand(rows, generator=g, device="cuda"))
    out = torch.empty(T, rows, device="cuda")
    rc = step._library().moe_q8_matmul(
        x.codes.data_ptr(), stride if T == 1 else 384, x.scales.data_ptr(), T, w.data_ptr(), stride if rows == 1 else 304,
        ws.data_ptr(), rows, cols, out.data_ptr(), 0, rows, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(out, product(x.codes[:, :cols], x.scales, w[:, :cols], ws, torch.float32))
