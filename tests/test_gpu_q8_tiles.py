"""The tiles of the 8-bit product against exact products on the GPU, whole outputs, bit for bit."""
import pytest
import torch

import expert_cache_host_amd as m
from expert_cache_host_amd import step
from q8_tile_cases import CASES

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tokens(x):
    """Codes and scales from the definition: the quotient of two float32 numbers that is no half lies further from one
    than binary64 rounds."""
    s = (x.double().abs().amax(1) / 127).float()
    return torch.round(x.double() / s.double()[:, None]), s


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


@pytest.mark.parametrize("i", range(len(CASES)))
def test_every_tile(i):
    _, T, rows, cols = CASES[i]
    g = gen(i)
    w = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda").to(torch.int8)
    ws = 1e-3 * (1 + torch.rand(rows, generator=g, device="cuda"))
    matrix = m.Q8Matrix(w, ws)
    # all types at the most steps of a tile, else in turn
    types = [torch.float32, torch.bfloat16, torch.float16]
    for dt in types if cols > 500 else types[i % 3:i % 3 + 1]:
        x = torch.randn(T, cols, generator=g, device="cuda").to(dt)
        codes, scales = tokens(x)
        want = product(codes, scales, w, ws, dt)
        q = m.q8_rows(x)
        assert torch.equal(q.codes[:, :cols].double(), codes) and torch.equal(q.scales, scales)
        # x of a wider buffer, the output between other columns
        wide = torch.full((T, cols + 8), float("nan"), device="cuda", dtype=dt)
        wide[:, 4:cols + 4] = x
        out = torch.full((T + 2, rows + 16), 77.0, device="cuda", dtype=dt)
        for _ in range(2):
            m.q8_matmul(wide[:, 4:cols + 4], matrix, out=out[1:T + 1, 5:rows + 5])
            assert torch.equal(out[1:T + 1, 5:rows + 5], want)
            assert (out[0] == 77).all() and (out[-1] == 77).all()
            assert (out[:, :5] == 77).all() and (out[:, rows + 5:] == 77).all()
            out[1:T + 1, 5:rows + 5] = 77
        assert torch.equal(m.q8_matmul(q, matrix, dtype=dt), want)


@pytest.mark.parametrize("T,cols,rows", [(512, 6144, 10240), (1024, 6144, 16384)])
def test_whole_tiles_of_a_prompt(T, cols, rows):
    """Sizes of many whole tiles and steps, in bfloat16, whose few digits make quotients that are halves: the scale has
    to be the quotient's rounding (a product with 1 / 127 is a step off in some rows, and such codes then differ)."""
    g = gen(T)
    x = (torch.randn(T, cols, generator=g, device="cuda") * (0.3 + torch.rand(T, 1, generator=g, device="cuda"))).bfloat16()
    x[3::50].clamp_(-3.96875, 3.96875)[:, 0] = 3.96875  # scale 1 / 32
    w = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda").to(torch.int8)
    ws = 4e-4 * (0.5 + torch.rand(rows, generator=g, device="cuda"))
    matrix = m.Q8Matrix(w, ws)
    codes, scales = tokens(x)
    assert scales[3] == 1 / 32 and (x[3].double() * 32 % 1 == 0.5).any()
    want = product(codes, scales, w, ws, torch.bfloat16)
    outs = [m.q8_matmul(x, matrix) for _ in range(6)]
    for out in outs:
        assert torch.equal(out, want)
