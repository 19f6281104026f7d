"""Every form of the products with operands that need every bit of their type
and with NaN in 8-bit rows; a norm of more rows than one launch takes.
"""
import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV
from test_gpu_block import check_linear

pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def product64(x, w):
    return x.double() @ w.double().t().contiguous()


def whole(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device=DEV).float()


def strided(t, pad, off):
    """t's values in a matrix with `pad` more elements a row, `off` elements in."""
    M, D = t.shape
    base = torch.zeros(M * (D + pad) + off + 8, dtype=t.dtype, device=t.device)
    v = base[off:off + M * (D + pad)].view(M, D + pad)[:, :D]
    v.copy_(t)
    return v


# every tile, split sums, operands copied to whole stages, and both row forms
WIDE = [(5, 100, 129), (24, 1024, 1024), (24, 515, 130), (70, 90, 515), (8, 256, 16383), (640, 2048, 1024), (1100, 2048, 999),
        (1500, 1500, 200), (2049, 2050, 200), (2500, 2048, 131), (4097, 4090, 264), (4100, 4097, 139), (4090, 4000, 272),
        (3900, 4090, 139)]


@pytest.mark.parametrize("dtype,most", [(F32, 1 << 17), (F16, 1 << 11), (BF16, 1 << 8)], ids=str)
@pytest.mark.parametrize("mnk", WIDE, ids=lambda t: "x".join(map(str, t)))
def test_operands_with_every_bit_of_their_type(mnk, dtype, most):
    """Whole numbers below 2^17 (fp32; 2^11 fp16, 2^8 bf16) against 0, 1 and -1,
    at most 64 of them not 0 in a row: sums below 2^23 are exact in fp32.  A path
    that kept fewer bits of an operand would be off."""
    M, N, K = mnk
    g = gen(M + K)
    x = torch.randint(1 - most, most, (M, K), generator=g, device=DEV).float()
    at = torch.randint(0, K, (N, 64), generator=g, device=DEV)
    w = torch.zeros(N, K, device=DEV)
    w.scatter_(1, at, torch.where(at % 2 == 0, 1.0, -1.0))
    assert torch.equal(x.to(dtype).float(), x)
    for a, b in ((x, w), (w, x)):
        ref = product64(a, b)
        for pad, off in ((0, 0), (3, 1)):
            y = ct.linear(strided(a.to(dtype), pad, off), strided(b.to(dtype), pad, off), out_dtype=F32)
            torch.cuda.synchronize()
            assert torch.equal(y.double(), ref), (mnk, pad)


# tiles of 256 x 256: their whole and their partial ones, operands on 16 bytes,
# off them, and copied
LARGEST = [(4090, 4000, 272), (3900, 4090, 139)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16, E4M3], ids=str)
@pytest.mark.parametrize("mnk", LARGEST, ids=lambda t: "x".join(map(str, t)))
def test_largest_tiles_are_exact(mnk, dtype):
    """Whole numbers with bias, gate and residual: one rounding at the end."""
    M, N, K = mnk
    g = gen(M + K)
    x, w, bias, gate, res = whole(g, M, K), whole(g, N, K), whole(g, N), whole(g, M, N), whole(g, M, N)
    ref = (product64(x, w) + bias.double()) * gate.double() + res.double()
    one = torch.ones(max(M, N), device=DEV)
    for pad, off in ((0, 0), (16, 16), (3, 1)):
        xd, wd = strided(x.to(dtype), pad, off), strided(w.to(dtype), pad, off)
        for out_dtype in (F32, F16, BF16):
            gd, rd = strided(gate.to(out_dtype), pad, off), strided(res.to(out_dtype), pad, off)
            if dtype == E4M3:
                y = ct.linear_q8(xd, one[:M], wd, one[:N], bias, gate=gd, residual=rd, out_dtype=out_dtype)
            else:
                y = ct.linear(xd, wd, bias, gate=gd, residual=rd, out_dtype=out_dtype)
            torch.cuda.synchronize()
            assert torch.equal(y, ref.to(out_dtype)), (mnk, dtype, pad, out_dtype)


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (F16, F16), (BF16, BF16), (E4M3, BF16), (E4M3, F16), (E4M3, F32)], ids=str)
def test_largest_tiles_with_everything(dtype, out_dtype):
    for act in ("gelu", "gelu_tanh", "silu"):
        check_linear(4090, 4000, 272, dtype, out_dtype, act, True, True, True, 6)


@pytest.mark.parametrize("out_dtype", [F16, BF16, F32], ids=str)
@pytest.mark.parametrize("M,N", [(3, 80), (70, 80), (300, 1000), (2100, 2050), (4200, 4100), (4090, 4000)])
def test_nan_in_8_bit_rows_reaches_its_row_and_column_alone(M, N, out_dtype):
    K = 192
    g = gen(13 + M)
    x = torch.randint(-2, 3, (M, K), generator=g, device=DEV).float()
    w = torch.randint(-2, 3, (N, K), generator=g, device=DEV).float()
    ref = product64(x, w)
    x[M // 2, 7], w[N // 3, 100] = float("nan"), float("nan")
    one = torch.ones(max(M, N), device=DEV)
    y = ct.linear_q8(x.to(E4M3), one[:M], w.to(E4M3), one[:N], out_dtype=out_dtype)
    torch.cuda.synchronize()
    hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    hit[M // 2], hit[:, N // 3] = True, True
    assert torch.equal(torch.isnan(y), hit)
    want = ref.to(out_dtype)  # whole numbers: one rounding
    assert torch.equal(y[~hit], want[~hit])


def test_rows_past_one_launch_with_a_residual():
    """2^21 rows are one launch: those behind take their own x, residual, h and y."""
    g = gen(62)
    M, D = 2_100_001, 96
    few, fres, gain = normal(g, 64, D).to(BF16), normal(g, 64, D).to(BF16), 1 + 0.1 * normal(g, D)
    many = lambda t: t.repeat(M // 64 + 1, 1)[:M]  # noqa: E731
    x, res = many(few), many(fres)
    for out_dtype in (BF16, E4M3):
        y, s, h = ct.rmsnorm(x, gain, res, out_dtype=out_dtype)
        y1, s1, h1 = ct.rmsnorm(few, gain, fres, out_dtype=out_dtype)
        torch.cuda.synchronize()
        bits = torch.uint8 if out_dtype == E4M3 else torch.int16
        assert torch.equal(h.view(torch.int16), many(h1.view(torch.int16)))
        assert torch.equal(y.view(bits), many(y1.view(bits)))
        assert s is None or torch.equal(s, s1.repeat(M // 64 + 1)[:M])
