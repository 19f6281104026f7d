"""Activations of the linear layers in fp32, by their relative error: the
negative tails, where the values are small but keep their digits, and large
and special values.  u = 2^-24, half a step of fp32.
"""
import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


# rows of x for a row form, and for tiles (partial and whole)
ROWS = [1, 24, 300]


def of_points(act, z, rows, out_dtype=torch.float32):
    """act at the points z (1-D), through a product whose sum is z itself."""
    w = torch.ones(80, 1, device=DEV)
    out = []
    for part in z.split(rows):
        y = ct.linear(part[:, None].contiguous(), w, act=act, out_dtype=out_dtype)
        torch.cuda.synchronize()
        nan = torch.isnan(y)
        assert torch.equal(nan, nan[:, :1].expand_as(y))
        assert torch.equal(y.masked_fill(nan, 0), y[:, :1].masked_fill(nan[:, :1], 0).expand_as(y))
        out.append(y[:, 0])
    return torch.cat(out).double()


@pytest.mark.parametrize("rows", ROWS)
def test_gelu_keeps_its_digits_in_the_negative_tail(rows):
    """z (1 + erf(z / sqrt 2)) / 2 = z q(-z) with q(a) = erfc(a / sqrt 2) / 2, which
    falls as exp(-a^2 / 2): the exponent, a constant and two products, is off by
    3 u of itself, 1.5 z^2 u of the value; what multiplies the exponential is
    fitted to 2.5 u and evaluated to 12 u (the reciprocal and 8 steps whose sum
    of magnitudes is twice the result), the exponential and the products add 6 u
    and the library's own erfc, were it used, 16 steps: 36 u hold either."""
    z = -torch.linspace(0.01, 12.0, 600, device=DEV)
    y = of_points("gelu", z, rows)
    zd = z.double()
    ref = 0.5 * zd * torch.erfc(-zd * 0.5 ** 0.5)
    tol = (1.5 * zd * zd + 36) * U * ref.abs()
    worst = float(((y - ref).abs() / tol).max())
    say(f"  gelu, {rows} rows: {worst:.3f} of the tolerance")
    assert worst <= 1.0


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows", ROWS)
def test_sigmoids_keep_their_digits_in_the_negative_tail(rows, act):
    """z / (1 + exp(-v)), v = z (silu) or sqrt(8 / pi) (z + 0.044715 z^3), taken as
    z e / (1 + e) with e = exp(v): e to 6 u beside what v itself is off by (0 for
    silu; two constants and five operations, 5 u |v|, for gelu_tanh), the
    reciprocal 2 u, two products and a sum 3 u, one for the rest.  Below exp(-87)
    the exponential's unit gives zeros: 2^-126 |z|."""
    z = -torch.linspace(0.01, 100.0 if act == "silu" else 11.0, 600, device=DEV)
    y = of_points(act, z, rows)
    zd = z.double()
    v = zd if act == "silu" else (8 / torch.pi) ** 0.5 * (zd + 0.044715 * zd ** 3)
    ref = zd * torch.exp(v) / (1 + torch.exp(v))
    tol = (12 + (0 if act == "silu" else 5 * v.abs())) * U * ref.abs() + 2.0 ** -126 * zd.abs()
    worst = float(((y - ref).abs() / tol).max())
    say(f"  {act}, {rows} rows: {worst:.3f} of the tolerance")
    assert worst <= 1.0


@pytest.mark.parametrize("rows", ROWS)
def test_activations_of_large_and_special_values(rows):
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([0.0, -0.0, 1e-30, 20.0, 100.0, 1e10, 3e38, inf, nan, -1e10, -3e38], device=DEV)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        y = of_points(act, z, rows)
        assert bool((y[:2] == 0).all()) and bool(torch.isnan(y[8])), act
        assert torch.equal(y[3:8], z[3:8].double()) or act == "silu"
        assert float(((y[3:7] - z[3:7].double()) / z[3:7].double()).abs().max()) < 1e-7 and float(y[7]) == inf, act
        assert abs(float(y[2]) / 1e-30 - (1.0 if act == "relu" else 0.5)) < 1e-6, act
        assert bool((y[9:] == 0).all()), act


