"""More refusals of the transformer-block entry points, before any HIP call:
the addresses here are never read."""
import os

import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

P = 1 << 20  # an aligned address that no call here reads


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(ct.LIB_PATH):
        from tensor_compiler_tiling_amd import build
        build.build()


LIN = dict(x=P, ldx=64, w=2 * P, ldw=64, y=3 * P, ldy=32, M=4, N=32, K=64, dtype=ct.CT_BF16, out_dtype=ct.CT_BF16, epi=None,
           workspace=None, workspace_bytes=0, stream=0)
Q8 = dict(x=P, ldx=64, xs=P, w=2 * P, ldw=64, ws=P, y=3 * P, ldy=32, M=4, N=32, K=64, out_dtype=ct.CT_BF16, epi=None,
          workspace=None, workspace_bytes=0, stream=0)
NORM = dict(x=P, ldx=64, residual=2 * P, ldr=64, gain=P, h=3 * P, ldh=64, y=4 * P, ldy=64, scale=None, M=4, D=64,
            dtype=ct.CT_BF16, out_dtype=ct.CT_BF16, eps=1e-6, stream=0)
QUANT = dict(x=P, ldx=64, q=2 * P, ldq=64, scale=P, M=4, D=64, dtype=ct.CT_BF16, stream=0)
CALLS = {"linear": (ct.ct_linear_fwd, LIN, "MNK"), "linear_q8": (ct.ct_linear_q8_fwd, Q8, "MNK"),
         "rmsnorm": (ct.ct_rmsnorm_fwd, NORM, "MD"), "quantize_rows": (ct.ct_quantize_rows, QUANT, "MD"),
         "workspace": (ct.ct_linear_workspace_bytes, dict(M=4, N=32, K=64, dtype=ct.CT_BF16), "MNK")}


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 64, (1 << 40) + 1, -(1 << 32)])
@pytest.mark.parametrize("call", list(CALLS))
def test_counts_past_32_bits_are_not_cut(call, n):
    """2^32 rows would be none, and 2^32 + 64 elements 64."""
    f, args, names = CALLS[call]
    for name in names:
        with pytest.raises(ValueError, match="32 bits"):
            f(**{**args, name: n})


@pytest.mark.parametrize("shape", [(1 << 32, 1), ((1 << 32) + 3, 1), (1, (1 << 32) + 1), (1 << 31, 1)], ids=str)
def test_helpers_refuse_counts_past_32_bits(shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device="meta")
    s = torch.empty(1, device="meta")
    for call in (lambda: ct.rmsnorm(x), lambda: ct.quantize_rows(x), lambda: ct.linear(x, x[:1]),
                 lambda: ct.linear_q8(q, s, q[:1], s)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


@pytest.mark.parametrize("over", [
    dict(y=P, out_dtype=ct.CT_E4M3, scale=P), dict(y=2 * P, out_dtype=ct.CT_E4M3, scale=P),
    dict(y=P, out_dtype=ct.CT_F32), dict(y=2 * P, out_dtype=ct.CT_F16),
    dict(y=P, ldy=72), dict(y=2 * P, ldy=128), dict(h=P, ldh=65), dict(h=2 * P, ldr=66),
    dict(y=P, ldy=72, M=2), dict(y=P, out_dtype=ct.CT_F32, M=1),
], ids=str)
def test_rmsnorm_refuses_to_write_over_rows_it_has_not_read(over):
    assert ct.ct_rmsnorm_fwd(**{**NORM, **over}) == ct.CT_ERR_INVALID_ARG
    assert "in the place of" in ct.ct_last_error()


@pytest.mark.parametrize("dtype", [ct.CT_F32, ct.CT_F16, ct.CT_BF16])
@pytest.mark.parametrize("M", [1, 4])
def test_quantize_rows_refuses_to_write_over_its_input(M, dtype):
    assert ct.ct_quantize_rows(**{**QUANT, "q": P, "M": M, "dtype": dtype, "ldq": 128}) == ct.CT_ERR_INVALID_ARG
    assert "in the place of" in ct.ct_last_error()


@pytest.mark.parametrize("ep", [dict(gate=3 * P, ldg=40), dict(residual=3 * P, ldr=33),
                                dict(gate=3 * P, ldg=32, residual=3 * P, ldr=64)], ids=str)
def test_products_refuse_a_gate_or_residual_in_place_with_another_stride(ep):
    e = ct.ct_linear_epilogue()
    for k, v in ep.items():
        setattr(e, k, v)
    assert ct.ct_linear_fwd(**{**LIN, "epi": e}) == ct.CT_ERR_INVALID_ARG
    assert "in the place of" in ct.ct_last_error()
    assert ct.ct_linear_q8_fwd(**{**Q8, "epi": e}) == ct.CT_ERR_INVALID_ARG
    assert "in the place of" in ct.ct_last_error()


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, args, _) in CALLS.items() for n in
                                       ("x", "w", "y", "q", "h", "residual", "xs", "ws", "gain", "scale") if args.get(n)])
def test_raw_entry_points_refuse_host_tensors(call, name):
    """A host address would be read by the kernel."""
    f, args, _ = CALLS[call]
    with pytest.raises(ValueError, match="on the GPU"):
        f(**{**args, name: torch.zeros(4, 64)})
    with pytest.raises(TypeError):
        f(**{**args, name: [0.0] * 256})


@pytest.mark.parametrize("mnk", [(1 << 30, 64, 64), (1 << 30, 512, 1), (1, 1 << 28, 64), (1 << 20, 1 << 20, 64)], ids=str)
def test_no_workspace_is_named_for_a_product_that_is_refused(mnk):
    M, N, K = mnk
    for dtype in (ct.CT_F32, ct.CT_F16, ct.CT_BF16):
        a = {**LIN, "M": M, "N": N, "K": K, "ldy": N, "dtype": dtype, "workspace": P, "workspace_bytes": 1 << 60}
        assert ct.ct_linear_fwd(**a) == ct.CT_ERR_UNSUPPORTED
        assert ct.ct_linear_workspace_bytes(M, N, K, dtype) == ct.CT_ERR_UNSUPPORTED
    assert ct.ct_linear_workspace_bytes(M, N, K, ct.CT_E4M3) == ct.CT_ERR_UNSUPPORTED
