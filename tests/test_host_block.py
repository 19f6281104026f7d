"""Refusals and host-side rules of the transformer-block entry points
(ct_rmsnorm_fwd, ct_quantize_rows, ct_linear_fwd, ct_linear_q8_fwd,
ct_linear_workspace_bytes): every bad argument is reported before any HIP
call, so the addresses here are never read."""
import ctypes
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
NORM = dict(x=P, ldx=64, residual=P, ldr=64, gain=P, h=2 * P, ldh=64, y=3 * P, ldy=64, scale=None, M=4, D=64,
            dtype=ct.CT_BF16, out_dtype=ct.CT_BF16, eps=1e-6, stream=0)
QUANT = dict(x=P, ldx=64, q=P, ldq=64, scale=P, M=4, D=64, dtype=ct.CT_BF16, stream=0)


def epi(**kw):
    e = ct.ct_linear_epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(K=-3), dict(dtype=7), dict(dtype=ct.CT_E4M3), dict(out_dtype=ct.CT_E4M3),
    dict(out_dtype=-1), dict(x=None), dict(w=None), dict(y=None), dict(ldx=63), dict(ldw=63), dict(ldy=31),
    dict(x=P + 1), dict(w=P + 1), dict(y=P + 1), dict(epi=epi(act=5)), dict(epi=epi(act=-1)),
    dict(epi=epi(gate=P, ldg=31)), dict(epi=epi(residual=P, ldr=0)), dict(epi=epi(gate=P + 1, ldg=32)),
    dict(epi=epi(bias=P + 2)), dict(dtype=ct.CT_F32, x=P + 2), dict(ldx=1 << 41),
], ids=str)
def test_linear_refuses(bad):
    assert ct.ct_linear_fwd(**{**LIN, **bad}) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


@pytest.mark.parametrize("same", [dict(y=P), dict(w=3 * P, y=3 * P)], ids=str)
def test_linear_refuses_to_write_over_its_operands(same):
    a = {**LIN, "x": P, "w": 2 * P, **same}
    assert ct.ct_linear_fwd(**a) == ct.CT_ERR_INVALID_ARG and "y must not be" in ct.ct_last_error()


def test_rmsnorm_refuses_one_place_for_h_and_y():
    assert ct.ct_rmsnorm_fwd(**{**NORM, "h": P, "y": P}) == ct.CT_ERR_INVALID_ARG
    assert "must not be the same" in ct.ct_last_error()


def test_linear_refuses_more_tiles_than_a_launch_takes():
    a = {**LIN, "M": 1 << 30, "x": P, "w": 2 * P, "y": 3 * P}
    assert ct.ct_linear_fwd(**a) == ct.CT_ERR_UNSUPPORTED
    b = {**LIN, "M": 1, "N": 1 << 28, "ldy": 1 << 28, "x": P, "w": 2 * P, "y": 3 * P}
    assert ct.ct_linear_fwd(**b) == ct.CT_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(xs=None), dict(ws=None), dict(xs=P + 2), dict(out_dtype=ct.CT_E4M3), dict(M=-1), dict(N=0), dict(K=0),
    dict(x=None), dict(ldx=63), dict(epi=epi(act=9)),
], ids=str)
def test_linear_q8_refuses(bad):
    assert ct.ct_linear_q8_fwd(**{**Q8, **bad}) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


@pytest.mark.parametrize("big", [
    dict(ldx=(8 << 20) // 2 + 8), dict(ldw=(8 << 20) // 2 + 8), dict(M=(1 << 30) + 1),
    dict(N=(1 << 30) + 1, ldy=1 << 31), dict(K=(1 << 29) + 1, ldx=1 << 30, ldw=1 << 30),
], ids=str)
def test_linear_says_what_it_cannot_do(big):
    assert ct.ct_linear_fwd(**{**LIN, **big}) == ct.CT_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(D=0), dict(dtype=ct.CT_E4M3), dict(dtype=9), dict(out_dtype=4), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(y=None), dict(ldx=63), dict(ldr=63),
    dict(ldh=63), dict(ldy=63), dict(residual=None), dict(scale=P), dict(out_dtype=ct.CT_E4M3), dict(gain=P + 1),
    dict(x=P + 1), dict(h=P + 1), dict(out_dtype=ct.CT_E4M3, scale=P + 2), dict(out_dtype=ct.CT_F32, y=P + 2),
], ids=str)
def test_rmsnorm_refuses(bad):
    assert ct.ct_rmsnorm_fwd(**{**NORM, **bad}) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


@pytest.mark.parametrize("bad", [dict(M=-1), dict(D=0), dict(dtype=ct.CT_E4M3), dict(x=None), dict(q=None),
                                 dict(scale=None), dict(ldx=63), dict(ldq=63), dict(x=P + 1)], ids=str)
def test_quantize_rows_refuses(bad):
    assert ct.ct_quantize_rows(**{**QUANT, **bad}) == ct.CT_ERR_INVALID_ARG


def test_no_rows_is_no_work():
    """An empty batch succeeds without looking at its (absent) pointers."""
    assert ct.ct_linear_fwd(**{**LIN, "M": 0, "x": None, "y": None}) == 0
    assert ct.ct_linear_q8_fwd(**{**Q8, "M": 0, "x": None, "xs": None, "y": None}) == 0
    assert ct.ct_rmsnorm_fwd(**{**NORM, "M": 0, "x": None, "y": None}) == 0
    assert ct.ct_quantize_rows(**{**QUANT, "M": 0, "x": None, "q": None, "scale": None}) == 0
    assert ct.ct_linear_workspace_bytes(0, 32, 64, ct.CT_BF16) == 0


def _split_shape():
    for M in (33, 48, 64, 96, 128, 200):
        need = ct.ct_linear_workspace_bytes(M, 512, 8192, ct.CT_BF16)
        if need > 0:
            return M, need
    raise AssertionError("no split product among these sizes")


def test_workspace_is_asked_for_and_checked():
    M, need = _split_shape()
    a = {**LIN, "M": M, "N": 512, "K": 8192, "ldx": 8192, "ldw": 8192, "ldy": 512}
    assert ct.ct_linear_fwd(**a) == ct.CT_ERR_INVALID_ARG
    assert str(need) in ct.ct_last_error()
    assert ct.ct_linear_fwd(**{**a, "workspace": P, "workspace_bytes": need - 1}) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_linear_fwd(**{**a, "workspace": P + 8, "workspace_bytes": need}) == ct.CT_ERR_INVALID_ARG


def test_workspace_bytes():
    f = ct.ct_linear_workspace_bytes
    assert f(1, 4096, 4096, ct.CT_BF16) == 0
    assert f(8192, 8192, 8192, ct.CT_E4M3) == 0
    for bad in ((-1, 4, 4, 0), (4, 0, 4, 0), (4, 4, 0, 0), (4, 4, 4, 8)):
        assert f(*bad) == ct.CT_ERR_INVALID_ARG
    assert f(4, 4, 1 << 30, ct.CT_F32) == ct.CT_ERR_UNSUPPORTED


def test_epilogue_struct_matches_the_header():
    """act, bias, gate, ldg, residual, ldr with C's natural alignment."""
    assert ctypes.sizeof(ct.ct_linear_epilogue) == 48
    assert [getattr(ct.ct_linear_epilogue, f).offset for f, _ in ct.ct_linear_epilogue._fields_] == [0, 8, 16, 24, 32, 40]


def test_helpers_refuse_host_tensors():
    x, w = torch.zeros(2, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ct.linear(x, w)
    with pytest.raises(ValueError):
        ct.rmsnorm(x)
    with pytest.raises(ValueError):
        ct.quantize_rows(x)
    with pytest.raises(ValueError):
        ct.linear_q8(x.to(torch.float8_e4m3fn), None, w.to(torch.float8_e4m3fn), None)
