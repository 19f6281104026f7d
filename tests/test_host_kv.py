"""Refusals and host-side rules of the key-value cache's entry points
(ct_kv_write, ct_kv_read, ct_kv_attention_fwd, ct_kv_attention_workspace_bytes):
every bad argument is reported before any HIP call, so the addresses here are
never read."""
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


CACHE = dict(k=P, v=2 * P, k_scale=None, v_scale=None, dtype=ct.CT_BF16, pages=10, heads=2, page=16, dim=64, ld_page=2048,
             ld_head=1024, ld_token=64, lds_page=0, lds_head=0, lds_token=0)
Q8 = dict(CACHE, dtype=ct.CT_E4M3, k_scale=3 * P, v_scale=4 * P, lds_page=32, lds_head=16, lds_token=1)
BATCH = dict(tokens=4, sequences=2, lens=5 * P, starts=None, table=6 * P, ldt=5, width=5)


def struct(cls, fields):
    c = cls()
    for k, v in fields.items():
        setattr(c, k, v)
    return c


def write(cache=CACHE, batch=BATCH, read=False, **kw):
    a = dict(k=7 * P, k_token=128, k_head=64, v=8 * P, v_token=128, v_head=64, dtype=ct.CT_BF16, stream=0)
    f = ct.ct_kv_read if read else ct.ct_kv_write
    return f(struct(ct.ct_kv_cache, cache), struct(ct.ct_kv_batch, batch), **{**a, **kw})


def attend(cache=CACHE, batch=BATCH, mask=None, **kw):
    a = dict(q=7 * P, q_token=256, q_head=64, y=8 * P, y_token=256, y_head=64, heads=4, dtype=ct.CT_BF16, scale=0.125,
             max_len=64, workspace=None, workspace_bytes=0, stream=0)
    m = struct(ct.ct_kv_mask, mask) if mask is not None else None
    return ct.ct_kv_attention_fwd(struct(ct.ct_kv_cache, cache), struct(ct.ct_kv_batch, batch), m, **{**a, **kw})


CALLS = {"write": write, "read": lambda *a, **kw: write(*a, read=True, **kw), "attend": attend}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=P + 8), dict(v=2 * P + 2), dict(dtype=ct.CT_F32), dict(dtype=9), dict(pages=0),
    dict(heads=0), dict(page=0), dict(dim=0), dict(pages=-1), dict(ld_page=0), dict(ld_head=-64), dict(ld_token=4),
    dict(ld_token=60), dict(ld_token=68), dict(ld_page=1 << 41), dict(ld_page=1024), dict(ld_head=960), dict(k_scale=P),
    dict(v_scale=P),
], ids=str)
def test_caches_that_are_refused(call, bad):
    assert CALLS[call](dict(CACHE, **bad)) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bad", [dict(k_scale=None), dict(v_scale=None), dict(k_scale=P + 2), dict(lds_page=0),
                                 dict(lds_token=-1), dict(lds_head=8), dict(ld_token=72)], ids=str)
def test_8_bit_caches_that_are_refused(call, bad):
    assert CALLS[call](dict(Q8, **bad)) == ct.CT_ERR_INVALID_ARG


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("big", [dict(dim=40), dict(dim=272, ld_token=512, ld_head=8192, ld_page=16384), dict(dim=8),
                                 dict(page=1 << 30, ld_token=64, ld_head=1 << 36, ld_page=1 << 37),
                                 dict(heads=(1 << 16) + 1, ld_page=1 << 27)], ids=str)
def test_caches_beyond_the_kernels(call, big):
    assert CALLS[call](dict(CACHE, **big)) == ct.CT_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(sequences=-1), dict(sequences=0), dict(tokens=5), dict(lens=None), dict(lens=5 * P + 2),
    dict(starts=P + 1), dict(table=P + 2), dict(width=0), dict(ldt=4), dict(table=None, sequences=11, tokens=11),
], ids=str)
def test_batches_that_are_refused(call, bad):
    assert CALLS[call](batch=dict(BATCH, **bad)) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


@pytest.mark.parametrize("call", list(CALLS))
def test_batches_beyond_the_kernels(call):
    assert CALLS[call](batch=dict(BATCH, tokens=1 << 25)) == ct.CT_ERR_UNSUPPORTED
    assert CALLS[call](batch=dict(BATCH, width=1 << 27, ldt=1 << 27)) == ct.CT_ERR_UNSUPPORTED
    assert CALLS[call](batch=dict(BATCH, starts=P, sequences=(1 << 24) + 1)) == ct.CT_ERR_UNSUPPORTED
    assert CALLS[call](batch=dict(BATCH, starts=P, sequences=(1 << 16) + 1)) == ct.CT_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", list(CALLS))
def test_null_structs_and_no_tokens(call):
    f = {"write": ct.ct_kv_write, "read": ct.ct_kv_read}.get(call)
    if f:
        assert f(None, None, P, 1, 1, P, 1, 1, 0, 0) == ct.CT_ERR_INVALID_ARG
        assert f(struct(ct.ct_kv_cache, CACHE), None, P, 1, 1, P, 1, 1, 0, 0) == ct.CT_ERR_INVALID_ARG
        assert CALLS[call](batch=dict(BATCH, tokens=0, lens=None, table=None), k=None, v=None) == 0
    else:
        assert ct.ct_kv_attention_fwd(None, None, None, P, 1, 1, P, 1, 1, 1, 2, 1.0, stream=0) == ct.CT_ERR_INVALID_ARG
        assert attend(batch=dict(BATCH, tokens=0, lens=None, table=None), q=None, y=None) == 0


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=7 * P + 1), dict(k_token=-1), dict(v_head=-64),
                                 dict(k_token=1 << 41), dict(dtype=ct.CT_E4M3), dict(dtype=-1), dict(k=P), dict(v=2 * P),
                                 dict(dtype=ct.CT_F32, v=8 * P + 2)], ids=str)
def test_rows_that_are_refused(read, bad):
    assert write(read=read, **bad) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


def test_one_place_for_keys_and_values_is_not_written():
    assert write(dict(CACHE, v=P)) == ct.CT_ERR_INVALID_ARG and "must not be the same" in ct.ct_last_error()


def test_one_place_for_both_scales_is_not_written():
    assert write(dict(Q8, v_scale=3 * P)) == ct.CT_ERR_INVALID_ARG and "k_scale and v_scale" in ct.ct_last_error()


def test_rows_read_to_one_place_are_refused():
    assert write(read=True, v=7 * P) == ct.CT_ERR_INVALID_ARG
    assert write(read=True, k_token=64) == ct.CT_ERR_INVALID_ARG
    assert write(read=True, v_head=32) == ct.CT_ERR_INVALID_ARG
    assert write(read=True, k_head=0) == ct.CT_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(y=None), dict(q=7 * P + 1), dict(y=8 * P + 1), dict(q_token=-4), dict(y_token=64), dict(y_head=32),
    dict(y_head=0), dict(heads=0), dict(heads=3), dict(heads=-2), dict(dtype=ct.CT_F32), dict(dtype=ct.CT_E4M3),
    dict(dtype=ct.CT_F16), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(max_len=-1), dict(y=7 * P), dict(y=P), dict(y=2 * P), dict(mask=dict(window=-1)), dict(mask=dict(sinks=-1, window=3)),
    dict(mask=dict(sinks=2)), dict(mask=dict(words=1)), dict(mask=dict(tree=P)), dict(mask=dict(tree=P + 4, words=1)),
    dict(mask=dict(tree=P, words=-1)),
], ids=str)
def test_attention_refuses(bad):
    assert attend(**bad) == ct.CT_ERR_INVALID_ARG
    assert ct.ct_last_error()


def test_attention_says_what_it_cannot_do():
    assert attend(scale=3e38) == ct.CT_ERR_UNSUPPORTED
    assert attend(batch=dict(BATCH, tokens=1 << 24), q_token=256) == ct.CT_ERR_UNSUPPORTED


def test_workspace_is_asked_for_and_checked():
    need = ct.ct_kv_attention_workspace_bytes(2, 2, 4, 2, 64, 65536)
    assert need > 0
    long = dict(CACHE, pages=5000)
    b = dict(BATCH, tokens=2, width=4096, ldt=4096)
    assert attend(long, b, max_len=65536) == ct.CT_ERR_INVALID_ARG and str(need) in ct.ct_last_error()
    assert attend(long, b, max_len=65536, workspace=P, workspace_bytes=need - 1) == ct.CT_ERR_INVALID_ARG
    assert attend(long, b, max_len=65536, workspace=P + 8, workspace_bytes=need) == ct.CT_ERR_INVALID_ARG


def test_workspace_bytes():
    f = ct.ct_kv_attention_workspace_bytes
    assert f(0, 3, 8, 2, 128) == 0
    assert f(8192, 1, 32, 8, 128, 8192) == 0
    for bad in ((-1, 1, 8, 2, 128), (1, -1, 8, 2, 128), (1, 1, 0, 2, 128), (1, 1, 8, 0, 128), (1, 1, 8, 3, 128), (1, 0, 8, 2, 128),
                (1, 1, 8, 2, 0), (1, 1, 8, 2, 128, -1), (1, 1, 8, 2, 128, 0, -1), (1, 1, 8, 2, 128, 0, 0, 1)):
        assert f(*bad) == ct.CT_ERR_INVALID_ARG, bad
    for big in ((1, 1, 8, 2, 120), (1, 1, 8, 2, 272), (1 << 26, 1, 8, 2, 128), (1 << 25, 1 << 25, 1, 1, 128), (1, 1, 1 << 17, 1, 128)):
        assert f(*big) == ct.CT_ERR_UNSUPPORTED, big
    assert f(1, 1, 8, 2, 128, 64, 0, 0, ct.CT_F32) == ct.CT_ERR_INVALID_ARG
    # a window bounds what there is to share
    assert f(1, 1, 8, 8, 128, 1 << 20, 128, 4) <= f(1, 1, 8, 8, 128, 1 << 20)


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, -(1 << 32)])
def test_counts_past_32_bits_are_not_cut(n):
    for name in ("tokens", "sequences", "heads", "kv_heads", "dim", "window", "sinks"):
        a = dict(tokens=1, sequences=1, heads=8, kv_heads=2, dim=128, max_len=0, window=4, sinks=0)
        with pytest.raises(ValueError, match="32 bits"):
            ct.ct_kv_attention_workspace_bytes(**{**a, name: n})


def test_structs_match_the_header():
    """C's natural alignment."""
    assert [getattr(ct.ct_kv_cache, f).offset for f, _ in ct.ct_kv_cache._fields_] == \
        [0, 8, 16, 24, 32, 36, 40, 44, 48, 56, 64, 72, 80, 88, 96]
    assert ctypes.sizeof(ct.ct_kv_cache) == 104
    assert [getattr(ct.ct_kv_batch, f).offset for f, _ in ct.ct_kv_batch._fields_] == [0, 4, 8, 16, 24, 32, 40]
    assert ctypes.sizeof(ct.ct_kv_batch) == 48
    assert [getattr(ct.ct_kv_mask, f).offset for f, _ in ct.ct_kv_mask._fields_] == [0, 4, 8, 16]
    assert ctypes.sizeof(ct.ct_kv_mask) == 24


def test_helpers_refuse_host_tensors():
    t = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ct.KVCache(t, t)
    with pytest.raises(ValueError, match="on the GPU"):
        ct.ct_kv_write(None, None, torch.zeros(1, 1, 64), 64, 64, P, 64, 64, 0, 0)


def test_caches_that_the_helper_refuses():
    m = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="meta")  # noqa: E731
    for k, v in ((m(2, 1, 16, 64), m(2, 1, 16, 32)), (m(2, 1, 16, 64), m(2, 1, 16, 64, dt=torch.float16)),
                 (m(2, 16, 64), m(2, 16, 64)), (m(2, 1, 16, 64, dt=torch.float32), m(2, 1, 16, 64, dt=torch.float32)),
                 (m(2, 4, 16, 64), m(2, 16, 4, 64).transpose(1, 2))):
        with pytest.raises(ValueError):
            ct.KVCache(k, v)
    e = m(2, 1, 16, 64, dt=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="scales"):
        ct.KVCache(e, e)
    with pytest.raises(ValueError, match="scales"):
        ct.KVCache(m(2, 1, 16, 64), m(2, 1, 16, 64), m(2, 1, 16), m(2, 1, 16))


def test_an_axis_of_one_has_no_layout():
    """k and v of the same layout whose axes of one differ in a stride that nothing
    uses: refused for where they are only."""
    for shape in ((3, 1, 16, 64), (1, 4, 16, 64), (3, 4, 1, 64), (1, 1, 1, 64)):
        n = shape[0] * shape[1] * shape[2] * 64
        st = [shape[1] * shape[2] * 64, shape[2] * 64, 64, 1]
        k = torch.empty(n, dtype=torch.bfloat16, device="meta").as_strided(shape, st)
        v = torch.empty(n, dtype=torch.bfloat16, device="meta").as_strided(shape, [s if m > 1 else 5 * s for s, m in zip(st, shape)])
        with pytest.raises(ValueError, match="on one device"):
            ct.KVCache(k, v)
