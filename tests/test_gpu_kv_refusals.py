"""Refusals of the key-value helpers that need tensors on the GPU, and calls at
their border that are taken."""
import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV
from _kv_helpers import BF16, E4M3, F16, F32, ints

pytestmark = pytest.mark.gpu


def parts(dtype=BF16, heads=2):
    c = ct.KVCache.empty(8, heads, 16, 64, dtype=dtype, device=DEV)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.view(torch.uint8).zero_()
    lens, table = ints([20, 9]), ints([[0, 1], [2, 3]])
    q = torch.ones(2, 4, 64, dtype=BF16, device=DEV)
    return c, lens, table, q


def test_attention_refuses():
    c, lens, table, q = parts()
    bits = torch.ones(2, dtype=torch.int64, device=DEV)
    for bad in (dict(max_len=-1), dict(max_len=-2 ** 40), dict(tree=bits[0]), dict(tree=bits.view(2, 1, 1)), dict(tree=bits[:1]),
                dict(tree=bits.int()), dict(tree=bits.cpu()), dict(tree=torch.ones(2, 4, dtype=torch.int64, device=DEV)[:, ::2]),
                dict(window=-1), dict(window=1 << 31), dict(sinks=-1, window=2), dict(out=q.float()), dict(out=q[:1]),
                dict(starts=ints([0, 2])), dict(starts=torch.zeros(3, dtype=torch.int64, device=DEV)), dict(table=table[:1]),
                dict(table=table.long()), dict(table=table.t()), dict(lens=lens.cpu()), dict(lens=lens.view(1, 2)),
                dict(lens=lens.float()), dict(q=q[0]), dict(q=q.half()[..., :48]), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            ct.kv_attention(**{**dict(q=q, cache=c, lens=lens, table=table), **bad})
    for bad in (dict(sinks=2), dict(scale=0.0), dict(scale=float("nan")), dict(out=q), dict(q=q.half()), dict(q=q[:, :3]),
                dict(lens=ints([20, 9, 3]), table=None), dict(lens=ints([1] * 9), table=None, q=torch.ones(9, 4, 64, dtype=BF16, device=DEV)),
                dict(out=q[:1].clone().expand(2, 4, 64))):
        with pytest.raises(ct.ConvTileError):
            ct.kv_attention(**{**dict(q=q, cache=c, lens=lens, table=table), **bad})


def test_writing_and_reading_refuse():
    c, lens, table, _ = parts(E4M3)
    k = torch.ones(2, 2, 64, dtype=BF16, device=DEV)
    for bad in (dict(k=k[0]), dict(k=k[:, :1]), dict(v=k.half()), dict(v=k[:1]), dict(k=k.cpu()), dict(k=k.transpose(0, 2)),
                dict(lens=lens.cpu()), dict(table=table[:, ::2][:, :0].long())):
        with pytest.raises(ValueError):
            ct.kv_write(**{**dict(cache=c, k=k, v=k, lens=lens, table=table), **bad})
    for bad in (dict(tokens=-1), dict(k=k[:1]), dict(k=k, dtype=F32), dict(tokens=1 << 31)):
        with pytest.raises(ValueError):
            ct.kv_read(**{**dict(cache=c, tokens=2, lens=lens, table=table), **bad})
    with pytest.raises(ct.ConvTileError):
        ct.kv_read(c, 2, lens, table, k=k, v=k)
    one = ct.KVCache(c.k, c.v, c.k_scale, c.k_scale)
    with pytest.raises(ct.ConvTileError, match="k_scale and v_scale"):
        ct.kv_write(one, k, k, lens, table)


def test_an_axis_of_one_of_any_stride():
    """One head, cut out of a wider tensor for k and by itself for v."""
    n = 6 * 16 * 64
    k = torch.zeros(n, dtype=F16, device=DEV).view(6, 16, 1, 64).transpose(1, 2)
    v = torch.zeros(n, dtype=F16, device=DEV).view(6, 1, 16, 64)
    assert k.stride() != v.stride()
    c = ct.KVCache(k, v)
    lens, table = ints([40]), ints([[5, 0, 2]])
    x, y = (torch.randn(40, 1, 64, device=DEV).half() for _ in range(2))
    ct.kv_write(c, x, y, lens, table)
    a, b = ct.kv_read(c, 40, lens, table)
    torch.cuda.synchronize()
    assert torch.equal(a, x) and torch.equal(b, y)
