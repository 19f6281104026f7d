"""GPU tests of attention over the key-value cache at widths, layouts and divisions
of the work beside those of test_gpu_kv_attention.py, against the definition in 64
bits (the tolerance's derivation stands at tolerance() in _kv_helpers.py)."""
import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV
from _kv_helpers import (BF16, E4M3, F16, F32, Setup, attention64, check_sequence, gen, ints, seen_causal, seen_tree, tolerance,
                         tree_bits)

pytestmark = pytest.mark.gpu

TYPES = [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)]
IDS = ["bf16", "f16", "bf16-e4m3", "f16-e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def compare(s, q, y, window=0, sinks=0, sees=None, name=""):
    for b, (length, new) in enumerate(s.seqs):
        if new == 0:
            continue
        k, v = s.held(b)
        see = seen_causal(length, new, window, sinks) if sees is None else seen_tree(length, new, window, sinks, sees[b])
        qb = q[s.first[b]:s.first[b + 1]]
        k = torch.where(k.isfinite(), k, torch.zeros_like(k))
        ref, size = attention64(qb, k, v, see, s.dim ** -0.5)
        tol = tolerance(torch.where(ref.isfinite(), ref, torch.zeros_like(ref)), size, qb, k, length, q.dtype, s.dim ** -0.5)
        check_sequence((name, b, length, new), y[s.first[b]:s.first[b + 1]].double(), ref, tol)


# new tokens and heads of a group: one row, 16 rows, a part of a tile, several tiles
ROWS = [(1, 1), (4, 4), (60, 1), (90, 4)]


@pytest.mark.parametrize("tree", [False, True], ids=["causal", "tree"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("new,group", ROWS)
@pytest.mark.parametrize("dim", [48, 64, 80, 96, 128, 160, 192, 240, 256])
def test_values_that_are_not_finite(dim, new, group, types, tree):
    """NaN and infinities in values that some rows see and others do not, in every
    head, at widths of and between the kernels' own; with a window and sinks too."""
    dtype, cdt = types
    seqs = [(300, new), (200, new)]
    s = Setup(seqs, 2, dim, 16, dtype, cdt, seed=dim + new)
    bad = [float("nan")] if cdt == E4M3 else [float("nan"), float("inf"), float("-inf")]
    g = torch.Generator().manual_seed(new + dim)
    for b, (length, _) in enumerate(seqs):
        # among all places, and among the new tokens', where rows differ by what they see
        for low in (0, length - new):
            for i in range(7):
                at = int(torch.randint(low, length, (1,), generator=g))
                s.v[b][at, i % 2, int(torch.randint(0, dim, (1,), generator=g))] = bad[i % len(bad)]
    s.write()
    q = torch.randn(s.tokens, 2 * group, dim, generator=gen(1), device=DEV).to(dtype)
    sees = bits = None
    if tree:
        sees = [torch.rand(new, new, generator=torch.Generator().manual_seed(b)) < 0.4 for b in range(2)]
        bits = torch.cat([tree_bits(x, (new + 63) // 64) for x in sees])
    for window, sinks in ((0, 0), (80, 3)):
        for longest in (None, 1):
            y = ct.kv_attention(q, s.cache, s.lens, s.table, max_len=longest, window=window, sinks=sinks, tree=bits)
            torch.cuda.synchronize()
            compare(s, q, y, window, sinks, sees, (window, longest))


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("new,group", ROWS[:3])
@pytest.mark.parametrize("dim", [32, 112, 144, 176, 208, 224, 240])
def test_widths_between_the_kernels_own(dim, new, group, types):
    dtype, cdt = types
    s = Setup([(700, new), (65, min(new, 65))], 2, dim, 24, dtype, cdt, seed=dim)
    s.write()
    q = torch.randn(s.tokens, 2 * group, dim, generator=gen(2), device=DEV).to(dtype)
    for window, sinks in ((0, 0), (70, 2)):
        y = ct.kv_attention(q, s.cache, s.lens, s.table, s.starts, window=window, sinks=sinks)
        torch.cuda.synchronize()
        compare(s, q, y, window, sinks)


def laid_out(shape, order, dtype):
    """A tensor of `shape` whose axes lie in memory in `order` (outermost first), full of NaN."""
    t = torch.full([shape[i] for i in order], float("nan"), dtype=F32, device=DEV).to(dtype)
    return t.permute([order.index(i) for i in range(len(shape))])


@pytest.mark.parametrize("cdt", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 5, 150])
@pytest.mark.parametrize("order,scales", [((1, 2, 0, 3), (1, 2, 0)), ((2, 0, 1, 3), (0, 1, 2)), ((0, 1, 2, 3), (2, 1, 0)),
                                          ((2, 1, 0, 3), (0, 2, 1)), ((1, 0, 2, 3), (2, 0, 1))], ids=str)
def test_any_order_of_the_axes(order, scales, new, cdt):
    """Pages or heads innermost, places outermost; scales in an order of their own."""
    pages, heads, page, dim = 13, 3, 24, 64
    k, v = (laid_out((pages, heads, page, dim), order, cdt) for _ in range(2))
    sk = [laid_out((pages, heads, page), scales, F32) for _ in range(2)] if cdt == E4M3 else [None, None]
    s = Setup([(200, new), (90, min(90, new))], heads, dim, page, BF16, cdt, seed=3)
    s.cache = ct.KVCache(k, v, *sk)
    s.table = torch.randperm(pages, generator=torch.Generator().manual_seed(4))[:12].to(torch.int32).to(DEV).view(2, 6)
    s.table = torch.cat([s.table, torch.full((2, 3), pages, dtype=torch.int32, device=DEV)], dim=1)  # the last columns name no page
    s.lens = ints([6 * page, 90])
    s.seqs = [(6 * page, new if new <= 6 * page else 6 * page), (90, min(90, new))]
    s.k[0], s.v[0] = s.k[0][:6 * page], s.v[0][:6 * page]
    first = [0, s.seqs[0][1], s.seqs[0][1] + s.seqs[1][1]]
    s.first, s.tokens, s.starts = first, first[-1], ints(first)
    s.write()
    q = torch.randn(s.tokens, 6, dim, generator=gen(5), device=DEV).to(BF16)
    y = ct.kv_attention(q, s.cache, s.lens, s.table, s.starts)
    rk, rv = ct.kv_read(s.cache, s.tokens, s.lens, s.table, s.starts, dtype=F32)
    torch.cuda.synchronize()
    compare(s, q, y)
    for b, (length, n) in enumerate(s.seqs):
        hk, hv = s.held(b)
        assert torch.equal(rk[first[b]:first[b + 1]].double(), hk[length - n:])
        assert torch.equal(rv[first[b]:first[b + 1]].double(), hv[length - n:])


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("length", [16384, 40000])
def test_as_many_parts_as_there_are(length, types):
    """One row of one head: 128 parts where the length has room for them, and fewer
    keys than the guide says, so that the last parts have none."""
    dtype, cdt = types
    s = Setup([(length, 1)], 1, 64, 64, dtype, cdt, seed=6)
    s.write()
    q = torch.randn(1, 1, 64, generator=gen(7), device=DEV).to(dtype)
    assert ct.ct_kv_attention_workspace_bytes(1, 1, 1, 1, 64, length, cache_dtype=ct.CT_E4M3) == 128 * 66 * 4
    for n in (length, length - 1, length // 2, 129, 1):
        y = ct.kv_attention(q, s.cache, ints([n]), s.table, max_len=length)
        torch.cuda.synchronize()
        k, v = (t[:n] for t in s.held(0))
        ref, size = attention64(q, k, v, seen_causal(n, 1, 0, 0), 64 ** -0.5)
        check_sequence(n, y.double(), ref, tolerance(ref, size, q, k, n, dtype, 64 ** -0.5))


@pytest.mark.parametrize("cdt", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_a_prompt_among_many_tokens(cdt):
    """The form and the parts follow averages: 300 single tokens, one of them over a
    long cache, beside a prompt of 700."""
    seqs = [(40 + i % 50, 1) for i in range(150)] + [(700, 700)] + [(6000, 1)] + [(30 + i % 9, 1) for i in range(149)]
    s = Setup(seqs, 1, 64, 64, BF16, cdt, seed=8)
    s.write()
    q = torch.randn(s.tokens, 4, 64, generator=gen(9), device=DEV).to(BF16)
    for window, sinks in ((0, 0), (33, 1)):
        y = ct.kv_attention(q, s.cache, s.lens, s.table, s.starts, window=window, sinks=sinks, max_len=6000)
        torch.cuda.synchronize()
        compare(s, q, y, window, sinks)


@pytest.mark.parametrize("new", [1, 40])
def test_a_shared_prefix_that_is_written_once(new):
    """Two sequences over one prefix's pages: the first writes them, the second its
    own tokens behind them."""
    s = Setup([(300, new), (320, new)], 2, 64, 16, BF16, E4M3, seed=10)
    shared = (300 - new) // 16
    s.table[1, :shared] = s.table[0, :shared]
    for x in (s.k, s.v):
        x[1][:shared * 16] = x[0][:shared * 16]
    own = 320 - shared * 16
    ct.kv_write(s.cache, torch.cat([s.k[0], s.k[1][-own:]]), torch.cat([s.v[0], s.v[1][-own:]]), s.lens, s.table,
                ints([0, 300, 300 + own]))
    q = torch.randn(2 * new, 8, 64, generator=gen(11), device=DEV).to(BF16)
    y = ct.kv_attention(q, s.cache, s.lens, s.table)
    torch.cuda.synchronize()
    compare(s, q, y)


@pytest.mark.parametrize("cdt", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_two_calls_at_once(cdt):
    """Two streams, a workspace each, over one cache."""
    s = Setup([(5000, 1), (300, 1)], 2, 128, 64, BF16, cdt, seed=12)
    s.write()
    qs = [torch.randn(2, 8, 128, generator=gen(13 + i), device=DEV).to(BF16) for i in range(2)]
    want = [ct.kv_attention(q, s.cache, s.lens, s.table) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, (q, st) in enumerate(zip(qs, streams)):
            got[i].append(ct.kv_attention(q, s.cache, s.lens, s.table, stream=st))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    compare(s, qs[0], want[0])


@pytest.mark.parametrize("types", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("dim", [112, 128, 192, 256])
@pytest.mark.parametrize("new,group", [(1, 1), (3, 4)])
def test_few_rows_of_one_sequence_with_a_long_table(new, group, dim, types):
    """What a guide of 2^19 keys and more in all heads chooses, on short lengths too:
    the table's further columns name a page of other values."""
    dtype, cdt = types
    s = Setup([(3000, new)], 8, dim, 64, dtype, cdt, seed=14)
    s.write()
    s.table = torch.cat([s.table, s.table[:, :1].expand(1, 1100)], dim=1).contiguous()
    q = torch.randn(new, 8 * group, dim, generator=gen(15), device=DEV).to(dtype)
    for window, sinks in ((0, 0), (1 << 18, 0), (70, 2)):
        y = ct.kv_attention(q, s.cache, s.lens, s.table, window=window, sinks=sinks)
        torch.cuda.synchronize()
        compare(s, q, y, window, sinks)
