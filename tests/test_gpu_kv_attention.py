"""GPU parity of attention over the key-value cache against its definition in
64 bits; the tolerance's derivation stands at tolerance() in _kv_helpers.py.
Every place of a cache that no token may see holds NaN, unless a test says
otherwise."""
import math

import pytest
import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV, say
from _kv_helpers import (BF16, E4M3, F16, Setup, attention64, check_sequence, gen, ints, seen_causal, seen_tree,
                         tolerance, tree_bits)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def compare(s, q, y, window=0, sinks=0, sees=None, scale=None, name=""):
    scale = scale or s.dim ** -0.5
    for b, (length, new) in enumerate(s.seqs):
        if new == 0:
            continue
        k, v = s.held(b)
        see = seen_causal(length, new, window, sinks) if sees is None else seen_tree(length, new, window, sinks, sees[b])
        qb = q[s.first[b]:s.first[b + 1]]
        ref, size = attention64(qb, k, v, see, scale)
        kk = torch.where(k.isfinite(), k, torch.zeros_like(k))
        tol = tolerance(torch.where(ref.isfinite(), ref, torch.zeros_like(ref)), size, qb, kk, length, q.dtype, scale)
        check_sequence((name, b, length, new), y[s.first[b]:s.first[b + 1]].double(), ref, tol)


def attend(s, q, window=0, sinks=0, starts=True, **kw):
    return ct.kv_attention(q, s.cache, s.lens, s.table, s.starts if starts else None, window=window, sinks=sinks, **kw)


TYPES = [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)]
IDS = ["bf16", "f16", "bf16-e4m3", "f16-e4m3"]

# sequences of (length, new), heads of the cache, group, dim, page, window, sinks, starts given
SHAPES = [
    # one token of one place; then lengths around a stage, a page and a part
    ([(1, 1)], 1, 1, 64, 16, 0, 0, False),
    ([(2, 1), (31, 1), (32, 1), (33, 1), (63, 1), (64, 1), (65, 1), (127, 1), (700, 1)], 2, 4, 128, 16, 0, 0, False),
    ([(1000, 1)], 1, 1, 16, 24, 0, 0, False),
    ([(517, 1), (4000, 1)], 3, 5, 48, 7, 0, 0, False),
    ([(9000, 1)], 2, 16, 128, 64, 0, 0, False),
    ([(300, 1), (20, 1)], 2, 3, 256, 32, 0, 0, False),
    ([(260, 1), (77, 1)], 1, 8, 192, 50, 0, 0, False),
    ([(515, 1)], 2, 2, 80, 1, 0, 0, False),
    # windows and sinks on single tokens: wider than the sequence, of one place, sinks alone past the window
    ([(500, 1), (40, 1), (3, 1)], 2, 4, 64, 16, 100, 4, False),
    ([(900, 1), (65, 1)], 1, 4, 128, 16, 1, 0, False),
    ([(900, 1), (130, 1)], 1, 4, 128, 64, 1, 70, False),
    ([(5000, 1), (1, 1)], 2, 8, 96, 32, 1024, 5, False),
    # a few tokens: 2 to 64 rows of a head
    ([(40, 2), (2, 2), (333, 2)], 2, 4, 128, 16, 0, 0, False),
    ([(300, 5), (5, 5)], 2, 5, 64, 16, 0, 0, False),
    ([(701, 7), (20, 7)], 1, 8, 128, 64, 50, 3, False),
    ([(513, 60), (60, 60)], 1, 1, 128, 64, 0, 0, False),
    ([(200, 30)], 2, 2, 256, 64, 0, 0, False),
    # prompts: whole, after a context, with windows; odd groups and widths
    ([(64, 64)], 1, 4, 64, 64, 0, 0, False),
    ([(257, 257), (1030, 257)], 2, 4, 128, 64, 0, 0, False),
    ([(129, 129)], 1, 7, 96, 16, 0, 0, False),
    ([(300, 300)], 1, 3, 256, 32, 0, 0, False),
    ([(200, 200)], 2, 1, 160, 50, 0, 0, False),
    ([(700, 300), (300, 300)], 1, 4, 128, 64, 64, 0, False),
    ([(700, 300), (2000, 300)], 1, 4, 80, 24, 130, 9, False),
    ([(600, 600)], 1, 2, 64, 16, 1, 1, False),
    # ragged: prompts beside single tokens and sequences without new ones
    ([(100, 37), (1, 1), (800, 1), (50, 0), (333, 333), (0, 0), (64, 64), (65, 2)], 2, 4, 128, 16, 0, 0, True),
    ([(100, 37), (1, 1), (800, 1), (50, 0), (333, 200), (0, 0), (64, 64), (65, 2)], 1, 6, 64, 64, 40, 5, True),
    ([(9, 1)] * 70 + [(200, 150)] + [(30, 1)] * 70, 1, 2, 64, 16, 0, 0, True),
    ([(3, 1), (70, 1), (2000, 2), (11, 0), (500, 1)], 2, 2, 128, 16, 0, 0, True),
]


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda t: f"{len(t[0])}x{t[0][-1]}_{'_'.join(map(str, t[1:]))}".replace(" ", ""))
def test_against_the_definition(shape, types):
    seqs, heads, group, dim, page, window, sinks, starts = shape
    dtype, cdt = types
    s = Setup(seqs, heads, dim, page, dtype, cdt, seed=len(seqs) + dim, order="token" if page == 16 else "head")
    s.write()
    q = (1.5 * torch.randn(s.tokens, heads * group, dim, generator=gen(5), device=DEV)).to(dtype)
    y = attend(s, q, window, sinks, starts)
    torch.cuda.synchronize()
    compare(s, q, y, window, sinks)
    # the same bits with every guide, and again
    for longest in (None, 1, max(n for n, _ in seqs)):
        z = attend(s, q, window, sinks, True, max_len=longest)
        torch.cuda.synchronize()
        compare(s, q, z, window, sinks, name=f"max_len {longest}")
        assert torch.equal(z, attend(s, q, window, sinks, True, max_len=longest))


def random_tree(n, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    sees = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        parent = i - 1 - int(torch.randint(0, min(i, 5) + 1, (1,), generator=g))
        if parent >= 0:
            sees[i] = sees[parent]
        sees[i, i] = True
    return sees


TREES = [
    ([(20, 4), (4, 4)], 1, 1, 64, 16, 0, 0), ([(300, 8), (8, 8), (70, 8)], 2, 2, 128, 64, 0, 0),
    ([(1000, 26), (150, 26)], 2, 4, 128, 64, 0, 0), ([(500, 64), (64, 64)], 1, 4, 96, 16, 0, 0),
    ([(300, 65), (129, 65)], 1, 2, 64, 24, 0, 0), ([(400, 130), (131, 130)], 1, 1, 128, 64, 0, 0),
    ([(200, 20), (60, 20)], 1, 4, 128, 16, 30, 4), ([(200, 40), (41, 40)], 1, 2, 64, 64, 3, 2),
    ([(150, 100), (101, 100)], 1, 1, 64, 64, 4, 120), ([(33, 30), (30, 30)], 2, 1, 256, 16, 2, 5),
]


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", TREES, ids=lambda t: f"{t[0][0]}_{'_'.join(map(str, t[1:]))}".replace(" ", ""))
def test_trees_against_the_definition(shape, types):
    seqs, heads, group, dim, page, window, sinks = shape
    dtype, cdt = types
    s = Setup(seqs, heads, dim, page, dtype, cdt, seed=dim + 1)
    s.write()
    q = (1.5 * torch.randn(s.tokens, heads * group, dim, generator=gen(6), device=DEV)).to(dtype)
    n = seqs[0][1]
    trees = [random_tree(n, 10 + b) for b in range(len(seqs))]
    # a chain too, whose window drops its own first nodes, and a matrix of any bits, with rows that see no node
    loose = torch.rand(n, n, generator=torch.Generator().manual_seed(3)) < 0.3
    loose[n // 2] = False
    for sees in (trees, [torch.ones(n, n, dtype=torch.bool).tril()] * len(seqs), [loose] * len(seqs)):
        for words in {(n + 63) // 64, (n + 63) // 64 + 1}:
            t = torch.cat([tree_bits(x, words) for x in sees])
            for flag in (True, False):
                y = attend(s, q, window, sinks, flag, tree=t[:, 0].contiguous() if words == 1 else t)
                torch.cuda.synchronize()
                compare(s, q, y, window, sinks, sees)


def test_ragged_trees():
    seqs = [(50, 5), (300, 0), (90, 70), (3, 3), (400, 1)]
    s = Setup(seqs, 2, 64, 16, BF16, BF16, seed=2)
    s.write()
    q = torch.randn(s.tokens, 4, 64, generator=gen(7), device=DEV).to(BF16)
    sees = [random_tree(n, n) for _, n in seqs]
    t = torch.cat([tree_bits(x, 2) for x in sees])
    # bits of nodes that a sequence does not have count as not set
    t[0, 0] |= 1 << 40
    t[0, 1] = -1
    y = attend(s, q, tree=t)
    torch.cuda.synchronize()
    compare(s, q, y, sees=sees)


def test_a_chain_is_the_causal_order():
    s = Setup([(300, 20), (40, 20)], 2, 128, 16, BF16, E4M3, seed=3)
    s.write()
    q = torch.randn(s.tokens, 8, 128, generator=gen(8), device=DEV).to(BF16)
    t = torch.cat([tree_bits(torch.ones(20, 20, dtype=torch.bool).tril(), 1)] * 2)
    for window, sinks in ((0, 0), (25, 3), (4, 2)):
        assert torch.equal(attend(s, q, window, sinks), attend(s, q, window, sinks, tree=t)), (window, sinks)


@pytest.mark.parametrize("tree", [False, True], ids=["causal", "tree"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("new,group", [(3, 4), (20, 3), (90, 4)])
def test_tokens_that_see_nothing_give_zeros(new, group, types, tree):
    """More new tokens than places in use: the first lie before the sequence."""
    dtype, cdt = types
    s = Setup([(new, new)] * 2, 2, 64, 16, dtype, cdt, seed=4)
    s.write()
    q = torch.randn(2 * new, 2 * group, 64, generator=gen(9), device=DEV).to(dtype)
    s.lens = ints([new - 2, 0])
    t = tree_bits(torch.zeros(2 * new, 2 * new, dtype=torch.bool), 3) if tree else None
    y = attend(s, q, starts=False, tree=t)
    torch.cuda.synchronize()
    assert bool((y[new:] == 0).all())
    assert bool((y[:2] == 0).all())
    assert bool(y.isfinite().all())
    if tree:
        assert bool((y == 0).all())
    else:
        assert bool((y[2:new] != 0).any(dim=2).all())


@pytest.mark.parametrize("types", TYPES[:2] + [(BF16, E4M3)], ids=IDS[:3])
@pytest.mark.parametrize("new,group", [(1, 4), (4, 4), (30, 2), (60, 1), (200, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_what_is_not_finite_counts_where_it_is_seen(new, group, types, window, sinks):
    dtype, cdt = types
    length = 300
    s = Setup([(length, new), (length, new)], 1, 128, 64, dtype, cdt, seed=6)
    bad = [float("nan")] if cdt == E4M3 else [float("nan"), float("inf"), float("-inf")]
    g = torch.Generator().manual_seed(new)
    for b in range(2):
        for _ in range(9):
            at = int(torch.randint(0, length, (1,), generator=g))
            s.v[b][at, 0, int(torch.randint(0, 128, (1,), generator=g))] = bad[at % len(bad)]
        # the last token's key is not finite: only it sees that
        s.k[b][length - 1, 0, 5] = bad[0]
    s.write()
    q = torch.randn(s.tokens, group, 128, generator=gen(10), device=DEV).to(dtype)
    y = attend(s, q, window, sinks)
    torch.cuda.synchronize()
    for b in range(2):
        assert bool(y[s.first[b + 1] - 1].isnan().all())
    keep = [t for b in range(2) for t in range(s.first[b], s.first[b + 1] - 1)]
    for b in range(2):
        if new == 1:
            continue
        k, v = s.held(b)
        k = torch.where(k.isfinite(), k, torch.zeros_like(k))
        see = seen_causal(length, new, window, sinks)[:-1]
        qb = q[s.first[b]:s.first[b + 1] - 1]
        ref, size = attention64(qb, k, v, see, 128 ** -0.5)
        tol = tolerance(torch.where(ref.isfinite(), ref, torch.zeros_like(ref)), size, qb, k, length, dtype, 128 ** -0.5)
        check_sequence(b, y[s.first[b]:s.first[b + 1] - 1].double(), ref, tol)
    say(f"  {len(keep)} tokens kept apart")


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("new", [1, 3, 100])
def test_scores_far_apart(new, types):
    """Weights that fall by hundreds of powers of two, and maxima that grow all along."""
    dtype, cdt = types
    s = Setup([(700, new)], 1, 64, 16, dtype, cdt, seed=7)
    ramp = torch.linspace(0.01, 6, 700, device=DEV)[:, None, None]
    s.k[0] = (torch.ones(700, 1, 64, device=DEV) * ramp + 0.01 * s.k[0].float()).to(dtype)
    s.write()
    for sign in (1.0, -1.0):
        q = (sign * 3 * torch.ones(new, 4, 64, device=DEV)).to(dtype)
        y = attend(s, q)
        torch.cuda.synchronize()
        compare(s, q, y)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 3.0])
def test_scale(scale):
    s = Setup([(333, 2)], 2, 64, 16, BF16, BF16, seed=8)
    s.write()
    q = torch.randn(2, 4, 64, generator=gen(11), device=DEV).to(BF16)
    y = attend(s, q, scale=scale)
    torch.cuda.synchronize()
    compare(s, q, y, scale=scale)


@pytest.mark.parametrize("new", [1, 40, 300])
def test_strides_and_rows_that_belong_to_nobody(new):
    seqs = [(400, new), (350, new)]
    s = Setup(seqs, 2, 96, 64, BF16, BF16, seed=9, order="token", extra=3)
    s.write()
    base = torch.randn(s.tokens + 7, 5 * 96 + 3, generator=gen(12), device=DEV).to(BF16)
    q = base[:, 1:1 + 4 * 96].view(s.tokens + 7, 4, 96)  # rows off 16 bytes, inside wider ones
    out = torch.full((4, s.tokens + 7, 98), 7.0, dtype=BF16, device=DEV).transpose(0, 1)[:, :, 1:97]
    starts = s.starts + 2
    got = ct.kv_attention(q, s.cache, s.lens, s.table, starts, out=out)
    torch.cuda.synchronize()
    assert got is out
    compare(s, q[2:2 + s.tokens], out[2:2 + s.tokens])
    assert bool((out[:2] == 7).all()) and bool((out[2 + s.tokens:] == 7).all())
    whole = out.transpose(0, 1)
    assert bool((torch.as_strided(whole, (4, s.tokens + 7, 1), (98 * (s.tokens + 7), 98, 1), 0) == 7).all())


def test_without_a_table():
    """A page a sequence."""
    s = Setup([(90, 1), (100, 1), (1, 1)], 2, 64, 100, F16, F16, seed=10, tables=False)
    s.write()
    q = torch.randn(3, 8, 64, generator=gen(13), device=DEV).to(F16)
    y = attend(s, q, starts=False)
    torch.cuda.synchronize()
    compare(s, q, y)


@pytest.mark.parametrize("new", [1, 70])
def test_pages_that_do_not_exist_are_read_as_the_first(new):
    s = Setup([(300, new)], 1, 64, 16, BF16, BF16, seed=11, filler=0.0)
    s.write()
    q = torch.randn(new, 4, 64, generator=gen(14), device=DEV).to(BF16)
    for bad in (-1, s.cache.pages, 2 ** 31 - 1, -2 ** 31):
        table = s.table.clone()
        table[0, 3] = bad
        first = s.table.clone()
        first[0, 3] = 0
        a = ct.kv_attention(q, s.cache, s.lens, table)
        b = ct.kv_attention(q, s.cache, s.lens, first)
        torch.cuda.synchronize()
        assert torch.equal(a, b), bad


def test_counts_that_do_not_fit_lead_nowhere():
    """Lengths past the table, starts out of order or past the tokens: other
    sequences keep their results."""
    s = Setup([(100, 2), (90, 2), (80, 2)], 1, 64, 16, BF16, BF16, seed=12, filler=0.0)
    s.write()
    q = torch.randn(6, 4, 64, generator=gen(15), device=DEV).to(BF16)
    good = attend(s, q)
    for lens in ([100, 2 ** 31 - 1, 80], [100, -5, 80], [100, 10 ** 6, 80]):
        y = ct.kv_attention(q, s.cache, ints(lens), s.table, s.starts)
        torch.cuda.synchronize()
        assert torch.equal(y[:2], good[:2]) and torch.equal(y[4:], good[4:]), lens
    guard = torch.full((10, 4, 64), 5.0, dtype=BF16, device=DEV)
    for starts in ([0, 2, 10 ** 6, 6], [-3, 2, 4, 2 ** 31 - 1], [0, 2, -7, 6]):  # the last gives rows to two sequences
        out = guard.clone()
        ct.kv_attention(q, s.cache, s.lens, s.table, ints(starts), out=out[2:8])
        torch.cuda.synchronize()
        assert torch.equal(out[:2], guard[:2]) and torch.equal(out[8:], guard[8:]), starts
        if starts[2] >= 0:
            assert torch.equal(out[2:4], good[:2]), starts


def test_far_places_of_a_large_pool():
    """Rows past 2^32 bytes of the pool, keys past 2^31 bytes of a head's stride."""
    pages, heads, page, dim = 70000, 4, 64, 128
    cache = ct.KVCache.empty(pages, heads, page, dim, dtype=F16)
    g = gen(16)
    table = ints([[69999, 5, 40000, 69000]])
    lens = ints([250])
    k, v = (torch.randn(250, heads, dim, generator=g, device=DEV).to(F16) for _ in range(2))
    for t in (cache.k, cache.v):
        for p in (69999, 5, 40000, 69000):
            t[p].fill_(float("nan"))
    ct.kv_write(cache, k, v, lens, table)
    rk, rv = ct.kv_read(cache, 250, lens, table)
    torch.cuda.synchronize()
    assert torch.equal(rk, k) and torch.equal(rv, v)
    for new in (1, 130):
        q = torch.randn(new, 8, dim, generator=g, device=DEV).to(F16)
        y = ct.kv_attention(q, cache, lens, table)
        torch.cuda.synchronize()
        ref, size = attention64(q, k.double(), v.double(), seen_causal(250, new, 0, 0), dim ** -0.5)
        check_sequence(new, y.double(), ref, tolerance(ref, size, q, k.double(), 250, F16, dim ** -0.5))


@pytest.mark.parametrize("cdt", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_a_prompt_in_chunks_and_tokens_one_by_one(cdt):
    """As a program serves: a prompt in chunks, then single tokens, each written
    and then attended; against the whole sequence at once, in 64 bits."""
    heads, group, dim, page = 2, 4, 128, 16
    total = 330
    s = Setup([(total, total)], heads, dim, page, BF16, cdt, seed=17)
    q = torch.randn(total, heads * group, dim, generator=gen(18), device=DEV).to(BF16)
    y = torch.empty_like(q)
    at = 0
    for n in [150, 96, 50] + [1] * 20 + [5] + [1] * 9:
        lens = ints([at + n])
        ct.kv_write(s.cache, s.k[0][at:at + n], s.v[0][at:at + n], lens, s.table)
        ct.kv_attention(q[at:at + n], s.cache, lens, s.table, out=y[at:at + n])
        at += n
    torch.cuda.synchronize()
    assert at == total
    compare(s, q, y)


@pytest.mark.parametrize("new", [1, 26])
@pytest.mark.parametrize("cdt", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_a_captured_step_follows_its_inputs(new, cdt):
    """Lengths, tables and rows are read at every replay; two graphs replayed
    at once keep apart."""
    seqs = [(900, new), (500, new), (40, new)]
    runs = []
    for seed in (19, 20):
        s = Setup(seqs, 2, 128, 64, BF16, cdt, seed=seed, filler=0.0)
        s.write()
        runs.append(dict(s=s, q=torch.randn(s.tokens, 8, 128, generator=gen(seed), device=DEV).to(BF16),
                         k=torch.randn(s.tokens, 2, 128, generator=gen(seed + 2), device=DEV).to(BF16),
                         lens=s.lens.clone(), stream=torch.cuda.Stream()))
    torch.cuda.synchronize()

    def step(r):
        ct.kv_write(r["s"].cache, r["k"], r["k"], r["lens"], r["s"].table)
        return ct.kv_attention(r["q"], r["s"].cache, r["lens"], r["s"].table, window=600, sinks=3)

    for r in runs:
        with torch.cuda.stream(r["stream"]):
            step(r)
            r["stream"].synchronize()
            r["graph"] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(r["graph"], stream=r["stream"]):
                r["y"] = step(r)
    torch.cuda.synchronize()
    for turn in range(4):
        for i, r in enumerate(runs):
            r["lens"].copy_(r["s"].lens - ints([turn, 3 * turn, 0]))
            r["q"].copy_(torch.randn(r["q"].shape, generator=gen(100 + 2 * turn + i), device=DEV).to(BF16))
            r["k"].mul_(-1)
        torch.cuda.synchronize()
        for r in runs:
            with torch.cuda.stream(r["stream"]):
                r["graph"].replay()
        torch.cuda.synchronize()
        for r in runs:
            got = r["y"].clone()
            want = step(r)
            torch.cuda.synchronize()
            assert torch.equal(got, want), turn


def test_another_stream():
    s = Setup([(2000, 1)], 2, 128, 64, BF16, BF16, seed=21)
    s.write()
    q = torch.randn(1, 8, 128, generator=gen(22), device=DEV).to(BF16)
    want = attend(s, q, starts=False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ct.kv_attention(q, s.cache, s.lens, s.table, stream=side)
    raw = ct.kv_attention(q, s.cache, s.lens, s.table, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)


def test_a_block_step():
    """The attention half of a block in the library's own calls, 8-bit cache: norm,
    fused projection, cache, attention, output projection onto the residual.
    Against 64 bits from the same 16-bit intermediate values; what remains is
    the output projection's sum (derived in test_gpu_block.py) on rows of
    attention that are themselves within their tolerance."""
    heads, group, dim, page, B = 2, 4, 64, 16, 5
    hq, width = heads * group, 256
    g = gen(23)
    x = torch.randn(B, width, generator=g, device=DEV).to(BF16)
    wqkv = (torch.randn((hq + 2 * heads) * dim, width, generator=g, device=DEV) * width ** -0.5).to(BF16)
    wo = (torch.randn(width, hq * dim, generator=g, device=DEV) * (hq * dim) ** -0.5).to(BF16)
    seqs = [(30 * (b + 1), 1) for b in range(B)]
    s = Setup(seqs, heads, dim, page, BF16, E4M3, seed=24)
    s.write()
    n, _, _ = ct.rmsnorm(x)
    qkv = ct.linear(n, wqkv)
    q = qkv[:, :hq * dim].view(B, hq, dim)
    k = qkv[:, hq * dim:(hq + heads) * dim].view(B, heads, dim)
    v = qkv[:, (hq + heads) * dim:].view(B, heads, dim)
    ct.kv_write(s.cache, k, v, s.lens, s.table)
    a = ct.kv_attention(q, s.cache, s.lens, s.table)
    y = ct.linear(a.view(B, hq * dim), wo, residual=x)
    torch.cuda.synchronize()
    for b in range(B):
        s.k[b][-1], s.v[b][-1] = k[b], v[b]
    compare(s, q, a)
    ref = a.view(B, -1).double() @ wo.double().t().contiguous() + x.double()
    size = a.view(B, -1).double().abs() @ wo.double().abs().t().contiguous()
    tol = 2 * (hq * dim + 4) * 2.0 ** -24 * size + 2 * 2.0 ** -24 * ref.abs() + 2.0 ** -8 * ref.abs()
    assert bool(((y.double() - ref).abs() <= tol).all())
    assert math.isfinite(float(y.float().sum()))


@pytest.mark.parametrize("new", [1, 40])
def test_pages_and_rows_that_are_shared(new):
    """Two sequences with one prefix's pages, and queries that are one row seen
    several times (no distance between tokens)."""
    s = Setup([(300, new), (300, new)], 2, 64, 16, BF16, E4M3, seed=25)
    shared = (300 - new) // 16
    s.table[1, :shared] = s.table[0, :shared]
    for x in (s.k, s.v):
        x[1][:shared * 16] = x[0][:shared * 16]
    s.write()  # both write the shared pages, with the same rows
    q = torch.randn(1, 8, 64, generator=gen(26), device=DEV).to(BF16).expand(2 * new, 8, 64)
    y = attend(s, q)
    torch.cuda.synchronize()
    compare(s, q, y)


@pytest.mark.parametrize("types", [(F16, E4M3), (F16, F16)], ids=["f16-e4m3", "f16"])
@pytest.mark.parametrize("new", [1, 50])
def test_rows_at_the_end_of_the_range(new, types):
    """Keys and values up to 60000 in fp16, whose codes stand for up to 61440; and
    rows near the least that fp16 holds."""
    dtype, cdt = types
    for size, qsize in ((60000.0, 3e-5), (1e-4, 60.0)):
        s = Setup([(200, new)], 1, 64, 16, dtype, cdt, seed=27)
        for x in (s.k, s.v):
            x[0].copy_((torch.rand(x[0].shape, generator=gen(28), device=DEV) * 2 - 1) * size)
            x[0][:, :, 0] = size
        s.write()
        q = (torch.randn(new, 4, 64, generator=gen(29), device=DEV) * qsize).to(dtype)
        y = attend(s, q)
        torch.cuda.synchronize()
        if size < 1 and cdt == E4M3:
            # Codes widen to half their value, which fp16 rounds by up to 2^-25 there: 2^-24 of
            # a value.  A score is off by 64 / 8 max |q| of those, a weight and their sum by a
            # factor of that each, the result by one more of V's own.
            k, v = s.held(0)
            ref, weight = attention64(q, k, v, seen_causal(200, new, 0, 0), 64 ** -0.5)
            off = 2.0 ** -24 * (1 + 2 * 8 * float(q.abs().max()) * weight)
            check_sequence(new, y.double(), ref, tolerance(ref, weight, q, k, 200, dtype, 64 ** -0.5) + off)
        else:
            compare(s, q, y)


def test_many_sequences():
    """20000 sequences, most of one token, counted through by every workgroup."""
    n = 20000
    lengths = [1 + (i * 7) % 5 for i in range(n)]
    new = [1 if i % 1000 else min(3, lengths[i]) for i in range(n)]
    k = torch.randn(n, 1, 8, 64, generator=gen(30), device=DEV).to(BF16)
    v = torch.randn(n, 1, 8, 64, generator=gen(31), device=DEV).to(BF16)
    cache = ct.KVCache(k, v)
    first = [0]
    for c in new:
        first.append(first[-1] + c)
    q = torch.randn(first[-1], 2, 64, generator=gen(32), device=DEV).to(BF16)
    y = ct.kv_attention(q, cache, ints(lengths), starts=ints(first))
    torch.cuda.synchronize()
    for i in [0, 1, 2, 63, 64, 999, 1000, 1001, 12000, 19998, 19999]:
        kk, vv = (t[i, :, :lengths[i]].transpose(0, 1).double() for t in (k, v))
        qi = q[first[i]:first[i + 1]]
        ref, size = attention64(qi, kk, vv, seen_causal(lengths[i], new[i], 0, 0), 64 ** -0.5)
        check_sequence(i, y[first[i]:first[i + 1]].double(), ref, tolerance(ref, size, qi, kk, lengths[i], BF16, 64 ** -0.5))
