"""A key-value cache in pages for the tests, and attention over it in 64 bits
from its definition: every tensor laid out from a list of sequences."""
from __future__ import annotations

import torch

from tensor_compiler_tiling_amd import convtile as ct

from _gpu_helpers import DEV

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def codes_of(v):
    """Rows of v (64 bits) as the values of their e4m3 codes, and their scales."""
    a = torch.where(v.isfinite(), v.abs(), torch.zeros_like(v)).amax(dim=-1).clamp_min(2.0 ** -100)
    s = torch.exp2(torch.floor(torch.log2(a)) - 8)
    s = torch.where(a > 448 * s, 2 * s, s)
    s = torch.where(a <= 224 * s, s / 2, s)
    assert bool((a <= 448 * s).all()) and bool((a > 224 * s).all())
    return (v / s[..., None]).float().to(E4M3), s.float()


class Setup:
    """Sequences of (length, new) tokens with keys and values of their own in
    `dtype`, in pages of a pool whose other places hold `filler`."""

    def __init__(self, seqs, heads, dim, page, dtype, cache_dtype, seed=0, order="head", tables=True, filler=float("nan"),
                 extra=0):
        g = gen(seed)
        self.seqs, self.heads, self.dim, self.page = seqs, heads, dim, page
        self.dtype, self.cache_dtype = dtype, cache_dtype
        width = max(1, max((n + page - 1) // page for n, _ in seqs)) + extra
        pages = len(seqs) * width + 2
        if not tables:
            assert width == 1
        shape = (pages, heads, page, dim) if order == "head" else (pages, page, heads, dim)

        def pool(shape, dt):
            t = torch.full(shape, filler, dtype=F32, device=DEV).to(dt)
            return t if order == "head" else t.transpose(1, 2)

        scales = [pool(shape[:3], F32) for _ in range(2)] if cache_dtype == E4M3 else [None, None]
        self.cache = ct.KVCache(pool(shape, cache_dtype), pool(shape, cache_dtype), *scales)
        self.table = torch.randperm(pages, generator=g, device=DEV)[:len(seqs) * width].view(len(seqs), width).to(torch.int32)
        if not tables:
            self.table = None
        self.lens = ints([n for n, _ in seqs])
        first = [0]
        for _, n in seqs:
            first.append(first[-1] + n)
        self.first, self.tokens = first, first[-1]
        self.starts = ints(first)
        self.k = [torch.randn(n, heads, dim, generator=g, device=DEV).to(dtype) for n, _ in seqs]
        self.v = [torch.randn(n, heads, dim, generator=g, device=DEV).to(dtype) for n, _ in seqs]

    def write(self):
        """All tokens, by the library: sequences as if every token were new."""
        n = [x for x, _ in self.seqs]
        starts = ints([sum(n[:i]) for i in range(len(n) + 1)])
        ct.kv_write(self.cache, torch.cat(self.k), torch.cat(self.v), self.lens, self.table, starts)

    def held(self, b):
        """What the cache stands for: keys and values of sequence b in 64 bits."""
        out = []
        for x in (self.k[b], self.v[b]):
            if self.cache_dtype == E4M3:
                q, s = codes_of(x.double())
                out.append(q.double() * s.double()[..., None])
            else:
                out.append(x.to(self.cache_dtype).double())
        return out


def seen_causal(length, new, window, sinks):
    """[new, length]: which places the tokens see."""
    at = torch.arange(length - new, length, device=DEV)[:, None]
    j = torch.arange(length, device=DEV)[None]
    see = j <= at
    if window:
        see &= (j > at - window) | (j < sinks)
    return see


def seen_tree(length, new, window, sinks, sees):
    """The same for drafted nodes; sees [new, new] on the host."""
    ctx = length - new
    out = torch.zeros(new, length, dtype=torch.bool)
    for i in range(new):
        nodes = [j for j in range(new) if bool(sees[i, j])]
        place = ctx + len(nodes) - 1
        for j in range(ctx):
            out[i, j] = not window or j > place - window or j < sinks
        for rank, j in enumerate(nodes):
            at = ctx + rank
            out[i, ctx + j] = not window or at > place - window or at < sinks
    return out.to(DEV)


def tree_bits(sees, words):
    """Rows of int64 words from sees [n, n] on the host."""
    n = sees.shape[0]
    bits = torch.zeros(n, words * 64, dtype=torch.int64)
    bits[:, :n] = sees.to(torch.int64)
    w = torch.ones(64, dtype=torch.int64) << torch.arange(64)
    return (bits.view(n, words, 64) * w).sum(dim=2).to(DEV)


def attention64(q, k, v, see, scale):
    """y and the size that errors are measured by, sum w |v| / sum w, of one
    sequence: q [n, heads * group, dim], k and v [length, heads, dim] in 64 bits.
    Values that are not finite count where they are seen, and only there."""
    n, hq, d = q.shape
    length, h, _ = k.shape
    g = hq // h
    fin = torch.where(v.isfinite(), v, torch.zeros_like(v))
    y = torch.zeros(n, hq, d, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(y)
    if length == 0:
        return y, size
    for j in range(h):
        x = q[:, j * g:(j + 1) * g].reshape(n * g, d).double()
        z = (x @ k[:, j].t().contiguous() * scale).view(n, g, length)
        z = z.masked_fill(~see[:, None], float("-inf"))
        top = z.amax(dim=2, keepdim=True)
        w = torch.exp(z - torch.where(top == float("-inf"), torch.zeros_like(top), top))
        total = w.sum(dim=2, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
        yj = (w.view(n * g, length) @ fin[:, j].contiguous()).view(n, g, d)
        size[:, j * g:(j + 1) * g] = (w.view(n * g, length) @ fin[:, j].abs().contiguous()).view(n, g, d)
        s = see.double()
        for bad, value in ((v[:, j].isnan(), float("nan")), (v[:, j] == float("inf"), float("inf")),
                           (v[:, j] == float("-inf"), float("-inf"))):
            hit = (s @ bad.double().contiguous() > 0)[:, None].expand(n, g, d)
            yj = torch.where(hit, yj + value, yj)
        y[:, j * g:(j + 1) * g] = yj
    return y, size


def tolerance(y, size, q, k, length, dtype, scale):
    """How far a result may be off (u = 2^-24, half a step of the type: h).

    - a score is a sum of dim products, exact in fp32, each addition off by at
      most 2 u of the partial sum: 2 (dim + 4) u scale sum |q k|; times log2 e,
      less the maximum (one rounding each, of values up to |z|): 4 u |z|.  With
      both at most e, a weight is off by a factor exp(e), and so is the sum of
      them: 2 e (1 + e) in all.  exp2 itself adds 2 u.
    - the weights are rounded to the type: h each, of sum w |v|.  In fp16 those
      below 2^-14 / 2^7 of the largest are off by up to 2^-32 of it instead.
    - the sums over `length` keys: 2 (length + 8) u each, in both.  Scalings by
      falling maxima and joins add 2 u for each 8 units of log2, at most 40 u.
    - the result's own rounding: h of it (2^-25 at least in fp16).
    """
    half = torch.finfo(dtype).eps / 2
    dim = q.shape[2]
    # the sum of |q k| is at most the norms' product
    zz = scale * float(q.double().norm(dim=2).amax()) * float(k.norm(dim=2).amax()) if k.numel() else 0.0
    e = (2 * (dim + 4) + 4 * 1.45) * U * zz
    rel = half + 2 * e * (1 + e) + 2 * U + 4 * (length + 8) * U + 40 * U
    tiny = 2.0 ** -25 if dtype == F16 else 0.0
    return rel * size + half * y.abs() + tiny + length * 2.0 ** -32 * size.amax()


def check_sequence(name, got, y, tol):
    bad_ref, bad_got = ~y.isfinite(), ~got.isfinite()
    assert torch.equal(bad_ref, bad_got), (name, "not finite", int(bad_ref.sum()), int(bad_got.sum()))
    assert torch.equal(y.isnan(), got.isnan()), name
    fin = ~bad_ref
    inf = bad_ref & ~y.isnan()
    assert torch.equal(y[inf] > 0, got[inf] > 0), name
    over = ((got - y).abs() - tol)[fin]
    if over.numel():
        assert float(over.max()) <= 0, (name, "over tolerance by", float(over.max()), "of", float(tol[fin].max()))
