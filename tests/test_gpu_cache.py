"""The quantized key-value cache on the GPU: writes and reads bit for bit against the oracle, attention
against a plain evaluation in 64 bits within bounds that are derived below."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
FORMATS = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 64), (256, 64), (256, 128), (256, 256)]
NBITS = [2, 4, 8]


@pytest.fixture(scope="module")
def hq():
    import weight_quantization_group_amd as hq

    hq.load_cache_library()
    return hq


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------

def bits16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def oracle_rows(x, nbits, gs):
    """(packed, scale, zero) of rows x [n, dim] by the oracle: the solve at 0 iterations."""
    kw = dict(iters=0)
    if x.dtype == torch.bfloat16:
        return oracle.quantize(bits16(x), nbits, gs, 1, dtype="bf16", **kw)
    return oracle.quantize(bits16(x), nbits, gs, 1, **kw)


def slot_rows(cache, side, slots):
    """The cache's (packed, scale, zero) of slots, as rows [tokens * heads, ...]."""
    page, place = slots // cache.page_size, slots % cache.page_size
    return [t[page, :, place].flatten(0, 1) for t in side]


def check_written(cache, K, V, slots):
    for side, x in ((cache.k, K), (cache.v, V)):
        packed, scale, zero = (t.cpu().numpy() for t in slot_rows(cache, side, slots))
        want = oracle_rows(x.reshape(-1, cache.dim), cache.nbits, cache.group_size)
        assert np.array_equal(scale, want[1])
        assert np.array_equal(zero, want[2])                   # by value: +0 and -0 alike
        assert np.array_equal(packed.view(np.uint32), want[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nbits", NBITS)
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_write_and_read_every_format(hq, dim, gs, nbits, dtype):
    dt, g = DTYPES[dtype], rng(dim + gs + nbits)
    heads, tokens = 3, 29
    c = hq.QuantizedCache.empty(5, 16, heads, dim, nbits, gs)
    slots = torch.randperm(80, device="cuda", generator=g)[:tokens]
    K = (torch.randn(tokens, heads, dim, device="cuda", generator=g) * 3).to(dt)
    V = torch.randn(tokens, heads, dim, device="cuda", generator=g).to(dt)
    back = hq.hqq_cache_write(c, K, V, slots, values=True)
    check_written(c, K, V, slots)
    K2, V2 = hq.hqq_cache_read(c, slots, dtype=dt)
    for side, got, again in ((c.k, K2, back[0]), (c.v, V2, back[1])):
        packed, scale, zero = (t.contiguous() for t in slot_rows(c, side, slots))
        want = hq.hqq_dequantize(packed, scale, zero, tokens * heads, dim, nbits, gs, 1, dtype=dt)
        assert torch.equal(got.view(-1, dim), want) and torch.equal(again, got)
        np_want = oracle.dequantize(packed.cpu().numpy().view(np.uint32), scale.cpu().numpy(), zero.cpu().numpy(),
                                    tokens * heads, dim, nbits, gs, 1, dtype="bf16" if dt == torch.bfloat16 else "f16")
        assert np.array_equal(bits16(got).reshape(-1, dim), np_want)


def edge_rows(dt, dim):
    """Groups that are constant, zero, tiny, huge, one value off, on the codes' half-way points."""
    t = torch.finfo(dt)
    rows = [torch.zeros(dim), -torch.zeros(dim), torch.full((dim,), 1.5), torch.full((dim,), -7.25),
            torch.linspace(-1, 1, dim), torch.arange(dim) % 2 * 1.0, (torch.arange(dim) % 31) * 0.5,
            torch.arange(dim) % 16 * 1.0 - 3, (torch.arange(dim) % 7) * 0.5 - 1.5,
            torch.where(torch.arange(dim) == 5, 1e4, 1e-3), torch.where(torch.arange(dim) == dim - 1, -1e4, 2.0),
            1000 + torch.arange(dim) % 3 * 1.0]
    if dt == torch.float16:
        rows += [torch.full((dim,), t.max) * torch.where(torch.arange(dim) % 2 == 0, 1.0, -1.0),
                 (torch.arange(dim) % 5) * 2.0 ** -24]
    else:
        rows += [torch.where(torch.arange(dim) % 2 == 0, 1e30, -1e30), (torch.arange(dim) % 5) * 2.0 ** -115]
    return torch.stack(rows).to(dt)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nbits", NBITS)
@pytest.mark.parametrize("dim,gs", [(64, 32), (128, 128), (256, 256)])
def test_write_edge_values(hq, dim, gs, nbits, dtype):
    x = edge_rows(DTYPES[dtype], dim).cuda()
    n = len(x)
    c = hq.QuantizedCache.empty(n, 16, 1, dim, nbits, gs)
    slots = torch.arange(n, device="cuda") * 16 + 3
    K, V = x[:, None], x.flip(0)[:, None].contiguous()
    back = hq.hqq_cache_write(c, K, V, slots, values=True)
    check_written(c, K, V, slots)
    got = hq.hqq_cache_read(c, slots, dtype=x.dtype)
    assert torch.equal(bits(got[0]), bits(back[0])) and torch.equal(bits(got[1]), bits(back[1]))
    constant = x.amax(1) == x.amin(1)
    assert torch.equal(got[0][constant, 0], x[constant])


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("tokens", [1, 2, 65, 700])
def test_write_parts_of_a_projection_and_skipped_tokens(hq, tokens):
    """K and V are cut from a wider tensor; tokens of slots outside the cache are skipped, and slots that no
    token names keep what they held, bit for bit."""
    g = rng(tokens)
    heads, dim, nbits, gs = 5, 96, 4, 32
    c = hq.QuantizedCache.empty(60, 16, heads, dim, nbits, gs)
    for side in (c.k, c.v):
        side[0].random_(-2 ** 31, 2 ** 31, generator=g)
        side[1].uniform_(0.5, 2, generator=g)
        side[2].uniform_(0, 15, generator=g)
    before = [t.clone() for t in c.k + c.v]
    wide = torch.randn(tokens, 3 * heads * dim + 8, device="cuda", generator=g).half()
    K = wide[:, 8 + heads * dim:8 + 2 * heads * dim].unflatten(1, (heads, dim))
    V = wide[:, 8 + 2 * heads * dim:].unflatten(1, (heads, dim))
    slots = torch.randperm(960, device="cuda", generator=g)[:tokens]
    bad = torch.tensor([-1, 960, -2 ** 63, 2 ** 63 - 1, 2 ** 40], device="cuda")
    skip = torch.rand(tokens, device="cuda", generator=g) < 0.2
    slots[skip] = bad[torch.randint(0, 5, (int(skip.sum()),), device="cuda", generator=g)]
    kept = ~skip
    back = hq.hqq_cache_write(c, K, V, slots, values=True)
    check_written(c, K[kept], V[kept], slots[kept])
    other = torch.ones(960, dtype=torch.bool, device="cuda")
    other[slots[kept]] = False
    for t, b in zip(c.k + c.v, before):
        assert torch.equal(t.transpose(1, 2).flatten(0, 1)[other], b.transpose(1, 2).flatten(0, 1)[other])
    got = hq.hqq_cache_read(c, slots)
    for i in range(2):
        assert torch.equal(got[i], back[i]) and not got[i][skip].any()


def test_heads_before_tokens(hq):
    """Any strides of tokens and heads: [heads, tokens, dim] seen as [tokens, heads, dim]."""
    g = rng(3)
    c, d = (hq.QuantizedCache.empty(4, 32, 4, 64, 8, 32) for _ in range(2))
    K, V = (torch.randn(4, 100, 64, device="cuda", generator=g).bfloat16().transpose(0, 1) for _ in range(2))
    slots = torch.arange(100, device="cuda")
    hq.hqq_cache_write(c, K, V, slots)
    hq.hqq_cache_write(d, K.contiguous(), V.contiguous(), slots)
    for a, b in zip(c.k + c.v, d.k + d.v):
        assert torch.equal(a, b)
    Q = torch.randn(4, 2, 64, device="cuda", generator=g).bfloat16().transpose(0, 1).repeat_interleave(2, 1)
    Q = torch.randn(8, 2, 64, device="cuda", generator=g).bfloat16().transpose(0, 1)
    table, n = torch.arange(4, device="cuda").int().expand(2, 4).contiguous(), torch.tensor([100, 7], device="cuda").int()
    a, b = hq.hqq_cache_attention(c, Q, table, n), hq.hqq_cache_attention(c, Q.contiguous(), table, n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_read_slots_twice_and_outside(hq):
    g = rng(4)
    c = hq.QuantizedCache.empty(6, 16, 2, 128, 2, 64)
    K, V = (torch.randn(96, 2, 128, device="cuda", generator=g).half() for _ in range(2))
    hq.hqq_cache_write(c, K, V, torch.arange(96, device="cuda"))
    all_k, all_v = hq.hqq_cache_read(c, torch.arange(96, device="cuda"))
    slots = torch.tensor([5, 5, 95, -1, 0, 96, 5, 2 ** 40, -2 ** 63, 17], device="cuda")
    inside = (slots >= 0) & (slots < 96)
    out = tuple(torch.full((10, 2, 128), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    got = hq.hqq_cache_read(c, slots, out=out)
    for t, every in zip(got, (all_k, all_v)):
        assert torch.equal(t[inside], every[slots[inside]]) and not t[~inside].any()
    assert got[0] is out[0]
    assert hq.hqq_cache_read(c, slots[:0])[0].shape == (0, 2, 128)
    fresh = hq.QuantizedCache.empty(6, 16, 2, 128, 2, 64)
    assert not hq.hqq_cache_read(fresh, torch.arange(96, device="cuda"))[0].any()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def decode(side, nbits, gs):
    """(codes, zero, 1 / scale) of rows [..., dim], 64 bits."""
    packed, scale, zero = side
    q = (packed.long()[..., None] >> torch.arange(0, 32, nbits, device=packed.device)) & ((1 << nbits) - 1)
    wide = lambda t: t.double().repeat_interleave(gs, -1)  # noqa: E731
    return q.flatten(-2).double(), wide(zero), 1.0 / wide(scale)


def reference(cache, Q, table, lengths, scale=None, window=0):
    """(out, lse) in 64 bits, and bounds of each one's error.

    With u = 2^-24 (half an fp32 step, relative), for a token t and group g of the keys
        s_t = scale * sum_g r (sum_d q c  -  z sum_d q):
    products of 11-bit q and codes are exact; every sum in fp32 has at most dim + 16 terms, and r, r z, the
    softmax scale and the exponent's argument add 8 roundings (1 / scale 2, its product with z, each group's
    scaling 2, the softmax scale 2, the argument 1), so
        |ds_t| <= (dim + 24) u scale sum_d |q| r (c + |z|)  +  4 u |s|max  =: d_t
    (q to 11 bits: fp16 is exact, bf16 too, down to 2^-31 of the row's largest, which the sum's own bound
    covers: dim 2^-31 < dim 2^-24 / 2).
    Weights: exp2 and its argument, 2^-22 together; the largest d: D.  Then
        |dlse| <= D + (n + 8) u + 2 u |lse|
        |dout| <= (2 D + 2^-21 + w) sum_t P_t r |c - z|  +  (n + 24) u sum_t P_t r (c + |z|) + half |out| + tiny
    with P the exact weights and w = 2^-11, the rounding of P r to 11 bits (fp16 outputs have a second operand for
    the rest, which the bound does not count on), with an exponent of its own down to 2^-25 of the largest or below,
    then absolute: `tiny` is 2^-29 of sum_t max(P r) (c + |z|)."""
    scale = 1.0 / math.sqrt(cache.dim) if scale is None else scale
    B, H, D = Q.shape
    G, u = H // cache.heads, 2.0 ** -24
    half = torch.finfo(Q.dtype).eps / 2
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * cache.page_size)
        t = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        page = table[b].long()[t // cache.page_size]
        there = (page >= 0) & (page < cache.pages)
        page, place = page[there], (t % cache.page_size)[there]
        if not len(page):
            continue
        for h in range(cache.heads):
            (kc, kz, kr), (vc, vz, vr) = (decode([a[page, h, place] for a in side], cache.nbits, cache.group_size)
                                          for side in (cache.k, cache.v))
            rows = slice(h * G, (h + 1) * G)
            q = Q[b, rows].double()
            S = q @ ((kc - kz) * kr).T * scale
            lse[b, rows] = torch.logsumexp(S, 1)
            P = torch.softmax(S, 1)
            v = (vc - vz) * vr
            out[b, rows] = P @ v
            d = (D + 24) * u * scale * (q.abs() @ (kr * (kc + kz.abs())).T) + 4 * u * S.abs().amax(1, keepdim=True)
            worst = d.amax(1, keepdim=True)
            tol_lse[b, rows] = worst[:, 0] + (len(t) + 8) * u + 2 * u * lse[b, rows].abs()
            mag = vr * (vc + vz.abs())
            tiny = 2.0 ** -29 * P.amax(1, keepdim=True) * vr.amax(0) * (vc + vz.abs()).sum(0)
            tol[b, rows] = (2 * worst + 2.0 ** -21 + 2.0 ** -11) * (P @ v.abs()) + (len(t) + 24) * u * (P @ mag) \
                + half * out[b, rows].abs() + tiny
    smallest = torch.finfo(Q.dtype).smallest_normal * torch.finfo(Q.dtype).eps
    return out, lse, tol + smallest, tol_lse


def check(cache, got, Q, table, lengths, **kw):
    out, lse, tol, tol_lse = reference(cache, Q, table, lengths, **kw)
    assert got[0].dtype == Q.dtype and got[0].shape == Q.shape and got[1].shape == Q.shape[:2]
    empty = lse == -math.inf
    assert torch.equal(got[1] == -math.inf, empty) and not got[0][empty].any()
    err = (got[1].double() - lse)[~empty].abs()
    assert bool((err <= tol_lse[~empty]).all()), float((err / tol_lse[~empty]).max())
    err = (got[0].double() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def filled(hq, g, pages, page_size, heads, dim, nbits, gs, spread=1.0):
    """A cache of random codes: scales of ranges around 1, zeros that put the values around 0."""
    def side():
        at = (pages, heads, page_size)
        packed = torch.randint(-2 ** 31, 2 ** 31, (*at, dim * nbits // 32), device="cuda", generator=g, dtype=torch.int64).int()
        qmax = (1 << nbits) - 1
        span = spread ** (2 * torch.rand(*at, dim // gs, device="cuda", generator=g) - 1) * 4
        zero = qmax * (0.5 + 0.3 * torch.randn(*at, dim // gs, device="cuda", generator=g))
        return packed, qmax / span, zero

    return hq.QuantizedCache(side(), side(), nbits, gs)


def batch_of(cache, g, dt, lengths, G, width=None, q=1.0):
    """Q, a table of distinct scattered pages (-1 past each length), lengths."""
    width = width or max(1, max(-(-n // cache.page_size) for n in lengths))
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(cache.pages, device="cuda", generator=g).int()
    at = 0
    for b, n in enumerate(lengths):
        k = -(-n // cache.page_size)
        table[b, :k] = free[at:at + k]
        at += k
    assert at <= cache.pages
    Q = (torch.randn(len(lengths), cache.heads * G, cache.dim, device="cuda", generator=g) * q).to(dt)
    return Q, table, torch.tensor(lengths, device="cuda").int()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nbits", NBITS)
@pytest.mark.parametrize("dim,gs", FORMATS)
def test_attention_every_format(hq, dim, gs, nbits, dtype):
    g = rng(dim * 3 + gs + nbits)
    c = filled(hq, g, 64, 16, 2, dim, nbits, gs)
    args = batch_of(c, g, DTYPES[dtype], [0, 1, 33, 300, 17, 128, 129], 3)
    check(c, hq.hqq_cache_attention(c, *args), *args)


@pytest.mark.parametrize("page_size", [16, 32, 64, 128, 256, 512, 1024])
def test_attention_lengths(hq, page_size):
    """Lengths at the edges of subtiles, tiles, workgroup steps and pages."""
    g = rng(page_size)
    lengths = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 1024, 1025, 1500]
    c = filled(hq, g, sum(-(-n // page_size) for n in lengths) + 2, page_size, 1, 128, 4, 64)
    args = batch_of(c, g, torch.float16, lengths, 2)
    check(c, hq.hqq_cache_attention(c, *args), *args)


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 15, 16, 17, 32, 40, 71])
@pytest.mark.parametrize("heads", [1, 3])
def test_attention_shared_heads(hq, G, heads):
    g = rng(G * 10 + heads)
    c = filled(hq, g, 40, 32, heads, 64, 8, 32)
    args = batch_of(c, g, torch.bfloat16, [200, 1, 450], G)
    check(c, hq.hqq_cache_attention(c, *args), *args)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 129, 500, 4000, 2 ** 40])
def test_attention_window(hq, window):
    g = rng(window % 1000)
    c = filled(hq, g, 300, 16, 2, 128, 8, 128)
    args = batch_of(c, g, torch.float16, [0, 1, 16, 100, 999, 1000, 513], 2)
    check(c, hq.hqq_cache_attention(c, *args, window=window), *args, window=window)


@pytest.mark.parametrize("scale", [0.5, 1e-3, 3.0])
def test_attention_scale(hq, scale):
    g = rng(6)
    c = filled(hq, g, 30, 16, 2, 96, 4, 32)
    args = batch_of(c, g, torch.float16, [100, 257], 4)
    check(c, hq.hqq_cache_attention(c, *args, softmax_scale=scale), *args, scale=scale)


@pytest.mark.parametrize("batch,length,heads,G", [(1, 20000, 1, 1), (1, 40001, 2, 5), (3, 9000, 4, 8), (70, 700, 2, 1),
                                                  (130, 300, 8, 2)])
def test_attention_split_over_the_length(hq, batch, length, heads, G):
    """Long sequences are cut into items and joined; batches of more than one wave's lanes are planned."""
    g = rng(batch)
    lengths = [length - (i * 37) % length for i in range(batch)]
    c = filled(hq, g, sum(-(-n // 64) for n in lengths), 64, heads, 64, 4, 64)
    args = batch_of(c, g, torch.float16, lengths, G)
    first = hq.hqq_cache_attention(c, *args)
    check(c, first, *args)
    again = hq.hqq_cache_attention(c, *args)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("batch,length,heads,G,dtype", [(70, 500, 40, 1, "fp16"), (3, 9000, 40, 2, "bf16"),
                                                        (200, 900, 16, 17, "bf16"), (1, 30000, 80, 1, "fp16")])
def test_attention_runs_that_cross_sequences(hq, batch, length, heads, G, dtype):
    """Many heads leave few runs to each, longer than a few steps: they go on from one sequence to the next,
    empty ones and single tokens among them."""
    g = rng(batch + heads)
    lengths = [max(0, length - (i * 131) % (length + 40)) for i in range(batch)]
    if batch > 3:
        lengths[1], lengths[2], lengths[-1] = 0, 1, 0
    c = filled(hq, g, sum(-(-n // 128) for n in lengths), 128, heads, 64, 4, 64)
    args = batch_of(c, g, DTYPES[dtype], lengths, G)
    got = hq.hqq_cache_attention(c, *args)
    some = torch.randperm(batch, device="cuda", generator=g)[:12].sort().values
    some = torch.unique(torch.cat([some, torch.tensor([0, min(1, batch - 1), batch - 1], device="cuda")]))
    rows = [t[some] for t in args]
    check(c, [t[some] for t in got], *rows)
    # and alone each sequence gives the same, within the rounding of another order of its sums
    one = some[0].item()
    alone = hq.hqq_cache_attention(c, *[t[one:one + 1] for t in args])
    check(c, alone, *[t[one:one + 1] for t in args])


@pytest.mark.parametrize("batch,most,heads,G,width", [
    (64, 40, 1, 1, 0), (65, 40, 1, 1, 0), (65, 900, 40, 1, 0), (128, 2000, 1, 3, 0), (129, 700, 4, 1, 0), (400, 60, 1, 1, 20), (1000, 60, 1, 2, 20),
    (1023, 200, 2, 1, 20), (1025, 130, 16, 2, 20), (4097, 100, 1, 1, 13), (5000, 33, 40, 1, 13)])
@pytest.mark.parametrize("long", [0, 9001])
def test_attention_many_sequences(hq, batch, most, heads, G, width, long):
    """The plan of more sequences than a wave's lanes, runs within sequences (many of them to a worker) and
    across: every row is written, and those of the first, the last, the longest and some others are right."""
    g = rng(batch + heads + long)
    lengths = torch.randint(0, most + 1, (batch,), generator=torch.Generator().manual_seed(batch)).tolist()
    lengths[0] = lengths[-1] = 0
    lengths[batch // 2], lengths[batch // 3] = most, long or most
    c = filled(hq, g, sum(-(-n // 64) for n in lengths), 64, heads, 64, 4, 32)
    args = batch_of(c, g, torch.bfloat16, lengths, G, width=max(width, -(-max(lengths) // 64)))
    got = torch.full_like(args[0], math.nan), torch.full(args[0].shape[:2], math.nan, device="cuda")
    hq.hqq_cache_attention(c, *args, out=got[0], lse=got[1])
    assert not got[0].isnan().any() and not got[1].isnan().any()
    some = torch.randperm(batch, device="cuda", generator=g)[:6].tolist() + [0, batch // 2, batch // 3, batch - 1]
    some = torch.tensor(sorted(set(some)), device="cuda")
    check(c, [t[some] for t in got], *[t[some] for t in args])
    again = hq.hqq_cache_attention(c, *args)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_attention_one_long_sequence_among_short_ones(hq):
    g = rng(7)
    lengths = [1, 0, 30000, 5, 0, 64, 129]
    c = filled(hq, g, 500, 64, 1, 128, 2, 32)
    args = batch_of(c, g, torch.bfloat16, lengths, 8)
    check(c, hq.hqq_cache_attention(c, *args), *args)
    assert torch.equal(args[2].cpu(), torch.tensor(lengths).int())


def test_attention_bad_pages_and_lengths(hq):
    """Tokens of a page outside the cache do not count; lengths outside the table are cut to it."""
    g = rng(8)
    c = filled(hq, g, 50, 16, 2, 128, 4, 64)
    Q, table, n = batch_of(c, g, torch.float16, [100, 100, 100, 100, 100, 100], 2, width=8)
    table[0, 0], table[1, 2], table[2, 6] = -1, 50, 2 ** 31 - 1
    table[3, :], table[4, 1:7:2] = -2 ** 31, 51
    got = hq.hqq_cache_attention(c, Q, table, n)
    check(c, got, Q, table, n)
    assert not got[0][3].any() and bool((got[1][3] == -math.inf).all())
    table[5, 7] = 3
    n = torch.tensor([100, -5, 128, 129, 2 ** 31 - 1, 10000], device="cuda").int()
    check(c, hq.hqq_cache_attention(c, Q, table, n), Q, table, n)


@pytest.mark.parametrize("window", [0, 40])
def test_attention_ignores_what_does_not_count(hq, window):
    """Infinities, NaN and zeros in the scales of tokens behind the last one, before the window and in
    other pages change nothing, bit for bit."""
    g = rng(9)
    for nbits, dim, gs, G in ((4, 128, 64, 4), (2, 96, 32, 1), (8, 64, 64, 20)):
        c = filled(hq, g, 60, 16, 2, dim, nbits, gs)
        Q, table, n = batch_of(c, g, torch.float16, [100, 1, 33, 250, 0], G)
        want = hq.hqq_cache_attention(c, Q, table, n, window=window)
        counts = torch.zeros(60 * 16, dtype=torch.bool, device="cuda")
        for b in range(5):
            t = torch.arange(max(0, int(n[b]) - window) if window else 0, int(n[b]), device="cuda")
            counts[table[b].long()[t // 16] * 16 + t % 16] = True
        poison = torch.tensor([math.inf, -math.inf, math.nan, 0.0, 1e-45, 3e38], device="cuda")
        for side in (c.k, c.v):
            for t in side[1:]:
                rows = t.transpose(1, 2).reshape(960, -1)
                rows[~counts] = poison[torch.randint(0, 6, rows[~counts].shape, device="cuda", generator=g)]
                t.copy_(rows.view(60, 16, 2, -1).transpose(1, 2))
        got = hq.hqq_cache_attention(c, Q, table, n, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_nan_and_infinity_stay_in_their_rows(hq):
    g = rng(10)
    c = filled(hq, g, 60, 16, 2, 128, 4, 64)
    Q, table, n = batch_of(c, g, torch.float16, [100, 333, 20], 4)
    want = hq.hqq_cache_attention(c, Q, table, n)
    Q[0, 1, 5], Q[1, 6, 100], Q[2, 0, 0] = math.nan, math.inf, -math.inf
    got = hq.hqq_cache_attention(c, Q, table, n)
    bad = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 6] = bad[2, 0] = True
    assert bool(got[0][bad].isnan().all()) and torch.equal(got[0][~bad], want[0][~bad])
    assert torch.equal(got[1][~bad], want[1][~bad]) and not bool(got[1][bad].isfinite().any())
    # a token's own: every head that reads it, no other
    Q, table, n = batch_of(c, g, torch.float16, [100, 333, 20], 4)
    want = hq.hqq_cache_attention(c, Q, table, n)
    c.v[1][table[1, 3], 1, 7, 0] = math.nan
    got = hq.hqq_cache_attention(c, Q, table, n)
    hit = torch.zeros_like(got[0], dtype=torch.bool)
    hit[1, 4:, :64] = True
    assert bool(got[0][hit].isnan().all()) and torch.equal(got[0][~hit], want[0][~hit])


@pytest.mark.parametrize("q", [1e-4, 30.0, 1e4])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_large_and_small(hq, dtype, q):
    """Scores far beyond fp16's range, or all alike; groups whose ranges differ by up to 2^20."""
    g = rng(11)
    for spread in (1.0, 1000.0):
        c = filled(hq, g, 80, 16, 2, 128, 4, 32, spread=spread)
        args = batch_of(c, g, DTYPES[dtype], [600, 5, 400], 4, q=q)
        check(c, hq.hqq_cache_attention(c, *args), *args)


def test_attention_bf16_beyond_fp16(hq):
    """Queries of 1e30 against keys of 1e-30, values of 1e30; a row of zeros and one of tiny values."""
    g = rng(12)
    c = filled(hq, g, 30, 16, 1, 128, 8, 64)
    c.k[1].mul_(1e30)
    c.v[1].mul_(1e-30)
    Q, table, n = batch_of(c, g, torch.bfloat16, [200, 100], 4)
    Q *= 1e30
    Q[0, 1] = 0.0
    Q[1, 2] = 1e-38
    check(c, hq.hqq_cache_attention(c, Q, table, n), Q, table, n)


def test_attention_constant_groups(hq):
    """Groups without a range (scale 1, zero -min) beside ordinary ones."""
    g = rng(13)
    c = hq.QuantizedCache.empty(20, 16, 2, 128, 4, 64)
    K, V = (torch.randn(300, 2, 128, device="cuda", generator=g).half() for _ in range(2))
    K[::3, :, :64] = 0.25
    V[::2, :, 64:] = -2.0
    V[5] = 0.0
    hq.hqq_cache_write(c, K, V, torch.arange(300, device="cuda"))
    Q = torch.randn(1, 6, 128, device="cuda", generator=g).half()
    table, n = torch.arange(20, device="cuda").int()[None], torch.tensor([300], device="cuda").int()
    check(c, hq.hqq_cache_attention(c, Q, table, n), Q, table, n)


def test_attention_does_not_depend_on_where_pages_are(hq):
    g = rng(14)
    c = filled(hq, g, 100, 16, 2, 128, 4, 64)
    Q, table, n = batch_of(c, g, torch.float16, [800, 333], 4)
    want = hq.hqq_cache_attention(c, Q, table, n)
    order = torch.randperm(100, device="cuda", generator=g)
    moved = hq.QuantizedCache(tuple(t[order].contiguous() for t in c.k), tuple(t[order].contiguous() for t in c.v), 4, 64)
    where = torch.argsort(order).int()
    got = hq.hqq_cache_attention(moved, Q, torch.where(table >= 0, where[table.clamp(min=0).long()], -1).int(), n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_far_pages(hq):
    """A cache whose codes take more than 2^32 bytes: the last pages are written, read and attended to."""
    pages, ps, heads, dim = 5000, 1024, 8, 128                 # 5.2e9 bytes of codes a side
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of device memory")

    def side():
        return (torch.empty(pages, heads, ps, dim // 4, dtype=torch.int32, device="cuda"),
                torch.empty(pages, heads, ps, 1, device="cuda"), torch.empty(pages, heads, ps, 1, device="cuda"))

    c, g = hq.QuantizedCache(side(), side(), 8, 128), rng(15)
    d = hq.QuantizedCache.empty(2, ps, heads, dim, 8, 128)
    K, V = (torch.randn(1500, heads, dim, device="cuda", generator=g).half() for _ in range(2))
    t = torch.arange(1500, device="cuda")
    far = torch.where(t < ps, (pages - 1) * ps + t, (pages - 3) * ps + t - ps)
    a, b = hq.hqq_cache_write(c, K, V, far, values=True), hq.hqq_cache_write(d, K, V, t, values=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = hq.hqq_cache_read(c, far), hq.hqq_cache_read(d, t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    Q, n = torch.randn(1, 16, dim, device="cuda", generator=g).half(), torch.tensor([1500], device="cuda").int()
    a = hq.hqq_cache_attention(c, Q, torch.tensor([[pages - 1, pages - 3]], device="cuda").int(), n)
    b = hq.hqq_cache_attention(d, Q, torch.tensor([[0, 1]], device="cuda").int(), n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# together, streams, graphs
# ---------------------------------------------------------------------------

def test_decode_steps(hq):
    """Two sequences grow: a prompt is written at once, then token by token; after each step the new
    token's attention over all of them, and at the end the prompt is read back."""
    g = rng(16)
    heads, G, dim = 2, 4, 128
    c = hq.QuantizedCache.empty(12, 32, heads, dim, 4, 64)
    table = torch.tensor([[3, 0, 7, 9], [11, 5, 2, 1]], device="cuda").int()
    lengths = [40, 0]

    def slots(b, t):
        return table[b].long()[t // 32] * 32 + t % 32

    K, V = (torch.randn(40, heads, dim, device="cuda", generator=g).half() for _ in range(2))
    at = slots(0, torch.arange(40, device="cuda"))
    prompt = hq.hqq_cache_write(c, K, V, at, values=True)
    for step in range(30):
        qkv = torch.randn(2, (G + 2) * heads * dim, device="cuda", generator=g).half()
        q, k, v = qkv.split([G * heads * dim, heads * dim, heads * dim], 1)
        new = torch.stack([slots(b, torch.tensor(lengths[b], device="cuda")) for b in range(2)])
        hq.hqq_cache_write(c, k.unflatten(1, (heads, dim)), v.unflatten(1, (heads, dim)), new)
        lengths = [n + 1 for n in lengths]
        n = torch.tensor(lengths, device="cuda").int()
        Q = q.unflatten(1, (G * heads, dim))
        got = hq.hqq_cache_attention(c, Q, table, n)
        if step % 7 == 0 or step == 29:
            check(c, got, Q, table, n)
    back = hq.hqq_cache_read(c, at)
    assert torch.equal(back[0], prompt[0]) and torch.equal(back[1], prompt[1])


def test_graph_and_streams(hq):
    """A captured decode step (write, attention, read) replays on new contents, beside eager work; calls on
    two streams with a workspace each give the same; a given workspace may hold anything."""
    g = rng(17)
    heads, G, dim = 2, 8, 128
    c = filled(hq, g, 400, 16, heads, dim, 4, 64)
    Q, table, n = batch_of(c, g, torch.float16, [3000, 1500, 7], G)
    K, V = (torch.randn(3, heads, dim, device="cuda", generator=g).half() for _ in range(2))
    last = (n - 1).long()
    slots = table.long().gather(1, (last // 16)[:, None])[:, 0] * 16 + last % 16
    size = hq.hqq_cache_attention_workspace(c, 3, heads * G, table.shape[1])
    ws = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    out, lse = torch.empty_like(Q), torch.empty(3, heads * G, device="cuda")

    def step(workspace, out=None, lse=None):
        hq.hqq_cache_write(c, K, V, slots)
        return (*hq.hqq_cache_attention(c, Q, table, n, out=out, lse=lse, workspace=workspace), *hq.hqq_cache_read(c, slots))

    step(ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(ws[0], out, lse)
    for i in range(4):
        Q.copy_(torch.randn(Q.shape, device="cuda", generator=g))
        K.copy_(torch.randn(K.shape, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in captured]
        for a, b in zip(mine, step(None)):
            assert torch.equal(a, b)
        check(c, mine[:2], Q, table, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, w in zip(streams, ws[1:]):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([hq.hqq_cache_attention(c, Q, table, n, workspace=w) for _ in range(3)])
    torch.cuda.synchronize()
    want = hq.hqq_cache_attention(c, Q, table, n)
    for runs in got:
        for r in runs:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


def test_graph_of_many_sequences(hq):
    """The plan that a call leaves in its workspace is that call's own: captured once, it is found anew for other
    lengths at every replay, whatever the workspace holds; two streams with a workspace each."""
    g = rng(19)
    c = filled(hq, g, 1200, 16, 3, 64, 8, 32)
    Q, table, n = batch_of(c, g, torch.bfloat16, [(i * 37) % 100 for i in range(200)], 2, width=50)
    size = hq.hqq_cache_attention_workspace(c, 200, 6, 50)
    ws = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    hq.hqq_cache_attention(c, Q, table, n, workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = hq.hqq_cache_attention(c, Q, table, n, workspace=ws[0])
    table.copy_(torch.randint(0, c.pages, table.shape, device="cuda", generator=g))
    for most in (0, 1, 40, 800, 100):
        n.copy_(torch.randint(0, most + 1, n.shape, device="cuda", generator=g))
        ws[0].fill_(most % 256)
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in captured]
        want = hq.hqq_cache_attention(c, Q, table, n)
        assert torch.equal(mine[0], want[0]) and torch.equal(mine[1], want[1])
        check(c, [t[::23] for t in mine], Q[::23], table[::23], n[::23])
    torch.cuda.synchronize()
    got = []
    for w, m in zip(ws[1:], (n, n.flip(0).contiguous())):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append((m, [hq.hqq_cache_attention(c, Q, table, m, workspace=w) for _ in range(3)]))
    torch.cuda.synchronize()
    for m, runs in got:
        want = hq.hqq_cache_attention(c, Q, table, m)
        for r in runs:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


def test_outputs_given(hq):
    """Rows beside a given output's keep what they held; the C call may leave out lse."""
    g = rng(18)
    c = filled(hq, g, 150, 16, 1, 64, 4, 32)
    Q, table, n = batch_of(c, g, torch.float16, [100, 1900], 3)
    want = hq.hqq_cache_attention(c, Q, table, n)
    room, row = torch.full((6, 3, 64), 7.0, device="cuda").half(), torch.full((8, 3), 7.0, device="cuda")
    got = hq.hqq_cache_attention(c, Q, table, n, out=room[2:4], lse=row[3:5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((room[:2] == 7).all()) and bool((room[4:] == 7).all()) and bool((row[:3] == 7).all()) and bool((row[5:] == 7).all())
    size = hq.hqq_cache_attention_workspace(c, 2, 3, table.shape[1])
    ws, out = torch.empty(max(16, size), dtype=torch.uint8, device="cuda"), torch.empty_like(Q)
    st = hq.load_cache_library().hqq_cache_attention(
        c._ptr, Q.data_ptr(), 3 * 64, 64, 2, 3, table.data_ptr(), table.shape[1], n.data_ptr(), 0.125, 0, 0,
        out.data_ptr(), None, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(out, want[0])


def test_nothing(hq):
    c = hq.QuantizedCache.empty(2, 16, 2, 64, 4, 32)
    none = torch.empty(0, 2, 64, device="cuda").half()
    assert hq.hqq_cache_write(c, none, none, torch.empty(0, dtype=torch.int64, device="cuda")) is None
    out, lse = hq.hqq_cache_attention(c, none, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                                      torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)


def test_binding_refuses(hq):
    """Wrong types, shapes, layouts and sizes raise before anything runs."""
    c = hq.QuantizedCache.empty(4, 16, 2, 128, 4, 64)
    K = torch.zeros(5, 2, 128, device="cuda").half()
    s = torch.arange(5, device="cuda")
    Q, table, n = torch.zeros(3, 4, 128, device="cuda").half(), torch.zeros(3, 2, device="cuda").int(), torch.ones(3, device="cuda").int()
    big = torch.zeros(3, 80, device="cuda").int()
    bad = [
        (TypeError, lambda: hq.hqq_cache_write(c, K.cpu(), K, s)),
        (TypeError, lambda: hq.hqq_cache_write(c, K.float(), K.float(), s)),
        (TypeError, lambda: hq.hqq_cache_write(c, K, K.bfloat16(), s)),
        (TypeError, lambda: hq.hqq_cache_write(c, K, K, s.int())),
        (ValueError, lambda: hq.hqq_cache_write(c, K, K, s[:4])),
        (ValueError, lambda: hq.hqq_cache_write(c, K, K[:, :1], s)),
        (ValueError, lambda: hq.hqq_cache_write(c, K[:, :1], K[:, :1], s)),
        (ValueError, lambda: hq.hqq_cache_write(c, K[..., :64], K[..., :64], s)),
        (ValueError, lambda: hq.hqq_cache_write(c, K.transpose(0, 2), K, s)),
        (ValueError, lambda: hq.hqq_cache_write(c, K[0], K[0], s)),
        (ValueError, lambda: hq.hqq_cache_write(c, torch.zeros(5, 2, 256, device="cuda").half()[..., ::2], K, s)),
        (hq.CacheError, lambda: hq.hqq_cache_write(c, torch.zeros(5 * 260, device="cuda").half().as_strided((5, 2, 128), (260, 128, 1)), K, s)),
        (hq.CacheError, lambda: hq.hqq_cache_write(c, torch.zeros(5 * 256 + 4, device="cuda").half()[4:].view(5, 2, 128), K, s)),
        (TypeError, lambda: hq.hqq_cache_read(c, s, dtype=torch.float32)),
        (TypeError, lambda: hq.hqq_cache_read(c, s.int())),
        (ValueError, lambda: hq.hqq_cache_read(c, s.view(5, 1))),
        (ValueError, lambda: hq.hqq_cache_read(c, s, out=(K[:4], K))),
        (hq.CacheError, lambda: hq.hqq_cache_read(c, s, out=(K, K))),
        (TypeError, lambda: hq.hqq_cache_read(c, s, out=(K, K.bfloat16()))),
        (ValueError, lambda: hq.hqq_cache_attention(c, Q, table[:2], n)),
        (ValueError, lambda: hq.hqq_cache_attention(c, Q, table, n[:2])),
        (TypeError, lambda: hq.hqq_cache_attention(c, Q, table.long(), n)),
        (TypeError, lambda: hq.hqq_cache_attention(c, Q, table, n.long())),
        (ValueError, lambda: hq.hqq_cache_attention(c, Q, table[0], n)),
        (ValueError, lambda: hq.hqq_cache_attention(c, Q, big[:, ::2], n)),
        (hq.CacheError, lambda: hq.hqq_cache_attention(c, Q[:, :3], table, n)),
        (hq.CacheError, lambda: hq.hqq_cache_attention(c, Q, table[:, :0], n)),
        (hq.CacheError, lambda: hq.hqq_cache_attention(c, Q, table, n, softmax_scale=0.0)),
        (hq.CacheError, lambda: hq.hqq_cache_attention(c, Q, table, n, window=-1)),
        (TypeError, lambda: hq.hqq_cache_attention(c, Q, table, n, out=Q.bfloat16())),
        (hq.CacheError, lambda: hq.hqq_cache_attention(c, Q, table, n, out=Q)),
        (ValueError, lambda: hq.hqq_cache_attention(c, Q, table, n, lse=torch.zeros(3, device="cuda"))),
        (TypeError, lambda: hq.hqq_cache_attention(c, Q, big, n, workspace=torch.zeros(10))),
        (hq.CacheError, lambda: hq.hqq_cache_attention(c, Q, big, n, workspace=torch.zeros(10, device="cuda"))),
        (hq.CacheError, lambda: hq.QuantizedCache.empty(4, 24, 2, 128, 4, 64)),
        (hq.CacheError, lambda: hq.QuantizedCache.empty(4, 16, 2, 160, 4, 32)),
        (ValueError, lambda: hq.QuantizedCache(c.k, (c.v[0], c.v[1], c.v[2][..., :1].contiguous()), 4, 64)),
        (ValueError, lambda: hq.QuantizedCache(c.k, (c.v[0][:3], *c.v[1:]), 4, 64)),
        (TypeError, lambda: hq.QuantizedCache(c.k, (c.v[0], c.v[1].half(), c.v[2]), 4, 64)),
        (ValueError, lambda: hq.QuantizedCache(c.k[:2], c.v, 4, 64)),
        (ValueError, lambda: hq.QuantizedCache(c.k, c.v, 3, 64)),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(AttributeError):
        c.k = c.v


# ---------------------------------------------------------------------------
# whole weights
# ---------------------------------------------------------------------------

def whole_bound(cache, Q, table, lengths):
    """(out, bound of its error) in 64 bits where each weight is held in two fp16 operands.

    Beside the terms of reference(): a weight p r times a power of two that brings the largest r of its
    group to 2^14 or more goes as the fp16 value next to it and that of the rest.  Together they are off by at
    most 2^-22 of it or, where the rest is subnormal, by 2^-25 with p <= 1, that is 2^-39 of the largest r in the
    frame of p (P's, the largest P being p = 1).  The zeros meet the unrounded weights.  A code stands in an fp16
    subnormal whose last place is 2^-24; products that are aligned by its exponent, 2^-14, lose at
    most u 2^10 / f of a code's unit each, f = 1, 16 or 64 being the place of the codes' last bit:
        |dout| <= (2 D + 2^-21) sum_t P_t |v_t|  +  2^-22 sum_t P_t r c  +  2^-39 max(P) max(r) sum_t c
                  +  (n + 24) u sum_t P_t r (c + |z|)  +  u 2^10 / f sum_t P_t r  +  half |out|"""
    B, H, D = Q.shape
    G, u = H // cache.heads, 2.0 ** -24
    f = {8: 1, 4: 16, 2: 64}[cache.nbits]
    half = torch.finfo(Q.dtype).eps / 2
    out, tol = (torch.zeros(B, H, D, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(B):
        t = torch.arange(int(lengths[b]), device="cuda")
        page, place = table[b].long()[t // cache.page_size], t % cache.page_size
        for h in range(cache.heads if len(t) else 0):
            (kc, kz, kr), (vc, vz, vr) = (decode([a[page, h, place] for a in side], cache.nbits, cache.group_size)
                                          for side in (cache.k, cache.v))
            rows = slice(h * G, (h + 1) * G)
            q = Q[b, rows].double() / math.sqrt(D)
            S = q @ ((kc - kz) * kr).T
            d = (D + 24) * u * (q.abs() @ (kr * (kc + kz.abs())).T) + 4 * u * S.abs().amax(1, keepdim=True)
            P = torch.softmax(S, 1)
            v = (vc - vz) * vr
            out[b, rows] = P @ v
            tol[b, rows] = (2 * d.amax(1, keepdim=True) + 2.0 ** -21) * (P @ v.abs()) + 2.0 ** -22 * (P @ (vr * vc)) \
                + 2.0 ** -39 * P.amax(1, keepdim=True) * vr.amax(0) * vc.sum(0) \
                + (len(t) + 24) * u * (P @ (vr * (vc + vz.abs()))) + u * 1024 / f * (P @ vr) + half * out[b, rows].abs()
    smallest = torch.finfo(Q.dtype).smallest_normal * torch.finfo(Q.dtype).eps
    return out, tol + smallest


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nbits", NBITS)
@pytest.mark.parametrize("dim,gs", [(64, 32), (96, 32), (128, 128), (256, 64)])
def test_attention_weights_are_whole(hq, dim, gs, nbits, dtype):
    """Few tokens of nearly even weight: some of their values cancel in some dims, where the output's own
    rounding is far below a weight's rounding to 11 bits (2^-11 of |v| beside a bound of about 2^-18)."""
    g = rng(dim + gs + 5 * nbits)
    lengths = [0] + [1, 2, 3, 4, 6, 9] * 5 + [33, 140, 1000]
    c = filled(hq, g, sum(-(-n // 16) for n in lengths), 16, 2, dim, nbits, gs)
    args = batch_of(c, g, DTYPES[dtype], lengths, 3, q=1 / 64)
    got = hq.hqq_cache_attention(c, *args)[0]
    out, tol = whole_bound(c, *args)
    err = (got.double() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("nbits", NBITS)
@pytest.mark.parametrize("place", [0, 40, 199])
def test_attention_a_wide_token_that_has_no_weight(hq, nbits, dtype, place):
    """One token with values 2^24 times the others' and a score some 60 below theirs: it takes nothing from
    the other tokens' weights but what the bound says."""
    g = rng(nbits + place)
    c = filled(hq, g, 13, 16, 1, 64, nbits, 32)
    Q, table, n = batch_of(c, g, DTYPES[dtype], [200], 4, q=1 / 64)
    page, at = int(table[0, place // 16]), place % 16
    Q[..., 0] = 8.0                                            # its key: -60 in the first group
    c.v[1][page, 0, at] *= 2.0 ** -24
    c.k[0][page, 0, at] = 0
    c.k[1][page, 0, at, 0], c.k[2][page, 0, at, 0] = 1.0, 60.0
    out, tol = whole_bound(c, Q, table, n)
    got = hq.hqq_cache_attention(c, Q, table, n)[0]
    err = (got.double() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("q,scale", [(1e-38, 1e-25), (1e-20, 1e-40), (1.0, 1e-45), (0.0, 1e-45), (1e-38, 2.0 ** 100)])
def test_attention_tiny_scores_beside_tokens_that_do_not_count(hq, q, scale):
    """softmax_scale times the query far below fp32's range: even weights for the tokens that count, in tiles
    with others too."""
    g = rng(20)
    c = filled(hq, g, 40, 16, 2, 128, 4, 64)
    Q, table, n = batch_of(c, g, torch.bfloat16, [100, 37, 0, 128, 1], 2)
    Q = (Q.float() * q).bfloat16()
    for window in (0, 33):
        check(c, hq.hqq_cache_attention(c, Q, table, n, softmax_scale=scale, window=window), Q, table, n, scale=scale,
              window=window)


@pytest.mark.parametrize("batch,most,heads,G,long", [(3, 9000, 40, 1, 0), (60, 700, 8, 2, 0), (70, 900, 40, 17, 0), (128, 40, 40, 1, 20000),
                                                     (600, 90, 16, 1, 9001), (3000, 20, 40, 2, 9001)])
def test_attention_workspace_of_just_its_bytes(hq, batch, most, heads, G, long):
    """Runs within sequences and across, fewer sequences than runs and more: what lies behind the workspace
    stays, whatever the workspace held."""
    g = rng(batch + most)
    lengths = torch.randint(0, most + 1, (batch,), generator=torch.Generator().manual_seed(batch)).tolist()
    lengths[batch // 2] = long or most
    c = filled(hq, g, sum(-(-n // 64) for n in lengths), 64, heads, 64, 4, 32)
    args = batch_of(c, g, torch.float16, lengths, G, width=max(13, -(-max(lengths) // 64)))
    size = hq.hqq_cache_attention_workspace(c, batch, heads * G, args[1].shape[1])
    assert size > 0 and size % 4 == 0
    room = torch.full((size // 4 + (1 << 20),), math.nan, device="cuda")
    want = hq.hqq_cache_attention(c, *args)
    got = hq.hqq_cache_attention(c, *args, workspace=room[:size // 4])
    assert bool(room[size // 4:].isnan().all())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    some = sorted({0, batch // 3, batch // 2, batch // 2 + 1, batch - 1} & set(range(batch)))
    check(c, [t[some] for t in got], *[t[some] for t in args])


CROSSING = [(96, 32, 2, "bf16"), (128, 32, 4, "fp16"), (256, 64, 8, "fp16"), (256, 128, 8, "bf16"), (64, 32, 2, "fp16"), (192, 64, 4, "bf16")]


@pytest.mark.parametrize("dim,gs,nbits,dtype", CROSSING)
@pytest.mark.parametrize("batch,most,heads,G,page_size", [(3, 9000, 40, 1, 64), (60, 1200, 20, 3, 16), (150, 500, 24, 1, 32),
                                                          (300, 700, 2, 17, 128)])
@pytest.mark.parametrize("window", [0, 333])
def test_attention_windows_and_formats_across_sequences(hq, dim, gs, nbits, dtype, batch, most, heads, G, page_size, window):
    """Runs that cross sequences, fewer and more of these than runs, planned by each wave and by a launch: every
    format's segments one behind the other in a workgroup's shared memory, and windows that begin inside a tile, where
    table entries before the window name no page."""
    g = rng(dim + batch + window)
    lengths = torch.randint(0, most + 1, (batch,), generator=torch.Generator().manual_seed(batch)).tolist()
    lengths[0], lengths[batch // 2], lengths[-1] = most, 0, most - 1
    pages = min(700, sum(-(-n // page_size) for n in lengths))
    c = filled(hq, g, pages, page_size, heads, dim, nbits, gs)
    width = max(-(-most // page_size), -(-800 // page_size))
    table = torch.randint(0, pages, (batch, width), device="cuda", generator=g).int()
    if window:
        first = (torch.tensor(lengths, device="cuda") - window).clamp(min=0)
        behind = torch.arange(width, device="cuda")[None] * page_size + page_size <= first[:, None]
        table[behind] = torch.tensor([-1, pages, 2 ** 31 - 1, -2 ** 31], device="cuda").int()[
            torch.randint(0, 4, table[behind].shape, device="cuda", generator=g)]
    Q = torch.randn(batch, heads * G, dim, device="cuda", generator=g).to(DTYPES[dtype])
    n = torch.tensor(lengths, device="cuda").int()
    got = torch.full_like(Q, math.nan), torch.full(Q.shape[:2], math.nan, device="cuda")
    hq.hqq_cache_attention(c, Q, table, n, window=window, out=got[0], lse=got[1])
    assert not got[0].isnan().any() and not got[1].isnan().any()
    some = torch.tensor(sorted({0, 1, batch // 2, batch // 2 + 1, batch - 1}), device="cuda")
    some = some[some < batch]
    check(c, [t[some] for t in got], Q[some], table[some], n[some], window=window)


def test_attention_of_several_new_tokens_of_a_sequence(hq):
    """One table row named several times with rising lengths: the tokens of a prompt's end, each seeing those
    before it."""
    g = rng(21)
    c = filled(hq, g, 90, 16, 2, 128, 4, 64)
    _, row, _ = batch_of(c, g, torch.float16, [1400], 4)
    table = row.repeat(9, 1)
    n = torch.arange(1392, 1401, device="cuda").int()
    Q = torch.randn(9, 8, 128, device="cuda", generator=g).half()
    for window in (0, 200):
        check(c, hq.hqq_cache_attention(c, Q, table, n, window=window), Q, table, n, window=window)


# ---------------------------------------------------------------------------
# the largest calls
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("heads", [1, 3, 1024])
def test_write_and_read_the_most_tokens(hq, heads):
    """2^26 rows: nearly all of them skipped, the first, the last and some between written and read back."""
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of device memory")
    g = rng(heads)
    tokens, dim = (1 << 26) // heads, 64
    c = hq.QuantizedCache.empty(20, 16, heads, dim, 4, 32)
    # rows that overlap: 8 values from one token, or head, to the next
    K, V = (torch.randn((tokens + heads) * 8 + dim, device="cuda", generator=g).half()
            .as_strided((tokens, heads, dim), (8, 8, 1)) for _ in range(2))
    some = torch.cat([torch.tensor([0, 1, 15, 16, tokens - 1, tokens - 17], device="cuda"),
                      torch.randint(20, tokens - 20, (250,), device="cuda", generator=g)]).unique()
    slots = torch.full((tokens,), -1, device="cuda")
    slots[some] = torch.randperm(320, device="cuda", generator=g)[:len(some)]
    hq.hqq_cache_write(c, K, V, slots)
    check_written(c, K[some], V[some], slots[some])
    got = hq.hqq_cache_read(c, slots)
    want = hq.hqq_cache_read(c, slots[some])
    for a, b in zip(got, want):
        assert torch.equal(a[some], b)
        a[some] = 0
        assert not a.view(torch.int64).any()
    with pytest.raises(hq.CacheError):
        more = torch.full((tokens + 1,), -1, device="cuda")
        hq.hqq_cache_write(c, K[:1].expand(tokens + 1, -1, -1), V[:1].expand(tokens + 1, -1, -1), more)


@pytest.mark.parametrize("place", [0, 1 << 19, (1 << 20) - 1])
def test_attention_of_the_longest_sequence(hq, place):
    """2^30 tokens, the table's pages all one but for one that takes all the weight: scores 60 or more above the
    others', whose 2^30 weights come to less than 2^30 e^-60 = 2^-56."""
    g = rng(22)
    c = filled(hq, g, 2, 1024, 1, 64, 2, 32)
    c.k[1].mul_(1e4)                                           # keys near 0, and one page's of 60 or more
    c.k[2][1, :, :, 0] -= 8.0 * 60 / 32 * c.k[1][1, :, :, 0]
    Q = torch.full((2, 3, 64), 1.0, device="cuda").bfloat16()
    table = torch.zeros(2, 1 << 20, dtype=torch.int32, device="cuda")
    table[0, place] = 1
    n = torch.tensor([1 << 30, 5], device="cuda").int()
    got = hq.hqq_cache_attention(c, Q, table, n)
    only = torch.tensor([[1], [0]], device="cuda").int(), torch.tensor([1024, 5], device="cuda").int()
    check(c, got, Q, *only)


@pytest.mark.parametrize("width", [1, 13])
def test_attention_of_the_most_sequences(hq, width):
    """2^15 sequences, whole and planned: empty ones, single tokens and a few long ones among them."""
    g = rng(23 + width)
    batch = 1 << 15
    c = filled(hq, g, 300, 64, 2, 64, 4, 32)
    n = torch.randint(0, 4, (batch,), device="cuda", generator=g).int()
    n[::4096] = width * 64
    n[-1] = width * 64 - 1
    table = torch.randint(0, 300, (batch, width), device="cuda", generator=g).int()
    Q = torch.randn(batch, 4, 64, device="cuda", generator=g).half()
    got = hq.hqq_cache_attention(c, Q, table, n)
    some = torch.cat([torch.arange(0, batch, 4096, device="cuda"), torch.tensor([1, 2, 4095, batch - 2, batch - 1], device="cuda")])
    check(c, [t[some] for t in got], Q[some], table[some], n[some])
    alone = torch.randint(0, batch, (100,), device="cuda", generator=g)
    parts = hq.hqq_cache_attention(c, Q[alone], table[alone], n[alone])
    short = n[alone] <= 128                                    # one step: one segment, whatever else runs
    assert torch.equal(parts[0][short], got[0][alone][short]) and torch.equal(parts[1][short], got[1][alone][short])
