"""Measured cases of the quantized key-value cache and the attention that reads it.

Keys and values of decoded tokens are held in pages, as packed codes with an fp32 scale and
zero per group of group_size consecutive values of a head (the library's axis = 1 format,
one row per page, head and token).  A slot is page * page_size + place in the page.

    write      scale = qmax / (max - min), zero = -(min * scale)  (1 and -min where max = min)
               code = clamp(round_half_even(x * scale + zero), 0, qmax), put at the tokens' slots;
               also the values (code - zero) / scale that the cache then stands for
    read       the values at given slots, rounded once; 0 at a slot below 0
    attention  one new token a sequence: s_t = softmax_scale * q . k_t over the sequence's last
               `window` tokens (all of them for 0), lse = log sum_t exp(s_t),
               out = sum_t exp(s_t - lse) v_t; a sequence of no tokens gives 0 and -inf.
               k_t and v_t are the values (code - zero) / scale, not rounded;
               q heads i * G .. i * G + G - 1 share key-value head i

All sums and products of the plain forms are fp32 and each output is rounded once.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    """The 7B decoder's heads (32 of 128), the 70B's (64 over 8 shared ones of 128), and other layouts."""
    def store(name, op, dtype, tokens, heads, dim, nbits, gs, page, fused=False, padded=False):
        return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "heads": heads, "dim": dim, "nbits": nbits,
                "gs": gs, "page": page, "fused": fused, "padded": padded}

    def attention(name, dtype, batch, q_heads, heads, dim, nbits, gs, page, length, ragged=False, window=0):
        return {"name": name, "op": "attention", "dtype": dtype, "batch": batch, "q_heads": q_heads, "heads": heads,
                "dim": dim, "nbits": nbits, "gs": gs, "page": page, "length": length, "ragged": ragged, "window": window}

    return [
        # a decode step of 32 sequences, one token each: latency counts
        store("write_decode", "write", "fp16", 32, 8, 128, 4, 64, 64),
        # a prompt, its keys and values cut from one fused projection
        store("write_prompt", "write", "bf16", 4096, 32, 128, 4, 64, 64, fused=True),
        # a padded batch, an odd number of heads, 8 bits in small groups
        store("write_ragged", "write", "fp16", 1237, 5, 96, 8, 32, 16, fused=True, padded=True),
        # a shared prefix, read back for the next prompt's attention
        store("read_prefix", "read", "fp16", 2048, 8, 128, 2, 32, 64, padded=True),
        # a long document, read back
        store("read_long", "read", "bf16", 32768, 8, 128, 4, 64, 64),
        # one user's next token: latency counts
        attention("attention_token", "fp16", 1, 32, 32, 128, 4, 64, 64, 700),
        # a served batch, every query head with its own keys and values
        attention("attention_batch_7b", "fp16", 32, 32, 32, 128, 4, 64, 64, 4096, ragged=True),
        # a served batch with shared heads
        attention("attention_batch_70b", "bf16", 64, 64, 8, 128, 4, 64, 64, 8192),
        # one token over a very long context
        attention("attention_long", "bf16", 1, 64, 8, 128, 4, 128, 256, 131072),
        # large heads at 8 bits, a sliding window
        attention("attention_window", "fp16", 8, 16, 4, 256, 8, 128, 32, 6000, ragged=True, window=4096),
        # small heads at 2 bits, small pages, odd counts, an empty sequence among them
        attention("attention_2bit", "bf16", 13, 21, 7, 64, 2, 32, 16, 3001, ragged=True),
        # all query heads over one shared head
        attention("attention_shared", "fp16", 24, 40, 1, 128, 8, 128, 16, 2500, ragged=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


FORMATS = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 64), (256, 64), (256, 128), (256, 256)]


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention"])
    dim, gs = rng.choice(FORMATS)
    c = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "heads": _spread(rng, 1, 40), "dim": dim,
         "nbits": rng.choice([2, 4, 4, 8]), "gs": gs, "page": rng.choice([16, 32, 64, 128, 256])}
    if op != "attention":
        c["tokens"] = _spread(rng, 1, 32768)
        while c["tokens"] > 1 and c["tokens"] * c["heads"] * dim > 32768 * 8 * 128:   # a fraction of the largest case
            c["tokens"] //= 2
        c["fused"], c["padded"] = rng.random() < 0.5, rng.random() < 0.5
        return c
    c["batch"] = _spread(rng, 1, 96)
    c["q_heads"] = c["heads"] * rng.choice([1, 1, 2, 3, 4, 7, 8, 16, 20])
    c["length"] = _spread(rng, 1, 131072)
    c["ragged"], c["window"] = rng.random() < 0.6, rng.choice([0, 0, 0, _spread(rng, 1, 8192)])
    while c["batch"] * c["length"] * c["heads"] * dim > 64 * 8192 * 8 * 128 // 4:
        if c["batch"] > 1:
            c["batch"] //= 2
        else:
            c["length"] //= 2
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _encode(x, nbits, gs):
    """Codes, scale and zero of rows x [..., dim] (fp32 values).  16-bit values on a group's grid lie half-way
    between two codes often, so the roundings are the format's: one of the quotient, one of x * scale + zero."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // gs, gs)
    lo, hi = g.amin(-1), g.amax(-1)
    same = hi == lo
    qmax = float((1 << nbits) - 1)
    one = torch.ones_like(hi)
    scale = torch.where(same, one, torch.div(qmax * one, torch.where(same, one, hi - lo)))
    zero = -(lo * scale)
    t = (g.double() * scale[..., None].double() + zero[..., None].double()).float()
    return t.round().clamp(0.0, qmax).reshape(x.shape), scale, zero


def _decode(codes, scale, zero, gs):
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // gs, gs)
    return ((g - zero[..., None]) / scale[..., None]).reshape(codes.shape)


def _shifts(nbits, device):
    return torch.arange(0, 32, nbits, dtype=torch.int32, device=device)


def _pack(codes, nbits):
    """Codes [..., dim] -> int32 words [..., dim * nbits / 32], lowest bits first."""
    q = codes.to(torch.int32).reshape(*codes.shape[:-1], -1, 32 // nbits)
    return (q << _shifts(nbits, q.device)).sum(-1, dtype=torch.int32)


def _unpack(words, nbits):
    q = (words[..., None] >> _shifts(nbits, words.device)) & ((1 << nbits) - 1)
    return q.to(torch.float32).reshape(*words.shape[:-1], -1)


def _lengths(c):
    """The sequences' lengths, before they are shuffled: a ragged batch has an empty one and a single token in it."""
    if not c["ragged"]:
        return [c["length"]] * c["batch"]
    n = [max(1, round(c["length"] * (i + 1) / c["batch"])) for i in range(c["batch"])]
    if c["batch"] >= 4:
        n[0], n[1] = 0, 1
    return n


def _seen(c):
    return [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]


def _pool(c, pages, normal, spread):
    """A side of the cache, its pages full of earlier tokens: (packed, scale, zero)."""
    shape = (pages, c["heads"], c["page"])
    packed = torch.empty(*shape, c["dim"] * c["nbits"] // 32, dtype=torch.int32, device="cuda")
    scale = torch.empty(*shape, c["dim"] // c["gs"], device="cuda")
    zero = torch.empty_like(scale)
    step = max(1, (1 << 25) // (c["heads"] * c["page"] * c["dim"]))
    for p in range(0, pages, step):
        at = slice(p, min(pages, p + step))
        x = (normal(at.stop - p, *shape[1:], c["dim"]) * spread).to(DTYPES[c["dtype"]]).float()
        codes, scale[at], zero[at] = _encode(x, c["nbits"], c["gs"])
        packed[at] = _pack(codes, c["nbits"])
    return packed, scale, zero


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    dt, H, D, P = DTYPES[c["dtype"]], c["heads"], c["dim"], c["page"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    # keys have a few channels of larger values; values have not
    spread = torch.ones(H, 1, D, device="cuda")
    spread[:, :, torch.randint(0, D, (max(1, D // 32),), device="cuda", generator=g)] = 4.0
    s = {"case": c}
    if c["op"] == "attention":
        n = torch.tensor(_lengths(c), device="cuda")[torch.randperm(c["batch"], device="cuda", generator=g)]
        width = max(1, -(-c["length"] // P))
        used = torch.arange(width, device="cuda") * P < n[:, None]
        pages = int(used.sum()) + 3
        table = torch.full((c["batch"], width), -1, dtype=torch.int32, device="cuda")
        table[used] = torch.randperm(pages, device="cuda", generator=g)[: pages - 3].int()
        s["table"], s["lengths"] = table, n.int()
        # heads from nearly even weights to a few tokens that take them all
        s["Q"] = (normal(c["batch"], c["q_heads"], D) * (0.3 + 2.0 * torch.rand(c["q_heads"], 1, device="cuda", generator=g))).to(dt)
    else:
        T = c["tokens"]
        if c["op"] == "write" and T <= 256:                   # one token of each of T sequences
            pages = T + 3
            s["slots"] = torch.randperm(pages, device="cuda", generator=g)[:T] * P + torch.randint(0, P, (T,), device="cuda", generator=g)
        else:                                                 # consecutive tokens over scattered pages
            pages = -(-T // P) + 3
            t = torch.arange(T, device="cuda")
            s["slots"] = torch.randperm(pages, device="cuda", generator=g)[t // P] * P + t % P
        if c["padded"]:
            s["slots"][torch.rand(T, device="cuda", generator=g) < 0.05] = -1
        if c["op"] == "write":
            if c["fused"]:                                    # queries, keys and values of one projection
                x = normal(T, 3, H, D)
                x[:, 1] *= spread[:, 0]
                x = x.to(dt)
                s["K"], s["V"] = x[:, 1], x[:, 2]
            else:
                s["K"], s["V"] = (normal(T, H, D) * spread[:, 0]).to(dt), normal(T, H, D).to(dt)
    s["k"], s["v"] = _pool(c, pages, normal, spread), _pool(c, pages, normal, torch.ones_like(spread))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _places(s):
    """(page, place) of each slot, and which slots are used."""
    keep = s["slots"] >= 0
    at = s["slots"].clamp(min=0)
    return at // s["case"]["page"], at % s["case"]["page"], keep


def _plain_write(s, x, side):
    c = s["case"]
    page, place, keep = _places(s)
    codes, scale, zero = _encode(x.float(), c["nbits"], c["gs"])
    packed, pool_scale, pool_zero = side
    page, place = page[keep], place[keep]
    packed[page, :, place] = _pack(codes, c["nbits"])[keep]
    pool_scale[page, :, place] = scale[keep]
    pool_zero[page, :, place] = zero[keep]
    return (_decode(codes, scale, zero, c["gs"]) * keep[:, None, None]).to(x.dtype)


def _plain_read(s, side):
    c = s["case"]
    page, place, keep = _places(s)
    packed, scale, zero = (t[page, :, place] for t in side)
    return (_decode(_unpack(packed, c["nbits"]), scale, zero, c["gs"]) * keep[:, None, None]).to(DTYPES[c["dtype"]])


def _plain_rows(s, side):
    """The values of every sequence's pages: [batch, heads, tokens, dim], fp32."""
    c = s["case"]
    packed, scale, zero = (t[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3) for t in side)
    return _decode(_unpack(packed, c["nbits"]), scale, zero, c["gs"])


def _plain(s):
    c = s["case"]
    if c["op"] == "write":
        k, v = _plain_write(s, s["K"], s["k"]), _plain_write(s, s["V"], s["v"])
        return {"k": k, "v": v, "k_scale": s["k"][1], "k_zero": s["k"][2], "v_scale": s["v"][1], "v_zero": s["v"][2]}
    if c["op"] == "read":
        return {"k": _plain_read(s, s["k"]), "v": _plain_read(s, s["v"])}
    B, H, D = c["batch"], c["heads"], c["dim"]
    q = s["Q"].float().view(B, H, c["q_heads"] // H, D).transpose(2, 3).contiguous()
    K = _plain_rows(s, s["k"])
    S = torch.matmul(K, q) * (1.0 / math.sqrt(D))             # [B, H, tokens, G]
    del K
    t, n = torch.arange(S.shape[2], device=S.device), s["lengths"][:, None]
    seen = t < n
    if c["window"]:
        seen = seen & (t >= n - c["window"])
    S = S.masked_fill(~seen[:, None, :, None], -math.inf)
    top = S.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    P = torch.exp(S - top)
    total = P.sum(2, keepdim=True)
    lse = (top + torch.log(total)).reshape(B, -1)
    P = (P / torch.where(total == 0, torch.ones_like(total), total)).transpose(2, 3).contiguous()
    out = torch.matmul(P, _plain_rows(s, s["v"]))             # [B, H, G, D]
    return {"out": out.reshape(B, -1, D).to(DTYPES[c["dtype"]]), "lse": lse}


def run(state):
    if not own:
        return _plain(state)
    import weight_quantization_group_amd as hq

    c = state["case"]
    cache = state.get("cache")
    if cache is None:                                         # a program's handle of its cache
        cache = state["cache"] = hq.QuantizedCache(state["k"], state["v"], c["nbits"], c["gs"])
    if c["op"] == "write":
        k, v = hq.hqq_cache_write(cache, state["K"], state["V"], state["slots"], values=True)
        return {"k": k, "v": v, "k_scale": cache.k[1], "k_zero": cache.k[2], "v_scale": cache.v[1], "v_zero": cache.v[2]}
    if c["op"] == "read":
        k, v = hq.hqq_cache_read(cache, state["slots"], dtype=DTYPES[c["dtype"]])
        return {"k": k, "v": v}
    out, lse = hq.hqq_cache_attention(cache, state["Q"], state["table"], state["lengths"], window=c["window"])
    return {"out": out, "lse": lse}


def work(case):
    """Each token's codes, scales and zeros, each input and each output once; two products of attention."""
    c = case
    row = c["heads"] * (c["dim"] * c["nbits"] / 8 + 8 * (c["dim"] // c["gs"]))    # bytes of a token's keys (or values)
    if c["op"] == "attention":
        tokens, queries = sum(_seen(c)), c["batch"] * c["q_heads"]
        return {"bytes": 2 * tokens * row + queries * (4 * c["dim"] + 4) + 4 * c["batch"],
                "flops": 4.0 * tokens * c["q_heads"] * c["dim"]}
    values = 2 * c["tokens"] * c["heads"] * c["dim"]
    moved = 2 * values * (2 if c["op"] == "write" else 1)                          # read: the values; write: the tokens too
    return {"bytes": 2 * c["tokens"] * row + moved + 8 * c["tokens"], "flops": 4.0 * values}


def exact(case, seed):
    """The definitions in 64 bits, a sequence and a head at a time."""
    c, s = case, prepare(case, seed)
    nb, gs = c["nbits"], c["gs"]

    def values(packed, scale, zero):                          # rows [..., words] -> [..., dim]
        w = torch.remainder(packed.to(torch.int64), 1 << 32)
        q = torch.stack([torch.remainder(torch.div(w, 1 << (j * nb), rounding_mode="floor"), 1 << nb) for j in range(32 // nb)], -1)
        q = q.flatten(-2).double()
        return (q - zero.double().repeat_interleave(gs, -1)) / scale.double().repeat_interleave(gs, -1)

    if c["op"] == "read":
        got = {}
        for name in ("k", "v"):
            rows = [t.transpose(1, 2).flatten(0, 1)[s["slots"].clamp(min=0)] for t in s[name]]
            got[name] = torch.where((s["slots"] >= 0)[:, None, None], values(*rows), 0.0)
        return got
    if c["op"] == "write":
        got = {}
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        page = torch.div(s["slots"][keep], c["page"], rounding_mode="floor")
        place = s["slots"][keep] - page * c["page"]
        for name, x in (("k", s["K"]), ("v", s["V"])):
            x = x.double().unflatten(-1, (-1, gs))
            least, range_ = x.min(-1).values, x.max(-1).values - x.min(-1).values
            scale = torch.where(range_ > 0, ((1 << nb) - 1) / range_, 1.0)
            zero = -least * scale
            # the code goes by the stored fp32 scale and zero, and by their fp32 fma: ties are frequent
            s32 = torch.where(range_ > 0, ((1 << nb) - 1) / range_.float().double(), 1.0).float()
            z32 = (-least * s32.double()).float()
            t = (x * s32[..., None].double() + z32[..., None].double()).float()
            q = torch.clamp(torch.round(t), 0, (1 << nb) - 1).double()
            back = ((q - z32[..., None].double()) / s32[..., None].double()).flatten(-2)
            got[name] = torch.zeros_like(back).index_copy(0, keep, back[keep])
            for what, pool, new in (("scale", s[name][1], scale), ("zero", s[name][2], zero)):
                pool = pool.double()
                pool[page, :, place] = new[keep]
                got["%s_%s" % (name, what)] = pool
        return got
    B, H, D = c["batch"], c["heads"], c["dim"]
    G = c["q_heads"] // H
    out = torch.zeros(B, c["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        t = torch.arange(first, n, device="cuda")
        page, place = s["table"][b].long()[t // c["page"]], t % c["page"]
        for h in range(H):
            K, V = (values(*(a[page, h, place] for a in s[name])) for name in ("k", "v"))
            S = s["Q"][b, h * G:(h + 1) * G].double() @ K.T / math.sqrt(D)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(S, 1)
            out[b, h * G:(h + 1) * G] = torch.softmax(S, 1) @ V
    return {"out": out, "lse": lse}
