"""Cases of the operators that keep long contexts in a small cache.

Next to the paged cache of 16- or 8-bit values and the attention over it, a server of long
contexts holds the cache in 4 bits and drops the positions that attention does not look at:

* ``store``  -- new keys and values written into a paged cache held in 4 bits (e2m1 codes, one
  power-of-two scale per token, head and 32 channels), and the same tokens read back;
* ``attend`` -- attention of each sequence's new tokens over such a cache, and (``lse``) the
  logarithm of each query row's sum of exponentials beside it;
* ``weigh``  -- the softmax weights that new tokens give to the cached positions, added up per
  position and key head;
* ``evict``  -- of each sequence and key head the last positions and the ones with the largest
  weights kept and moved to the front of other pages.

Shapes are those of this library's benchmark models (56 and 96 heads of 128 channels) or generic
ones.
"""
import math
import random

import torch

own = False

#: Types of activations and of a 16-bit cache.
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
#: Largest finite value of the 8-bit type.
E4M3_MAX = 448.0
#: Values of the 4-bit codes: a sign bit above these magnitudes.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
#: Channels that share one scale.
GROUP = 32


def listed():
    return [
        # one decoding step of 64 sequences: 64 tokens, each to a page of its own; a call's latency
        dict(op="store", name="store 64 tokens x 96 heads", T=64, heads=96, dim=128, page=16, skip=False, type="f16"),
        # a long prompt's keys and values, padding tokens among them: the most bytes
        dict(op="store", name="store 4095 tokens x 56 heads", T=4095, heads=56, dim=128, page=64, skip=True, type="bf16"),
        # a short prefix, heads of 80 channels: the last group is half of one
        dict(op="store", name="store 333 tokens x 8 heads of 80", T=333, heads=8, dim=80, page=32, skip=True, type="bf16"),
        # one sequence that decodes: latency, and one short axis to split
        dict(op="attend", name="attend 1 token over 1000", S=1, q=1, q_low=1, len=1000, len_low=1000, heads=32, kv=8,
             dim=128, page=16, cache="e2m1", type="f16", window=0, lse=False),
        # a batch of 64 ragged sequences that decode, heads not shared: the most bytes
        dict(op="attend", name="attend 64 x 1 token over 2048", S=64, q=1, q_low=1, len=2048, len_low=100, heads=96, kv=96,
             dim=128, page=16, cache="e2m1", type="f16", window=0, lse=True),
        # a chunk of a long prompt over what came before it: matrix products
        dict(op="attend", name="attend 2048 tokens over 16384", S=1, q=2048, q_low=2048, len=16384, len_low=16384, heads=32,
             kv=8, dim=128, page=64, cache="e2m1", type="bf16", window=0, lse=True),
        # prompts' chunks of all lengths and decoding sequences in one call, a sliding window
        dict(op="attend", name="attend 16 x 0-300 tokens over 5000", S=16, q=300, q_low=0, len=5000, len_low=0, heads=16,
             kv=4, dim=64, page=16, cache="e2m1", type="f16", window=1024, lse=False),
        # a small batch that decodes over an 8-bit cache: a call's latency
        dict(op="weigh", name="weigh 3 x 1 token over 1500", S=3, q=1, q_low=1, len=1500, len_low=700, heads=32, kv=8,
             dim=128, page=16, cache="e4m3", type="f16", window=0),
        # the same batch of 64 as above: every key once
        dict(op="weigh", name="weigh 64 x 1 token over 2048", S=64, q=1, q_low=1, len=2048, len_low=100, heads=96, kv=96,
             dim=128, page=16, cache="e2m1", type="f16", window=0),
        # a prompt's last part, whose attention says which positions of the whole are kept: matrix products
        dict(op="weigh", name="weigh 1500 tokens over 8000", S=1, q=1500, q_low=1500, len=8000, len_low=8000, heads=32, kv=8,
             dim=128, page=64, cache="bf16", type="bf16", window=0),
        # one long context cut to a quarter
        dict(op="evict", name="evict 16384 to 4096", S=1, len=16384, len_low=16384, keep=4096, recent=512, kv=8, dim=128,
             page=16, cache="f16"),
        # a ragged batch cut to what it may hold; some sequences are shorter than that
        dict(op="evict", name="evict 64 x 100-4096 to 1024", S=64, len=4096, len_low=100, keep=1024, recent=100, kv=8,
             dim=128, page=32, cache="e4m3"),
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "weigh", "weigh", "evict"])
    kind = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 80, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        heads = _between(rng, 1, 96)
        T = _between(rng, 1, min(16384, 4095 * 56 // heads))
        return dict(op=op, T=T, heads=heads, dim=dim, page=page, skip=rng.random() < 0.5, type=kind)
    if op == "evict":
        S = _between(rng, 1, 64)
        length = _between(rng, 64, min(32768, 262144 // S))
        keep = _between(rng, max(1, length // 16), max(1, length // 2))
        return dict(op=op, S=S, len=length, len_low=_between(rng, 1, length), keep=keep, recent=rng.randint(0, keep),
                    kv=rng.choice([1, 2, 4, 8]), dim=dim, page=page, cache=rng.choice([kind, "e4m3"]))
    kv, share = rng.choice([1, 2, 4, 8, 8, 12]), rng.choice([1, 2, 4, 8])
    more = dict(cache="e2m1", lse=rng.random() < 0.5) if op == "attend" else dict(cache=rng.choice([kind, "e4m3", "e2m1"]))
    window = rng.choice([0, 0, 0, 300])
    if rng.random() < 0.5:  # decoding
        S = _between(rng, 1, 64)
        length = _between(rng, 16, min(32768, 131072 // S))
        return dict(op=op, S=S, q=1, q_low=1, len=length, len_low=_between(rng, 1, length), heads=kv * share, kv=kv, dim=dim,
                    page=page, type=kind, window=window, **more)
    S = _between(rng, 1, 8)  # chunks
    length = _between(rng, 64, (16384 if op == "attend" else 8192) // S)
    q = _between(rng, 2, min(length, 1024))
    heads = min(32, kv * share)
    return dict(op=op, S=S, q=q, q_low=rng.randint(0, q), len=length, len_low=rng.randint(q, length), heads=heads // share * share,
                kv=heads // share, dim=dim, page=page, type=kind, window=window, **more)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, type=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(type)


def _lengths(c):
    """Host lists: each sequence's new tokens and its length with them, the same for every seed."""
    r = random.Random(c["S"])
    new = [r.randint(c["q_low"], c["q"]) if "q" in c else 0 for _ in range(c["S"])]
    length = [max(n, r.randint(c["len_low"], c["len"])) for n in new]
    new[0], length[0] = c.get("q", 0), max(c.get("q", 0), c["len"])
    return new, length


def _scale_row(dim):
    """Scales of one head vector of a 4-bit cache: one for 32 channels, rounded up to 2, 4 or 8."""
    return 2 if dim <= 64 else 4 if dim <= 128 else 8


def _code(a):
    """Index of the e2m1 magnitude nearest to a >= 0, ties to the even one."""
    return ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() +
            (a >= 3.5).byte() + (a > 5.0).byte())


def _pages(c, g, pages, cache, heads):
    """A pool of `pages` pages as earlier steps left it: normal keys and values."""
    shape = (pages, heads, c["page"], c["dim"])
    if cache in TYPES:
        return dict(k=torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).to(TYPES[cache]),
                    v=torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).to(TYPES[cache]), ks=None, vs=None)
    out = {}
    for n in ("k", "v"):
        if cache == "e4m3":  # codes of normal values of many sizes: a token's scale says where its largest value lies
            out[n] = (torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) * 80) \
                .clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            out[n + "s"] = torch.exp2(torch.randint(-8, -5, shape[:3], generator=g, device="cuda").float())
        else:  # pairs of codes of normal values, drawn from a table of 65536
            x = _normal((2, 65536), g) * 2.2
            x = _code(x.abs()) | (x < 0).byte() << 3
            at = torch.randint(0, 65536, shape[:3] + (c["dim"] // 2,), generator=g, device="cuda", dtype=torch.int32)
            out[n] = (x[0] | x[1] << 4)[at]
            out[n + "s"] = torch.randint(125, 127, shape[:3] + (_scale_row(c["dim"]),), generator=g, device="cuda",
                                         dtype=torch.uint8)
    return out


def _shuffled(count, g):
    return torch.randperm(count, generator=g, device="cuda").to(torch.int32)


def _slots(c, pages, g):
    """T slots on whole pages in any order (as an allocator hands them out); some of no token."""
    T, page = c["T"], c["page"]
    order = _shuffled(pages, g)[:(T + page - 1) // page].long()
    t = torch.arange(T, device="cuda")
    slots = (order[t // page] * page + t % page).to(torch.int32)
    if c["skip"]:
        slots = torch.where((torch.rand(T, generator=g, device="cuda") < 0.1) & (t > 0), torch.full_like(slots, -1), slots)
    return slots


def _tables(needs, pages, g):
    """Tables of the given numbers of pages, row after row, for each list: no page twice."""
    order, at, tables = _shuffled(pages, g), 0, []
    for need in needs:
        table = torch.zeros((len(need), max(1, max(need))), device="cuda", dtype=torch.int32)
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        tables.append(table)
    return tables


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "store":
        pages = (c["T"] + c["page"] - 1) // c["page"] + 3
        if c["T"] <= 64:  # into a pool in use; a decoding batch writes one token to a page
            pages = max(pages, c["T"] + 3)
        s = dict(c, **_pages(c, g, pages, "e2m1", c["heads"]), slots=_slots(c, pages, g))
        kind, shape = TYPES[c["type"]], (c["T"], c["heads"], c["dim"])
        if c["T"] <= 64:
            at = _shuffled(pages, g)[:c["T"]]
            s["slots"] = torch.where(s["slots"] < 0, s["slots"], at * c["page"] + at % c["page"])
        # keys and values are slices of one product's output, as they are in a decoder layer
        qkv = _normal((c["T"], 3, c["heads"], c["dim"]), g)
        qkv *= torch.exp(_normal((c["T"], 3, 1, 1), g))
        qkv = qkv.to(kind)
        s["new_k"], s["new_v"] = qkv[:, 1], qkv[:, 2]
        s["out_k"], s["out_v"] = (torch.empty(shape, device="cuda", dtype=kind) for _ in range(2))
        if own:
            import unstructured_sparse_skinny_amd as L
            s["cache_"] = L.Cache(s["k"], s["v"], s["ks"], s["vs"])
        return s
    new, length = _lengths(c)
    page = c["page"]
    needs = [[(n + page - 1) // page for n in length]]
    if c["op"] == "evict":
        needs.append([(c["keep"] + page - 1) // page] * c["S"])
    pages = sum(map(sum, needs)) + 1
    s = dict(c, **_pages(c, g, pages, c["cache"], c["kv"]))
    tables = _tables(needs, pages, g)
    s["table"] = tables[0]
    s["length"] = torch.tensor(length, device="cuda", dtype=torch.int32)
    if c["op"] != "attend":
        # sums of weights of many sizes, an earlier step's before `weigh`; positions that nobody looked at have none
        w = torch.exp(_normal((pages, c["kv"], page), g) * (2 if c["op"] == "evict" else 1) - 1)
        w *= c["heads"] / c["kv"] / c["len"] if c["op"] == "weigh" else 1
        s["weight"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.05, torch.zeros_like(w), w)
    if c["op"] == "evict":
        s["to"] = tables[1]
        s["kept"] = torch.empty((c["S"], c["kv"], c["keep"]), device="cuda", dtype=torch.int32)
    else:
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        s["q_most"], s["T"] = max(new), sum(new)
        s["start"] = torch.tensor(start, device="cuda", dtype=torch.int32)
        s["query"] = (_normal((s["T"], c["heads"], c["dim"]), g) * 1.5).to(TYPES[c["type"]])
        s["out"] = torch.empty_like(s["query"])
        s["row_lse"] = torch.empty((s["T"], c["heads"]), device="cuda") if c.get("lse") else None
        if c["op"] == "weigh":  # what the layer's attention said about its rows
            score = _scores(s)
            s["row_lse"] = _rows(s, _log_sum(score)[..., None])[..., 0].contiguous()
    if own:
        import unstructured_sparse_skinny_amd as L
        s["cache_"] = L.Cache(s["k"], s["v"], s["ks"], s["vs"])
        if c["op"] == "attend":
            s["handle"] = L.lscd_attention_create(c["heads"], c["kv"], c["dim"])
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    if own:
        import unstructured_sparse_skinny_amd as L
        if s["op"] == "store":
            L.lscd_cache_write(s["cache_"], s["new_k"], s["new_v"], s["slots"])
            L.lscd_cache_read(s["cache_"], s["slots"], s["out_k"], s["out_v"])
            return [s["out_k"], s["out_v"], s["k"], s["v"], s["ks"], s["vs"]]
        if s["op"] == "attend":
            L.lscd_attention(s["handle"], s["cache_"], s["query"], s["start"], s["length"], s["table"], s["out"],
                             window=s["window"], lse=s["row_lse"])
            return [s["out"], s["row_lse"]] if s["lse"] else [s["out"]]
        if s["op"] == "weigh":
            L.lscd_cache_weigh(s["cache_"], s["query"], s["row_lse"], s["start"], s["length"], s["table"], s["weight"],
                               window=s["window"])
            return s["weight"]
        L.lscd_cache_evict(s["cache_"], s["weight"], s["length"], s["table"], s["keep"], s["recent"], to=s["to"],
                           kept=s["kept"])
        return [x for x in (s["k"], s["v"], s["ks"], s["vs"], s["weight"], s["kept"]) if x is not None]
    if s["op"] == "store":
        _plain_write(s["new_k"], s["slots"], s["k"], s["ks"])
        _plain_write(s["new_v"], s["slots"], s["v"], s["vs"])
        kind = TYPES[s["type"]]
        return [_plain_read(s["k"], s["ks"], s["slots"], s["dim"], kind),
                _plain_read(s["v"], s["vs"], s["slots"], s["dim"], kind), s["k"], s["v"], s["ks"], s["vs"]]
    if s["op"] == "attend":
        return _plain_attend(s)
    if s["op"] == "weigh":
        return _plain_weigh(s)
    return _plain_evict(s)


def _plain_write(new, slots, pages, scales):
    """Each token, head and 32 channels: scale = the least power of two with max |x| / scale <= 6 (1 where all
    are zero), held as its exponent + 127; code = x / scale rounded to the nearest e2m1 value, ties to even;
    two codes a byte, the even channel's in the low half."""
    T, heads, dim = new.shape
    groups = (dim + GROUP - 1) // GROUP
    x = torch.zeros((T, heads, groups * GROUP), device="cuda", dtype=torch.float32)
    x[:, :, :dim] = new.float()
    x = x.reshape(T, heads, groups, GROUP)
    most = x.abs().amax(dim=3)
    fraction, exponent = torch.frexp(most / 6.0)
    exponent = torch.where(most > 0, exponent - (fraction == 0.5).int(), torch.zeros_like(exponent)).clamp(min=-126)
    x = torch.ldexp(x, -exponent[..., None])
    code = (_code(x.abs()) | torch.signbit(x).byte() << 3).reshape(T, heads, groups * GROUP)[:, :, :dim]
    code = code[:, :, 0::2] | code[:, :, 1::2] << 4
    scale = (exponent + 127).byte()
    # a token of no slot writes what is there already: the first slot's own values stay
    page, keep = pages.shape[2], slots >= 0
    at = torch.where(keep, slots, slots.max()).long()
    here = torch.argmax(slots)
    pages[at // page, :, at % page] = torch.where(keep[:, None, None], code, code[here])
    scales[at // page, :, at % page, :groups] = torch.where(keep[:, None, None], scale, scale[here])


def _values(code, scale, dim):
    """The values of 4-bit codes [..][dim / 2] with their scales [..][groups], in 32 bits."""
    table = torch.tensor(E2M1, device="cuda")
    x = torch.stack([table[(code & 15).int()], table[(code >> 4).int()]], dim=-1).flatten(-2)
    by = torch.exp2(scale[..., :(dim + GROUP - 1) // GROUP].float() - 127)
    return x * by.repeat_interleave(GROUP, dim=-1)[..., :dim]


def _plain_read(pages, scales, slots, dim, kind):
    """Code times scale in the model's type; zeros where there is no slot."""
    page, at = pages.shape[2], slots.clamp(min=0).long()
    x = _values(pages[at // page, :, at % page], scales[at // page, :, at % page], dim)
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).to(kind)


def _cached(s, which):
    """The keys ("k") or values ("v") of each sequence's pages in order, in 32 bits: [sequence][head][token][channel]."""
    pages, scales, t = s[which], s[which + "s"], s["table"].long()
    if s["cache"] == "e2m1":
        x = _values(pages[t], scales[t], s["dim"])
    elif s["cache"] == "e4m3":
        x = pages.view(torch.uint8)[t].view(pages.dtype).float() * scales[t][..., None]
    else:
        x = pages[t].float()
    S, wide = t.shape
    return x.permute(0, 2, 1, 3, 4).reshape(S, s["kv"], wide * s["page"], s["dim"])


def _padded(s, rows):
    """Rows [T][heads][..] of new tokens by sequence: [S][kv][share][most][..]; rows behind a sequence's last are any."""
    i = torch.arange(s["q_most"], device="cuda")
    x = rows[(s["start"][:-1, None] + i).clamp(max=s["T"] - 1).long()]
    x = x.reshape(s["S"], s["q_most"], s["kv"], s["heads"] // s["kv"], -1)
    return x.permute(0, 2, 3, 1, 4)


def _rows(s, x):
    """The reverse of _padded: [T][heads][..]."""
    x = x.permute(0, 3, 1, 2, 4).reshape(s["S"], s["q_most"], s["heads"], -1)
    t, start = torch.arange(s["T"], device="cuda"), s["start"].long()
    at = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return x[at, t - start[at]]


def _scores(s):
    """q.k / sqrt(dim) [S][kv][share][most][positions], -infinity where it is not seen: token i of a sequence's n new
    ones stands at position p = length - n + i and sees the positions j with j <= p and, with a window, j > p - window."""
    S, most, kv, share, dim = s["S"], s["q_most"], s["kv"], s["heads"] // s["kv"], s["dim"]
    q = _padded(s, s["query"].float()).reshape(S, kv, share * most, dim)
    score = torch.matmul(q, _cached(s, "k").transpose(2, 3)).mul_(1.0 / math.sqrt(dim)).reshape(S, kv, share, most, -1)
    length, new = s["length"].long(), (s["start"][1:] - s["start"][:-1]).long()
    i, j = torch.arange(most, device="cuda"), torch.arange(score.shape[-1], device="cuda")
    p = (length - new)[:, None, None] + i[:, None]
    sees = (j <= p) & (j < length[:, None, None]) & (i[:, None] < new[:, None, None])
    if s["window"]:
        sees &= j > p - s["window"]
    return score.masked_fill_(~sees[:, None, None], -math.inf)


def _log_sum(score):
    """ln of the sum of exp over the last axis; -infinity where nothing is seen."""
    most = score.amax(dim=-1, keepdim=True).clamp_(min=-3e38)
    return (score - most).exp_().sum(dim=-1).log_() + most[..., 0]


def _plain_attend(s):
    """Softmax of the scores over the positions seen, times the values; zeros where there is none."""
    S, most, kv, share, dim = s["S"], s["q_most"], s["kv"], s["heads"] // s["kv"], s["dim"]
    score = _scores(s)
    top = score.amax(dim=-1, keepdim=True).clamp_(min=-3e38)
    score = score.sub_(top).exp_()
    total = score.sum(dim=-1, keepdim=True)
    o = torch.matmul(score.reshape(S, kv, share * most, -1), _cached(s, "v")).reshape(S, kv, share, most, dim)
    o = _rows(s, torch.where(total > 0, o / total, torch.zeros_like(o))).to(TYPES[s["type"]])
    return [o, _rows(s, total.log() + top)[..., 0]] if s["lse"] else [o]


def _plain_weigh(s):
    """weight of position j and key head h: the sum over the rows of the head's query heads of exp(score - lse); new
    tokens' positions start from it, it is added to the others'."""
    score, lse = _scores(s), _padded(s, s["row_lse"])
    p = torch.where(lse > -math.inf, score.sub_(lse.clamp(min=-3e38)).exp_(), torch.zeros_like(lse)).sum(dim=(2, 3))
    length, new = s["length"].long(), (s["start"][1:] - s["start"][:-1]).long()
    j = torch.arange(p.shape[-1], device="cuda")
    i, at = ((j < length[:, None]) & (new > 0)[:, None]).nonzero().unbind(1)
    page, row = s["table"].long()[i, at // s["page"]], at % s["page"]
    old = (at < (length - new)[i])[:, None].float() * s["weight"][page, :, row]
    s["weight"][page, :, row] = old + p[i, :, at]
    return s["weight"]


def _plain_evict(s):
    """Each sequence and head: the last `recent` positions and those of the others with the largest weights, the lower
    position where they are equal, `keep` in all (every one of a shorter sequence), in order into the pages of `to`."""
    S, kv, page, keep = s["S"], s["kv"], s["page"], s["keep"]
    t, length = s["table"].long(), s["length"].long()[:, None, None]
    w = s["weight"][t].permute(0, 2, 1, 3).reshape(S, kv, -1)
    j = torch.arange(w.shape[-1], device="cuda")
    w = w.masked_fill(j >= length - s["recent"], math.inf).masked_fill(j >= length, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :keep]
    order = order.masked_fill(order >= length, 1 << 40)
    kept = torch.full((S, kv, keep), 1 << 40, device="cuda", dtype=torch.int64)
    kept[..., :order.shape[-1]] = torch.sort(order, dim=-1)[0]
    i, h, n = (kept < 1 << 40).nonzero().unbind(1)
    at, to = kept[i, h, n], s["to"].long()[i, n // page]
    page_, row, to_row = t[i, at // page], at % page, n % page
    for x in (s["k"], s["v"], s["ks"], s["vs"], s["weight"]):
        if x is not None:  # (indexing is by bytes: it has no 8-bit float form)
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[to, h, to_row] = x[page_, h, row]
    s["kept"].copy_(kept.masked_fill(kept >= 1 << 40, -1))
    return [x for x in (s["k"], s["v"], s["ks"], s["vs"], s["weight"], s["kept"]) if x is not None]


# ------------------------------------------------------------------ what a pass cannot do without


def _positions(new, length, window):
    """(positions that some token of the sequence sees, pairs of a token and a position that it sees)"""
    first = length - new
    pairs = sum(min(first + i + 1, window or length) for i in range(new))
    seen = (length if not window else min(length, window + new - 1)) if new else 0
    return seen, pairs


def _row_bytes(c, cache):
    """Bytes of one position and head of keys or of values: values and scales."""
    return {"e2m1": c["dim"] // 2 + (c["dim"] + GROUP - 1) // GROUP, "e4m3": c["dim"] + 4}.get(cache, 2 * c["dim"])


def work(case):
    c = case
    if c["op"] == "store":
        # a token's 16-bit values in, codes and scales out, and back; the slots
        row = _row_bytes(c, "e2m1")
        return {"bytes": 4 * c["T"] * (c["heads"] * (2 * c["dim"] + row) + 1), "flops": 8 * c["T"] * c["heads"] * c["dim"]}
    new, length = _lengths(c)
    row = _row_bytes(c, c["cache"])
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in length)
        # weights read; kept positions read and written with theirs; their numbers
        return {"bytes": c["kv"] * (4 * sum(length) + kept * (2 * (2 * row) + 4 + 4)), "flops": c["kv"] * sum(length)}
    parts = [_positions(a, b, c["window"]) for a, b in zip(new, length)]
    seen, pairs, rows = sum(p[0] for p in parts), sum(p[1] for p in parts), sum(new) * c["heads"]
    if c["op"] == "weigh":
        # keys, queries, their sums; a weight read (of old positions) and written
        weights = sum(2 * p[0] - n for p, n in zip(parts, new))
        return {"bytes": c["kv"] * (seen * row + 4 * weights) + rows * (2 * c["dim"] + 4), "flops": 2 * pairs * c["heads"] * c["dim"]}
    return {"bytes": 2 * c["kv"] * seen * row + rows * (4 * c["dim"] + (4 if c["lse"] else 0)),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def _wide(codes, scales, dim):
    """Values of a 4-bit pool in 64 bits, from the format: sign, two bits of exponent, one of fraction."""
    c = torch.empty(codes.shape[:-1] + (dim,), device="cuda", dtype=torch.int64)
    c[..., 0::2], c[..., 1::2] = (codes & 15).long(), (codes >> 4).long()
    e, f = (c >> 1) & 3, (c & 1).double()
    x = torch.where(e > 0, (1 + f / 2) * torch.exp2((e - 1).double()), f / 2)
    by = torch.exp2(scales.double() - 127)
    return torch.where(c > 7, -x, x) * by[..., torch.arange(dim, device="cuda") // GROUP]


def _exact_store(new, slots, dim):
    """The values that the tokens are read back as: each group's scale, and its values' distance to every e2m1 value."""
    x = torch.where((slots >= 0)[:, None, None], new.double(), torch.zeros((), device="cuda", dtype=torch.float64))
    grid = torch.tensor(E2M1[:8], device="cuda", dtype=torch.float64)
    even = torch.arange(8, device="cuda") % 2 == 0
    out = torch.empty_like(x)
    for a in range(0, dim, GROUP):
        y = x[:, :, a:a + GROUP]
        most = y.abs().amax(dim=2, keepdim=True)
        power = torch.ceil(torch.log2(most / 6.0))
        power = torch.where(most <= 6.0 * torch.exp2(power - 1), power - 1, power)
        scale = torch.where(most > 0, torch.exp2(power.clamp(min=-126)), torch.ones_like(most))
        best, value = torch.full_like(y, math.inf), torch.zeros_like(y)
        for i in range(8):
            far = ((y / scale).abs() - grid[i]).abs()
            nearer = (far < best) | ((far == best) & even[i])
            best, value = torch.where(nearer, far, best), torch.where(nearer, grid[i], value)
        out[:, :, a:a + GROUP] = torch.copysign(value, y) * scale
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if s["op"] == "store":
        return [_exact_store(s["new_k"], s["slots"], s["dim"]), _exact_store(s["new_v"], s["slots"], s["dim"])] + [None] * 4
    page, kv, dim = s["page"], s["kv"], s["dim"]
    length = s["length"].tolist()
    if s["op"] == "evict":
        pools = [x for x in (s["k"], s["v"], s["ks"], s["vs"], s["weight"]) if x is not None]
        out = [x.double() for x in pools]
        for i, n in enumerate(length):
            first = max(0, n - s["recent"])
            pos = torch.arange(n, device="cuda")
            at, keep = s["table"][i].long()[pos // page], min(n, s["keep"])
            for h in range(kv):
                w = s["weight"][at, h, pos % page].double()
                # ranked by weight, the lower position first among equals, the last ones before all
                rank = torch.argsort(-w[:first], stable=True)
                mine = torch.cat([rank[:keep - (n - first)] if n - first < keep else rank[:0], pos[max(first, n - keep):]])
                mine = mine.sort()[0]
                to = s["to"][i].long()[torch.arange(keep, device="cuda") // page]
                for x, y in zip(pools, out):
                    y[to, h, torch.arange(keep, device="cuda") % page] = (
                        x.view(torch.uint8)[at[mine], h, mine % page].view(x.dtype).double()
                        if x.dtype == torch.float8_e4m3fn else x[at[mine], h, mine % page].double())
        return out + [None]
    start, share = s["start"].tolist(), s["heads"] // kv
    out = torch.zeros((s["T"], s["heads"], dim), device="cuda", dtype=torch.float64)
    lse = torch.full((s["T"], s["heads"]), -math.inf, device="cuda", dtype=torch.float64)
    weight = s["weight"].double() if s["op"] == "weigh" else None
    for i in range(s["S"]):
        a, b, n = start[i], start[i + 1], length[i]
        if a == b or n == 0:
            continue
        pos = torch.arange(n, device="cuda")
        at = s["table"][i].long()[pos // page]
        p = n - (b - a) + torch.arange(b - a, device="cuda")[:, None]
        hidden = (pos > p) | ((pos <= p - s["window"]) if s["window"] else (pos < 0))
        for h in range(kv):
            def values(n):
                x, by = s[n][:, h], s[n + "s"]
                if s["cache"] == "e2m1":
                    return _wide(x[at, pos % page], by[at, h, pos % page], dim)
                x = x.view(torch.uint8).reshape(x.shape[0], page, -1)[at, pos % page].view(s[n].dtype).double()
                return x if by is None else x * by[at, h, pos % page].double()[:, None]

            k, v = values("k"), values("v") if s["op"] == "attend" else None
            got = torch.zeros(n, device="cuda", dtype=torch.float64)
            for f in range(h * share, (h + 1) * share):
                z = (s["query"][a:b, f].double() @ k.t() / math.sqrt(dim)).masked_fill(hidden, -math.inf)
                if s["op"] == "weigh":
                    got += torch.nan_to_num(torch.exp(z - s["row_lse"][a:b, f, None].double())).sum(dim=0)
                else:
                    lse[a:b, f] = torch.logsumexp(z, dim=1)
                    out[a:b, f] = torch.softmax(z, dim=1) @ v
            if s["op"] == "weigh":
                weight[at, h, pos % page] = torch.where(pos < n - (b - a), weight[at, h, pos % page], 0.0) + got
    if s["op"] == "weigh":
        return weight
    return [out, lse] if s["lse"] else [out]
