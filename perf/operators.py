"""The paged INT4 KV cache's operators as measured cases: inputs, plain forms and exact values.

Five operators of one serving path, on caches whose keys and values are held in 4 bits, one group
of 128 per (token, head) vector:

  append   new keys and values are quantized into their slots of the cache, and read back
  attend   attention of new tokens over the cache: single tokens, a few drafted ones, prompts
  weigh    the attention weight that every cached token received, summed over queries and heads
  evict    the cached tokens with the smallest accumulated weight leave, the others move up

A case's sizes (sequence lengths among them) follow from the case alone, its values from the seed.
With `own` false the operators run as elementary torch operations in 32 bits; with `own` true as
this package's entry points.
"""
import math

import torch

own = False

DIM = 128          # elements of a (token, head) vector: one quantization group
DEV = "cuda"


# ------------------------------------------------------------------------------ cases

def _case(name, op, batch, new, ctx, q_heads, kv_heads, page, layout, ragged=0, idle=0, causal=True,
          fused=False, budget=0, recent=0, prev=False):
    """new: tokens of a sequence that are new (its queries); ctx: cached tokens before them; both
    shrink from sequence to sequence by up to `ragged` percent. idle: sequences at the end with
    nothing in the cache. fused: q (k, v) are column slices of one projection's output."""
    return {"name": name, "op": op, "batch": batch, "new": new, "ctx": ctx, "q_heads": q_heads,
            "kv_heads": kv_heads, "page": page, "layout": layout, "ragged": ragged, "idle": idle,
            "causal": causal, "fused": fused, "budget": budget, "recent": recent, "prev": prev}


def listed():
    return [
        # one new token for each of 64 sequences: what a decode step writes; latency counts
        _case("append 64 tokens", "append", 64, 1, 4000, 8, 8, 64, "head", 60, fused=True),
        # ragged prompts behind cached prefixes, into small pages that start and end anywhere
        _case("append prompts", "append", 9, 4000, 37, 8, 8, 16, "token", 70, fused=True),
        # the smallest call: one sequence, one token, a head for every query head
        _case("decode 1x1000", "attend", 1, 1, 999, 32, 32, 16, "head"),
        # a serving batch in mid-flight: ragged lengths, two padded slots, 8 query heads a key head
        _case("decode 64x8192 ragged", "attend", 64, 1, 8191, 64, 8, 64, "head", 50, idle=2,
              fused=True),
        # long documents in a contiguous cache laid out as the cache quantizer writes it
        _case("decode 2x131072", "attend", 2, 1, 131071, 64, 8, 131072, "token"),
        # five drafted tokens a sequence, odd lengths, pages that end inside a tile
        _case("verify 16x5", "attend", 16, 5, 2996, 32, 8, 24, "head", 30),
        # a whole prompt at once
        _case("prompt 1x4096", "attend", 1, 4096, 0, 64, 8, 64, "head", fused=True),
        # chunks of prompts behind their cached beginnings, odd sizes, a head for every query head
        _case("chunks 6x700", "attend", 6, 700, 4300, 32, 32, 16, "token", 50),
        # every decode step's contribution to the eviction score
        _case("weigh decode 64x8192", "weigh", 64, 1, 8191, 64, 8, 64, "head", 50, idle=1,
              prev=True),
        # the score of a prompt's own tokens
        _case("weigh prompt 1x4096", "weigh", 1, 4096, 0, 64, 8, 64, "head"),
        # a batch that outgrew its budget
        _case("evict 64x2048", "evict", 64, 0, 2048, 8, 8, 64, "head", 25, budget=1024,
              recent=256),
        # one long document cut to a window, odd sizes, token-major pages
        _case("evict 1x65537", "evict", 1, 0, 65537, 8, 8, 16, "token", budget=4097, recent=501),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 32])
    group = rng.choice([1, 2, 3, 4, 7, 8]) if kv_heads < 32 else 1
    page = rng.choice([1, 8, 16, 24, 64, 100, 256])
    layout = rng.choice(["head", "token"])
    ragged = rng.choice([0, 30, 60, 90])
    batch = _log(rng, 1, 64)
    if op == "evict":
        most = min(65537, 64 * 2048 * 8 // (batch * kv_heads))
        ctx = _log(rng, 2, max(3, most))
        budget = rng.randint(1, ctx)
        return {k: v for k, v in _case(
            "", op, batch, 0, ctx, kv_heads, kv_heads, page, layout, ragged, budget=budget,
            recent=rng.randint(0, budget)).items() if k != "name"}
    kind = rng.choice(["single", "few", "many"])
    if kind == "many":
        batch = min(batch, 12)
    new = {"single": 1, "few": rng.randint(2, 8), "many": _log(rng, 9, 4096)}[kind]
    heads = kv_heads * group
    cached = 2 * 131072 * 8 // (batch * kv_heads)          # vectors of the listed long case
    scores = 4096 * 2048 * 64 // (batch * new * heads)     # scores of the listed prompt
    most = max(1, min(131072, cached, scores) - new)
    new = min(new, max(1, min(cached, scores)))
    ctx = _log(rng, 1, most) - 1
    if op == "append":
        new = min(new, max(1, 36000 * 8 // (batch * kv_heads)))
        ctx = min(ctx, 8192)
    return {k: v for k, v in _case(
        "", op, batch, new, ctx, heads, kv_heads, page, layout, ragged,
        idle=rng.choice([0, 0, 1]) if op == "attend" and batch > 1 else 0,
        causal=op == "append" or rng.random() < 0.8, fused=rng.random() < 0.5,
        prev=op == "weigh" and rng.random() < 0.5).items() if k != "name"}


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence."""
    out = []
    for i in range(case["batch"]):
        cut = case["ragged"] * ((i * 37 + 11) % 101 if i else 0)      # the first is the longest
        new = case["new"] - case["new"] * cut // 10100
        ctx = case["ctx"] - case["ctx"] * cut // 10100
        idle = i >= case["batch"] - case["idle"]
        out.append((new, 0 if idle else ctx + new))
    return out


def work(case):
    lens = _lengths(case)
    new, cached = sum(n for n, _ in lens), sum(c for _, c in lens)
    hq, h = case["q_heads"], case["kv_heads"]
    code = DIM // 2 + 4
    if case["op"] == "append":
        # fp16 vectors in, codes and scales out, and those read back as fp16 vectors
        return {"bytes": new * h * 2 * (2 * 2 * DIM + 2 * code), "flops": new * h * 2 * DIM * 4}
    if case["op"] == "evict":
        kept = sum(min(c, case["budget"]) for _, c in lens)
        # the scores in; of the kept tokens codes, scales and scores moved (read and written), the
        # positions out, and the moved vectors read back as fp16
        return {"bytes": h * (4 * cached + kept * (2 * 2 * code + 4 + 4 + 2 * (code + 2 * DIM))),
                "flops": h * cached * 4}
    pairs = 0
    for n, c in lens:
        if not case["causal"]:
            pairs += n * c
        elif c >= n:
            pairs += n * c - n * (n - 1) // 2
    q_bytes = new * hq * DIM * 2
    if case["op"] == "attend":
        return {"bytes": cached * h * 2 * code + 2 * q_bytes + new * hq * 4,
                "flops": 4 * DIM * pairs * hq}
    return {"bytes": cached * h * (code + 4 + (4 if case["prev"] else 0)) + q_bytes + new * hq * 4,
            "flops": 2 * DIM * pairs * hq}


# ------------------------------------------------------------------------------ inputs

def _quantize(x):
    """The cache's encoding of vectors x [..., 128]: codes uint8 [..., 64], scales [...]."""
    x = x.float()
    amax = x.abs().amax(-1)
    seven = torch.full_like(amax, 7)     # a number there would be multiplied by a reciprocal
    scale = amax / seven
    inv = torch.where(amax == 0, 0, seven / amax)
    q = torch.round(x * inv[..., None]).to(torch.int32) & 15
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), scale


def _codes(q4):
    """Signed codes, as float32 [..., 128], of packed bytes [..., 64]."""
    q = torch.stack((q4 & 15, q4 >> 4), -1).flatten(-2).to(torch.float32)
    return torch.where(q >= 8, q - 16, q)


def _vectors(gen, *shape):
    """Keys or values: normal, with a size of its own for each vector and a few large elements."""
    x = torch.randn(*shape, generator=gen, device=DEV)
    x *= torch.exp(0.3 * torch.randn(*shape[:-1], 1, generator=gen, device=DEV))
    x[..., 5] *= 4
    x[..., 77] *= 3
    return x.half()


def _pool(case, pages, gen):
    """A pool of pages with every slot filled: (k4, ks, v4, vs), shaped [page, slot, head, ...]."""
    ps, h = case["page"], case["kv_heads"]
    lead = (pages, h, ps) if case["layout"] == "head" else (pages, ps, h)
    out = []
    for _ in range(2):
        if gen is None:
            q4 = torch.zeros(*lead, DIM // 2, dtype=torch.uint8, device=DEV)
            s = torch.zeros(*lead, device=DEV)
        else:
            q4, s = _quantize(_vectors(gen, *lead, DIM))
        out += [q4.transpose(1, 2), s.transpose(1, 2)] if case["layout"] == "head" else [q4, s]
    return out


def _table(case, lens, gen):
    """Pages of each sequence [batch, most pages], shuffled; -1 behind its last. And their number."""
    need = [-(-n // case["page"]) for n in lens]
    total = sum(need) + 2
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = torch.tensor(need, device=DEV)
    inside = torch.arange(table.shape[1], device=DEV)[None] < at[:, None]
    table[inside] = order[: sum(need)]
    return table, total


def _starts(counts):
    s = [0]
    for c in counts:
        s.append(s[-1] + c)
    return torch.tensor(s, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    lens = _lengths(case)
    hq, h = case["q_heads"], case["kv_heads"]
    kv = [c for _, c in lens]
    table, pages = _table(case, kv, gen)
    s = {"case": case, "table": table, "kv_lens": torch.tensor(kv, dtype=torch.int32, device=DEV),
         "max_len": max(kv), "scale": DIM ** -0.5}
    if case["op"] == "evict":
        return _prepare_evict(case, s, kv, pages, gen)
    new = [n for n, _ in lens]
    rows = sum(new)
    s["cu_q"], s["rows"], s["max_q"] = _starts(new), rows, max(new)
    s["pool"] = _pool(case, pages, None if case["op"] == "append" else gen)
    # the new tokens' vectors, as slices of one projection's output or as tensors of their own
    if case["op"] == "append":
        if case["fused"]:
            x = torch.cat([_vectors(gen, rows, 3 * h, DIM)], 1)
            s["k"], s["v"] = x[:, h:2 * h], x[:, 2 * h:]
        else:
            s["k"], s["v"] = _vectors(gen, rows, h, DIM), _vectors(gen, rows, h, DIM)
    else:
        wide = hq + 2 * h if case["fused"] else hq
        x = 1.5 * torch.randn(rows, wide, DIM, generator=gen, device=DEV)
        s["q"] = x.half()[:, :hq]
    if case["op"] == "weigh":
        s["lse"] = _attend(s)[1]
        shape = (case["batch"], h, s["max_len"])
        s["prev"] = torch.rand(shape, generator=gen, device=DEV) if case["prev"] else None
        s["sums"] = torch.zeros(shape, device=DEV)
    if own:
        from w4a4_mixed_precision_b200 import atom
        s["cache"] = atom.KV4Cache(*s["pool"])
        s["batch"] = atom.KV4Batch(s["table"], s["kv_lens"], s["cu_q"], max_q=s["max_q"])
    return s


def _prepare_evict(case, s, kv, pages, gen):
    h, budget = case["kv_heads"], case["budget"]
    shape = (case["batch"], h, s["max_len"])
    # accumulated weights: most tokens little, a few much, many never looked at (ties at zero)
    w = torch.rand(shape, generator=gen, device=DEV).pow(8) * 50
    s["weights"] = torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.3, 0.0, w)
    s["pool"] = _pool(case, pages, gen)
    kept = [min(c, budget) for c in kv]
    s["to_table"], to_pages = _table(case, kept, gen)
    s["to_pool"] = _pool(case, to_pages, None)
    s["to_lens"] = torch.zeros(case["batch"], dtype=torch.int32, device=DEV)
    s["cu_q"], s["rows"] = _starts(kept), sum(kept)
    s["kept"] = torch.zeros(case["batch"], h, budget, dtype=torch.int32, device=DEV)
    s["to_weights"] = torch.zeros(case["batch"], h, budget, device=DEV)
    if own:
        from w4a4_mixed_precision_b200 import atom
        none = torch.zeros(case["batch"] + 1, dtype=torch.int32, device=DEV)
        s["cache"] = atom.KV4Cache(*s["pool"])
        s["batch"] = atom.KV4Batch(s["table"], s["kv_lens"], none, max_q=0)
        s["to_cache"] = atom.KV4Cache(*s["to_pool"])
        s["to_batch"] = atom.KV4Batch(s["to_table"], s["to_lens"], s["cu_q"], max_q=budget)
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "append":
        seq, pos = _positions(s["cu_q"], s["kv_lens"], s["rows"])
        page, slot = _slots(s["table"], s["case"]["page"], seq, pos)
        k4, ks, v4, vs = s["pool"]
        for x, q4, sc in ((s["k"], k4, ks), (s["v"], v4, vs)):
            q4[page, slot], sc[page, slot] = _quantize(x)
        return _read(s["pool"], page, slot)
    if op == "attend":
        return _attend(s)
    return _weigh(s) if op == "weigh" else _evict(s)


def _run_own(s, op):
    from w4a4_mixed_precision_b200 import atom
    causal = s["case"]["causal"]
    if op == "append":
        atom.atom_kv4_append(s["k"], s["v"], s["cache"], s["batch"])
        return atom.atom_kv4_gather(s["cache"], s["batch"], s["rows"])
    if op == "attend":
        return atom.atom_kv4_attention(s["q"], s["cache"], s["batch"], causal=causal,
                                       scale=s["scale"])
    if op == "weigh":
        return atom.atom_kv4_attention_weights(s["q"], s["lse"], s["cache"], s["batch"], s["sums"],
                                               prev=s["prev"], causal=causal, scale=s["scale"])
    kept, weights = atom.atom_kv4_evict(s["weights"], s["cache"], s["batch"], s["case"]["budget"],
                                        s["case"]["recent"], s["to_cache"], s["to_table"],
                                        s["to_lens"], kept=s["kept"], new_weights=s["to_weights"])
    k, v = atom.atom_kv4_gather(s["to_cache"], s["to_batch"], s["rows"])
    return kept, s["to_lens"], weights, k, v


# ------------------------------------------------------------------------------ plain forms

def _positions(cu_q, kv_lens, rows):
    """Sequence and position in it of each new token: the last ones of their sequences."""
    row = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(cu_q.long(), row, right=True) - 1
    return seq, (kv_lens[seq] - cu_q[seq + 1] + row).long()


def _slots(table, page_size, seq, pos):
    return table[seq, pos // page_size].long(), pos % page_size


def _read(pool, page, slot):
    """(k, v) fp16 [..., heads, 128] of slots of the cache."""
    k4, ks, v4, vs = pool
    return tuple((_codes(q4[page, slot]) * sc[page, slot][..., None]).half()
                 for q4, sc in ((k4, ks), (v4, vs)))


def _cached(s, which):
    """Keys (0) or values (1) of all sequences, float32 [batch, heads, most tokens, 128]."""
    pos = torch.arange(s["max_len"], device=DEV)[None]
    seq = torch.arange(s["case"]["batch"], device=DEV)[:, None]
    page, slot = _slots(s["table"], s["case"]["page"], seq, pos)
    page = page.clamp(min=0)
    q4, sc = s["pool"][2 * which], s["pool"][2 * which + 1]
    x = _codes(q4[page, slot]) * sc[page, slot][..., None]
    return x.transpose(1, 2)


def _scores(s):
    """Scores float32 [batch, kv heads, group, most queries, most tokens], -inf where masked, and
    the rows' places [batch, most queries]."""
    c = s["case"]
    b, h, g = c["batch"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    i = torch.arange(s["max_q"], device=DEV)[None]
    count = (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    row = (s["cu_q"][:-1, None] + torch.minimum(i, (count - 1).clamp(min=0))).clamp(max=s["rows"] - 1)
    q = s["q"][row.long()].float().view(b, s["max_q"], h, g, DIM).permute(0, 2, 3, 1, 4)
    keys = _cached(s, 0)
    x = (q.reshape(b, h, g * s["max_q"], DIM) @ keys.transpose(-1, -2)).view(
        b, h, g, s["max_q"], s["max_len"])
    x *= s["scale"]
    pos = torch.arange(s["max_len"], device=DEV)
    last = s["kv_lens"][:, None] - (count - 1 - i if c["causal"] else 0)   # tokens a query may see
    seen = (pos < last[..., None]) & (pos < s["kv_lens"][:, None, None]) & (i < count)[..., None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    return x, row, count


def _attend(s):
    c = s["case"]
    b, h = c["batch"], c["kv_heads"]
    g = c["q_heads"] // h
    x, row, count = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    x = torch.exp_(x.sub_(top))
    total = x.sum(-1, keepdim=True)
    out = (x.view(b, h, g * s["max_q"], -1) @ _cached(s, 1)).view(b, h, g, s["max_q"], DIM)
    out = torch.where(total > 0, out / total, 0).permute(0, 3, 1, 2, 4)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)
    seq, _ = _positions(s["cu_q"], s["kv_lens"], s["rows"])
    at = torch.arange(s["rows"], device=DEV) - s["cu_q"][seq]
    return (out[seq, at].reshape(s["rows"], h * g, DIM).half(),
            lse[seq, at].reshape(s["rows"], h * g))


def _weigh(s):
    c = s["case"]
    b, h = c["batch"], c["kv_heads"]
    g = c["q_heads"] // h
    x, row, count = _scores(s)
    lse = s["lse"][row.long()].view(b, s["max_q"], h, g).permute(0, 2, 3, 1)
    lse = torch.where(lse == -math.inf, math.inf, lse)     # a row that saw nothing gives nothing
    w = torch.exp_(x.sub_(lse[..., None])).sum((2, 3))
    if s["prev"] is not None:
        w = w + s["prev"]
    inside = torch.arange(s["max_len"], device=DEV) < s["kv_lens"][:, None, None]
    s["sums"].copy_(torch.where(inside, w, s["sums"]))
    return s["sums"]


def _evict(s):
    c = s["case"]
    budget, n = c["budget"], s["max_len"]
    lens = s["kv_lens"][:, None, None].long()
    new = lens.clamp(max=budget)
    recent = new.clamp(max=c["recent"])
    pos = torch.arange(n, device=DEV)[None, None]
    old = pos < lens - recent                               # those that have to earn their place
    w = torch.where(old, s["weights"], -1.0)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, pos.expand_as(order))
    keep = torch.where(old, rank < new - recent, pos < lens)
    kept = torch.sort(torch.where(keep, pos, n), dim=-1).values[..., :budget]
    if kept.shape[-1] < budget:
        kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=n)
    inside = torch.arange(budget, device=DEV) < new
    kept = torch.where(inside, kept, -1)
    s["kept"].copy_(kept)
    s["to_lens"].copy_(new[:, 0, 0])
    at = kept.clamp(min=0)
    w = s["weights"].gather(-1, at)
    s["to_weights"].copy_(torch.where(inside, w, s["to_weights"]))
    # the kept vectors' slots, and the slots that they move to
    seq, to = _positions(s["cu_q"], s["to_lens"], s["rows"])
    head = torch.arange(c["kv_heads"], device=DEV)[None]
    page, slot = _slots(s["table"], c["page"], seq[:, None], at[seq, :, to])
    to_page, to_slot = _slots(s["to_table"], c["page"], seq, to)
    for x, y in zip(s["pool"], s["to_pool"]):
        y[to_page, to_slot] = x[page, slot, head]
    k, v = _read(s["to_pool"], to_page, to_slot)
    return s["kept"], s["to_lens"], s["to_weights"], k, v


# ------------------------------------------------------------------------------ exact values

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return tuple(_exact_round_trip(s[x]) for x in ("k", "v"))
    if case["op"] == "evict":
        return _exact_evict(s)
    batch, hq, h = case["batch"], case["q_heads"], case["kv_heads"]
    out = torch.zeros(s["rows"], hq, DIM, dtype=torch.float64, device=DEV)
    lse = torch.full((s["rows"], hq), -math.inf, dtype=torch.float64, device=DEV)
    sums = torch.zeros(batch, h, s["max_len"], dtype=torch.float64, device=DEV)
    start = s["cu_q"].tolist()
    for b, (new, length) in enumerate(_lengths(case)):
        if length == 0 or new == 0:
            continue
        keys, values = (_exact_sequence(s, b, length, w) for w in (0, 1))
        limit = torch.full((new,), length, device=DEV)
        if case["causal"]:
            limit = length - new + 1 + torch.arange(new, device=DEV)
        hidden = torch.arange(length, device=DEV)[None] >= limit[:, None]
        mine = slice(start[b], start[b] + new)
        for head in range(hq):
            kv = head // (hq // h)
            x = s["q"][mine, head].double() @ keys[kv].T * s["scale"]
            x[hidden] = -math.inf
            z = torch.logsumexp(x, -1)
            if case["op"] == "attend":
                lse[mine, head] = z
                p = torch.nan_to_num(torch.exp(x - z[:, None]), nan=0.0)
                out[mine, head] = p @ values[kv]
            else:
                given = s["lse"][mine, head].double()
                p = torch.where((given == -math.inf)[:, None], 0, torch.exp(x - given[:, None]))
                sums[b, kv, :length] += p.sum(0)
        if case["op"] == "weigh" and s["prev"] is not None:
            sums[b, :, :length] += s["prev"][b, :, :length].double()
    return (out, lse) if case["op"] == "attend" else sums


def _exact_values(q4, scale):
    low, high = (q4 & 15).double(), (q4 >> 4).double()
    low[low > 7] -= 16
    high[high > 7] -= 16
    x = torch.empty(*q4.shape[:-1], DIM, dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = low, high
    return x * scale.double()[..., None]


def _exact_sequence(s, b, length, which):
    """Keys or values of one sequence, float64 [heads, length, 128]."""
    q4, scale = s["pool"][2 * which], s["pool"][2 * which + 1]
    pages = s["table"][b, : -(-length // s["case"]["page"])].long()
    q4, scale = (x[pages].flatten(0, 1)[:length].transpose(0, 1) for x in (q4, scale))
    return _exact_values(q4, scale)


def _exact_round_trip(x):
    """The codes are whole numbers set by 32-bit steps (scale amax/7, inverse 7/amax, ties to even);
    each code times its scale is exact in 64 bits."""
    x = x.float()
    amax = x.abs().max(-1, keepdim=True).values
    inv = torch.full_like(amax, 7.0) / amax
    inv[amax == 0] = 0
    scale = amax / torch.full_like(amax, 7.0)
    return torch.round(x * inv).double() * scale.double()


def _exact_evict(s):
    c = s["case"]
    kept = torch.full((c["batch"], c["kv_heads"], c["budget"]), -1, dtype=torch.int64)
    weights = torch.zeros(c["batch"], c["kv_heads"], c["budget"], dtype=torch.float64)
    all_w = s["weights"].double().cpu()
    lens, keys, values = [], [], []
    for b, length in enumerate(s["kv_lens"].tolist()):
        n = min(length, c["budget"])
        last = min(n, c["recent"])
        lens.append(n)
        k, v = (_exact_sequence(s, b, length, w) for w in (0, 1))
        at = []
        for h in range(c["kv_heads"]):
            w = all_w[b, h, : length - last]
            best = torch.argsort(-w, stable=True)[: n - last].sort().values
            at.append(torch.cat([best, torch.arange(length - last, length)]))
            kept[b, h, :n] = at[-1]
            weights[b, h, :n] = all_w[b, h, at[-1]]
        at = torch.stack(at).to(DEV)[..., None].expand(-1, -1, DIM)
        keys.append(k.gather(1, at).transpose(0, 1))
        values.append(v.gather(1, at).transpose(0, 1))
    return (kept.int(), torch.tensor(lens, dtype=torch.int32), weights, torch.cat(keys),
            torch.cat(values))
