"""What the shared-prefix decode, the cross attention and the page operators cost, and what they return.

``run`` makes one pass of an operator: in elementary torch operations, or (``own``) by the library's entry points.
Lengths, group sizes and parents follow from the case alone; values follow from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- the cases
def _shared(name, **kw):
    c = {"name": name, "op": "shared", "paged": True, "page": 16, "P": 1, "B": 16, "Q": 1, "lone": 0, "H_q": 64, "H_kv": 8, "d": 128,
         "dtype": "bf16", "prefix": 4096, "own_rows": 256, "ragged": False, "lens": 1}
    c.update(kw)
    return c


def _cross(name, **kw):
    c = {"name": name, "op": "cross", "E": 16, "tokens": 1, "S": 512, "H_q": 64, "H_kv": 8, "d": 64, "dtype": "bf16", "ragged": True, "lens": 1}
    c.update(kw)
    return c


def _pages(name, **kw):
    c = {"name": name, "op": "pages", "kind": "beam", "groups": 16, "width": 4, "rows": 4096, "page": 16, "new_rows": 1, "H_kv": 8, "d": 128,
         "dtype": "bf16", "spare": 0.25, "lens": 1}
    c.update(kw)
    return c


def listed():
    return [
        # a few samples of a short prompt, float32: the call's own latency
        _shared("shared tiny f32", paged=False, page=0, B=4, H_q=8, H_kv=2, d=64, dtype="f32", prefix=192, own_rows=24),
        # 16 samples of one prompt on the Llama-2-70B-shaped layer, in a paged cache
        _shared("shared samples", B=16, prefix=4096, own_rows=256),
        # a long system prompt under a large batch of conversations
        _shared("shared system prompt", B=128, prefix=16384, own_rows=512, ragged=True, page=64, lens=3),
        # several prompts of different lengths, contiguous caches, two sequences that share nothing
        _shared("shared prompts ragged", paged=False, page=0, P=6, B=64, lone=2, H_q=32, prefix=8191, own_rows=1001, ragged=True, lens=4),
        # four drafted tokens of each sequence are checked at once, one key/value head
        _shared("shared drafts mqa", P=2, B=32, Q=4, H_q=32, H_kv=1, prefix=8192, own_rows=512, ragged=True, page=128, lens=5),
        # decoding of an encoder-decoder model (T5-XXL-shaped heads), one token per input
        _cross("cross one token", E=32, H_kv=64, S=512),
        # beam search: four beams of each input
        _cross("cross beams", E=16, tokens=4, S=2048, lens=2),
        # target sequences of unequal length against inputs of unequal length
        _cross("cross targets ragged", E=8, tokens=509, S=2047, H_q=32, d=128, lens=3),
        # whole long targets at once
        _cross("cross long", E=4, tokens=1024, S=4096, d=128, ragged=False),
        # float32, odd sizes
        _cross("cross f32", E=5, tokens=61, S=777, H_q=12, H_kv=4, dtype="f32", lens=4),
        # one step of a beam search over a paged cache: beams take their parents' pages, each gets room for a row
        _pages("pages beam step"),
        # finished sequences leave, the pages that stay move to the front of the pool
        _pages("pages compact", kind="compact", groups=48, width=4, rows=4096, spare=0.5, lens=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "cross", "cross", "pages"])
    heads = rng.choice([(64, 8), (32, 8), (32, 1), (8, 2), (12, 4), (64, 64), (40, 8), (24, 1)])
    lens = rng.randrange(1, 1 << 20)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "shared":
        paged = rng.random() < 0.6
        B = _log(rng, 2, 96)
        c = {"op": op, "paged": paged, "page": rng.choice([8, 16, 64, 128, 256]) if paged else 0, "P": rng.randint(1, max(1, min(8, B // 2))), "B": B,
             "Q": rng.choice([1, 1, 1, 2, 5]), "lone": rng.choice([0, 0, 1]), "H_q": heads[0], "H_kv": heads[1], "d": rng.choice([64, 128]),
             "dtype": dtype, "prefix": _log(rng, 130, 12000), "own_rows": _log(rng, 20, 1500), "ragged": True, "lens": lens}
        while c["P"] * c["prefix"] * c["H_kv"] * c["d"] > 70e6 or c["B"] * c["own_rows"] * c["H_kv"] * c["d"] > 60e6:
            c["prefix"], c["own_rows"] = max(130, c["prefix"] // 2), max(20, c["own_rows"] // 2)
            if c["prefix"] == 130 and c["own_rows"] == 20:
                break
        if dtype == "f32":
            c["B"], c["prefix"] = min(c["B"], 24), min(c["prefix"], 2500)
            c["P"] = min(c["P"], c["B"] // 2)
        return c
    if op == "cross":
        c = {"op": op, "E": _log(rng, 1, 48), "tokens": _log(rng, 1, 800), "S": _log(rng, 33, 4000), "H_q": heads[0], "H_kv": heads[1],
             "d": rng.choice([64, 128]), "dtype": dtype, "ragged": True, "lens": lens}
        while c["E"] * c["tokens"] * c["S"] * c["H_q"] > (2e8 if dtype == "f32" else 8e8) or c["E"] * c["S"] * c["H_kv"] * c["d"] > 60e6:
            c["tokens"], c["S"] = max(1, c["tokens"] // 2), max(33, c["S"] * 3 // 4)
            if c["tokens"] == 1 and c["S"] == 33:
                break
        return c
    return {"op": op, "kind": rng.choice(["beam", "compact"]), "groups": _log(rng, 2, 48), "width": rng.choice([1, 2, 4, 6]), "rows": _log(rng, 40, 4000),
            "page": rng.choice([8, 16, 32, 64]), "new_rows": rng.choice([1, 1, 3, 17]), "H_kv": heads[1] if heads[1] < 64 else 8, "d": rng.choice([64, 128]),
            "dtype": dtype if dtype == "bf16" else "f32", "spare": rng.choice([0.2, 0.5, 0.8]), "lens": lens}


# ------------------------------------------------------------------------------- what follows from a case
def _cut(rnd, total, parts, ragged):
    """`total` things in `parts` runs, each of at least one."""
    if not ragged or parts == 1:
        at = [total * i // parts for i in range(parts + 1)]
    else:
        at = [0] + sorted(rnd.sample(range(1, total), parts - 1)) + [total]
    return at


def _shared_plan(c):
    rnd = random.Random(c["lens"])
    at = [c["lone"] + x for x in _cut(rnd, c["B"] - c["lone"], c["P"], c["ragged"])]
    step = c["page"] if c["paged"] else 1
    prefix = [(rnd.randint(c["prefix"] // 2, c["prefix"]) if c["ragged"] else c["prefix"]) // step * step for _ in range(c["P"])]
    low = c["Q"] if c["Q"] > 1 else 0
    tail = [rnd.randint(low, max(low, c["own_rows"])) if c["ragged"] else max(low, c["own_rows"]) for _ in range(c["B"])]
    return at, prefix, tail


def _cross_plan(c):
    rnd = random.Random(c["lens"])
    tokens = [rnd.randint(min(1, c["tokens"]), c["tokens"]) if c["ragged"] else c["tokens"] for _ in range(c["E"])]
    states = [rnd.randint(c["S"] // 4, c["S"]) if c["ragged"] else c["S"] for _ in range(c["E"])]
    if c["ragged"] and c["E"] > 4:
        states[rnd.randrange(c["E"])] = 0  # an input of no states
    return [sum(tokens[:e]) for e in range(c["E"] + 1)], states


def _pages_plan(c):
    """Block tables of groups of sequences that share the pages of their common rows, the counts, and what happens next."""
    rnd = random.Random(c["lens"])
    ps, W, n = c["page"], c["width"], c["groups"] * c["width"]
    max_pages = -(-(c["rows"] + c["new_rows"]) // ps) + 1
    table, lens, used = np.full((n, max_pages), -1, np.int32), np.zeros(n, np.int32), 0
    for g in range(c["groups"]):
        rows = rnd.randint(c["rows"] // 2, c["rows"])
        common = rnd.randint(rows // 2, rows) // ps
        for w in range(W):
            need = -(-rows // ps)
            table[g * W + w, :common] = np.arange(used, used + common)
            mine = used + common + w * (need - common)
            table[g * W + w, common:need] = np.arange(mine, mine + need - common)
            lens[g * W + w] = rows
        used += common + W * (need - common)
    n_pages = int((used + n * (1 + -(-c["new_rows"] // ps))) * (1 + c["spare"])) + 8
    place = np.random.RandomState(c["lens"] % (1 << 31)).permutation(n_pages).astype(np.int32)
    held = table >= 0
    table[held] = place[table[held]]
    refs = np.bincount(table[held], minlength=n_pages).astype(np.int32)
    parents = np.array([(i // W) * W + rnd.randrange(W) for i in range(n)], np.int32)
    done = np.array(sorted(rnd.sample(range(n), max(1, n // 3))), np.int32)
    if n > 4:
        parents[rnd.randrange(n)] = -1  # a beam that ends
    return table, lens, refs, parents, done


# ------------------------------------------------------------------------------------------------ inputs
def _normal(shape, gen, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dtype = case, DTYPES[case["dtype"]]
    s = {"case": c, "scale": case["d"] ** -0.5}
    if c["op"] == "shared":
        at, prefix, tail = _shared_plan(c)
        s.update(group_start=_int(at), members=max(b - a for a, b in zip(at, at[1:])))
        s["q"] = _normal((c["B"], c["H_q"], c["d"]) if c["Q"] == 1 else (c["B"], c["Q"], c["H_q"], c["d"]), gen, 1.0, dtype)
        if not c["paged"]:
            s.update(prefix_lens=_int(prefix), seq_lens=_int(tail))
            for n in ("k_prefix", "v_prefix"):
                s[n] = _normal((c["P"], max(1, c["prefix"]), c["H_kv"], c["d"]), gen, 1.0, dtype)
            for n in ("k_cache", "v_cache"):
                s[n] = _normal((c["B"], max(c["Q"], c["own_rows"]), c["H_kv"], c["d"]), gen, 1.0, dtype)
            return s
        ps = c["page"]
        group = [next((g for g in range(c["P"]) if at[g] <= b < at[g + 1]), -1) for b in range(c["B"])]
        head = [prefix[g] if g >= 0 else 0 for g in group]
        max_pages = max(-(-(h + max(c["Q"], c["own_rows"])) // ps) for h in head)
        first = np.cumsum([0] + [p // ps for p in prefix])
        table, used = np.full((c["B"], max_pages), -1, np.int32), int(first[-1])
        for b, g in enumerate(group):
            k = head[b] // ps
            if g >= 0:
                table[b, :k] = np.arange(first[g], first[g] + k)
            more = -(-tail[b] // ps)
            table[b, k:k + more] = np.arange(used, used + more)
            used += more
        place = np.random.RandomState(c["lens"] % (1 << 31)).permutation(used + 3).astype(np.int32)
        table[table >= 0] = place[table[table >= 0]]
        s.update(block_table=_int(table), seq_lens=_int([h + t for h, t in zip(head, tail)]), shared_rows=_int(prefix))
        for n in ("k_pool", "v_pool"):
            s[n] = _normal((used + 3, ps, c["H_kv"], c["d"]), gen, 1.0, dtype)
        return s
    if c["op"] == "cross":
        at, states = _cross_plan(c)
        s.update(q_start=_int(at), enc_lens=_int(states), longest=max(b - a for a, b in zip(at, at[1:])))
        s["q"] = _normal((at[-1], c["H_q"], c["d"]), gen, 1.0, dtype)
        for n in ("k_enc", "v_enc"):
            s[n] = _normal((c["E"], c["S"], c["H_kv"], c["d"]), gen, 1.0, dtype)
        return s
    table, lens, refs, parents, done = _pages_plan(c)
    s.update(table=_int(table), lens=_int(lens), refs=_int(refs), parents=_int(parents), done=_int(done))
    s.update(table_next=torch.empty_like(s["table"]), lens_next=torch.empty_like(s["lens"]))
    for n in ("k_pool", "v_pool"):
        s[n] = _normal((len(refs), c["page"], c["H_kv"], c["d"]), gen, 1.0, dtype)
    return s


# ------------------------------------------------------------------------------------------- plain forms
def _part(q, k, v, lens, scale):
    """Attention of q [G, H_kv, R, d] over k, v [G, L, H_kv, d], row i of group g over its first lens[g, i] rows ([G, 1 or R]), left
    unfinished: the largest score, the sum of exponentials and the weighted sum of values."""
    x = torch.matmul(q.float(), k.float().permute(0, 2, 3, 1)) * scale
    seen = torch.arange(k.shape[1], device=q.device) < lens[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(x - torch.where(m == -math.inf, 0.0, m)), 0.0)
    return m, e.sum(-1, keepdim=True), torch.matmul(e, v.float().permute(0, 2, 1, 3))


def _finish(parts):
    top = parts[0][0]
    for m, _, _ in parts[1:]:
        top = torch.maximum(top, m)
    top = torch.where(top == -math.inf, 0.0, top)
    total = sum(torch.exp(m - top) * n for m, n, _ in parts)
    out = sum(torch.exp(m - top) * o for m, _, o in parts)
    return torch.where(total > 0, out / torch.where(total > 0, total, 1.0), 0.0)


def _by_heads(q, H_kv):
    """[G, T, H_q, d] as [G, H_kv, T * r, d]."""
    G, T, H_q, d = q.shape
    return q.view(G, T, H_kv, H_q // H_kv, d).permute(0, 2, 1, 3, 4).reshape(G, H_kv, T * (H_q // H_kv), d)


def _by_tokens(o, T):
    G, H_kv, R, d = o.shape
    return o.view(G, H_kv, T, R // T, d).permute(0, 2, 1, 3, 4).reshape(G, T, H_kv * (R // T), d)


def _plain_shared(s):
    c = s["case"]
    B, Q, r, start = c["B"], c["Q"], c["H_q"] // c["H_kv"], s["group_start"].long()
    q = s["q"].view(B, Q, c["H_q"], c["d"])
    b = torch.arange(B, device=q.device)
    group = torch.searchsorted(start, b, right=True) - 1
    inside = (group >= 0) & (group < c["P"])
    group = group.clamp(0, c["P"] - 1)
    slot = (b - start[group]).clamp(0, s["members"] - 1)
    if c["paged"]:
        ps, shared = c["page"], s["shared_rows"].long()
        first = torch.arange(max(1, c["prefix"] // ps), device=q.device)
        pages = s["block_table"].long()[start[:-1]][:, first.clamp(max=s["block_table"].shape[1] - 1)].clamp(min=0)
        kp, vp = (s[n][pages].flatten(1, 2) for n in ("k_pool", "v_pool"))
        prefix = shared
        head = torch.where(inside, shared[group], 0)
        more = torch.arange(-(-max(c["Q"], c["own_rows"]) // ps), device=q.device)
        pages = s["block_table"].long().gather(1, (head[:, None] // ps + more).clamp(max=s["block_table"].shape[1] - 1)).clamp(min=0)
        ko, vo = (s[n][pages].flatten(1, 2) for n in ("k_pool", "v_pool"))
        tail = s["seq_lens"].long() - head
    else:
        kp, vp, ko, vo = s["k_prefix"], s["v_prefix"], s["k_cache"], s["v_cache"]
        prefix, tail = s["prefix_lens"].long(), s["seq_lens"].long()
    grouped = torch.zeros((c["P"], s["members"], Q, c["H_q"], c["d"]), dtype=q.dtype, device=q.device)
    grouped[group[inside], slot[inside]] = q[inside]
    m, n, o = _part(_by_heads(grouped.flatten(1, 2), c["H_kv"]), kp, vp, prefix[:, None], s["scale"])
    back = lambda t: torch.where(inside[:, None, None, None, None], t.view(c["P"], c["H_kv"], s["members"], Q * r, -1)[group, :, slot][:, :, None], 0.0)[:, :, 0]  # noqa: E731
    m = torch.where(inside[:, None, None, None], back(m), -math.inf)
    token = torch.arange(Q, device=q.device).repeat_interleave(r)
    own_part = _part(_by_heads(q, c["H_kv"]), ko, vo, tail[:, None] - (Q - 1) + token, s["scale"])
    return _by_tokens(_finish([(m, back(n), back(o)), own_part]), Q).view(s["q"].shape)


def _plain_cross(s):
    c, q, start = s["case"], s["q"], s["q_start"].long()
    i = torch.arange(q.shape[0], device=q.device)
    e = torch.searchsorted(start, i, right=True) - 1
    padded = torch.zeros((c["E"], s["longest"], c["H_q"], c["d"]), dtype=q.dtype, device=q.device)
    padded[e, i - start[e]] = q
    o = _finish([_part(_by_heads(padded, c["H_kv"]), s["k_enc"], s["v_enc"], s["enc_lens"].long()[:, None], s["scale"])])
    return _by_tokens(o, s["longest"])[e, i - start[e]]


def _plain_copy(s, pairs):
    pairs = pairs[pairs[:, 0] >= 0].long()
    for n in ("k_pool", "v_pool"):
        s[n][pairs[:, 1]] = s[n][pairs[:, 0]]


def _in_order(flags):
    """The numbers of the true flags in ascending order, at the front of a list as long as the flags."""
    rank = torch.cumsum(flags, 0) - 1
    found = torch.full((flags.shape[0] + 1,), -1, dtype=torch.long, device=flags.device)
    found[torch.where(flags, rank, flags.shape[0])] = torch.arange(flags.shape[0], device=flags.device)
    return found[:-1]


def _plain_beam(s):
    c, table, parents = s["case"], s["table"], s["parents"].long()
    ps, B, n_pages = c["page"], table.shape[0], s["refs"].shape[0]
    live = parents >= 0
    children = torch.zeros(B + 1, dtype=torch.int32, device=table.device).index_add_(0, torch.where(live, parents, B), live.int())[:-1]
    at = torch.where(table >= 0, table, n_pages).long()
    refs = torch.cat([s["refs"], s["refs"][:1]]).index_add_(0, at.flatten(), (children - 1)[:, None].expand_as(table).flatten())[:-1]
    table = torch.where(live[:, None], table[parents.clamp(min=0)], -1)
    lens = torch.where(live, s["lens"][parents.clamp(min=0)], 0)
    # room for new_rows rows of each sequence
    first, last = lens.long() // ps, (lens.long() + c["new_rows"] - 1) // ps
    slots = first[:, None] + torch.arange((c["new_rows"] - 1) // ps + 2, device=table.device)
    wanted = (slots <= last[:, None]) & (last < table.shape[1])[:, None]
    page = table.long().gather(1, slots.clamp(max=table.shape[1] - 1))
    count = refs[page.clamp(min=0)]
    shared = wanted & (page >= 0) & (count > 1)
    p = torch.where(shared, page, -1).flatten()
    earlier = ((p[:, None] == p[None, :]) & torch.ones(p.numel(), p.numel(), dtype=torch.bool, device=p.device).tril(-1)).sum(1).view_as(page)
    fresh = shared & (earlier < count - 1)  # the last holder keeps the page
    need = fresh | (wanted & (page < 0))
    total = torch.cumsum(need.sum(1), 0)
    free = refs == 0
    need = need & (total <= free.sum())[:, None]
    fresh = fresh & need
    rank = (torch.cumsum(need.flatten().long(), 0) - 1).view_as(page)
    given = torch.where(need, _in_order(free)[rank.clamp(min=0)], -1)
    refs = torch.cat([refs, refs[:1]])
    refs.index_add_(0, torch.where(fresh, page, n_pages).flatten(), torch.full_like(page, -1, dtype=torch.int32).flatten())
    refs[torch.where(need, given, n_pages).flatten()] = 1
    wide = torch.cat([table, table[:, :1].expand(-1, slots.shape[1])], 1)
    wide.scatter_(1, torch.where(need, slots, table.shape[1] + torch.arange(slots.shape[1], device=table.device)), given.int())
    moved = fresh[:, 0] & (lens % ps > 0)
    pairs = torch.stack([torch.where(moved, page[:, 0], -1), torch.where(moved, given[:, 0], -1)], 1).int()
    _plain_copy(s, pairs)
    return {"table": wide[:, :table.shape[1]].contiguous(), "lens": lens, "refs": refs[:-1], "pairs": pairs, "k": s["k_pool"], "v": s["v_pool"]}


def _plain_compact(s):
    n_pages, done = s["refs"].shape[0], s["done"].long()
    gone = s["table"][done]
    refs = torch.cat([s["refs"], s["refs"][:1]])
    refs = refs.index_add_(0, torch.where(gone >= 0, gone, n_pages).long().flatten(), torch.full_like(gone, -1).flatten())[:-1]
    table, lens = s["table"].index_fill(0, done, -1), s["lens"].index_fill(0, done, 0)
    live, number = refs > 0, torch.arange(n_pages, device=refs.device)
    n_live = live.sum()
    src, dst = _in_order(live & (number >= n_live)), _in_order(~live & (number < n_live))
    moved = src >= 0
    to = torch.cat([number, number[:1]])
    to[torch.where(moved, src, n_pages)] = dst
    back = torch.cat([number, number[:1]])
    back[torch.where(moved, dst, n_pages)] = src
    refs = torch.where(number < n_live, refs[back[:-1]], 0)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], -1).int()
    pairs = torch.stack([torch.where(moved, src, -1), torch.where(moved, dst, -1)], 1)[:max(1, n_pages // 2)].int()
    _plain_copy(s, pairs)
    return {"table": table, "lens": lens, "refs": refs, "pairs": pairs, "live": n_live.int().view(1), "k": s["k_pool"], "v": s["v_pool"]}


# ---------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import grouped_query_attention_decode_b200 as gqa

        if c["op"] == "shared" and c["paged"]:
            return gqa.decode_shared_paged(s["q"], s["k_pool"], s["v_pool"], s["block_table"], s["seq_lens"], s["group_start"], s["shared_rows"], s["scale"])
        if c["op"] == "shared":
            return gqa.decode_shared(s["q"], s["k_prefix"], s["v_prefix"], s["prefix_lens"], s["group_start"], s["k_cache"], s["v_cache"], s["seq_lens"], s["scale"])
        if c["op"] == "cross":
            return gqa.cross_attend(s["q"], s["k_enc"], s["v_enc"], s["enc_lens"], s["q_start"], s["scale"])
        refs = s["refs"].clone()
        if c["kind"] == "beam":
            table, lens = s["table_next"], s["lens_next"]
            gqa.pages_fork(s["parents"], s["table"], s["lens"], table, lens, refs)
            pairs = gqa.pages_reserve(table, lens, refs, c["new_rows"], c["page"])
            gqa.pages_copy(s["k_pool"], s["v_pool"], pairs)
            return {"table": table, "lens": lens, "refs": refs, "pairs": pairs, "k": s["k_pool"], "v": s["v_pool"]}
        table, lens = s["table"].clone(), s["lens"].clone()
        gqa.pages_free(s["done"], table, lens, refs)
        pairs, live = gqa.pages_compact(table, refs)
        gqa.pages_copy(s["k_pool"], s["v_pool"], pairs)
        return {"table": table, "lens": lens, "refs": refs, "pairs": pairs, "live": live, "k": s["k_pool"], "v": s["v_pool"]}
    if c["op"] == "shared":
        return _plain_shared(s)
    if c["op"] == "cross":
        return _plain_cross(s)
    return _plain_beam(s) if c["kind"] == "beam" else _plain_compact(s)


def work(case):
    c, size = case, 4 if case["dtype"] == "f32" else 2
    if c["op"] == "shared":
        at, prefix, tail = _shared_plan(c)
        rows = sum(prefix) + sum(tail)
        seen = sum((at[g + 1] - at[g]) * prefix[g] for g in range(c["P"])) + sum(tail)
        return {"bytes": 2 * rows * c["H_kv"] * c["d"] * size + c["B"] * c["Q"] * c["H_q"] * c["d"] * (size + 4), "flops": 4 * c["Q"] * c["H_q"] * c["d"] * seen}
    if c["op"] == "cross":
        at, states = _cross_plan(c)
        return {"bytes": 2 * sum(states) * c["H_kv"] * c["d"] * size + at[-1] * c["H_q"] * c["d"] * (size + 4),
                "flops": 4 * c["H_q"] * c["d"] * sum((at[e + 1] - at[e]) * states[e] for e in range(c["E"]))}
    table, lens, refs, parents, done = _pages_plan(c)
    page, state = 2 * c["page"] * c["H_kv"] * c["d"] * size, 4 * (2 * table.size + 2 * refs.size + 2 * lens.size)
    if c["kind"] == "beam":
        count = np.bincount(parents[parents >= 0], minlength=len(lens))
        part = lens % c["page"] > 0
        pages = int((count - 1).clip(0)[part].sum())  # each child but one of a sequence whose last page is not full
    else:
        refs = refs - np.bincount(table[done][table[done] >= 0], minlength=len(refs))
        pages = int((refs[int((refs > 0).sum()):] > 0).sum())
    return {"bytes": 2 * pages * page + state, "flops": 0}


# ------------------------------------------------------------------------------------------ in 64 bits
def _attend64(q, k, v, scale):
    """q [T, H_q, d] over all rows of k, v [n, H_kv, d], head by group of heads."""
    T, H_q, d = q.shape
    if k.shape[0] == 0:
        return torch.zeros((T, H_q, d), dtype=torch.float64, device=q.device)
    r = H_q // k.shape[1]
    out = torch.empty((T, H_q, d), dtype=torch.float64, device=q.device)
    for j in range(k.shape[1]):
        w = torch.softmax(q[:, j * r:(j + 1) * r].double().reshape(T * r, d) @ k[:, j].double().T * scale, -1)
        out[:, j * r:(j + 1) * r] = (w @ v[:, j].double()).view(T, r, d)
    return out


def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None  # whole numbers and copies
    s = prepare(c, seed)
    if c["op"] == "cross":
        at, states = _cross_plan(c)
        if 4 * c["H_q"] * c["d"] * at[-1] * c["S"] > 1e12:
            return None
        return torch.cat([_attend64(s["q"][at[e]:at[e + 1]], s["k_enc"][e, :states[e]], s["v_enc"][e, :states[e]], s["scale"]) for e in range(c["E"])])
    at, prefix, tail = _shared_plan(c)
    q = s["q"].view(c["B"], c["Q"], c["H_q"], c["d"])
    outs = []
    for b in range(c["B"]):
        g = next((g for g in range(c["P"]) if at[g] <= b < at[g + 1]), -1)
        head = prefix[g] if g >= 0 else 0
        if c["paged"]:
            n = head + tail[b]
            pages = s["block_table"][b, :-(-n // c["page"])].long()
            k, v = (s[x][pages].flatten(0, 1)[:n] for x in ("k_pool", "v_pool"))
        else:
            k, v = (torch.cat([s[x][max(g, 0), :head], s[y][b, :tail[b]]]) for x, y in (("k_prefix", "k_cache"), ("v_prefix", "v_cache")))
        n = k.shape[0]
        outs.append(torch.stack([_attend64(q[b, j:j + 1], k[:max(0, n - c["Q"] + 1 + j)], v[:max(0, n - c["Q"] + 1 + j)], s["scale"])[0] for j in range(c["Q"])]))
    return torch.stack(outs).view(s["q"].shape)
