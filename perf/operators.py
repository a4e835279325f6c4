"""The serving operators around the decode step: what is measured, on which cases.

  prefill   attention of chunks of new tokens over the paged expanded cache (GQA path)
  append    the new tokens' latent rows into the pages of the latent cache, of the expanded
            cache (their per-group projections) and of the RoPE keys
  fork      sequences forked (full pages shared, the last partial page copied), extended by
            new tokens, and freed again: one round of parallel sampling or beam search
  compact   a fragmented pool's live pages moved to its front, page tables rewritten

`own` False computes each in its plain form (elementary torch operations in fp32, rounded
once); True makes the calls of this package.
"""
import math
import random

import torch

own = False

PAGE = 64
D_LATENT, D_ROPE, D_NOPE, D_V = 512, 64, 128, 128
D_QK, D_ROW, D_KV = D_NOPE + D_ROPE, D_LATENT + D_ROPE, D_NOPE + D_V
SCALE = 1.0 / math.sqrt(D_QK)
BF16 = torch.bfloat16


# ------------------------------------------------------------------ the cases

def listed():
    """Layer shapes: 32 heads over 8 groups, 128 over 8, and 128 over 4 (the package's own
    configurations); lengths around its workloads' 256 .. 64K."""
    return [
        # five draft tokens of one short conversation are verified: the smallest call
        dict(name="prefill_verify_h32_l256", op="prefill", heads=32, groups=8, batch=1, new=5, new_hi=5,
             ctx=251, ctx_hi=251, full=0, lens_seed=1),
        # a whole prompt, nothing cached before it
        dict(name="prefill_prompt_h128_l8192", op="prefill", heads=128, groups=8, batch=1, new=8192, new_hi=8192,
             ctx=0, ctx_hi=0, full=0, lens_seed=2),
        # one chunk of a long document, far into it
        dict(name="prefill_chunk2k_h128_ctx32k", op="prefill", heads=128, groups=8, batch=1, new=2048, new_hi=2048,
             ctx=32768, ctx_hi=32768, full=0, lens_seed=3),
        # a mixed serving batch: one chunk of a prompt beside sequences that each add one token
        dict(name="prefill_mixed_h128_b32", op="prefill", heads=128, groups=8, batch=32, new=1, new_hi=1,
             ctx=2048, ctx_hi=8192, full=1021, lens_seed=4),
        # a batch of ragged prompts of the small layer
        dict(name="prefill_ragged_h32_b16", op="prefill", heads=32, groups=8, batch=16, new=130, new_hi=2047,
             ctx=0, ctx_hi=0, full=0, lens_seed=5),
        # draft verification for a batch, 32 heads to a group
        dict(name="prefill_verify_h128_g4_b32", op="prefill", heads=128, groups=4, batch=32, new=3, new_hi=8,
             ctx=3500, ctx_hi=4096, full=0, lens_seed=6),
        # the tokens of one decode step with two tokens to a sequence
        dict(name="append_step_h128_b64", op="append", heads=128, groups=8, batch=64, new=2, new_hi=2,
             ctx=300, ctx_hi=1024, latent=True, lens_seed=7),
        # the tokens of a prefill batch
        dict(name="append_prompts_h128_8k", op="append", heads=128, groups=8, batch=7, new=900, new_hi=1500,
             ctx=0, ctx_hi=700, latent=True, lens_seed=8),
        # one conversation continued in four ways
        dict(name="fork_h32_1x4", op="fork", heads=32, groups=8, parents=1, children=4, ctx=250, ctx_hi=250,
             lens_seed=9),
        # a batch of prompts, each sampled eight times
        dict(name="fork_h128_32x8", op="fork", heads=128, groups=8, parents=32, children=8, ctx=500, ctx_hi=1500,
             lens_seed=10),
        # a small pool after a few sequences have ended
        dict(name="compact_h32_p64", op="compact", heads=32, groups=8, pages=64, live=0.45, batch=5, lens_seed=11),
        # a large pool, two fifths live
        dict(name="compact_h128_p2048", op="compact", heads=128, groups=8, pages=2048, live=0.4, batch=48,
             lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "append", "fork", "compact"])
    heads, groups = rng.choice([(32, 8), (128, 8), (128, 4), (64, 8)])
    seed = rng.randrange(1 << 30)
    if op == "prefill":
        while True:
            batch = _log_int(rng, 1, 48)
            new = _log_int(rng, 1, 4096)
            ctx = rng.choice([0, _log_int(rng, 1, 40000)])
            case = dict(op=op, heads=heads, groups=groups, batch=batch, new=max(1, new // 3), new_hi=new,
                        ctx=ctx // 2, ctx_hi=ctx, full=rng.choice([0, 0, _log_int(rng, 16, 1500)]), lens_seed=seed)
            w = work(case)
            if w["flops"] <= 5.5e12 and w["bytes"] <= 2e9 and sum(_lengths(case)[0]) <= 16384:
                return case
    if op == "append":
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 8000 // batch))
        ctx = rng.choice([0, _log_int(rng, 1, 1200)])
        return dict(op=op, heads=heads, groups=groups, batch=batch, new=max(1, new // 2), new_hi=new, ctx=ctx // 2,
                    ctx_hi=ctx, latent=rng.choice([True, True, False]), lens_seed=seed)
    if op == "fork":
        parents = _log_int(rng, 1, 32)
        ctx = _log_int(rng, 20, 1500)
        return dict(op=op, heads=heads, groups=groups, parents=parents, children=rng.randint(1, 8), ctx=ctx // 2,
                    ctx_hi=ctx, lens_seed=seed)
    return dict(op=op, heads=heads, groups=groups, pages=_log_int(rng, 48, 2048), live=round(rng.uniform(0.1, 0.8), 3),
                batch=rng.randint(2, 48), lens_seed=seed)


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence; `full` > 0 gives
    the first sequence a chunk of that many."""
    rng = random.Random(case["lens_seed"])
    new = [rng.randint(case["new"], case["new_hi"]) for _ in range(case["batch"])]
    ctx = [rng.randint(case["ctx"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case.get("full"):
        new[0] = case["full"]
    return new, [n + c for n, c in zip(new, ctx)]


def _fork_lengths(case):
    rng = random.Random(case["lens_seed"])
    lens = [rng.randint(max(1, case["ctx"]), case["ctx_hi"]) for _ in range(case["parents"])]
    grow = [rng.randint(0, 9) for _ in range(case["parents"] * (1 + case["children"]))]
    return lens, grow


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    heads, groups = case["heads"], case["groups"]
    row = groups * D_KV * 2 + D_ROPE * 2              # one token of the expanded cache
    page = PAGE * (D_ROW * 2 + row)                   # one page of all caches
    if case["op"] == "prefill":
        new, lens = _lengths(case)
        pairs = sum(n * (2 * length - n + 1) // 2 for n, length in zip(new, lens))
        return {"bytes": sum(lens) * row + sum(new) * heads * (D_QK * 2 + D_V * 2 + 4),
                "flops": 2.0 * heads * pairs * (D_QK + D_V)}
    if case["op"] == "append":
        n = sum(_lengths(case)[0])
        return {"bytes": n * (D_ROW * 2 * (2 if case["latent"] else 1) + row) + groups * D_LATENT * D_KV * 2,
                "flops": 2.0 * n * groups * D_LATENT * D_KV}
    if case["op"] == "fork":
        lens, grow = _fork_lengths(case)
        copied = sum(1 for x in lens if x % PAGE) * case["children"]
        return {"bytes": copied * 2 * page + sum(_pages(x) for x in lens) * case["children"] * 12, "flops": 0}
    live = _compact_layout(case)[1]
    moved = sum(1 for p in live if p >= len(live))
    return {"bytes": moved * 2 * page + case["pages"] * 8, "flops": 0}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(lens, max_pages, pool):
    """Page table rows from the list of pages `pool`, in order; unused entries 0."""
    at, rows = 0, []
    for n in lens:
        k = _pages(n)
        rows.append(pool[at:at + k] + [0] * (max_pages - k))
        at += k
    return _i32(rows)


def _caches(gen, groups, pages, latent=True):
    n = pages * PAGE
    return {"latent": _randn(gen, pages, PAGE, D_ROW) if latent else None,
            "kv": _randn(gen, groups, n, D_KV), "rope": _randn(gen, n, D_ROPE)}


def _weights(gen, groups):
    return {k: (torch.randn(groups, D_LATENT, D_NOPE, generator=gen, device="cuda") / math.sqrt(D_LATENT)).to(BF16)
            for k in ("w_uk", "w_uv")}


def _compact_layout(case):
    """(page lists of the sequences, live pages): each sequence shares its first pages with the
    one before it in half of the cases, as after a fork."""
    rng = random.Random(case["lens_seed"])
    order = list(range(case["pages"]))
    rng.shuffle(order)
    target = max(1, int(case["pages"] * case["live"]))
    live, seqs = order[:target], []
    cut = sorted(rng.randint(0, target) for _ in range(case["batch"] - 1))
    for a, b in zip([0] + cut, cut + [target]):
        shared = seqs[-1][:rng.randint(0, len(seqs[-1]))] if seqs and rng.random() < 0.5 else []
        seqs.append(shared + live[a:b])
    return seqs, live


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    st = {"case": case, "groups": case["groups"], "heads": case["heads"]}
    if case["op"] in ("prefill", "append"):
        new, lens = _lengths(case)
        need = [_pages(x) for x in lens]
        pages = sum(need) + 3
        pool = list(range(pages))
        rng.shuffle(pool)
        st.update(new=new, lens=lens, pages=pages, table=_table(lens, max(need), pool), seqlens=_i32(lens))
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st.update(starts=_i32(starts), total=starts[-1])
        st.update(_caches(gen, case["groups"], pages, latent=case["op"] == "append" and case["latent"]))
        if case["op"] == "prefill":
            st["q"] = _randn(gen, starts[-1], case["heads"], D_QK)
        else:
            st["rows"] = _randn(gen, starts[-1], D_ROW)
            st.update(_weights(gen, case["groups"]))
    elif case["op"] == "fork":
        lens, grow = _fork_lengths(case)
        parents, kids = case["parents"], case["parents"] * case["children"]
        need = [_pages(x) for x in lens]
        pages = sum(need) + kids + sum(1 for _ in grow) + 5
        pool = list(range(pages))
        rng.shuffle(pool)
        width = max(need) + 2
        refs = [0] * pages
        for p in pool[:sum(need)]:
            refs[p] = 1
        st.update(pages=pages, table=_table(lens + [0] * kids, width, pool), seqlens=_i32(lens + [0] * kids),
                  refs=_i32(refs), forks=_i32([[i % parents, parents + i] for i in range(kids)]),
                  grow=_i32([0] * parents + grow[parents:]),
                  gone=_i32(list(range(parents, parents + kids))),
                  pairs=torch.full((kids, 2), -1, dtype=torch.int32, device="cuda"))
        st.update(_caches(gen, case["groups"], pages))
    else:
        seqs, _ = _compact_layout(case)
        refs = [0] * case["pages"]
        for s in seqs:
            for p in s:
                refs[p] += 1
        width = max(1, max(len(s) for s in seqs))
        lens = [max(0, len(s) * PAGE - rng.randint(0, PAGE - 1)) if s else 0 for s in seqs]
        st.update(pages=case["pages"], table=_i32([s + [0] * (width - len(s)) for s in seqs]), seqlens=_i32(lens),
                  refs=_i32(refs))
        st.update(_caches(gen, case["groups"], case["pages"]))
        st.update(table_out=torch.zeros_like(st["table"]), refs_out=torch.zeros_like(st["refs"]),
                  pairs=torch.full((max(1, case["pages"] // 2), 2), -1, dtype=torch.int32, device="cuda"),
                  counts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a program that calls the package keeps beside its tensors: the dimensions, the index,
    the output buffers, the split plan of these lengths."""
    from decode_attention_06_b200 import gqla
    st["dims"] = gqla.make_dims(st["heads"], st["groups"])
    st["ws"] = gqla.new_workspace()
    if "refs" in st:
        st["pool"] = gqla.make_page_pool(st["table"], st["seqlens"], st["refs"])
    else:
        st["kvi"] = gqla.make_kv_index(st["table"], st["seqlens"], st["pages"])
    if st["case"]["op"] == "prefill":
        splits = gqla.plan_prefill(st["dims"], st["new"], st["lens"])
        st["bufs"] = gqla.PrefillBuffers(st["dims"], st["total"], splits)


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return {"prefill": _own_prefill, "append": _own_append, "fork": _own_fork, "compact": _own_compact}[op](st)
    return {"prefill": _prefill, "append": _append, "fork": _fork, "compact": _compact}[op](st)


def _own_prefill(st):
    from decode_attention_06_b200 import gqla
    out, lse = gqla.prefill_step(st["dims"], st["bufs"], st["q"], st["starts"], st["kvi"], st["kv"], st["rope"])
    return {"out": out, "lse": lse}


def _own_append(st):
    from decode_attention_06_b200 import gqla
    gqla.gqla_append_cache(st["dims"], st["rows"], st["starts"], st["kvi"], st["ws"], latent_cache=st["latent"],
                           w_uk=st["w_uk"], w_uv=st["w_uv"], kv_expanded=st["kv"], k_rope=st["rope"])
    return {"latent": st["latent"], "kv": st["kv"], "rope": st["rope"]}


def _own_fork(st):
    from decode_attention_06_b200 import gqla
    pool, ws = st["pool"], st["ws"]
    gqla.gqla_fork_sequences(pool, st["forks"], st["pairs"], ws)
    gqla.gqla_copy_pages(st["dims"], st["pairs"], st["pages"], ws, latent_cache=st["latent"], kv_expanded=st["kv"],
                         k_rope=st["rope"])
    gqla.gqla_extend_sequences(pool, st["grow"], ws)
    grown = (st["seqlens"].clone(), st["refs"].clone())
    gqla.gqla_free_sequences(pool, st["gone"], ws)
    return _fork_result(st, grown)


def _own_compact(st):
    from decode_attention_06_b200 import gqla
    gqla.gqla_compact_pages(st["pool"], st["table_out"], st["refs_out"], st["pairs"], st["counts"], st["ws"])
    gqla.gqla_copy_pages(st["dims"], st["pairs"], st["pages"], st["ws"], latent_cache=st["latent"],
                         kv_expanded=st["kv"], k_rope=st["rope"])
    return _compact_result(st)


def _fork_result(st, grown):
    return {"table": st["table"], "grown_len": grown[0], "grown_refs": grown[1], "len": st["seqlens"],
            "refs": st["refs"], "pairs": st["pairs"], "latent": st["latent"], "kv": st["kv"], "rope": st["rope"]}


def _compact_result(st):
    return {"table": st["table_out"], "refs": st["refs_out"], "pairs": st["pairs"], "counts": st["counts"],
            "latent": st["latent"], "kv": st["kv"], "rope": st["rope"]}


# ------------------------------------------------------------------ the plain forms

def _slots(st, b):
    """Cache slots of the tokens of sequence b, in order."""
    t = torch.arange(st["lens"][b], device="cuda")
    return st["table"][b].long()[t // PAGE] * PAGE + t % PAGE


def _prefill(st):
    heads, groups = st["heads"], st["groups"]
    per = heads // groups
    out = torch.empty(st["total"], heads, D_V, dtype=BF16, device="cuda")
    lse = torch.empty(st["total"], heads, dtype=torch.float32, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
        slots = _slots(st, b)
        kv = st["kv"][:, slots].float()                                     # [g][L][256]
        rope = st["rope"][slots].float().expand(groups, length, D_ROPE)
        key, value = torch.cat([kv[..., :D_NOPE], rope], -1), kv[..., D_NOPE:]
        rows = max(1, min(n, (1 << 29) // (heads * length)))                # scores of at most 2 GB at a time
        for i in range(0, n, rows):
            m = min(rows, n - i)
            q = st["q"][at + i:at + i + m].float().view(m, groups, per, D_QK).permute(1, 0, 2, 3)
            s = torch.matmul(q.reshape(groups, m * per, D_QK), key.transpose(1, 2)).view(groups, m, per, length) * SCALE
            seen = torch.arange(length, device="cuda") <= (length - n + i + torch.arange(m, device="cuda"))[:, None]
            s = s.masked_fill(~seen[None, :, None, :], -math.inf)
            top = s.amax(-1, keepdim=True)
            p = (s - top).exp()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul((p / total).view(groups, m * per, length), value)
            out[at + i:at + i + m] = o.view(groups, m, per, D_V).permute(1, 0, 2, 3).reshape(m, heads, D_V).to(BF16)
            lse[at + i:at + i + m] = (top + total.log()).view(groups, m, per).permute(1, 0, 2).reshape(m, heads)
        at += n
    return {"out": out, "lse": lse}


def _append(st):
    starts, lens = st["starts"].long(), st["seqlens"].long()
    row = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(starts, row, right=True) - 1
    pos = lens[b] - (starts[b + 1] - row)
    slot = st["table"].long()[b, pos // PAGE] * PAGE + pos % PAGE
    if st["latent"] is not None:
        st["latent"].view(-1, D_ROW)[slot] = st["rows"]
    c = st["rows"][:, :D_LATENT].float()
    w = torch.cat([st["w_uk"], st["w_uv"]], -1).float()                     # [g][512][256]
    st["kv"][:, slot] = torch.matmul(c, w).to(BF16)
    st["rope"][slot] = st["rows"][:, D_LATENT:]
    return {"latent": st["latent"], "kv": st["kv"], "rope": st["rope"]}


def _free_pages(refs):
    """All pages, the free ones first, each half in ascending order."""
    return torch.sort((refs > 0).to(torch.int32), stable=True).indices


def _copy(st, moves, src, dst):
    """Pages src -> dst of every cache where `moves` says so; the other entries repeat the first
    that moves (with none, page 0 is written with itself)."""
    first = moves.to(torch.int32).argmax()
    src, dst = (torch.where(moves, x, torch.where(moves.any(), x[first], 0)).long() for x in (src, dst))
    st["latent"][dst] = st["latent"][src]
    kv = st["kv"].view(st["groups"], -1, PAGE, D_KV)
    kv[:, dst] = kv[:, src]
    rope = st["rope"].view(-1, PAGE, D_ROPE)
    rope[dst] = rope[src]


def _count(st, table, used):
    """How many of the entries that `used` marks name each page."""
    where = torch.where(used, table.long(), st["pages"]).reshape(-1)
    hits = torch.zeros(st["pages"] + 1, dtype=torch.int32, device="cuda")
    return hits.index_add_(0, where, torch.ones_like(where, dtype=torch.int32))[:-1]


def _fork(st):
    table, lens, refs = st["table"], st["seqlens"], st["refs"]
    parent, child = st["forks"][:, 0].long(), st["forks"][:, 1].long()
    col = torch.arange(table.shape[1], device="cuda")
    plen = lens[parent]
    part = plen % PAGE != 0
    fresh = _free_pages(refs)[(torch.cumsum(part, 0) - 1).clamp(min=0)].to(torch.int32)
    last = (_pages(plen) - 1).clamp(min=0).long()
    src = table[parent, last]
    rows = torch.where(part[:, None] & (col == last[:, None]), fresh[:, None], table[parent])
    used = col < _pages(plen)[:, None]
    table[child] = torch.where(used, rows, table[child])
    st["pairs"].copy_(torch.where(part[:, None], torch.stack([src, fresh], 1), -1))
    refs += _count(st, rows, used)
    lens[child] = plen
    _copy(st, part, src, fresh)
    # extend: the pages that each sequence lacks, the lowest free ones, sequence after sequence
    old, want = _pages(lens), _pages(lens + st["grow"])
    before = torch.cumsum(want - old, 0) - (want - old)
    take = (col >= old[:, None]) & (col < want[:, None])
    which = (before[:, None] + col - old[:, None]).clamp(0, st["pages"] - 1)
    table.copy_(torch.where(take, _free_pages(refs)[which.long()].to(torch.int32), table))
    refs += _count(st, table, take)
    lens += st["grow"]
    grown = (lens.clone(), refs.clone())
    gone = st["gone"].long()
    refs -= _count(st, table[gone], col < _pages(lens[gone])[:, None])
    lens[gone] = 0
    return _fork_result(st, grown)


def _compact(st):
    refs = st["refs"]
    used = refs > 0
    page = torch.arange(st["pages"], device="cuda")
    live = used.sum()
    high = used & (page >= live)                     # live pages that move ...
    hole = ~used & (page < live)                     # ... and the free ones they move to: as many
    src = torch.sort((~high).to(torch.int32), stable=True).indices
    dst = torch.sort((~hole).to(torch.int32), stable=True).indices
    moves = high.sum()
    half = st["pairs"].shape[0]
    moving = torch.arange(half, device="cuda") < moves
    st["pairs"].copy_(torch.where(moving[:, None], torch.stack([src, dst], 1)[:half], -1))
    new = page.clone()
    new[src] = torch.where(torch.arange(st["pages"], device="cuda") < moves, dst, src)
    col = torch.arange(st["table"].shape[1], device="cuda")
    inside = col < _pages(st["seqlens"])[:, None]
    st["table_out"].copy_(torch.where(inside, new[st["table"].long()], st["table"].long()))
    st["refs_out"].zero_()
    st["refs_out"].index_add_(0, new, torch.where(used, refs, 0))
    st["counts"].copy_(torch.stack([live, moves]))
    _copy(st, moving, src[:half], dst[:half])
    return _compact_result(st)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """From the definitions, head by head and in float64: the softmax over the visible tokens, the
    projections of the appended rows. Page moves compute no numbers."""
    if case["op"] in ("fork", "compact"):
        return None
    st = prepare(case, seed)
    slot_of = lambda b, t: st["table"][b, t // PAGE].long() * PAGE + t % PAGE  # noqa: E731
    if case["op"] == "append":
        kv, rope = st["kv"].double(), st["rope"].double()
        latent = None if st["latent"] is None else st["latent"].double().view(-1, D_ROW)
        at = 0
        for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
            slot = slot_of(b, torch.arange(length - n, length, device="cuda"))
            rows = st["rows"][at:at + n].double()
            for g in range(case["groups"]):
                kv[g, slot, :D_NOPE] = rows[:, :D_LATENT] @ st["w_uk"][g].double()
                kv[g, slot, D_NOPE:] = rows[:, :D_LATENT] @ st["w_uv"][g].double()
            rope[slot] = rows[:, D_LATENT:]
            if latent is not None:
                latent[slot] = rows
            at += n
        return {"latent": None if latent is None else latent.view(st["latent"].shape), "kv": kv, "rope": rope}
    if work(case)["flops"] > 2e13:
        return None
    out = torch.empty(st["total"], case["heads"], D_V, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["total"], case["heads"], dtype=torch.float64, device="cuda")
    at, per = 0, case["heads"] // case["groups"]
    for b, (n, length) in enumerate(zip(st["new"], st["lens"])):
        slot = slot_of(b, torch.arange(length, device="cuda"))
        rope = st["rope"][slot].double()
        for g in range(case["groups"]):
            kv = st["kv"][g, slot].double()
            step = max(1, (1 << 28) // (length * per))
            for i in range(0, n, step):
                q = st["q"][at + i:min(at + i + step, at + n), g * per:(g + 1) * per].double()
                m = q.shape[0]
                s = torch.einsum("mhd,td->mht", q[..., :D_NOPE], kv[:, :D_NOPE])
                s += torch.einsum("mhd,td->mht", q[..., D_NOPE:], rope)
                s /= math.sqrt(D_QK)
                last = torch.arange(length - n + i, length - n + i + m, device="cuda")
                s.masked_fill_(torch.arange(length, device="cuda")[None, None, :] > last[:, None, None], -math.inf)
                z = torch.logsumexp(s, -1)
                lse[at + i:at + i + m, g * per:(g + 1) * per] = z
                out[at + i:at + i + m, g * per:(g + 1) * per] = torch.einsum(
                    "mht,td->mhd", (s - z[..., None]).exp_(), kv[:, D_NOPE:])
        at += n
    return {"out": out, "lse": lse}
