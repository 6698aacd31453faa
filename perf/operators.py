"""Cases of the speculative / multimodal serving operators of the paged cache.

Each case is one call (or the few calls of one step) that a serving program
makes: attention of a chunk of new rows over the paged cache, cross attention
to an encoder's cached states, the append that rotates by positions of several
axes, the return of pages behind rejected draft tokens, and the compaction of
a fragmented page pool.  ``run`` computes a case with elementary torch
operations, or, when ``own`` is true, with the library's entry points.
"""
import math
import random

import torch

own = False

HEAD_DIM = 64
HALF = HEAD_DIM // 2
POOL_MAX_SEQS = 1024          # growth marks at the end of a pool state
BF, I32 = torch.bfloat16, torch.int32


# ---- cases ------------------------------------------------------------------

def _attention(kind, name, batch, rows, lens, heads, page, sizes):
    """rows, lens: the least and the most query rows and cached tokens of a
    sequence, drawn from seed ``sizes``; heads: query and KV heads."""
    return dict(name=name, kind=kind, batch=batch, min_rows=rows[0],
                max_rows=rows[1], min_len=lens[0], max_len=lens[1],
                q_heads=heads[0], kv_heads=heads[1], page=page, sizes=sizes)


def listed():
    return [
        # a speculative step of a handful of short conversations (latency)
        _attention("chunk", "chunk_tiny", 4, (1, 5), (16, 100), (32, 8),
                   16, 1),
        # verification of 8 draft tokens per sequence, the decode batch
        _attention("chunk", "chunk_verify", 64, (8, 8), (2048, 2048), (32, 8),
                   16, 2),
        # 4 draft tokens over the longest contexts
        _attention("chunk", "chunk_long", 8, (4, 4), (131072, 131072), (32, 8),
                   16, 3),
        # continuous batching: single tokens, drafts and prompt chunks at once
        _attention("chunk", "chunk_mixed", 64, (1, 512), (16, 8192), (32, 4),
                   32, 4),
        # one decoder token per sequence over encoder states (speech, images)
        _attention("cross", "cross_step", 64, (1, 1), (375, 1500), (16, 16),
                   16, 5),
        # decoder prompts over encoder states
        _attention("cross", "cross_prompt", 32, (224, 448), (1500, 1500),
                   (16, 16), 16, 6),
        # one new token per sequence of a multimodal batch
        dict(name="mrope_step", kind="mrope", tokens=64, q_heads=32,
             kv_heads=8, page=16, axes=3, interleaved=False,
             max_position=32768),
        # a prompt chunk with images, 16 sequences x 512 tokens
        dict(name="mrope_chunk", kind="mrope", tokens=8192, q_heads=32,
             kv_heads=8, page=16, axes=3, interleaved=True,
             max_position=32768),
        # rejected draft tokens of the decode batch go back
        dict(name="truncate_verify", kind="truncate", batch=64, min_len=1024,
             max_len=2048, drop=8, shared=0.0, page=16, sizes=7),
        # a large batch falls back to checkpoints of any length
        dict(name="truncate_many", kind="truncate", batch=1024, min_len=16,
             max_len=4096, drop=4096, shared=0.25, page=16, sizes=8),
        # a small pool after a few sequences ended
        dict(name="compact_small", kind="compact", pages=1024, used=600,
             moves=128, batch=24, layers=2, kv_heads=8, page=16),
        # the decode batch's pool, half used, a quarter of it out of place
        dict(name="compact_large", kind="compact", pages=16384, used=8192,
             moves=2048, batch=64, layers=2, kv_heads=8, page=16),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["chunk", "chunk", "cross", "cross", "mrope", "truncate",
                       "compact"])
    page = rng.choice([16, 32])
    if kind in ("chunk", "cross"):
        batch = _logint(rng, 1, 64)
        hkv = rng.choice([1, 2, 4, 8, 16] if kind == "cross" else
                         [1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 8])
        # tokens in the cache of the whole batch, and visible pairs, stay
        # below those of the largest listed case
        top = min(131072 if kind == "chunk" else 8192,
                  8 * 131072 // batch)
        most = _logint(rng, 1, top)
        rows = _logint(rng, 1, max(1, min(512, 2 ** 27 // (most * batch
                                                           * hq))))
        if kind == "chunk":
            rows = min(rows, most)
        case = _attention(kind, "", batch, (_logint(rng, 1, rows), rows),
                          (_logint(rng, 1, most), most), (hq, hkv), page,
                          rng.randrange(1 << 30))
        del case["name"]
        return case
    if kind == "mrope":
        hkv = rng.choice([1, 2, 4, 8])
        return dict(kind=kind, tokens=_logint(rng, 1, 8192),
                    q_heads=hkv * rng.choice([1, 2, 4, 8]), kv_heads=hkv,
                    page=page, axes=rng.choice([1, 2, 3, 4]),
                    interleaved=rng.random() < 0.5,
                    max_position=_logint(rng, 8192, 131072))
    if kind == "truncate":
        most = _logint(rng, 16, 4096)
        return dict(kind=kind, batch=_logint(rng, 1, 1024),
                    min_len=_logint(rng, 1, most), max_len=most,
                    drop=_logint(rng, 1, most),
                    shared=rng.choice([0.0, 0.25, 0.5]), page=page,
                    sizes=rng.randrange(1 << 30))
    pages = _logint(rng, 64, 16384)
    used = rng.randint(1, pages - 1)
    return dict(kind=kind, pages=pages, used=used,
                moves=rng.randint(0, min(used, pages - used, 2048)),
                batch=_logint(rng, 1, 64), layers=rng.choice([1, 2]),
                kv_heads=rng.choice([2, 8]), page=page)


def _sizes(case):
    """(query rows, cached tokens) of every sequence, fixed by the case."""
    rng = random.Random(case["sizes"])
    lens = [_logint(rng, case["min_len"], case["max_len"])
            for _ in range(case["batch"])]
    if case["kind"] == "truncate":
        drop = [rng.randint(0, min(case["drop"], n)) for n in lens]
        twin = [s > 0 and rng.random() < case["shared"]
                for s in range(case["batch"])]
        # a twin shares every page of its left neighbour
        for s in range(1, case["batch"]):
            if twin[s]:
                lens[s] = lens[s - 1]
                drop[s] = min(drop[s], lens[s])
        return lens, drop, twin
    rows = [_logint(rng, case["min_rows"], case["max_rows"])
            for _ in range(case["batch"])]
    if case["kind"] == "chunk":
        lens = [max(n, t) for n, t in zip(lens, rows)]
    return rows, lens


def work(case):
    kind = case["kind"]
    if kind in ("chunk", "cross"):
        rows, lens = _sizes(case)
        hq, hkv = case["q_heads"], case["kv_heads"]
        kv = 2 * sum(lens) * hkv * HEAD_DIM * 2
        qo = 2 * sum(rows) * hq * HEAD_DIM * 2
        if kind == "chunk":
            pairs = sum(t * (c - t) + t * (t + 1) // 2
                        for t, c in zip(rows, lens))
        else:
            pairs = sum(t * c for t, c in zip(rows, lens))
        return {"bytes": kv + qo, "flops": 4 * HEAD_DIM * hq * pairs}
    if kind == "mrope":
        hq, hkv = case["q_heads"], case["kv_heads"]
        t = case["tokens"]
        row = HEAD_DIM * 2
        # q in and out, k and v in and into their slots, slots, positions,
        # and the angles of the positions met (at most one table row a token
        # and axis, of which the pairs together use one row's worth)
        return {"bytes": t * (2 * hq * row + 4 * hkv * row + 4
                              + 4 * case["axes"] + 2 * HALF * 4),
                "flops": 6 * t * (hq + hkv) * HALF}
    if kind == "truncate":
        lens, drop, _ = _sizes(case)
        ps = case["page"]
        gone = sum(-(-n // ps) - -(-(n - d) // ps)
                   for n, d in zip(lens, drop))
        # contexts and new lengths in, contexts out; per dropped table entry
        # the entry in and out, its count in and out and its stack entry
        return {"bytes": 12 * case["batch"] + 20 * gone, "flops": 0}
    ps, hkv = case["page"], case["kv_heads"]
    page_bytes = ps * hkv * HEAD_DIM * 2
    # every count and used table entry in, moved counts, entries and moves out,
    # the stack out; K and V of every moved page in and out, in each layer
    ints = (case["pages"] + case["used"] + 5 * case["moves"]
            + case["pages"] - case["used"])
    pools = 4 * case["layers"] * case["moves"] * page_bytes
    return {"bytes": 4 * ints + pools, "flops": 0}


# ---- inputs -----------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda",
                       dtype=torch.float32).to(BF)


def _ints(values):
    return torch.tensor(values, dtype=I32, device="cuda")


def _tables(gen, counts, width, num_pages):
    """Block tables [len(counts)][width]: the pages of a shuffled pool in
    order, -1 behind each sequence's last."""
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(I32)
    cnt = torch.tensor(counts, device="cuda")
    start = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(width, device="cuda")
    idx = (start[:, None] + col).clamp_(max=num_pages - 1)
    return torch.where(col < cnt[:, None], perm[idx],
                       torch.full_like(perm[:1], -1)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    st = {"case": case}
    if kind in ("chunk", "cross"):
        rows, lens = _sizes(case)
        hq, hkv = case["q_heads"], case["kv_heads"]
        ps = case["page"]
        counts = [-(-n // ps) for n in lens]
        num_pages = sum(counts)
        qsl = [0]
        for t in rows:
            qsl.append(qsl[-1] + t)
        st.update(
            rows=rows, lens=lens, starts=qsl, scale=1 / math.sqrt(HEAD_DIM),
            q=_normal(gen, qsl[-1], hq, HEAD_DIM),
            k_pool=_normal(gen, num_pages, ps, hkv, HEAD_DIM),
            v_pool=_normal(gen, num_pages, ps, hkv, HEAD_DIM),
            tables=_tables(gen, counts, max(counts), num_pages),
            context_lens=_ints(lens), query_start_loc=_ints(qsl),
            err=torch.zeros(1, dtype=I32, device="cuda"))
        st["out"] = torch.empty_like(st["q"])
        if own:
            from paged_kv_cache_376_b200 import _lib as tv
            st["workspace"] = tv.chunk_workspace(case["batch"], max(rows), hq,
                                                 hkv)
        return st
    if kind == "mrope":
        hq, hkv = case["q_heads"], case["kv_heads"]
        t, ps = case["tokens"], case["page"]
        num_pages = -(-t // ps)
        # rows of one fused projection: q heads, k heads, v heads of a token
        qkv = _normal(gen, t, (hq + 2 * hkv) * HEAD_DIM)
        q, k, v = qkv.split([hq * HEAD_DIM, hkv * HEAD_DIM, hkv * HEAD_DIM], 1)
        # text and images in turn: a text token stands at one position on
        # every axis, an image token at its own place of a 24 x 24 grid
        base = torch.randint(0, case["max_position"] - 64, (), generator=gen,
                             device="cuda")
        i = torch.arange(t, device="cuda")
        image = (i // 576) % 2 == 1
        first = base // 2 + 48 * (i // 576)
        offset = torch.stack([i * 0, (i % 576) // 24, i % 24, i % 7])
        pos = torch.where(image, first + offset,
                          first + (i % 576) // 16)[:case["axes"]]
        pos = pos.clamp(max=case["max_position"] - 1)
        if case["interleaved"]:
            axis = torch.arange(HALF, device="cuda") % case["axes"]
        else:
            axis = torch.arange(HALF, device="cuda") * case["axes"] // HALF
        angle = (torch.arange(case["max_position"], device="cuda",
                              dtype=torch.float64)[:, None]
                 * 500000.0 ** (-torch.arange(HALF, device="cuda",
                                              dtype=torch.float64) / HALF))
        slots = torch.randperm(num_pages * ps, generator=gen, device="cuda")
        st.update(
            q=q.unflatten(1, (hq, HEAD_DIM)),
            k=k.unflatten(1, (hkv, HEAD_DIM)),
            v=v.unflatten(1, (hkv, HEAD_DIM)),
            positions=pos.to(I32).contiguous(), pair_axis=axis.to(I32),
            slots=slots[:t].to(I32).contiguous(),
            cos_sin=torch.stack([angle.cos(), angle.sin()], 1).float()
            .contiguous(),
            k_pool=_normal(gen, num_pages, ps, hkv, HEAD_DIM),
            v_pool=_normal(gen, num_pages, ps, hkv, HEAD_DIM),
            q_out=torch.empty(t, hq, HEAD_DIM, dtype=BF, device="cuda"),
            err=torch.zeros(1, dtype=I32, device="cuda"))
        return st
    if kind == "truncate":
        lens, drop, twin = _sizes(case)
        ps, b = case["page"], case["batch"]
        counts = [0 if twin[s] else -(-lens[s] // ps) for s in range(b)]
        num_pages = sum(counts) + sum(counts) // 4 + 1
        width = -(-max(lens) // ps)
        bt = _tables(gen, counts, width, num_pages)
        group = torch.tensor([s for s in range(b)], device="cuda")
        own_row = torch.tensor(twin, device="cuda")
        src = torch.cummax(torch.where(own_row, torch.zeros_like(group),
                                       group), 0).values
        bt = bt[src].contiguous()
        _pool_ints(st, num_pages, ps, bt, _ints(lens))
        st["new_lens"] = _ints([n - d for n, d in zip(lens, drop)])
        st["err"] = torch.zeros(1, dtype=I32, device="cuda")
        return st
    # compact: `moves` used pages lie at or above page `used`, the other used
    # pages and `moves` free ones below it, in shuffled order
    pages, used, moves = case["pages"], case["used"], case["moves"]
    hkv, ps, b = case["kv_heads"], case["page"], case["batch"]
    low = torch.randperm(used, generator=gen, device="cuda")[:used - moves]
    high = used + torch.randperm(pages - used, generator=gen,
                                 device="cuda")[:moves]
    ids = torch.cat([low, high])
    ids = ids[torch.randperm(used, generator=gen, device="cuda")].to(I32)
    cut = [used * s // b for s in range(b + 1)]
    counts = [cut[s + 1] - cut[s] for s in range(b)]
    width = max(counts)
    col = torch.arange(width, device="cuda")
    cnt = torch.tensor(counts, device="cuda")
    idx = (torch.tensor(cut[:-1], device="cuda")[:, None] + col).clamp_(
        max=used - 1)
    bt = torch.where(col < cnt[:, None], ids[idx],
                     torch.full_like(ids[:1], -1)).contiguous()
    lens = [n * ps - min(n, 1) * (s % ps) for s, n in enumerate(counts)]
    _pool_ints(st, pages, ps, bt, _ints(lens))
    st["pools"] = [(_normal(gen, pages, ps, hkv, HEAD_DIM),
                    _normal(gen, pages, ps, hkv, HEAD_DIM))
                   for _ in range(case["layers"])]
    st["moves"] = torch.zeros(2, max(1, pages // 2), dtype=I32, device="cuda")
    st["num_moves"] = torch.zeros(1, dtype=I32, device="cuda")
    st["err"] = torch.zeros(1, dtype=I32, device="cuda")
    return st


def _pool_ints(st, num_pages, ps, bt, lens):
    """The pool state of these tables beside them in one buffer, and a copy of
    it: ``run`` starts from the copy, since the call changes them in place."""
    b, width = bt.shape
    nstate = 4 + 4 * num_pages + POOL_MAX_SEQS
    pad = [-(-n // 4) * 4 for n in (nstate, b * width, b)]
    buf = torch.zeros(sum(pad), dtype=I32, device="cuda")
    state = buf[:nstate]
    tables = buf[pad[0]:pad[0] + b * width].view(b, width)
    ctx = buf[pad[0] + pad[1]:pad[0] + pad[1] + b]
    tables.copy_(bt)
    ctx.copy_(lens)
    held = torch.arange(width, device="cuda") < (lens[:, None] + ps - 1) // ps
    ref = torch.bincount(bt[held].long(), minlength=num_pages)
    free = (ref == 0).nonzero().flatten().flip(0)
    state[0] = free.numel()
    state[3] = ps
    state[4:4 + free.numel()] = free.to(I32)
    state[4 + num_pages:4 + 2 * num_pages] = ref.to(I32)
    st.update(num_pages=num_pages, page=ps, ints=buf, ints0=buf.clone(),
              state=state, tables=tables, context_lens=ctx)


# ---- one pass ---------------------------------------------------------------

def run(state):
    kind = state["case"]["kind"]
    if kind in ("chunk", "cross"):
        return _run_attention(state, kind == "chunk")
    if kind == "mrope":
        return _run_mrope(state)
    if kind == "truncate":
        return _run_truncate(state)
    return _run_compact(state)


def _run_attention(st, causal):
    out = st["out"]
    if own:
        from paged_kv_cache_376_b200 import _lib as tv
        call = tv.tv_paged_chunk if causal else tv.tv_paged_cross_attention
        call(out, st["q"], st["query_start_loc"], st["k_pool"], st["v_pool"],
             st["tables"], st["context_lens"], st["scale"], max(st["rows"]),
             workspace=st["workspace"], err=st["err"])
        return out
    ps, hkv = st["k_pool"].shape[1:3]
    hq = out.shape[1]
    g = hq // hkv
    for s, (t, c) in enumerate(zip(st["rows"], st["lens"])):
        r0 = st["starts"][s]
        ids = st["tables"][s, :-(-c // ps)].long()
        k = st["k_pool"][ids].flatten(0, 1)[:c].float().transpose(0, 1)
        v = st["v_pool"][ids].flatten(0, 1)[:c].float().transpose(0, 1)
        q = st["q"][r0:r0 + t].float().view(t, hkv, g, HEAD_DIM)
        q = q.permute(1, 0, 2, 3).reshape(hkv, t * g, HEAD_DIM)
        x = torch.matmul(q, k.transpose(1, 2)) * st["scale"]
        if causal:
            last = torch.arange(t * g, device="cuda") // g + (c - t)
            hidden = torch.arange(c, device="cuda") > last[:, None]
            x = x.masked_fill(hidden, float("-inf"))
        x = torch.exp(x - x.amax(-1, keepdim=True))
        o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
        o = o.view(hkv, t, g, HEAD_DIM).permute(1, 0, 2, 3)
        out[r0:r0 + t] = o.reshape(t, hq, HEAD_DIM).to(BF)
    return out


def _run_mrope(st):
    if own:
        from paged_kv_cache_376_b200 import _lib as tv
        tv.tv_kv_append_mrope(st["q_out"], st["q"], st["k"], st["v"],
                              st["slots"], st["positions"], st["pair_axis"],
                              st["k_pool"], st["v_pool"], st["cos_sin"],
                              err=st["err"])
        return st["q_out"], st["k_pool"], st["v_pool"]
    pair = torch.arange(HALF, device="cuda")
    pos = st["positions"].long()[st["pair_axis"].long()].t()    # [T][32]
    c = st["cos_sin"][pos, 0, pair][:, None]
    s = st["cos_sin"][pos, 1, pair][:, None]

    def rotated(x):
        a, b = x[..., :HALF].float(), x[..., HALF:].float()
        return torch.cat([a * c - b * s, b * c + a * s], -1).to(BF)

    st["q_out"].copy_(rotated(st["q"]))
    slots = st["slots"].long()
    st["k_pool"].flatten(0, 1)[slots] = rotated(st["k"])
    st["v_pool"].flatten(0, 1)[slots] = st["v"]
    return st["q_out"], st["k_pool"], st["v_pool"]


def _run_truncate(st):
    st["ints"].copy_(st["ints0"])
    state, bt, ctx, new = (st["state"], st["tables"], st["context_lens"],
                           st["new_lens"])
    if own:
        from paged_kv_cache_376_b200 import _lib as tv
        tv.tv_pool_truncate(state, bt, ctx, new, err=st["err"])
        return state, bt, ctx
    n, ps = st["num_pages"], st["page"]
    col = torch.arange(bt.shape[1], device="cuda")
    gone = ((col >= ((new + ps - 1) // ps)[:, None])
            & (col < ((ctx + ps - 1) // ps)[:, None]))
    ref = state[4 + n:4 + 2 * n]
    page = torch.where(gone, bt, n).flatten().long()
    lost = torch.zeros(n + 1, dtype=I32, device="cuda").index_add_(
        0, page, torch.ones_like(page, dtype=I32))[:n]
    freed = (lost > 0) & (ref == lost)
    ref -= lost
    # freed pages go onto the stack in ascending order
    rank = torch.cumsum(freed, 0)
    place = torch.where(freed, state[0] + rank - 1, n)
    stack = torch.cat([state[4:4 + n], state[:1]])
    stack[place] = torch.where(freed, torch.arange(n, device="cuda"),
                               stack[n].long()).to(I32)
    state[4:4 + n] = stack[:n]
    state[0] += rank[-1].to(I32)
    bt.masked_fill_(gone, -1)
    ctx.copy_(new)
    return state, bt, ctx


def _run_compact(st):
    st["ints"].copy_(st["ints0"])
    state, bt, ctx = st["state"], st["tables"], st["context_lens"]
    moves, count = st["moves"], st["num_moves"]
    if own:
        from paged_kv_cache_376_b200 import _lib as tv
        (k0, v0), rest = st["pools"][0], st["pools"][1:]
        tv.tv_pool_compact(state, bt, ctx, moves, count, k_pool=k0, v_pool=v0,
                           err=st["err"])
        for k, v in rest:
            tv.tv_page_copy(k, v, moves[0], moves[1], num_pairs=count,
                            err=st["err"])
    else:
        n, ps = st["num_pages"], st["page"]
        cap = moves.shape[1]
        ids = torch.arange(n, device="cuda")
        ref = state[4 + n:4 + 2 * n]
        held = ref > 0
        used = held.sum()
        src = held & (ids >= used)
        dst = ~held & (ids < used)
        num = src.sum()
        # i-th page to move goes to the i-th free page below `used`
        pad = moves[:, :1].expand(2, 1)
        lists = torch.cat([moves, pad], 1)
        lists[0, torch.where(src, torch.cumsum(src, 0) - 1, cap)] = ids.to(I32)
        lists[1, torch.where(dst, torch.cumsum(dst, 0) - 1, cap)] = ids.to(I32)
        moves.copy_(lists[:, :cap])
        count.copy_(num[None])
        valid = torch.arange(cap, device="cuda") < num
        a = torch.where(valid, moves[0], n).long()
        b = torch.where(valid, moves[1], n).long()
        where = torch.arange(n + 1, device="cuda", dtype=I32)
        where[a] = b.to(I32)
        where[n] = -1
        live = (torch.arange(bt.shape[1], device="cuda")
                < ((ctx + ps - 1) // ps)[:, None])
        bt.copy_(torch.where(live, where[bt.clamp(min=0).long()], bt))
        more = torch.cat([ref, ref[:1] * 0])
        more[b] = more[a]
        more[a] = 0
        ref.copy_(more[:n])
        place = n - 1 - ids                      # n-1, n-2, ... , used
        stack = state[4:4 + n]
        stack.copy_(torch.where(ids < n - used, place.to(I32), stack))
        state[0] = (n - used).to(I32)
        num_moves = st["case"]["moves"]
        for k, v in st["pools"]:
            k[moves[1, :num_moves].long()] = k[moves[0, :num_moves].long()]
            v[moves[1, :num_moves].long()] = v[moves[0, :num_moves].long()]
    return [state, bt, ctx, moves, count] + [p for kv in st["pools"]
                                             for p in kv]


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    kind = case["kind"]
    if kind == "truncate":
        return None          # whole numbers only
    st = prepare(case, seed)
    f64 = torch.float64
    if kind == "compact":
        n = st["num_pages"]
        ref = st["ints0"][4 + n:4 + 2 * n].tolist()
        used = sum(r > 0 for r in ref)
        src = [p for p in range(used, n) if ref[p] > 0]
        dst = [p for p in range(used) if ref[p] == 0]
        src, dst = (torch.tensor(x, dtype=torch.long, device="cuda")
                    for x in (src, dst))
        pools = []
        for p in (p for kv in st["pools"] for p in kv):
            pools.append(p.to(f64))
            pools[-1].index_copy_(0, dst, pools[-1][src])
        return [None] * 5 + pools
    if kind == "mrope":
        # angles from the definition, not from the 32-bit table
        inv = torch.tensor([500000.0 ** (-i / HALF) for i in range(HALF)],
                           dtype=f64, device="cuda")
        axis = st["pair_axis"].long()
        theta = st["positions"].to(f64)[axis, :].T * inv

        def turn(x):
            z = torch.complex(x[..., :HALF].to(f64), x[..., HALF:].to(f64))
            z = z * torch.polar(torch.ones_like(theta), theta).unsqueeze(1)
            return torch.cat((z.real, z.imag), dim=-1)

        kp = st["k_pool"].to(f64).flatten(0, 1)
        vp = st["v_pool"].to(f64).flatten(0, 1)
        kp.index_copy_(0, st["slots"].long(), turn(st["k"]))
        vp.index_copy_(0, st["slots"].long(), st["v"].to(f64))
        shape = st["k_pool"].shape
        return turn(st["q"]), kp.view(shape), vp.view(shape)
    ps, hkv = case["page"], case["kv_heads"]
    res = torch.zeros(st["q"].shape, dtype=f64, device="cuda")
    flat_k = st["k_pool"].view(-1, hkv, HEAD_DIM)
    flat_v = st["v_pool"].view(-1, hkv, HEAD_DIM)
    for s in range(case["batch"]):
        lo, hi = st["starts"][s], st["starts"][s + 1]
        n = st["lens"][s]
        j = torch.arange(n, device="cuda")
        slot = st["tables"][s].long()[j // ps] * ps + j % ps
        keys, vals = flat_k[slot].to(f64), flat_v[slot].to(f64)
        for h in range(case["q_heads"]):
            kv = h * hkv // case["q_heads"]
            w = st["q"][lo:hi, h].to(f64) @ keys[:, kv].T / 8.0
            if kind == "chunk":
                w = w + torch.triu(torch.full_like(w, -math.inf),
                                   diagonal=n - (hi - lo) + 1)
            w = torch.exp(w - torch.logsumexp(w, dim=1, keepdim=True))
            res[lo:hi, h] = w @ vals[:, kv]
    return res
