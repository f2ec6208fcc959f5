"""The serving operators measured: page tables and slot maps, the K/V store, packed prompt attention, decode
attention over a shared prefix, and rules on logits.

listed() and draw() give cases, prepare() their inputs, run() one pass: the plain form, or with `own` the calls of
the package.  work() counts what a pass cannot do without, exact() gives its result in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decode step of 16 rows (8 variations, each a conditional and an unconditional row) in pages of 256
        dict(name="map_step_16", op="map", requests=16, fresh=1, fresh_to=1, cached=40, cached_to=9000, page=256),
        # a batch of ragged prompts entering an empty cache
        dict(name="map_prompts_256", op="map", requests=256, fresh=17, fresh_to=2048, cached=0, cached_to=0, page=64),
        # the new token of 16 rows, one layer
        dict(name="store_step_16", op="store", tokens=16, kv_heads=8, dim=128, page=256, type="bf16"),
        # a packed batch of prompts, one layer
        dict(name="store_prompts_16k", op="store", tokens=16387, kv_heads=8, dim=128, page=64, type="f16"),
        # a conditional and an unconditional prompt of usual length
        dict(name="prompt_pair_300", op="prompt", requests=2, fresh=237, fresh_to=300, cached=0, cached_to=0,
             heads=32, kv_heads=8, dim=128, type="bf16"),
        # ragged prompts, some continuing a cached part, in the shape of the small decoder's heads
        dict(name="prompt_ragged_16", op="prompt", requests=16, fresh=61, fresh_to=2048, cached=0, cached_to=900,
             heads=16, kv_heads=16, dim=64, type="f16"),
        # two histories at the cap of 9000 frames
        dict(name="prompt_pair_9000", op="prompt", requests=2, fresh=9000, fresh_to=9000, cached=0, cached_to=0,
             heads=32, kv_heads=8, dim=128, type="bf16"),
        # four variations right after a prompt of 300 tokens
        dict(name="prefix_start_4", op="prefix", requests=4, prefix=300, own=1, own_to=40, page=256,
             heads=32, kv_heads=8, dim=128, type="bf16"),
        # 16 variations far into a song that continues a given one
        dict(name="prefix_song_16", op="prefix", requests=16, prefix=4500, own=700, own_to=4500, page=256,
             heads=32, kv_heads=8, dim=128, type="bf16"),
        # many short continuations of one long context, small pages
        dict(name="prefix_batch_128", op="prefix", requests=128, prefix=9001, own=5, own_to=700, page=16,
             heads=32, kv_heads=8, dim=128, type="f16"),
        # the frame draw's logits (16384 codes and the end token) of a conditional pair, 1500 frames in
        dict(name="rules_frame_2", op="rules", rows=2, vocab=16385, history=1500, bias=16, masks=1, type="f32"),
        # a full vocabulary for a large batch
        dict(name="rules_vocab_192", op="rules", rows=192, vocab=200000, history=4096, bias=300, masks=24, type="f32"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["map", "store", "prompt", "prefix", "rules"])
    heads, kv_heads = rng.choice([(32, 8), (16, 16), (4, 2), (16, 1), (24, 4), (8, 8)])
    shape = dict(heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]), type=rng.choice(["bf16", "f16"]))
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "map":
        fresh = rng.choice([1, _spread(rng, 1, 200)])
        return dict(op=op, requests=_spread(rng, 1, 256), fresh=fresh, fresh_to=fresh if fresh == 1 else _spread(rng, fresh, 2048),
                    cached=rng.choice([0, _spread(rng, 1, 500)]), cached_to=_spread(rng, 500, 9000), page=page)
    if op == "store":
        return dict(op=op, tokens=_spread(rng, 1, 16387), kv_heads=kv_heads, dim=shape["dim"], page=page, type=shape["type"])
    if op == "prompt":
        requests = _spread(rng, 1, 32)
        longest = min(9000, int(9000 * math.sqrt(2.0 * 32 / (requests * heads))))
        fresh = _spread(rng, 1, longest // 2)
        return dict(op=op, requests=requests, fresh=fresh, fresh_to=_spread(rng, fresh, longest // 2),
                    cached=0, cached_to=rng.choice([0, _spread(rng, 1, longest // 2)]), **shape)
    if op == "prefix":
        low = _spread(rng, 1, 1000)
        requests = _spread(rng, 1, 128)
        return dict(op=op, requests=requests, prefix=_spread(rng, 16, 9000), own=low,
                    own_to=_spread(rng, low, max(low, min(4500, 90000 // requests))), page=page, **shape)
    return dict(op=op, rows=_spread(rng, 1, 192), vocab=_spread(rng, 500, 200000), history=_spread(rng, 1, 4096),
                bias=rng.choice([0, _spread(rng, 1, 300)]), masks=rng.choice([0, 1, 3]), type=rng.choice(["f32", "bf16", "f16"]))


def _lengths(n, low, high):
    """n whole numbers from low to high, even over the logarithm, in a mixed order."""
    if low == high or n == 1:
        return [high] * n
    a = max(low, 1)
    v = [int(round(a * (high / a) ** (i / (n - 1)))) for i in range(n)]
    if low == 0:
        v[0] = 0
    step = next(s for s in (7, 5, 3, 11, 13, 1) if math.gcd(s, n) == 1)
    return [v[(i * step + n // 2) % n] for i in range(n)]


def _fresh_cached(case):
    n = case["requests"]
    fresh = _lengths(n, case["fresh"], case["fresh_to"])
    cached = _lengths(n, min(case["cached"], case["cached_to"]), case["cached_to"])
    return fresh, cached[1:] + cached[:1]


def _ceil(a, b):
    return -(-a // b)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case)
    op = case["op"]
    if op in ("map", "prompt"):
        fresh, cached = _fresh_cached(case)
        total = sum(fresh)
    if op == "map":
        # every request's row of the table holds the pages of its cached tokens; the other pages of the pool are free
        n, page = case["requests"], case["page"]
        have = [_ceil(c, page) for c in cached]
        used = sum(have)
        wanted = sum(_ceil(c + f, page) for c, f in zip(cached, fresh)) - used
        n_pages = used + wanted + 64
        pages = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((n, max(_ceil(c + f, page) for c, f in zip(cached, fresh)) + 2), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(table.shape[1], device="cuda")
        table[at < _int32(have)[:, None]] = pages[:used]
        rows = -(-total // 16) * 16  # the maps are padded to a whole number of 16 tokens
        state.update(fresh=_int32(fresh), cached=_int32(cached), free=pages[used:].contiguous(), table=table, n_pages=n_pages,
                     cu=torch.empty(n + 1, dtype=torch.int32, device="cuda"), lens=torch.empty(n, dtype=torch.int32, device="cuda"),
                     positions=torch.empty(rows, dtype=torch.int32, device="cuda"), seqs=torch.empty(rows, dtype=torch.int32, device="cuda"),
                     slots=torch.empty(rows, dtype=torch.int64, device="cuda"), taken=torch.empty(1, dtype=torch.int32, device="cuda"))
    elif op == "store":
        t, hk, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
        n_pages = _ceil(t, page) + 3
        slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:t]
        qkv = torch.randn(t, 2 * hk, d, generator=g, device="cuda").to(TYPES[case["type"]])  # the projection's k and v columns
        pool = torch.zeros(n_pages, 2, hk, page, d, dtype=TYPES[case["type"]], device="cuda")
        state.update(k=qkv[:, :hk], v=qkv[:, hk:], slots=slots, pool=pool)
    elif op == "prompt":
        hq, hk, d, kind = case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
        keys = [f + c for f, c in zip(fresh, cached)]
        cu_q = torch.tensor([0] + fresh).cumsum(0).to(torch.int32).cuda()
        cu_k = torch.tensor([0] + keys).cumsum(0).to(torch.int32).cuda() if max(cached) else None
        q = torch.randn(total, hq, d, generator=g, device="cuda").to(kind)  # after the per-head norm: entries of size one
        k = torch.randn(sum(keys), hk, d, generator=g, device="cuda").to(kind)
        v = torch.randn(sum(keys), hk, d, generator=g, device="cuda").to(kind)
        state.update(q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, longest=(max(fresh), max(keys)), out=torch.empty_like(q),
                     lse=torch.empty(total, hq, device="cuda"))
    elif op == "prefix":
        n, hq, hk, d, kind, page = case["requests"], case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]], case["page"]
        lens = _lengths(n, case["own"], case["own_to"])
        np_, most = _ceil(case["prefix"], page), _ceil(max(lens), page)
        n_pages = np_ + sum(_ceil(x, page) for x in lens) + 5
        pages = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
        own_pages = _int32([_ceil(x, page) for x in lens])
        table[torch.arange(most, device="cuda") < own_pages[:, None]] = pages[np_:n_pages - 5]
        pool = torch.randn(n_pages, 2, hk, page, d, generator=g, device="cuda", dtype=torch.float32).to(kind)
        q = torch.randn(n, hq, d, generator=g, device="cuda").to(kind)
        state.update(q=q, pool=pool, pages=pages[:np_].contiguous(), table=table, lens=_int32(lens), out=torch.empty_like(q),
                     lse=torch.empty(n, hq, device="cuda"))
        if own:
            from autoregressive_audio_token_b200 import ops
            size = ops.m3_attn_prefix_workspace(n, hq, hk, d, np_, page, most)
            state.update(workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    else:
        r, n = case["rows"], case["vocab"]
        logits = (3 * torch.randn(r, n, generator=g, device="cuda")).to(TYPES[case["type"]])
        # tokens come again and again: squared uniform numbers favour the low ones
        history = (torch.rand(r, case["history"], generator=g, device="cuda").square() * n).to(torch.int32).clamp_(max=n - 1)
        hist_len = torch.randint(case["history"] // 2, case["history"] + 1, (r,), generator=g, device="cuda").to(torch.int32)
        u = lambda low, high: low + (high - low) * torch.rand(r, generator=g, device="cuda")  # noqa: E731
        state.update(logits=logits, history=history, hist_len=hist_len, repetition=u(1.0, 1.5), frequency=u(0.0, 0.3), presence=u(0.0, 0.6),
                     bias_ids=None, bias=None, mask=None, mask_row=None, out=torch.empty_like(logits))
        if case["bias"]:
            nb = min(case["bias"], n)
            state.update(bias_ids=torch.rand(r, n, generator=g, device="cuda").topk(nb).indices.to(torch.int32),
                         bias=4 * torch.randn(r, nb, generator=g, device="cuda"))
        if case["masks"]:
            words = _ceil(n, 32)
            mask = torch.randint(-2**31, 2**31, (case["masks"], words), generator=g, device="cuda").to(torch.int32)
            mask_row = torch.randint(0, case["masks"], (r,), generator=g, device="cuda").to(torch.int32)
            mask_row[r // 2:][:1] = -1  # one row without a grammar
            state.update(mask=mask, mask_row=mask_row)
    return state


def run(s):
    return {"map": _map, "store": _store, "prompt": _prompt, "prefix": _prefix, "rules": _rules}[s["op"]](s)


def _map(s):
    if own:
        from autoregressive_audio_token_b200 import ops
        ops.m3_kv_map(s["fresh"], s["cached"], s["free"], s["table"], s["page"], s["n_pages"], s["cu"], s["positions"],
                      s["slots"], s["seqs"], s["lens"], s["taken"])
        return {n: s[n] for n in ("table", "cu", "positions", "slots", "seqs", "lens", "taken")}
    fresh, cached, free, table, page = s["fresh"], s["cached"], s["free"], s["table"], s["page"]
    lens = fresh + cached
    cu = torch.cat([fresh.new_zeros(1), fresh.cumsum(0, dtype=torch.int32)])
    have = (cached + page - 1) // page
    need = (((lens + page - 1) // page).clamp(max=table.shape[1]) - have).clamp(min=0)
    first = need.cumsum(0, dtype=torch.int32) - need
    at = torch.arange(table.shape[1], device="cuda", dtype=torch.int32) - have[:, None]
    new = (at >= 0) & (at < need[:, None])
    place = first[:, None] + at
    page_of = torch.where(place < free.numel(), free[place.clamp(0, free.numel() - 1)], -1)
    table = torch.where(new, page_of, table)
    token = torch.arange(s["slots"].numel(), device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(cu[1:], token, right=True)
    there = token < cu[-1]
    seq = seq.clamp(max=fresh.numel() - 1)
    pos = cached[seq] + token - cu[seq]
    col = pos // page
    number = table[seq, col.clamp(0, table.shape[1] - 1)].long()
    good = there & (col < table.shape[1]) & (number >= 0) & (number < s["n_pages"])
    slots = torch.where(good, number * page + pos % page, -1)
    return {"table": table, "cu": cu, "positions": torch.where(there, pos, -1), "slots": slots,
            "seqs": torch.where(there, seq, -1).to(torch.int32), "lens": lens, "taken": need.sum(0, keepdim=True, dtype=torch.int32)}


def _store(s):
    if own:
        from autoregressive_audio_token_b200 import ops
        ops.m3_kv_store(s["k"], s["v"], s["slots"], s["pool"])
        return s["pool"]
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    s["pool"][page, 0, :, at] = s["k"]
    s["pool"][page, 1, :, at] = s["v"]
    return s["pool"]


def _prompt(s):
    if own:
        from autoregressive_audio_token_b200 import ops
        ops.m3_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["out"], s["lse"], cu_k=s["cu_k"])
        return {"out": s["out"], "lse": s["lse"]}
    q, k, v, cu_q = s["q"], s["k"], s["v"], s["cu_q"]
    cu_k = cu_q if s["cu_k"] is None else s["cu_k"]
    lq, lk = s["longest"]
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    # the sequences padded to the longest: [requests, heads, length, dim]
    iq, ik = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda")
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    at_q = (cu_q[:-1, None] + iq).clamp(max=q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1)
    qp = q[at_q].float().mul_(d ** -0.5).transpose(1, 2).unflatten(1, (hk, hq // hk))
    kp = k[at_k].float().transpose(1, 2).unsqueeze(2)
    vp = v[at_k].float().transpose(1, 2).unsqueeze(2)
    w = qp @ kp.transpose(-1, -2)
    last = iq + (nk - nq)[:, None]  # each query's own position among the keys
    seen = ik <= last[:, :, None]
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp_(min=-1e30)
    w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w @ vp) / total.clamp(min=1e-30)
    lse = torch.log(total).add_(top).squeeze(-1)
    rows = (iq < nq[:, None]).flatten().nonzero_static(size=q.shape[0]).squeeze(1)  # the padded rows that are queries, in order
    o = o.flatten(1, 2).transpose(1, 2).flatten(0, 1)[rows]
    lse = lse.flatten(1, 2).transpose(1, 2).flatten(0, 1)[rows]
    return {"out": o.to(q.dtype), "lse": lse}


def _prefix(s):
    if own:
        from autoregressive_audio_token_b200 import ops
        ops.m3_attn_prefix(s["q"], s["pool"], s["pages"], s["prefix"], s["table"], s["lens"], s["out"], s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    q, pool, lens = s["q"], s["pool"], s["lens"]
    n, hq, d = q.shape
    hk = pool.shape[2]
    shared = pool[s["pages"]].float()  # [pages, 2, heads, page, dim]
    shared = shared.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :s["prefix"]]
    each = pool[s["table"].clamp(min=0)].float()  # [rows, pages, 2, heads, page, dim]
    each = each.permute(2, 0, 3, 1, 4, 5).flatten(3, 4)
    qf = q.float().mul_(d ** -0.5).unflatten(1, (hk, hq // hk))
    w_shared = torch.einsum("bhgd,hpd->bhgp", qf, shared[0])
    w_each = qf @ each[0].transpose(-1, -2)
    there = torch.arange(w_each.shape[-1], device="cuda") < lens[:, None]
    w_each = w_each.masked_fill(~there[:, None, None], -math.inf)
    top = torch.maximum(w_shared.amax(-1, keepdim=True), w_each.amax(-1, keepdim=True))
    w_shared, w_each = (w_shared - top).exp_(), (w_each - top).exp_()
    total = w_shared.sum(-1, keepdim=True) + w_each.sum(-1, keepdim=True)
    v_each = torch.where(there[:, None, :, None], each[1], 0.0)
    o = (torch.einsum("bhgp,hpd->bhgd", w_shared, shared[1]) + w_each @ v_each) / total
    return {"out": o.flatten(1, 2).to(q.dtype), "lse": (torch.log(total) + top).flatten(1)}


def _rules(s):
    if own:
        from autoregressive_audio_token_b200 import ops
        ops.m3_logit_rules(s["logits"], s["out"], history=s["history"], hist_len=s["hist_len"], repetition=s["repetition"],
                           frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"],
                           mask=s["mask"], mask_row=s["mask_row"])
        return s["out"]
    x = s["logits"].float()
    r, n = x.shape
    counted = torch.arange(s["history"].shape[1], device="cuda") < s["hist_len"][:, None]
    count = torch.zeros(r, n, dtype=torch.int32, device="cuda").scatter_add_(1, s["history"].long(), counted.to(torch.int32))
    rep, seen = s["repetition"][:, None], count > 0
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - torch.where(seen, s["presence"][:, None], 0.0)
    if s["bias"] is not None:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        i = torch.arange(n, device="cuda")
        bits = s["mask"][s["mask_row"].clamp(min=0)]
        allowed = ((bits[:, i >> 5] >> (i & 31)) & 1).bool() | (s["mask_row"] < 0)[:, None]
        x = x.masked_fill(~allowed, -math.inf)
    return x.to(s["logits"].dtype)


def work(case):
    op = case["op"]
    size = 4 if case.get("type") == "f32" else 2
    if op == "map":
        fresh, cached = _fresh_cached(case)
        page, total = case["page"], sum(fresh)
        new = sum(_ceil(c + f, page) - _ceil(c, page) for c, f in zip(cached, fresh))
        # lengths in, sums and lengths out, free pages in, table entries out, a token's position, sequence and slot out
        return {"bytes": 16.0 * case["requests"] + 8.0 * new + 16.0 * total, "flops": 4.0 * total}
    if op == "store":
        return {"bytes": case["tokens"] * (4.0 * case["kv_heads"] * case["dim"] * size + 8), "flops": 0}
    if op == "prompt":
        fresh, cached = _fresh_cached(case)
        pairs = sum(f * c + f * (f + 1) / 2 for f, c in zip(fresh, cached))
        tq, tk = sum(fresh), sum(fresh) + sum(cached)
        return {"bytes": 2.0 * case["dim"] * size * (tq * case["heads"] + tk * case["kv_heads"]) + 4.0 * tq * case["heads"],
                "flops": 4.0 * case["heads"] * case["dim"] * pairs}
    if op == "prefix":
        n, lens = case["requests"], _lengths(case["requests"], case["own"], case["own_to"])
        return {"bytes": 2.0 * size * case["dim"] * (case["kv_heads"] * (case["prefix"] + sum(lens)) + n * case["heads"]) + 4.0 * n * case["heads"],
                "flops": 4.0 * case["heads"] * case["dim"] * (n * case["prefix"] + sum(lens))}
    values = float(case["rows"]) * case["vocab"]
    masks = case["masks"] * case["vocab"] / 8.0
    return {"bytes": 2.0 * size * values + masks + case["rows"] * (3.0 * case["history"] + 8.0 * case["bias"]), "flops": 4.0 * values}


def exact(case, seed):
    op = case["op"]
    if op == "map":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "store":
        # slot by slot, from the pool's flat view of rows of `dim` numbers
        n, two, hk, page, d = s["pool"].shape
        rows = torch.zeros(n * two * hk * page, d, dtype=torch.float64, device="cuda")
        head = torch.arange(hk, device="cuda")
        at = ((s["slots"] // page * two)[:, None] * hk + head) * page + (s["slots"] % page)[:, None]
        rows[at.flatten()] = s["k"].double().flatten(0, 1)
        rows[(at + hk * page).flatten()] = s["v"].double().flatten(0, 1)
        return rows.view(n, two, hk, page, d)
    if op == "prompt":
        cu_q = s["cu_q"].tolist()
        cu_k = cu_q if s["cu_k"] is None else s["cu_k"].tolist()
        q, k, v = s["q"], s["k"], s["v"]
        group = q.shape[1] // k.shape[1]
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
        for a, b, ka, kb in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
            for h in range(q.shape[1]):
                kd, vd = k[ka:kb, h // group].double(), v[ka:kb, h // group].double()
                z = q[a:b, h].double() @ kd.T / math.sqrt(q.shape[2])
                z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(kb - ka - (b - a) + 1), -math.inf)
                out[a:b, h] = torch.softmax(z, 1) @ vd
                lse[a:b, h] = torch.logsumexp(z, 1)
        return {"out": out, "lse": lse}
    if op == "prefix":
        q, pool, lens = s["q"], s["pool"], s["lens"].tolist()
        group = q.shape[1] // pool.shape[2]
        out, lse = [], []
        for b, own_len in enumerate(lens):
            own_pages = s["table"][b, : _ceil(own_len, case["page"])]
            parts = []
            for pages, count in ((s["pages"], case["prefix"]), (own_pages, own_len)):
                kv = pool[pages.long()].double()  # [pages, 2, heads, page, dim]
                parts.append(torch.cat(list(kv), dim=2)[:, :, :count] if len(pages) else kv.new_zeros(2, pool.shape[2], 0, pool.shape[4]))
            kd, vd = torch.cat(parts, dim=2).repeat_interleave(group, dim=1)
            z = torch.einsum("hd,hpd->hp", q[b].double(), kd) / math.sqrt(q.shape[2])
            out.append(torch.einsum("hp,hpd->hd", torch.softmax(z, 1), vd))
            lse.append(torch.logsumexp(z, 1))
        return {"out": torch.stack(out), "lse": torch.stack(lse)}
    x = s["logits"].double()
    for r in range(x.shape[0]):
        used, times = s["history"][r, : int(s["hist_len"][r])].long().unique(return_counts=True)
        y, rep = x[r, used], s["repetition"][r].double()
        y = torch.where(y > 0, y / rep, y * rep) - s["frequency"][r].double() * times - s["presence"][r].double()
        x[r, used] = y
        if s["bias"] is not None:
            x[r].index_add_(0, s["bias_ids"][r].long(), s["bias"][r].double())
        if s["mask"] is not None and s["mask_row"][r] >= 0:
            words = s["mask"][s["mask_row"][r].long()].long()
            bits = (words[:, None] >> torch.arange(32, device="cuda")) & 1
            x[r, bits.flatten()[: x.shape[1]] == 0] = -math.inf
    return x
