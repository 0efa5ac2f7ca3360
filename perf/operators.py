"""The attention that follows the indexer, and the cache around it: cases, plain forms and definitions.

Five operators of one serving step:

  tables   request lengths -> row and key offsets, block-table entries, slots and visible lengths
  store    new tokens written into the paged caches by slot (latent + rotary part, or K and V)
  latent   attention over one shared latent vector a token (absorbed form), whole prefix or selected keys
  paged    grouped-query attention over a paged K/V cache, whole prefix or selected 128-key blocks

``run`` takes what ``prepare`` gives and makes one pass: in elementary torch operations where ``own`` is
false, through the framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
LATENT, ROPE = 512, 64           # a latent token: 512 shared values (keys and values), 64 rotary ones (keys only)
DK = LATENT + ROPE
D = 128                          # head size of the paged K/V cache
BLOCK = 128                      # keys of one selectable block


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 running requests: every request gets one token, a few get a new page
        dict(name="tables_decode", op="tables", reqs=64, new_lo=1, new_hi=1, cached_lo=1, cached_hi=16384, page=64),
        # a large mixed step: thousands of requests, most decoding, prompts of up to 255 tokens among them
        dict(name="tables_mixed", op="tables", reqs=2048, new_lo=0, new_hi=255, cached_lo=0, cached_hi=32768, page=64),
        # the new latents of one decode step
        dict(name="store_latent_decode", op="store", kind="latent", tokens=64, kv_heads=1, page=64, pages=1024, dtype="bf16"),
        # a prefill chunk's keys and values, four KV heads, pages of 128
        dict(name="store_kv_prefill", op="store", kind="kv", tokens=32768, kv_heads=4, page=128, pages=512, dtype="bf16"),
        # the smallest call: one new token of a short request, the 16 heads of one shard
        dict(name="latent_single", op="latent", reqs=1, rows=1, heads=16, len_lo=777, len_hi=777, page=64, topk=0, dtype="fp16"),
        # the indexer's verify step: 4 rows over 16,384 keys, each row its own top-2048 keys
        dict(name="latent_verify_top2048", op="latent", reqs=1, rows=4, heads=64, len_lo=16384, len_hi=16384, page=64, topk=2048,
             dtype="bf16"),
        # long contexts read whole: 16 requests, one new token each, all 128 heads on this GPU
        dict(name="latent_long_decode", op="latent", reqs=16, rows=1, heads=128, len_lo=30001, len_hi=119999, page=64, topk=0,
             dtype="bf16"),
        # a prefill chunk after the indexer: every row attends to its own 2048 keys of a 32k context
        dict(name="latent_prefill_top2048", op="latent", reqs=1, rows=1024, heads=128, len_lo=32768, len_hi=32768, page=64, topk=2048,
             dtype="bf16"),
        # the smallest call: one new token of a short request, 32 query heads on 4 KV heads
        dict(name="paged_single", op="paged", reqs=1, rows=1, heads=32, kv_heads=4, len_lo=333, len_hi=333, page=128, topk=0, dtype="fp16"),
        # a verify step of 16 requests, 4 rows each, ragged contexts read whole
        dict(name="paged_verify", op="paged", reqs=16, rows=4, heads=32, kv_heads=4, len_lo=8191, len_hi=32768, page=128, topk=0,
             dtype="bf16"),
        # block-sparse decode: each KV head reads its 16 selected blocks of 128 keys
        dict(name="paged_decode_16_blocks", op="paged", reqs=64, rows=1, heads=32, kv_heads=4, len_lo=1000, len_hi=8192, page=128,
             topk=16, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "latent", "latent", "paged", "paged"])
    page = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "tables":
        new_lo = rng.choice([0, 1])
        return dict(op=op, reqs=_log_int(rng, 1, 2048), new_lo=new_lo, new_hi=max(1, _log_int(rng, 1, 255)), cached_lo=rng.choice([0, 1]),
                    cached_hi=_log_int(rng, 1, 32768), page=page)
    if op == "store":
        kind = rng.choice(["latent", "kv"])
        tokens = _log_int(rng, 1, 32768)
        pages = -(-tokens // page) + _log_int(rng, 1, 256)
        return dict(op=op, kind=kind, tokens=tokens, kv_heads=1 if kind == "latent" else rng.choice([1, 2, 4]), page=page, pages=pages,
                    dtype=dtype)
    if op == "latent":
        heads = rng.choice([8, 16, 20, 32, 64, 128])
        if rng.random() < 0.5:  # whole prefix
            hi = _log_int(rng, 1, 100000)
            reqs, rows = _log_int(rng, 1, 24), rng.choice([1, 1, 2, 4])
            reqs = max(1, min(reqs, 1200000 // hi, 200000000 // (hi * rows * heads)))
            return dict(op=op, reqs=reqs, rows=rows, heads=heads, len_lo=max(rows, hi // rng.choice([1, 2, 16])), len_hi=max(rows, hi),
                        page=page, topk=0, dtype=dtype)
        rows, topk, reqs = _log_int(rng, 1, 1024), _log_int(rng, 1, 2048), rng.choice([1, 1, 3, 16])
        reqs = max(1, min(reqs, 250000000 // (rows * topk * heads)))
        hi = max(rows, _log_int(rng, 64, 32768))
        return dict(op=op, reqs=reqs, rows=rows, heads=heads, len_lo=max(rows, hi // 2), len_hi=hi, page=page, topk=topk, dtype=dtype)
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 5, 8, 16])
    hi = _log_int(rng, 1, 32768)
    if rng.random() < 0.5:
        reqs, rows = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 4])
        reqs = max(1, min(reqs, 1200000 // (hi * kv_heads)))
        return dict(op=op, reqs=reqs, rows=rows, heads=kv_heads * group, kv_heads=kv_heads, len_lo=max(rows, hi // rng.choice([1, 2, 16])),
                    len_hi=max(rows, hi), page=page, topk=0, dtype=dtype)
    reqs, rows, topk = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 4]), _log_int(rng, 1, 32)
    reqs = max(1, min(reqs, 1200000 // (rows * topk * BLOCK * kv_heads)))
    return dict(op=op, reqs=reqs, rows=rows, heads=kv_heads * group, kv_heads=kv_heads, len_lo=max(rows, hi // 2), len_hi=max(rows, hi),
                page=page, topk=topk, dtype=dtype)


def _spread(n, lo, hi, step):
    """n whole numbers over [lo, hi], the same for the same arguments, both ends among them."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _coprime(n):
    s = max(1, int(n * 0.618))
    while math.gcd(s, n) != 1:
        s += 1
    return s


def _lens(case):
    return _spread(case["reqs"], case["len_lo"], case["len_hi"], _coprime(case["reqs"]))


def _new(case):
    """Two of three requests decode one token (or none), the third brings a prompt's."""
    n = _spread(case["reqs"], case["new_lo"], case["new_hi"], _coprime(case["reqs"]))
    return [v if i % 3 == 0 else min(max(case["new_lo"], 1), case["new_hi"]) for i, v in enumerate(n)]


def work(case):
    op = case["op"]
    if op == "tables":
        rows, b = sum(_new(case)), case["reqs"]
        return {"bytes": 8 * rows + 16 * b + 8 * (rows // case["page"] + b), "flops": 0}
    if op == "store":
        row = DK if case["kind"] == "latent" else 2 * D * case["kv_heads"]
        return {"bytes": case["tokens"] * (2 * 2 * row + 4), "flops": 0}
    heads, rows, lens = case["heads"], case["rows"], _lens(case)
    kv, dk, dv, key = (1, DK, LATENT, 2 * DK) if op == "latent" else (case["kv_heads"], D, D, 4 * D)
    per = case["topk"] * (1 if op == "latent" else BLOCK)
    size = flops = 0
    for n in lens:
        seen = [n - rows + i + 1 if not per else min(per, n - rows + i + 1) for i in range(rows)]
        size += kv * key * min(n, sum(seen) if per else n)
        flops += 2 * heads * (dk + dv) * sum(seen)
    t = rows * len(lens)
    return {"bytes": size + 2 * t * heads * (dk + dv) + 4 * t * heads + 4 * t * case["topk"] * (1 if op == "latent" else kv), "flops": flops}


# ------------------------------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _randn(shape, g, dtype, by=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return x if by == 1.0 else x.mul_(by)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "tables":
        page, b = case["page"], case["reqs"]
        new = _int32(_new(case))
        cached = _spread(b, case["cached_lo"], case["cached_hi"], _coprime(b))
        shift = int(torch.randint(0, b, (1,), generator=g, device=DEV))
        cached = _int32(cached[shift:] + cached[:shift])
        has = (cached + page - 1) // page
        width = int(has.max()) + -(-case["new_hi"] // page) + 1
        total = b * width
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = perm.view(b, width).clone()
        held = torch.arange(width, device=DEV)[None, :] < has[:, None]
        s.update(cached=cached, new=new, free=table[~held].contiguous(), table=torch.where(held, table, -1), rows=sum(_new(case)),
                 page=page, num_pages=total)
    elif case["op"] == "store":
        n, page, pages, h = case["tokens"], case["page"], case["pages"], case["kv_heads"]
        dt = _dtype(case)
        s.update(slots=torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32), page=page)
        if case["kind"] == "latent":
            s.update(first=_randn((n, LATENT), g, dt), second=_randn((n, ROPE), g, dt),
                     cache=torch.zeros((pages, page, DK), dtype=dt, device=DEV))
        else:
            s.update(first=_randn((n, h, D), g, dt), second=_randn((n, h, D), g, dt),
                     cache=torch.zeros((pages, h, page, D), dtype=dt, device=DEV),
                     vcache=torch.zeros((pages, h, page, D), dtype=dt, device=DEV))
    else:
        s.update(_attention_inputs(case, g))
    if own:  # the descriptor of pointers and sizes that a serving program keeps beside its buffers
        s["handle"] = _handle(s)
    return s


def _attention_inputs(case, g):
    latent, dt, page, rows, heads = case["op"] == "latent", _dtype(case), case["page"], case["rows"], case["heads"]
    lens, b = _lens(case), case["reqs"]
    need = [-(-n // page) for n in lens]
    width, pages = max(need), sum(need) + 3
    t = b * rows
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    k_len = _int32(lens)
    start = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    start[1:] = torch.cumsum(_int32(need), 0)
    j = torch.arange(width, device=DEV, dtype=torch.int32)[None, :]
    held = j < _int32(need)[:, None]
    table = torch.where(held, perm[torch.where(held, start[:-1, None] + j, 0).long()], -1).to(torch.int32)
    cu_k = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    cu_k[1:] = torch.cumsum(k_len, 0)
    # row i of a request sees all but its last rows-1-i keys: itself and what came before it
    vis = (k_len[:, None] - rows + 1 + torch.arange(rows, device=DEV, dtype=torch.int32)[None, :]).reshape(t).to(torch.int32)
    s = dict(page=page, table=table.contiguous(), cu_q=_int32([rows * i for i in range(b + 1)]), cu_k=cu_k, k_len=k_len, vis=vis, lens=lens)
    if latent:
        s["scale"] = DK ** -0.5
        s["q"] = _randn((t, heads, DK), g, dt, 2.0)
        s["cache"] = _randn((pages, page, DK), g, dt)
    else:
        s["scale"] = D ** -0.5
        s["q"] = _randn((t, heads, D), g, dt, 2.0)
        s["cache"] = _randn((pages, case["kv_heads"], page, D), g, dt)
        s["vcache"] = _randn((pages, case["kv_heads"], page, D), g, dt)
    # what lies past a request's last key was never written
    for name in ("cache", "vcache"):
        if name in s:
            last = table.gather(1, (_int32(need) - 1)[:, None].long())[:, 0].long()
            dead = torch.arange(page, device=DEV)[None, :] >= (k_len - (_int32(need) - 1) * page)[:, None]
            pg = last[:, None].expand(b, page)[dead]
            off = torch.arange(page, device=DEV)[None, :].expand(b, page)[dead]
            if latent:
                s[name][pg, off] = math.nan
            else:
                s[name][pg, :, off] = math.nan
    if case["topk"]:
        kv, k = (1, case["topk"]) if latent else (case["kv_heads"], case["topk"])
        units = vis.long() if latent else (vis.long() + BLOCK - 1) // BLOCK  # keys, or blocks, that a row may choose
        most = int(units.max())
        score = torch.rand((kv, t, most), generator=g, device=DEV)
        score = score.masked_fill(torch.arange(most, device=DEV)[None, None, :] >= units[None, :, None], -1.0)
        val, pick = score.topk(min(k, most), dim=2)
        pick = torch.where(val >= 0, pick, -1).to(torch.int32)
        if pick.shape[2] < k:
            pick = torch.cat([pick, torch.full((kv, t, k - pick.shape[2]), -1, dtype=torch.int32, device=DEV)], 2)
        s["pick"] = (pick[0] if latent else pick).contiguous()
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"tables": _plain_tables, "store": _plain_store, "latent": _plain_attention, "paged": _plain_attention}[s["case"]["op"]](s)


def _handle(s):
    from fp4_sparse_attention_gb300 import binding

    case = s["case"]
    if case["op"] not in ("latent", "paged"):
        return None
    return binding.DeviceAttention(
        q=s["q"], k=s["cache"], v=s.get("vcache"), cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"], block_table=s["table"],
        visible_len=s["vis"], max_seqlen_q=case["rows"], max_seqlen_k=case["len_hi"], scale=s["scale"], indices=s.get("pick"))


def _run_own(s):
    from fp4_sparse_attention_gb300 import binding

    op = s["case"]["op"]
    if op == "tables":
        cu_q, cu_k, visible, slots, taken = binding.fp4idx_build_tables(s["cached"], s["new"], s["table"], s["free"], s["page"], s["rows"])
        return cu_q, cu_k, s["table"], visible, slots, taken
    if op == "store":
        if s["case"]["kind"] == "latent":
            binding.fp4idx_store_latent(s["first"], s["second"], s["slots"], s["cache"])
            return s["cache"]
        binding.fp4idx_store_kv(s["first"], s["second"], s["slots"], s["cache"], s["vcache"])
        return s["cache"], s["vcache"]
    if op == "latent":
        return binding.fp4idx_latent_attention(s["handle"])
    return binding.fp4idx_paged_attention(s["handle"])


def _plain_tables(s):
    cached, new, table, free, page = s["cached"], s["new"], s["table"], s["free"], s["page"]
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    total = cached + new
    cu_q = torch.cat([zero, torch.cumsum(new, 0).to(torch.int32)])
    cu_k = torch.cat([zero, torch.cumsum(total, 0).to(torch.int32)])
    has, need = (cached + page - 1) // page, (total + page - 1) // page
    upto = torch.cumsum(need - has, 0)
    first = upto - (need - has)
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    fresh = (j >= has[:, None]) & (j < need[:, None])
    at = torch.where(fresh, first[:, None] + j - has[:, None], 0)
    table = torch.where(fresh, free[at], table)
    t = torch.arange(s["rows"], device=DEV, dtype=torch.int32)
    req = torch.searchsorted(cu_q[1:], t, right=True)
    pos = cached[req] + t - cu_q[req]
    slots = table[req, (pos // page).long()] * page + pos % page
    return cu_q, cu_k, table, pos + 1, slots.to(torch.int32), upto[-1:].to(torch.int32)


def _plain_store(s):
    at, page, cache = s["slots"].long(), s["page"], s["cache"]
    if s["case"]["kind"] == "latent":
        cache.view(-1, DK)[at] = torch.cat([s["first"], s["second"]], 1)
        return cache
    cache[at // page, :, at % page] = s["first"]
    s["vcache"][at // page, :, at % page] = s["second"]
    return cache, s["vcache"]


def _plain_attention(s):
    """softmax(scale * q k^T) v over each row's keys, in 32 bits.  Groups: X requests (or rows, with selected
    keys) x KV heads; a group's R query rows share its n gathered keys."""
    case, q, page, table, vis = s["case"], s["q"], s["page"], s["table"], s["vis"]
    latent, rows, heads, b = case["op"] == "latent", case["rows"], case["heads"], case["reqs"]
    kv = 1 if latent else case["kv_heads"]
    t, grp = b * rows, heads // kv
    if case["topk"]:
        pick = s["pick"][None] if latent else s["pick"]
        pos = pick.permute(1, 0, 2).long()                                                  # [T, kv, k]
        if not latent:
            pos = torch.where(pos[..., None] >= 0, pos[..., None] * BLOCK + torch.arange(BLOCK, device=DEV), -1).flatten(2)
        seen = (pos >= 0) & (pos < vis[:, None, None])
        req = torch.arange(t, device=DEV)[:, None, None] // rows
        mask = seen[:, :, None, :]                                                          # [X, kv, R, n]
        qg = q.float().view(t, kv, grp, -1)
    else:
        n = case["len_hi"]
        pos = torch.arange(n, device=DEV)[None, None, :].expand(b, kv, n)
        seen = pos < s["k_len"][:, None, None]
        req = torch.arange(b, device=DEV)[:, None, None]
        mask = (pos[:, :, None, :] < vis.view(b, 1, rows, 1)).repeat_interleave(grp, 2)
        qg = q.float().view(b, rows, kv, grp, -1).transpose(1, 2).flatten(2, 3)
    at = torch.where(seen, pos, 0)
    pg = torch.where(seen, table[req, at // page].long(), 0)
    head = torch.arange(kv, device=DEV)[None, :, None]
    off = at % page
    pick_rows = (lambda c: c[pg, off]) if latent else (lambda c: c[pg, head, off])
    k = torch.where(seen[..., None], pick_rows(s["cache"]).float(), 0.0)
    v = k[..., :LATENT] if latent else torch.where(seen[..., None], pick_rows(s["vcache"]).float(), 0.0)
    w = torch.matmul(qg, k.transpose(2, 3)).mul_(s["scale"])
    w.masked_fill_(~mask, -math.inf)
    top = w.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = w.sub_(top).exp_()
    total = w.sum(3, keepdim=True)
    out = torch.matmul(w, v) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top)[..., 0]
    if not case["topk"]:
        out = out.view(b, kv, rows, grp, -1).transpose(1, 2)
        lse = lse.view(b, kv, rows, grp).transpose(1, 2)
    return out.reshape(t, heads, -1).to(q.dtype), lse.reshape(t, heads)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] in ("tables", "store"):
        return None  # whole numbers, and copies
    s = prepare(case, seed)
    heads, rows, page = case["heads"], case["rows"], s["page"]
    latent = case["op"] == "latent"
    kv = 1 if latent else case["kv_heads"]
    grp, t = heads // kv, case["reqs"] * rows
    out = torch.zeros((t, heads, LATENT if latent else D), dtype=torch.float64, device=DEV)
    lse = torch.full((t, heads), -math.inf, dtype=torch.float64, device=DEV)

    def gather(cache, slot, h):
        flat = cache if latent else cache[:, h]
        return flat[slot // page, slot % page].double()

    for b in range(case["reqs"]):
        n = s["lens"][b]
        pages = s["table"][b].long()
        for h in range(kv):
            cols = slice(h * grp, (h + 1) * grp)
            if not case["topk"]:
                where = torch.arange(n, device=DEV)
                slot = pages[where // page] * page + where % page
                keys = gather(s["cache"], slot, h)
                vals = keys[:, :LATENT] if latent else gather(s["vcache"], slot, h)
                for i in range(rows):
                    r, m = b * rows + i, n - rows + 1 + i
                    logit = s["q"][r, cols].double() @ keys[:m].T * s["scale"]
                    lse[r, cols] = torch.logsumexp(logit, 1)
                    out[r, cols] = torch.softmax(logit, 1) @ vals[:m]
                continue
            for i0 in range(0, rows, 32):
                r = torch.arange(b * rows + i0, b * rows + min(rows, i0 + 32), device=DEV)
                chosen = (s["pick"] if latent else s["pick"][h])[r].long()
                if not latent:
                    chosen = torch.where(chosen[:, :, None] < 0, -1, chosen[:, :, None] * BLOCK + torch.arange(BLOCK, device=DEV))
                    chosen = chosen.reshape(len(r), -1)
                ok = (chosen >= 0) & (chosen < s["vis"][r].long()[:, None])
                where = chosen.clamp(0, n - 1)
                slot = pages[where // page] * page + where % page
                keys = gather(s["cache"], slot, h)
                vals = keys[..., :LATENT] if latent else gather(s["vcache"], slot, h)
                vals = vals.masked_fill(~ok[..., None], 0.0)
                logit = torch.einsum("rhd,rnd->rhn", s["q"][r][:, cols].double(), keys) * s["scale"]
                logit = logit.masked_fill(~ok[:, None, :], -math.inf)
                lse[r, cols] = torch.logsumexp(logit, 2)
                out[r, cols] = torch.einsum("rhn,rnd->rhd", torch.exp(logit - lse[r, cols][..., None]), vals)
    return out, lse
