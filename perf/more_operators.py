"""Requests that share a prefix: the page operations that make and undo the sharing, and the attention
that reads a shared prefix once for all of them.

Five operators over the paged caches of one serving program:

  attend   grouped-query attention of groups of requests whose first prefix_len positions are the same keys
  fork     children that continue a parent: table rows shared, a page of their own for the unfinished page
  copy     pages of several caches copied by (source, destination) lists
  release  requests dropped or cut back, and the list of pages that no request holds any more
  compact  the highest pages in use moved into the lowest free ones: tables and copy lists

``run`` takes what ``prepare`` gives and makes one pass: in elementary torch operations where ``own`` is
false, through the framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
D = 128                          # head size of the paged K/V cache
LATENT = 576                     # a token of the latent cache: 512 shared values and 64 rotary ones
INDEX = 68                       # a token of the fused MXFP4 index cache: 64 bytes of codes, 4 of scales


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: two continuations of one short prompt, a token each
        dict(name="attend_pair", op="attend", groups=1, reqs=2, rows=1, heads=16, kv_heads=2, prefix_lo=200, prefix_hi=200, own_lo=1,
             own_hi=31, page=64, dtype="fp16"),
        # 64 samples drawn from one long prompt, each some way on its own
        dict(name="attend_samples", op="attend", groups=1, reqs=64, rows=1, heads=32, kv_heads=4, prefix_lo=32768, prefix_hi=32768, own_lo=1,
             own_hi=1024, page=128, dtype="bf16"),
        # a verify step: 8 system prompts, 6 conversations on each, 4 rows a conversation, odd lengths, 5 heads a K/V head
        dict(name="attend_verify", op="attend", groups=8, reqs=6, rows=4, heads=40, kv_heads=8, prefix_lo=1001, prefix_hi=9001, own_lo=5,
             own_hi=1999, page=64, dtype="bf16"),
        # four prompts of 512 rows behind one system prompt, prefilled in one step
        dict(name="attend_prefill", op="attend", groups=1, reqs=4, rows=512, heads=32, kv_heads=8, prefix_lo=8191, prefix_hi=8191, own_lo=512,
             own_hi=640, page=64, dtype="bf16"),
        # four samples started from one prompt
        dict(name="fork_samples", op="fork", parents=1, forks=4, others=12, len_lo=1000, len_hi=1000, page=64),
        # a large sampling job: 64 prompts, 31 children each
        dict(name="fork_many", op="fork", parents=64, forks=1984, others=0, len_lo=1, len_hi=32767, page=64),
        # the unfinished pages of a few forks, in one layer's latent and index cache
        dict(name="copy_unfinished", op="copy", pairs=8, pages=256, layers=1, page=64),
        # moves of a compaction, four layers
        dict(name="copy_moves", op="copy", pairs=1500, pages=4096, layers=4, page=64),
        # four of 64 running requests end
        dict(name="release_few", op="release", reqs=64, shared=1, gone=4, len_lo=1, len_hi=16384, spare=4096, page=64),
        # a job of 2,048 requests on shared prompts ends a third of them, in a pool of several hundred thousand pages
        dict(name="release_many", op="release", reqs=2048, shared=8, gone=700, len_lo=1, len_hi=32768, spare=100000, page=64),
        # a small pool, nearly empty: all of its pages move down
        dict(name="compact_small", op="compact", reqs=32, shared=1, gone=0, len_lo=1, len_hi=2048, spare=4096, page=128, moves=1024),
        # the large job's pool in one step, with a budget of moves
        dict(name="compact_large", op="compact", reqs=2048, shared=8, gone=0, len_lo=1, len_hi=32768, spare=300000, page=64, moves=65536),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "fork", "copy", "release", "compact"])
    page = rng.choice([64, 128])
    if op == "attend":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        heads = kv_heads * group
        prefix, more = _log_int(rng, 1, 65536), _log_int(rng, 1, 2048)
        # no more than the largest listed case: products, keys read, requests
        rows = max(1, min(rng.choice([1, 1, 1, 2, 4, _log_int(rng, 1, 512)]), 400000000 // ((prefix + more + 512) * heads)))
        mine = rows + more
        groups = max(1, min(_log_int(rng, 1, 16), 800000 // (prefix * kv_heads), 500000000 // ((prefix + mine) * rows * heads)))
        reqs = max(1, min(_log_int(rng, 1, 128), 800000 // (mine * kv_heads * groups), 500000000 // ((prefix + mine) * rows * heads * groups)))
        return dict(op=op, groups=groups, reqs=reqs, rows=rows, heads=heads, kv_heads=kv_heads,
                    prefix_lo=max(1, prefix // rng.choice([1, 2, 8])), prefix_hi=prefix, own_lo=rng.choice([rows, (rows + mine) // 2]), own_hi=mine,
                    page=page, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "fork":
        parents = _log_int(rng, 1, 64)
        return dict(op=op, parents=parents, forks=_log_int(rng, 1, 1984), others=rng.choice([0, 7]), len_lo=1, len_hi=_log_int(rng, 1, 32767),
                    page=page)
    if op == "copy":
        layers = rng.choice([1, 2, 3, 4])
        pairs = _log_int(rng, 1, 6000 // layers * 64 // page)
        return dict(op=op, pairs=pairs, pages=2 * pairs + _log_int(rng, 1, 256), layers=layers, page=page)
    reqs = _log_int(rng, 1, 2048)
    c = dict(op=op, reqs=reqs, shared=rng.choice([1, 2, 8]), gone=0, len_lo=1, len_hi=_log_int(rng, 1, 32768), spare=_log_int(rng, 1, 100000),
             page=page)
    if op == "release":
        c["gone"] = rng.randint(0, reqs)
    else:
        c["moves"] = _log_int(rng, 1, 65536)
    return c


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi] in a fixed mixed order, both ends among them."""
    if n == 1:
        return [hi]
    step = max(1, int(n * 0.618))
    while math.gcd(step, n) != 1:
        step += 1
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _attend_lens(case):
    """Prefix of each group, and of each request what it has behind it."""
    own_lens = _spread(case["groups"] * case["reqs"], case["own_lo"], case["own_hi"])
    return _spread(case["groups"], case["prefix_lo"], case["prefix_hi"]), own_lens


def work(case):
    op, page = case["op"], case["page"]
    if op == "attend":
        prefix, mine = _attend_lens(case)
        rows, heads, kv, t = case["rows"], case["heads"], case["kv_heads"], case["rows"] * len(mine)
        keys = sum(prefix) + sum(mine)
        seen = sum(rows * (prefix[i // case["reqs"]] + n) - rows * (rows - 1) // 2 for i, n in enumerate(mine))
        return {"bytes": keys * kv * 4 * D + 4 * t * heads * D + 4 * t * heads, "flops": 4 * heads * D * seen}
    if op == "fork":
        lens = _spread(case["parents"], case["len_lo"], case["len_hi"])
        held = sum(-(-n // page) for n in lens)
        new = sum(-(-lens[i % case["parents"]] // page) for i in range(case["forks"]))
        return {"bytes": 4 * (held + new + 6 * case["forks"]), "flops": 0}
    if op == "copy":
        return {"bytes": case["pairs"] * (2 * case["layers"] * page * (2 * LATENT + INDEX) + 8), "flops": 0}
    lens = _spread(case["reqs"], case["len_lo"], case["len_hi"])
    held = sum(-(-n // page) for n in lens)
    if op == "release":
        return {"bytes": 4 * (held + case["reqs"] + 2 * case["gone"] + _pool(case)), "flops": 0}
    return {"bytes": 4 * (2 * held + case["reqs"] + 2 * case["moves"]), "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs
def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _randn(shape, g, dtype, by=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return x if by == 1.0 else x.mul_(by)


def _sums(x):
    out = torch.zeros(len(x) + 1, dtype=torch.int32, device=DEV)
    out[1:] = torch.cumsum(x, 0)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"attend": _attend_inputs, "fork": _fork_inputs, "copy": _copy_inputs, "release": _pool_inputs, "compact": _pool_inputs}[case["op"]](case, g)
    s.update(case=case, page=case["page"])
    if own:  # the descriptors of pointers and sizes that a serving program keeps beside its buffers
        _handles(s)
    return s


def _tables(lens, common, owner, page, g, spare, extra=0):
    """Block table of requests whose first `common` pages are those of request `owner`, and the pool's size."""
    b = len(lens)
    need = (lens + page - 1) // page
    mine = torch.where(torch.arange(b, device=DEV) == owner, 0, common)     # first page of its own
    start = _sums((need - mine).clamp(min=0)).long()
    total = int(start[-1])
    width = int(need.max()) + extra
    perm = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(max(1, width), device=DEV)[None, :]
    first = torch.where(j < mine[:, None], start[:-1][owner][:, None] + j, start[:-1, None] + j - mine[:, None])
    held = j < need[:, None]
    table = torch.where(held, perm[torch.where(held, first, 0)], -1).to(torch.int32)
    return table.contiguous(), perm[total:].contiguous(), total + spare


def _attend_inputs(case, g):
    dt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
    page, rows, kv, per = case["page"], case["rows"], case["kv_heads"], case["reqs"]
    prefix, mine = _attend_lens(case)
    b = len(mine)
    t = b * rows
    prefix_len, owner = _int32(prefix), torch.arange(b, device=DEV) // per * per
    shared = prefix_len.repeat_interleave(per)
    lens = shared + _int32(mine)
    table, _, pages = _tables(lens, shared // page, owner, page, g, 3)
    q = _randn((t, case["heads"], D), g, dt, 2.0)
    k, v = _randn((pages, kv, page, D), g, dt), _randn((pages, kv, page, D), g, dt)
    # every request has its own copy of the page that the prefix ends in
    part = (shared % page).long()
    at = (shared // page).long()[:, None]
    held = table.gather(1, at)[:, 0].long()
    source = held[owner]
    off = torch.arange(page, device=DEV)[None, :]
    for x in (k, v):
        copied = (off < part[:, None])[:, None, :, None]
        x[held] = torch.where(copied, x[source], x[held])
    # what lies past a request's last key was never written
    last = table.gather(1, ((lens - 1) // page).long()[:, None])[:, 0].long()
    dead = (off > ((lens - 1) % page)[:, None])[:, None, :, None]
    for x in (k, v):
        x[last] = torch.where(dead, math.nan, x[last])
    vis = (lens[:, None] - rows + 1 + torch.arange(rows, device=DEV, dtype=torch.int32)[None, :]).reshape(t).to(torch.int32)
    return dict(q=q, k=k, v=v, table=table, prefix=prefix, mine=mine, prefix_len=prefix_len, lens=lens, vis=vis, cu_k=_sums(lens),
                cu_q=_int32([rows * i for i in range(b + 1)]), groups=_int32([per * i for i in range(case["groups"] + 1)]),
                most=max(p + mine[i * per + j] for i, p in enumerate(prefix) for j in range(per)), scale=D ** -0.5)


def _fork_inputs(case, g):
    page, n, forks = case["page"], case["parents"], case["forks"]
    reqs = n + forks + case["others"]
    lens = _int32(_spread(n, case["len_lo"], case["len_hi"]))
    row = torch.randperm(reqs, generator=g, device=DEV).to(torch.int32)      # parents, children, rows that are neither
    cached = torch.zeros(reqs, dtype=torch.int32, device=DEV)
    cached[row[:n].long()] = lens
    cached[row[n + forks:].long()] = 1
    table, free, pages = _tables(cached, torch.zeros_like(cached), torch.arange(reqs, device=DEV), page, g, forks + 1, extra=1)
    parent = row[torch.arange(forks, device=DEV) % n]
    return dict(cached=cached, table=table, free=free, pages=pages, parent=parent.contiguous(), child=row[n:n + forks].contiguous())


def _copy_inputs(case, g):
    pages, n, page = case["pages"], case["pairs"], case["page"]
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    caches = []
    for _ in range(case["layers"]):
        caches.append(_randn((pages, page, LATENT), g, torch.bfloat16))
        caches.append(torch.randint(0, 256, (pages, 1, page * INDEX), generator=g, device=DEV, dtype=torch.uint8))
    return dict(caches=caches, src=perm[:n].contiguous(), dst=perm[n:2 * n].contiguous())


def _pool(case):
    """Pages of the pool: those of the requests, a shared prompt's once, and the spare ones."""
    page, lens = case["page"], _spread(case["reqs"], case["len_lo"], case["len_hi"])
    total = 0
    for i, n in enumerate(lens):
        owner = i // case["shared"] * case["shared"]
        common = 0 if i == owner else min(n, lens[owner]) // 2 // page
        total += -(-n // page) - common
    return total + case["spare"]


def _pool_inputs(case, g):
    page, b = case["page"], case["reqs"]
    lens = _int32(_spread(b, case["len_lo"], case["len_hi"]))
    i = torch.arange(b, device=DEV)
    owner = i // case["shared"] * case["shared"]
    common = torch.where(i == owner, 0, torch.minimum(lens, lens[owner]) // 2 // page)  # half of the shorter one is shared
    table, _, pages = _tables(lens, common, owner, page, g, case["spare"], extra=1)
    s = dict(cached=lens, table=table, pages=pages)
    if case["op"] == "release":
        gone = torch.randperm(b, generator=g, device=DEV)[:case["gone"]]
        keep = torch.where(torch.arange(len(gone), device=DEV) % 3 == 0, lens[gone] // 3, 0)  # one in three is only cut back
        s.update(gone=gone.to(torch.int32), keep=keep.to(torch.int32))
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"attend": _own_attend, "fork": _own_fork, "copy": _own_copy, "release": _own_release, "compact": _own_compact}[op](s)
    return {"attend": _plain_attend, "fork": _plain_fork, "copy": _plain_copy, "release": _plain_release, "compact": _plain_compact}[op](s)


def _handles(s):
    from fp4_sparse_attention_gb300 import binding

    case = s["case"]
    if case["op"] == "attend":
        s["handle"] = binding.DeviceSharedAttention(
            q=s["q"], k=s["k"], v=s["v"], cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"], block_table=s["table"], visible_len=s["vis"],
            max_seqlen_q=case["rows"], max_seqlen_k=s["most"], scale=s["scale"], group_offsets=s["groups"], prefix_len=s["prefix_len"],
            max_group_rows=case["rows"] * case["reqs"])
    elif case["op"] == "copy":
        s["handle"] = binding.DevicePages(s["caches"])


def _own_attend(s):
    from fp4_sparse_attention_gb300 import binding

    return binding.fp4idx_shared_prefix_attention(s["handle"])


def _own_fork(s):
    from fp4_sparse_attention_gb300 import binding

    src, dst, taken = binding.fp4idx_fork_requests(s["parent"], s["child"], s["cached"], s["table"], s["free"], s["page"], num_pages=s["pages"])
    return s["cached"], s["table"], src, dst, taken


def _own_copy(s):
    from fp4_sparse_attention_gb300 import binding

    binding.fp4idx_copy_pages(s["handle"], s["src"], s["dst"])
    return s["caches"]


def _own_release(s):
    from fp4_sparse_attention_gb300 import binding

    free, count = binding.fp4idx_release_pages(s["gone"], s["cached"], s["table"], s["page"], s["pages"], keep_len=s["keep"])
    return s["cached"], free, count


def _own_compact(s):
    from fp4_sparse_attention_gb300 import binding

    table, src, dst, count, extent = binding.fp4idx_compact_pages(s["cached"], s["table"], s["page"], s["pages"], s["case"]["moves"],
                                                                  out_table=torch.empty_like(s["table"]))
    return table, src, dst, count, extent


def _plain_attend(s):
    """softmax(scale * q k^T) v in 32 bits, group by group: the prefix through the group's first request, then
    what each request has of its own, all requests at once."""
    case, page, table = s["case"], s["page"], s["table"]
    rows, heads, kv, per = case["rows"], case["heads"], case["kv_heads"], case["reqs"]
    grp, n_rows = heads // kv, case["rows"] * case["reqs"]
    head = torch.arange(kv, device=DEV)[None, :, None]
    outs, lses = [], []
    for i, n in enumerate(s["prefix"]):
        first = i * per
        pos = torch.arange(n, device=DEV)
        pg, off = table[first].long()[pos // page], pos % page
        k, v = s["k"][pg, :, off].float(), s["v"][pg, :, off].float()                                # [n, kv, D]
        q = s["q"][first * rows:first * rows + n_rows].float().view(n_rows, kv, grp, D)
        vis = s["vis"][first * rows:first * rows + n_rows]
        w = torch.matmul(q.permute(1, 0, 2, 3).flatten(1, 2), k.permute(1, 2, 0)).mul_(s["scale"])   # [kv, rows * grp, n]
        w.masked_fill_((pos[None, :] >= vis[:, None]).repeat_interleave(grp, 0)[None], -math.inf)
        # the requests' own keys
        m = max(s["mine"][first:first + per])
        at = n + torch.arange(m, device=DEV)[None, :].expand(per, m)
        there = at < s["lens"][first:first + per, None]
        at = torch.where(there, at, 0)
        pg = table[first:first + per].gather(1, (at // page).long())
        pg = torch.where(there, pg, 0).long()[:, None, :]
        off = (at % page)[:, None, :]
        k2 = torch.where(there[:, None, :, None], s["k"][pg, head, off].float(), 0.0)                # [per, kv, m, D]
        v2 = torch.where(there[:, None, :, None], s["v"][pg, head, off].float(), 0.0)
        q2 = q.view(per, rows, kv, grp, D).transpose(1, 2).flatten(2, 3)                             # [per, kv, rows * grp, D]
        w2 = torch.matmul(q2, k2.transpose(2, 3)).mul_(s["scale"])
        unseen = (n + torch.arange(m, device=DEV))[None, None, :] >= vis.view(per, rows, 1)
        w2.masked_fill_(unseen.repeat_interleave(grp, 1)[:, None], -math.inf)
        w = w.view(kv, per, rows * grp, n).transpose(0, 1)
        top = torch.maximum(w.amax(3, keepdim=True), w2.amax(3, keepdim=True))
        top = torch.where(top == -math.inf, 0.0, top)
        w, w2 = (w - top).exp_(), (w2 - top).exp_()
        total = w.sum(3, keepdim=True) + w2.sum(3, keepdim=True)
        out = torch.matmul(w.transpose(0, 1).flatten(1, 2), v.permute(1, 0, 2)).view(kv, per, rows * grp, D).transpose(0, 1)
        out = (out + torch.matmul(w2, v2)) / torch.where(total > 0, total, 1.0)
        lse = (total.log() + top)[..., 0]
        outs.append(out.view(per, kv, rows, grp, D).transpose(1, 2).reshape(n_rows, heads, D).to(s["q"].dtype))
        lses.append(lse.view(per, kv, rows, grp).transpose(1, 2).reshape(n_rows, heads))
    return torch.cat(outs), torch.cat(lses)


def _plain_fork(s):
    page, table, cached, parent, child = s["page"], s["table"], s["cached"], s["parent"].long(), s["child"].long()
    n = cached[parent]
    full, part = n // page, n % page > 0
    before = torch.cumsum(part, 0)
    new = s["free"][torch.where(part, before - 1, 0)]
    rows = table[parent]
    source = rows.gather(1, torch.where(part, full, 0).long()[:, None])[:, 0]
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    rows = torch.where((j == full[:, None]) & part[:, None], new[:, None], rows)
    table[child] = torch.where(j < (full + part)[:, None], rows, table[child])
    cached[child] = n
    return cached, table, torch.where(part, source, -1), torch.where(part, new, -1), before[-1:].to(torch.int32)


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for c in s["caches"]:
        c[dst] = c[src]
    return s["caches"]


def _held(s):
    """Which table entries are held, and which pages of the pool some entry names."""
    need = (s["cached"] + s["page"] - 1) // s["page"]
    held = torch.arange(s["table"].shape[1], device=DEV)[None, :] < need[:, None]
    live = torch.zeros(s["pages"] + 1, dtype=torch.bool, device=DEV)
    live[torch.where(held, s["table"], s["pages"]).long()] = True
    return held, live[:-1]


def _listed(mask, at, width):
    """The indices where mask holds, index i at place at[i], -1 behind them."""
    out = torch.full((width + 1,), -1, dtype=torch.int32, device=DEV)
    out[torch.where(mask, at, width)] = torch.arange(len(mask), dtype=torch.int32, device=DEV)
    out[width] = -1
    return out[:width]


def _plain_release(s):
    gone = s["gone"].long()
    s["cached"][gone] = torch.minimum(s["cached"][gone], s["keep"])
    _, live = _held(s)
    rank = torch.cumsum(~live, 0)
    return s["cached"], _listed(~live, rank - 1, s["pages"]), rank[-1:].to(torch.int32)


def _plain_compact(s):
    held, live = _held(s)
    most, page_id = s["case"]["moves"], torch.arange(s["pages"], device=DEV)
    upto = torch.cumsum(live, 0)
    n = upto[-1]
    above, hole = n - upto, page_id - upto                      # pages in use above a page; free ones below a free page
    movers = live & (page_id >= n)
    count = torch.minimum(movers.sum(), torch.tensor(most, device=DEV))
    src = _listed(movers & (above < count), above, most)
    dst = _listed(~live & (page_id < n) & (hole < count), hole, most)
    to = torch.arange(s["pages"] + 1, dtype=torch.int32, device=DEV)
    to[torch.where(src >= 0, src, s["pages"]).long()] = dst
    table = torch.where(held, to[torch.where(held, s["table"], 0).long()], s["table"])
    left = movers & (above >= count)                            # pages that the budget leaves where they are
    extent = torch.where(left, page_id + 1, 0).amax().maximum(n)
    return table, src, dst, count.to(torch.int32).view(1), extent.to(torch.int32).view(1)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] != "attend":
        return None  # whole numbers, and copies
    s = prepare(case, seed)
    rows, heads, kv, page = case["rows"], case["heads"], case["kv_heads"], s["page"]
    grp, t = heads // kv, len(s["mine"]) * case["rows"]
    out = torch.zeros((t, heads, D), dtype=torch.float64, device=DEV)
    lse = torch.full((t, heads), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(len(s["mine"])):  # each request by itself, through its own table row
        n = s["prefix"][b // case["reqs"]] + s["mine"][b]
        where = torch.arange(n, device=DEV)
        pages, r = s["table"][b].long()[where // page], slice(b * rows, (b + 1) * rows)
        for h in range(kv):
            hs = slice(h * grp, (h + 1) * grp)
            keys, vals = s["k"][pages, h, where % page].double(), s["v"][pages, h, where % page].double()
            logit = torch.einsum("rgd,nd->rgn", s["q"][r, hs].double(), keys) * s["scale"]
            logit = logit.masked_fill(where[None, None, :] >= s["vis"][r].long()[:, None, None], -math.inf)
            lse[r, hs] = torch.logsumexp(logit, 2)
            out[r, hs] = torch.einsum("rgn,nd->rgd", torch.exp(logit - lse[r, hs][..., None]), vals)
    return out, lse
