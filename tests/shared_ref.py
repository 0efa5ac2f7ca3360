"""Plain Python forms of the page operations of include/fp4idx.h, and cases of attention whose requests
share a prefix (the attention itself is held to tests/attention_ref.py, which knows nothing of sharing)."""
import math

import torch

from tests import attention_ref as R

ERR_PAGE_RANGE, ERR_LENGTHS, ERR_REQUESTS = 0x1, 0x8, 0x10


# ---------------------------------------------------------------- pages
def fork(parent, child, fork_len, cached, table, free, page, num_pages):
    """Lists in; (cached, table, src, dst, taken, error bits) out."""
    cached, table, reqs, stride = list(cached), [list(r) for r in table], len(cached), len(table[0])
    old_len, old = list(cached), [list(r) for r in table]
    src, dst, err, used = [], [], 0, 0

    def there(i):
        return 0 <= parent[i] < reqs and 0 <= child[i] < reqs

    parents = {parent[i] for i in range(len(parent)) if there(i)}
    named = set()
    for i in range(len(parent)):
        src.append(-1)
        dst.append(-1)
        if parent[i] < 0 or child[i] < 0:
            continue
        if not there(i):
            err |= ERR_REQUESTS
            continue
        n = max(0, old_len[parent[i]])
        if fork_len is not None:
            n = min(n, max(0, fork_len[i]))
        full, part = n // page, n % page > 0
        fits = full + part <= stride
        refused = child[i] in named or child[i] in parents
        named.add(child[i])
        if not fits:
            err |= ERR_LENGTHS
        if refused:
            err |= ERR_REQUESTS
        new = -1
        if fits and part:
            new = max(-1, free[used]) if used < len(free) else -1
            used += 1
        if refused or not fits:
            continue
        table[child[i]][:full] = old[parent[i]][:full]
        cached[child[i]] = n
        if part:
            table[child[i]][full] = new
            at = old[parent[i]][full]
            if new < 0:
                err |= ERR_LENGTHS
            if not 0 <= at < num_pages:
                err |= ERR_PAGE_RANGE
            elif new >= 0:
                src[-1], dst[-1] = at, new
    return cached, table, src, dst, min(used, len(free)), err


def in_use(cached, table, page, num_pages):
    """(set of pages that held entries name, error bits)"""
    live, err = set(), 0
    for n, row in zip(cached, table):
        held = -(-max(0, n) // page)
        if held > len(row):
            err |= ERR_LENGTHS
        for x in row[:held]:
            if 0 <= x < num_pages:
                live.add(x)
            else:
                err |= ERR_PAGE_RANGE
    return live, err


def release(requests, keep, cached, table, page, num_pages):
    """(cached, free list, number, error bits)"""
    cached, err = list(cached), 0
    for i, b in enumerate(requests):
        if b >= len(cached):
            err |= ERR_REQUESTS
        elif b >= 0:
            cached[b] = min(cached[b], max(0, keep[i]) if keep is not None else 0)
    live, bits = in_use(cached, table, page, num_pages)
    free = [x for x in range(num_pages) if x not in live]
    return cached, free + [-1] * (num_pages - len(free)), len(free), err | bits


def compact(cached, table, page, num_pages, max_moves):
    """(table, src, dst, moves, extent, error bits)"""
    live, err = in_use(cached, table, page, num_pages)
    n = len(live)
    src = sorted((x for x in live if x >= n), reverse=True)[:max_moves]
    dst = [x for x in range(n) if x not in live][:len(src)]
    to = dict(zip(src, dst))
    out = []
    for length, row in zip(cached, table):
        held = -(-max(0, length) // page)
        out.append([to.get(x, x) if j < held else x for j, x in enumerate(row)])
    extent = max((to.get(x, x) for x in live), default=-1) + 1
    pad = [-1] * (max_moves - len(src))
    return out, src + pad, dst + pad, len(src), extent, err


# ---------------------------------------------------------------- attention
def make_shared(seed, groups, heads, kv_heads, page=64, **kw):
    """groups: [(prefix, [(rows, keys of its own), ...]), ...].  A case of attention_ref whose requests' pages are
    shared below the prefix, and their copies of the page that it ends in hold the same values."""
    q_lens = [r for _, reqs in groups for r, _ in reqs]
    k_lens = [max(0, n + own) for n, reqs in groups for _, own in reqs]
    junk = kw.get("junk", math.nan)
    c = R.make_case(seed, q_lens, k_lens, heads=heads, kv_heads=kv_heads, page=page, **kw)
    b = 0
    for n, reqs in groups:
        first = c["pages"][b] if reqs else []
        for i in range(1, len(reqs)):
            mine, common = c["pages"][b + i], min(n, k_lens[b], k_lens[b + i])
            for j in range(common // page):
                for x in (c["k"], c["v"]):
                    x[mine[j]] = junk  # held by nobody
                mine[j] = first[j]
            if common % page:
                j = common // page
                for x in (c["k"], c["v"]):
                    x[mine[j], :, :common % page] = x[first[j], :, :common % page]
        b += len(reqs)
    c["groups"] = groups
    return c


def group_arguments(c, device="cuda"):
    """group_offsets, prefix_len and max_group_rows of a case of make_shared."""
    counts = [len(reqs) for _, reqs in c["groups"]]
    return dict(group_offsets=R.offsets(counts, device),
                prefix_len=torch.tensor([n for n, _ in c["groups"]], dtype=torch.int32, device=device),
                max_group_rows=max([sum(r for r, _ in reqs) for _, reqs in c["groups"]] + [1]))
