"""Plain 64-bit implementation of the attention calls (include/fp4idx.h), row by row and without
tiles, and the error bound their results are held to."""
import math

import torch


def visible(c, b, t):
    """Positions row t of request b sees: [0, result)."""
    k_len = c["k_lens"][b]
    if c.get("visible_len") is not None:
        v = int(c["visible_len"][t])
    elif c.get("causal"):
        q0 = sum(c["q_lens"][:b])
        off = int(c["qo_offset"][b]) if c.get("qo_offset") is not None else k_len - c["q_lens"][b]
        v = t - q0 + off + 1
    else:
        v = k_len
    return max(0, min(v, k_len))


def keys_of(c, b, t, hk):
    """Logical positions row t attends to with K/V head hk, in list order (repeats kept)."""
    vis = visible(c, b, t)
    if c.get("indices") is None:
        pos = list(range(vis))
    elif c["v"] is None:
        pos = [int(s) for s in c["indices"][t].tolist() if 0 <= s < vis]
    else:
        pos = [s for i in c["indices"][hk, t].tolist() if i >= 0
               for s in range(128 * i, min(128 * i + 128, vis))]
    page = c["page"]
    row = c["pages"][b]  # physical page of every logical page
    return [s for s in pos if 0 <= row[s // page] < c["k"].shape[0]]


def reference(c):
    """(out [T,H,dv], lse [T,H], bound_out, bound_lse) in float64.

    The bounds: the weights are rounded once to the operand type (unit roundoff u; below the
    type's normal range by at most `tiny`, relative to a largest weight of at least 1), so the
    sum is off by at most u * sum w|v| + n * tiny * max|v|; the result is rounded once (u); the
    fp32 score of dk products is off by at most e = dk * 2^-23 * sum|q k| * scale, which scales
    every weight by at most 1 + 2e, numerator and denominator alike; fp32 sums of n terms and
    the exponential add (n + 64) * 2^-23 of sum w|v| at most, and of the logarithm's argument.
    """
    latent = c["v"] is None
    q, dev = c["q"].double(), c["q"].device
    T, H, dk = q.shape
    dv = 512 if latent else 128
    kv = 1 if latent else c["k"].shape[1]
    g = H // kv
    u, tiny = (2.0 ** -8, 0.0) if c["q"].dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)
    out = torch.zeros((T, H, dv), dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    t = 0
    for b, n_rows in enumerate(c["q_lens"]):
        pages = torch.tensor(c["pages"][b] or [0], device=dev)
        for _ in range(n_rows):
            for hk in range(kv):
                pos = torch.tensor(keys_of(c, b, t, hk), dtype=torch.long, device=dev)
                if not len(pos):
                    continue
                pg, off = pages[pos // c["page"]], pos % c["page"]
                k = (c["k"][pg, off] if latent else c["k"][pg, hk, off]).double()
                v = k[:, :512] if latent else c["v"][pg, hk, off].double()
                hs = slice(hk * g, (hk + 1) * g)
                s = q[t, hs] @ k.T * c["scale"]
                top = s.amax(1, keepdim=True)
                top = torch.where(top == -math.inf, torch.zeros_like(top), top)
                w = torch.exp(s - top)
                total = w.sum(1, keepdim=True)
                some = total[:, 0] > 0
                p = w / torch.where(total > 0, total, torch.ones_like(total))
                out[t, hs] = p @ v
                lse[t, hs] = torch.where(some | total[:, 0].isnan(), total.log()[:, 0] + top[:, 0], lse[t, hs])
                e = dk * 2.0 ** -23 * abs(c["scale"]) * (q[t, hs].abs() @ k.abs().T).amax(1, keepdim=True)
                n = len(pos)
                spread = p @ v.abs()
                b_out[t, hs] = (u + 2 * e + (n + 64) * 2.0 ** -23) * spread + u * out[t, hs].abs() \
                    + n * tiny * v.abs().amax()
                b_lse[t, hs] = (e + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * (top.abs() + total.log().abs()))[:, 0]
            t += 1
    return out, lse, b_out, b_lse


def make_case(seed, q_lens, k_lens, heads, kv_heads=None, page=64, dtype=torch.bfloat16, visibility="causal",
              select=0, spare=3, device="cpu", scale=None, gain=2.0, junk=math.nan):
    """Seeded inputs: kv_heads None for latent attention.  Cache contents nobody sees are `junk`."""
    g = torch.Generator().manual_seed(seed)
    latent = kv_heads is None
    dk = 576 if latent else 128
    T, B = sum(q_lens), len(q_lens)
    need = [-(-n // page) for n in k_lens]
    perm = torch.randperm(sum(need) + spare, generator=g).tolist()
    pages, at = [], 0
    for n in need:
        pages.append(perm[at:at + n])
        at += n
    P = len(perm)
    shape = (P, page, dk) if latent else (P, kv_heads, page, dk)
    c = dict(q_lens=q_lens, k_lens=k_lens, page=page, pages=pages, scale=dk ** -0.5 if scale is None else scale)
    c["q"] = (torch.randn((T, heads, dk), generator=g) * gain).to(dtype)
    c["k"] = torch.randn(shape, generator=g).to(dtype)
    c["v"] = None if latent else torch.randn(shape, generator=g).to(dtype)
    for x in (c["k"], c["v"]):
        if x is None:
            continue
        for p in perm[at:]:
            x[p] = junk
        for b, n in enumerate(k_lens):
            if n % page:
                if latent:
                    x[pages[b][-1], n % page:] = junk
                else:
                    x[pages[b][-1], :, n % page:] = junk
    if visibility == "lens":  # any length, 0 and past the end among them
        v = [int(torch.randint(-1, k + 3, (1,), generator=g)) for b, k in enumerate(k_lens) for _ in range(q_lens[b])]
        c["visible_len"] = torch.tensor(v, dtype=torch.int32)
    elif visibility == "offset":
        c["causal"] = True
        c["qo_offset"] = torch.tensor([max(0, k - q - 5) for q, k in zip(q_lens, k_lens)], dtype=torch.int32)
    else:
        c["causal"] = visibility == "causal"
    if select:
        rows = [b for b, n in enumerate(q_lens) for _ in range(n)]
        kv = 1 if latent else kv_heads
        idx = torch.full((kv, T, select), -1, dtype=torch.int32)
        for t, b in enumerate(rows):
            most = k_lens[b] if latent else -(-k_lens[b] // 128)
            for h in range(kv):
                pick = torch.randperm(most, generator=g)[:select].to(torch.int32)
                idx[h, t, :len(pick)] = pick
                idx[h, t] = idx[h, t][torch.randperm(select, generator=g)]  # -1 anywhere
        c["indices"] = idx[0].contiguous() if latent else idx
    for name in ("q", "k", "v", "visible_len", "qo_offset", "indices"):
        if c.get(name) is not None:
            c[name] = c[name].to(device)
    return c


def table_of(c, extra=2):
    """block_table [B, stride] int32; unused entries are out of range."""
    width = max([len(r) for r in c["pages"]] + [1]) + extra
    rows = [r + [10 ** 6] * (width - len(r)) for r in c["pages"]]
    return torch.tensor(rows, dtype=torch.int32, device=c["q"].device)


def offsets(lens, device):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)
