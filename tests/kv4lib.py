"""Plain 64-bit forms of the 4-bit KV cache's operators for the tests: the
layout byte by byte, E2M1 rounding by distance, softmax and eviction from their
definitions.  Nothing here calls the package."""
import math

import torch

F64 = torch.float64
MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)


def page_bytes(dim, page):
    return page * dim * 17 // 16


def quantize(x):
    """(values [..., D] float64, codes [..., D] uint8, scales [..., D/32] uint8)
    of x; NaN counts as 0, infinities saturate and do not count for the scale."""
    x = x.to(F64)
    b = x.unflatten(-1, (-1, 32))
    finite = torch.where(torch.isfinite(b), b, 0.0)
    top = finite.abs().amax(-1, keepdim=True)
    f, e = torch.frexp(top)  # top = f * 2^e, f in [0.5, 1)
    e = torch.where(f < 0.875, e - 3, e - 2).to(F64)  # least e with top < 7 * 2^e
    e = torch.where(top == 0, -126.0, e).clamp(-126, 125)
    y = torch.where(torch.isnan(b), 0.0, b) * torch.exp2(-e)
    y = y.clamp(-100.0, 100.0)
    grid, a = MAGNITUDES.to(x.device), y.abs()
    low = (a[..., None] >= grid[1:]).sum(-1)
    high = (low + 1).clamp(max=7)
    down, up = a - grid[low], grid[high] - a
    mag = torch.where((up < down) | ((up == down) & (low % 2 == 1)), high, low)  # a tie goes to the even code
    sign = torch.signbit(y)
    codes = (mag + 8 * sign).to(torch.uint8)
    value = grid[mag] * torch.where(sign, -1.0, 1.0) * torch.exp2(e)
    return value.flatten(-2), codes.flatten(-2), (e + 127).to(torch.uint8).squeeze(-1)


def places(dim, page, t):
    """Byte offsets in one head's page bytes of token t: K codes [D/2], V codes
    [D/2], K scales [D/32], V scales [D/32]."""
    half, n32, wide = page * dim // 2, dim // 32, dim // 16
    c = torch.arange(0, dim, 2)
    blk = torch.arange(n32)
    return (t * (dim // 2) + c // 2, half + ((t // 4 * 16 + c // wide) * 4 + t % 4) * n32 + c % wide // 2,
            2 * half + t * n32 + blk, 2 * half + page * n32 + (t // 4 * n32 + blk) * 4 + t % 4)


def write(pages, dim, pg, t, head, k, v):
    """Quantized rows k, v [D] into page pg, slot t (pages on the host)."""
    page = pages.shape[2] * 16 // (17 * dim)
    at = places(dim, page, t)
    for x, code_at, scale_at in ((k, at[0], at[2]), (v, at[1], at[3])):
        _, c, s = quantize(x)
        pages[pg, head, code_at] = c[0::2] | c[1::2] << 4
        pages[pg, head, scale_at] = s


def values(pages, dim):
    """float64 K, V [n_pages, H, P, D] of a pool on the host."""
    n, h, size = pages.shape
    page = size * 16 // (17 * dim)
    out = [torch.empty(n, h, page, dim, dtype=F64) for _ in range(2)]
    for t in range(page):
        at = places(dim, page, t)
        for which in (0, 1):
            byte = pages[:, :, at[which]]
            code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).long()
            mag = MAGNITUDES[code & 7] * torch.where(code >= 8, -1.0, 1.0).to(F64)
            s = pages[:, :, at[2 + which]].to(F64)
            scale = torch.where(s == 255, math.nan, torch.exp2(s - 127))
            out[which][:, :, t] = (mag.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
    return out


def slots_of(table, b, n, page):
    where = torch.arange(n)
    return table[b].long()[where // page], where % page


def attention(q, pages, table, lens, cu, dim, scale, mass=None):
    """64-bit out, lse, mass and, per output, the magnitudes that error bounds
    need: big = (sum p|v|, sum |v|) and the largest sum |q||k| * scale of a row."""
    k_all, v_all = values(pages, dim)
    page = k_all.shape[2]
    rows, heads, _ = q.shape
    kv = k_all.shape[1]
    g = heads // kv
    out = torch.zeros(rows, heads, dim, dtype=F64)
    big = torch.zeros(2, rows, heads, dim, dtype=F64)
    mag = torch.zeros(rows, heads, dtype=F64)
    lse = torch.full((rows, heads), -math.inf, dtype=F64)
    mass = None if mass is None else mass.to(F64).clone()
    for b in range(len(lens)):
        n, r0, r1 = int(lens[b]), int(cu[b]), int(cu[b + 1])
        m = r1 - r0
        pg, t = slots_of(table, b, n, page)
        last = n - m + torch.arange(m)
        hidden = torch.arange(n)[None] > last[:, None]
        for h in range(heads):
            k, v = k_all[pg, h // g, t], v_all[pg, h // g, t]
            x = (q[r0:r1, h].to(F64) @ k.T) * scale
            x = x.masked_fill(hidden, -math.inf)
            a = (q[r0:r1, h].to(F64).abs() @ k.abs().T) * scale
            z = torch.logsumexp(x, -1) if n else torch.full((m,), -math.inf, dtype=F64)
            p = torch.where(hidden, 0.0, torch.exp(x - z[:, None]))
            out[r0:r1, h] = p @ v
            big[0, r0:r1, h] = p @ v.abs()
            big[1, r0:r1, h] = v.abs().sum(0)
            lse[r0:r1, h] = z
            if n:
                mag[r0:r1, h] = a.masked_fill(hidden, 0.0).amax(-1)
            if mass is not None:
                mass[pg, h // g, t] += p.sum(0)
    return out, lse, mass, big, mag


def attention_bounds(q, dim, lens, out, big, mag, rows=0):
    """Largest error of out and of ln p that the kernels' arithmetic allows.

    A logit is a sum of D exact products in 32 bits (each addition off by at
    most 2^-24 of sum |q||k|), times scale log2 e (two roundings), then 2^x
    (a few units of 2^-23): |d ln p| <= (D + 4) 2^-24 sum|q||k| scale + 2^-21
    for the weight and the same for the sum that divides it.  The weights
    enter the second product as two BF16 terms (16 bits, 2^-16), or, for BF16
    queries with many `rows` (tokens x heads of a group) of a sequence, rounded
    to BF16 once: each weight is then off by 2^-8 of itself at most and the
    result by 2^-8 sum p|v|.  The sum over
    the slots is in 32 bits (L 2^-24), and the result is rounded once to the
    output's type.  A weight below 2^-126 relative to its row's largest is 0 in
    32 bits (2^-126 sum |v|), as is what BF16 leaves of it (as much again)."""
    longest = max([int(n) for n in lens] + [1])
    d = 2 * ((dim + 4) * 2.0 ** -24 * mag + 2.0 ** -21)
    final = torch.finfo(q.dtype).eps / 2
    weight = 2.0 ** -8 if q.dtype == torch.bfloat16 and rows > (16 if dim == 256 else 64) else 2.0 ** -16
    tol = final * out.abs() * (1 + 2.0 ** -8) + (d[..., None] + weight + longest * 2.0 ** -24) * big[0] * 1.01
    tol = tol + 2.0 ** -125 * big[1]
    # below the type's normal range a rounding is half a subnormal step
    return tol + torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps, d


def evict(pages, table, lens, mass, pos, next_pos, budget, sinks, recent, dim):
    """Lens, pages, mass, pos after eviction (host tensors, copies)."""
    page = pages.shape[2] * 16 // (17 * dim)
    pages, mass, pos, lens = pages.clone(), mass.clone(), pos.clone(), lens.clone()
    old = pages.clone(), mass.clone(), pos.clone()
    for b in range(len(lens)):
        n = int(lens[b])
        if n <= budget:
            continue
        pg, t = slots_of(table, b, n, page)
        for h in range(pages.shape[1]):
            keys = []
            for i, (w, p) in enumerate(zip(old[1][pg, h, t].tolist(), old[2][pg, h, t].tolist())):
                safe = p < sinks or p >= int(next_pos[b]) - recent
                # protected slots rank equal, above all others
                keys.append((0, 0.0, False, i) if safe else (1, math.inf if math.isnan(w) else -w, math.isnan(w), i))
            kept = sorted(range(n), key=lambda i: keys[i])[:budget]
            inside = set(kept)
            holes = [i for i in range(budget) if i not in inside]
            movers = sorted(i for i in kept if i >= budget)
            assert len(holes) == len(movers)
            if not holes:
                continue
            at = [places(dim, page, x) for x in range(page)]  # by slot in the page
            at = torch.stack([torch.cat(x) for x in at])
            to, fr = torch.tensor(holes), torch.tensor(movers)
            pages[pg[to][:, None], h, at[t[to]]] = old[0][pg[fr][:, None], h, at[t[fr]]]
            mass[pg[to], h, t[to]] = old[1][pg[fr], h, t[fr]]
            pos[pg[to], h, t[to]] = old[2][pg[fr], h, t[fr]]
        lens[b] = budget
    return lens, pages, mass, pos


def table_of(lens, page, n_pages, seed):
    """A shuffled block table (host int32) for sequences of `lens` slots."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-int(n) // page) for n in lens]
    order = torch.randperm(n_pages, generator=g)[:sum(per)].to(torch.int32)
    table = torch.full((len(lens), max(per + [1])), 0, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table
