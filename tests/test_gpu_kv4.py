"""The 4-bit KV cache on the GPU against plain 64-bit forms (kv4lib): the
encoder and decoder byte for byte, attention within bounds derived from its
arithmetic, eviction exactly, and all four in a row.

Pools start filled with 0xFF bytes, whose scales mean NaN: what a call must not
look at shows in its results."""
import math

import numpy as np
import pytest
import torch

import kv4lib as R

pytestmark = pytest.mark.gpu

sz = pytest.importorskip("lossless_kv_cache_splitzip_amd")
DEV = "cuda"
BF, HF, E5 = torch.bfloat16, torch.float16, torch.float8_e5m2


def _pool(n_pages, kv, dim, page):
    return torch.full((n_pages, kv, R.page_bytes(dim, page)), 255, dtype=torch.uint8, device=DEV)


def _cu(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)


def _rows(rows, heads, dim, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads, dim, generator=g) * torch.exp(spread * torch.randn(rows, heads, dim // 32, 1, generator=g)
                                                              ).expand(-1, -1, -1, 32).flatten(2)
    return x.to(dtype)


def _filled(lens, kv, dim, page, seed, extra=3):
    """A pool with every sequence's slots appended; (pages, table, lens, k, v) with k, v per sequence."""
    n_pages = sum(-(-n // page) for n in lens) + extra
    table = R.table_of(lens, page, n_pages, seed)
    pages = _pool(n_pages, kv, dim, page)
    total = sum(lens)
    k, v = _rows(total, kv, dim, BF, seed + 1, 0.3), _rows(total, kv, dim, BF, seed + 2, 0.3)
    ln = torch.tensor(lens, dtype=torch.int32)
    if total:
        sz.kv4_append(pages, k.to(DEV), v.to(DEV), table.to(DEV), ln.to(DEV), cu=_cu(lens).to(DEV), max_new=max(lens))
    return pages, table, ln


# ---------------------------------------------------------------- append, read
@pytest.mark.parametrize("dim,page,kv,dtype,before,new", [
    (128, 16, 8, BF, [0, 5, 33], [17, 1, 30]),
    (128, 64, 1, HF, [3], [130]),
    (64, 16, 3, BF, [0, 15, 16, 17], [1, 1, 1, 1]),
    (64, 256, 2, E5, [250, 0], [13, 0]),
    (256, 32, 2, HF, [31, 2], [6, 64]),
    (256, 16, 1, E5, [1], [2]),
    (128, 128, 4, E5, [127, 0, 4], [2, 129, 3]),
    (64, 32, 5, HF, [0], [1]),
    (256, 128, 1, BF, [0, 100], [1, 257]),
])
def test_append_matches_the_layout_and_read_gives_it_back(dim, page, kv, dtype, before, new):
    print(f"case append dim={dim} page={page} kv={kv} {dtype} {before}+{new}", flush=True)
    lens = [a + b for a, b in zip(before, new)]
    n_pages = sum(-(-n // page) for n in lens) + 2
    table = R.table_of(lens, page, n_pages, 5)
    total = sum(new)
    # K and V as slices of one projection's output
    x = _rows(total, 3 * kv, dim, torch.float32, 7, 2.0).clamp(-5e4, 5e4).to(dtype)
    k, v = x[:, kv:2 * kv], x[:, 2 * kv:]
    positions = torch.arange(total, dtype=torch.int32) * 3 + 11
    pages = _pool(n_pages, kv, dim, page)
    mass = torch.full((n_pages, kv, page), 7.5, device=DEV)
    pos = torch.full((n_pages, kv, page), -1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    want, wm, wp = pages.cpu(), mass.cpu(), pos.cpu()
    kq, vq = torch.empty(total, kv, dim, dtype=R.F64), torch.empty(total, kv, dim, dtype=R.F64)
    kf, vf, at = k.float(), v.float(), 0
    for b in range(len(lens)):
        for i in range(new[b]):
            slot = before[b] + i
            pg, t = int(table[b, slot // page]), slot % page
            for h in range(kv):
                R.write(want, dim, pg, t, h, kf[at, h], vf[at, h])
                kq[at, h], vq[at, h] = R.quantize(kf[at, h])[0], R.quantize(vf[at, h])[0]
            wm[pg, :, t], wp[pg, :, t] = 0.0, positions[at]
            at += 1
    args = (table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    sz.kv4_append(pages, xd[:, kv:2 * kv], xd[:, 2 * kv:], *args, cu=_cu(new).to(DEV), positions=positions.to(DEV),
                  mass=mass, pos=pos, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(pages.cpu(), want)
    assert torch.equal(mass.cpu(), wm) and torch.equal(pos.cpu(), wp)
    # back: exact in BF16; rows behind the last sequence stay
    out = [torch.full((total + 3, kv, dim), 9.0, dtype=BF, device=DEV) for _ in range(2)]
    sz.kv4_read(pages, *args, dim, cu=_cu(new).to(DEV), n_tokens=total + 3, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for got, ref in zip(out, (kq, vq)):
        assert torch.equal(got[:total].cpu().double(), ref)
        assert bool((got[total:] == 9.0).all())
    hk, hv = sz.kv4_read(pages, *args, dim, cu=_cu(new).to(DEV), n_tokens=total, dtype=HF)
    assert torch.equal(hk.cpu(), kq.to(HF)) and torch.equal(hv.cpu(), vq.to(HF))


@pytest.mark.parametrize("dim,kv,dtype,page", [
    (64, 1, BF, 16), (64, 1, E5, 256), (128, 1, HF, 64), (64, 2, E5, 16), (64, 3, BF, 32), (64, 4, HF, 16), (256, 1, BF, 128)])
def test_many_rows_of_few_heads_as_in_small_calls(dim, kv, dtype, page):
    """One call of 70,000 rows and calls of 5000 rows give the same bytes, positions and weights; one sequence has
    page numbers outside the pool, some have no rows."""
    before, new = [5, 0, 7, 0, 130, 1, 2], [30001, 1, 0, 38999, 4, 1002, 3]
    lens = [a + b for a, b in zip(before, new)]
    print(f"case narrow dim={dim} kv={kv} {dtype} page={page}", flush=True)
    n_pages = sum(-(-n // page) for n in lens) + 2
    table = R.table_of(lens, page, n_pages, 17)
    table[5, 1] = n_pages  # the second page's rows of one sequence have no place
    total, cu = sum(new), _cu(new)
    k, v = (_rows(total, kv, dim, torch.float32, s, 2.0).clamp(-5e4, 5e4).to(dtype).to(DEV) for s in (3, 4))
    positions = (torch.arange(total, dtype=torch.int32) * 5 + 2).to(DEV)
    table = table.to(DEV)
    got = []
    for step in (total, 5000):
        pages = _pool(n_pages, kv, dim, page)
        mass = torch.full((n_pages, kv, page), 7.5, device=DEV)
        pos = torch.full((n_pages, kv, page), -1, dtype=torch.int32, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = [torch.full((total + 3, kv, dim), 9.0, dtype=BF, device=DEV) for _ in range(2)]
        for lo in range(0, total, step):
            hi = min(lo + step, total)
            part = [max(0, min(hi, int(cu[b + 1])) - max(lo, int(cu[b]))) for b in range(len(new))]
            done = [max(0, min(hi, int(cu[b + 1])) - int(cu[b])) for b in range(len(new))]
            ln = torch.tensor([a + d for a, d in zip(before, done)], dtype=torch.int32, device=DEV)
            c = _cu(part).to(DEV)
            sz.kv4_append(pages, k[lo:hi], v[lo:hi], table, ln, cu=c, positions=positions[lo:hi], mass=mass, pos=pos,
                          status=status)
            n = hi - lo + (3 if hi == total else 0)
            sz.kv4_read(pages, table, ln, dim, cu=c, n_tokens=n, out=[o[lo:lo + n] for o in out])
        torch.cuda.synchronize()
        assert int(status.item()) != 0
        got.append((pages, mass, pos, *out))
    for one, many in zip(*got):
        assert torch.equal(one, many)
    off = int(cu[5])
    k_out = got[0][3]
    assert bool((k_out[off + page - 1:off + min(2 * page - 1, 1002)] == 9.0).all())
    kq = R.quantize(k[:off + page - 1].float())[0]
    assert torch.equal(k_out[:off + page - 1].double(), kq)
    hk, _ = sz.kv4_read(got[0][0], table, torch.tensor(lens, dtype=torch.int32, device=DEV), dim, cu=cu.to(DEV),
                        n_tokens=total, dtype=HF)
    assert torch.equal(hk[:off + page - 1], kq.to(HF))


@pytest.mark.parametrize("dtype", [HF, E5])
def test_every_pattern_of_the_other_types(dtype):
    """Each FP16 or E5M2 pattern as the first of a block of 2, -1.5, .. times it, and beside ones."""
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits.to(torch.int16).view(HF) if dtype == HF else bits[:256].to(torch.uint8).view(E5)
    n = bits.numel()
    x = torch.zeros(n, 2, 64)
    x[:, 0] = bits.float()[:, None] * torch.linspace(-1, 1, 64)
    x[:, 0, 0] = x[:, 0, 32] = bits.float()
    x[:, 1, :32] = torch.linspace(0, 2, 32)
    x[:, 1, 7] = bits.float()
    x = x.to(dtype)
    pages = _pool(n // 256, 2, 64, 256)
    table = torch.arange(n // 256, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    sz.kv4_append(pages, x.to(DEV), x.to(DEV), table, lens, cu=cu)
    k, v = sz.kv4_read(pages, table, lens, 64, cu=cu, n_tokens=n)
    want = R.quantize(x.float())[0]
    assert torch.equal(k.cpu().double(), want) and torch.equal(v.cpu().double(), want)


def test_every_bf16_pattern_and_the_borders():
    # each of the 65,536 BF16 patterns as the largest of a block whose other
    # values sit at its rounding borders
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    x = torch.zeros(65536, 1, 64, dtype=BF)
    x[:, 0, 0] = bits
    for i in range(1, 32):
        x[:, 0, i] = (bits.float() * (i / 32.0)).to(BF)
    x[:, 0, 32:] = x[:, 0, :32].flip(-1)
    n = x.shape[0]
    pages = _pool(n // 256, 1, 64, 256)
    table = torch.arange(n // 256, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sz.kv4_append(pages, x.to(DEV), x.flip(0).contiguous().to(DEV), table, lens, cu=cu, status=status)
    k, v = sz.kv4_read(pages, table, lens, 64, cu=cu, n_tokens=n)
    torch.cuda.synchronize()
    want = R.quantize(x.float())[0]
    assert int(status.item()) == sz.E_NONFINITE
    assert torch.equal(k.cpu().double(), want) and torch.equal(v.cpu().double(), want.flip(0))
    ok = torch.isfinite(x).all(-1, keepdim=True).expand_as(x)
    # no value of a block is further off than 2^e, a seventh of the block's bound
    top = x.float().unflatten(-1, (2, 32)).abs().amax(-1, keepdim=True).double()
    err = (want - x.double()).unflatten(-1, (2, 32)).abs()
    fine = (top < 1.75 * 2.0 ** 127) & (top >= 2.0 ** -120) & ok.unflatten(-1, (2, 32))
    assert bool((err <= top * (2 / 7) * 1.0000001)[fine].all())


def test_non_finite_values_are_stored_as_the_header_says():
    x = torch.ones(4, 1, 64, dtype=BF)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 5] = math.nan, math.inf, -math.inf
    pages = _pool(1, 1, 64, 16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([4], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for y, code in ((torch.ones_like(x), 0), (x, sz.E_NONFINITE)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        sz.kv4_append(pages, y.to(DEV), torch.ones_like(y).to(DEV), table, lens, cu=cu, status=status)
        k, _ = sz.kv4_read(pages, table, lens, 64, cu=cu, n_tokens=4)
        torch.cuda.synchronize()
        assert int(status.item()) == code
        assert torch.equal(k.cpu().double(), R.quantize(y.float())[0])
    k = k.cpu().float()
    assert k[0, 0, 3] == 0 and k[1, 0, 40] == 1.5 and k[2, 0, 5] == -1.5 and k[3, 0, 0] == 1.0


def test_many_sequences_some_without_rows():
    """More sequences than a wave has lanes, rows of none, one and several."""
    g = torch.Generator().manual_seed(9)
    new = torch.randint(0, 4, (200,), generator=g).tolist()
    new[0], new[63], new[64], new[199] = 0, 3, 0, 0
    before = torch.randint(0, 40, (200,), generator=g).tolist()
    lens = [a + b for a, b in zip(before, new)]
    kv, dim, page = 3, 64, 16
    n_pages = sum(-(-n // page) for n in lens)
    table = R.table_of(lens, page, n_pages, 10)
    pages = torch.zeros(n_pages, kv, R.page_bytes(dim, page), dtype=torch.uint8, device=DEV)
    ln = torch.tensor(lens, dtype=torch.int32)
    k, v = _rows(sum(lens), kv, dim, BF, 11, 0.3), _rows(sum(lens), kv, dim, BF, 12, 0.3)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    sz.kv4_append(pages, k.to(DEV), v.to(DEV), table.to(DEV), ln.to(DEV), cu=_cu(lens).to(DEV), status=st)
    rk, rv = sz.kv4_read(pages, table.to(DEV), ln.to(DEV), dim, cu=_cu(new).to(DEV), n_tokens=sum(new), status=st)
    assert int(st.item()) == 0
    keep = torch.cat([torch.arange(e - m, e) for e, m in zip(np.cumsum(lens).tolist(), new)])
    assert torch.equal(rk.cpu().double(), R.quantize(k.float())[0][keep])
    assert torch.equal(rv.cpu().double(), R.quantize(v.float())[0][keep])
    q = _rows(sum(new), 6, dim, BF, 13)
    mass = torch.zeros(n_pages, kv, page, device=DEV)
    out, lse = sz.kv4_attention(q.to(DEV), pages, table.to(DEV), ln.to(DEV), cu=_cu(new).to(DEV), max_new=3, mass=mass,
                                return_lse=True, status=st)
    assert int(st.item()) == 0
    ro, rl, rm, big, mag = R.attention(q, pages.cpu(), table, ln, _cu(new), dim, dim ** -0.5, torch.zeros(n_pages, kv, page))
    tol, d = R.attention_bounds(q, dim, lens, ro, big, mag)
    assert bool(((out.cpu().double() - ro).abs() <= tol).all())
    assert bool(((mass.cpu().double() - rm).abs() <= (float(d.max()) + 6 * 2.0 ** -24) * rm + 2.0 ** -23 * rm).all())
    # long ones among short ones are cut, the short ones are not
    budget = 20
    nxt = torch.full((200,), 1000, dtype=torch.int32)
    pos = torch.zeros(n_pages, kv, page, dtype=torch.int32)
    want = R.evict(pages.cpu(), table, ln, mass.cpu(), pos, nxt, budget, 0, 0, dim)
    d = [t.to(DEV) for t in (pages, table, ln, mass, pos, nxt)]
    sz.kv4_evict(*d, dim, budget)
    assert torch.equal(d[2].cpu(), want[0]) and torch.equal(d[0].cpu(), want[1])


# ------------------------------------------------------------------- attention
def _attend_case(lens, new, kv, group, dim, page, dtype, seed, scale=None, mass=True, q_gain=1.0, max_len=None,
                 strided=False):
    pages, table, ln = _filled(lens, kv, dim, page, seed)
    rows, heads = sum(new), kv * group
    scale = dim ** -0.5 if scale is None else scale
    q = (_rows(rows, heads, dim, torch.float32, seed + 3, 0.2) * q_gain).to(dtype)
    qd = q.to(DEV)
    if strided:
        wide = torch.zeros(rows, heads + 2, dim + 8, dtype=dtype, device=DEV)
        wide[:, 1:-1, :dim] = qd
        qd = wide[:, 1:-1, :dim]
    m_in = torch.rand(pages.shape[0], kv, page, generator=torch.Generator().manual_seed(seed)) * 3
    m_out = torch.full_like(m_in, -2.0).to(DEV)
    out = torch.full((rows + 2, heads, dim), 5.0, dtype=dtype, device=DEV)
    lse = torch.full((rows + 2, heads), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pad = torch.zeros(2, heads, dim, dtype=dtype, device=DEV)
    q_all = torch.cat([qd, pad]) if not strided else None
    if strided:
        out, lse, q_all = out[:rows], lse[:rows], qd
    sz.kv4_attention(q_all, pages, table.to(DEV), ln.to(DEV), cu=_cu(new).to(DEV), max_new=max(new + [0]), scale=scale,
                     max_len=max_len, mass=m_in.to(DEV) if mass else None, mass_out=m_out if mass else None, out=out,
                     lse=lse, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ro, rl, rm, big, mag = R.attention(q, pages.cpu(), table, ln, _cu(new), dim, scale, m_in)
    tol, d = R.attention_bounds(q, dim, lens, ro, big, mag, max(new + [0]) * group)
    err = (out[:rows].cpu().double() - ro).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if not strided:
        assert bool((out[rows:] == 5.0).all()) and bool((lse[rows:] == 5.0).all())
    got = lse[:rows].cpu().double()
    empty = rl == -math.inf
    assert torch.equal(got == -math.inf, empty)
    assert bool((out[:rows].cpu()[empty] == 0).all())
    # lse: the error of a logit, and a rounding of it
    assert bool(((got - rl).abs() <= d + 2.0 ** -22 * rl.abs() + 2.0 ** -21)[~empty].all())
    if mass:
        seen = torch.zeros(pages.shape[0], page, dtype=torch.bool)
        for b, n in enumerate(lens):
            pg, t = R.slots_of(table, b, n, page)
            seen[pg, t] = True
        got = m_out.cpu().double()
        sel = seen[:, None].expand_as(got)
        assert bool((got[~sel] == -2.0).all())
        # each weight is off by d relative; the sum over the rows in 32 bits, and the final addition
        worst = float(d.max()) + max(new + [1]) * group * 2.0 ** -24
        tol = worst * (rm - m_in.double()).abs() + 2.0 ** -23 * rm.abs()
        assert bool(((got - rm).abs() <= tol)[sel].all()), float(((got - rm).abs() / tol)[sel].max())
    return out


SMALL = [
    # lens, new, kv, group, dim, page, dtype
    ([1], [1], 1, 1, 64, 16, BF),
    ([1, 2, 31, 32, 33], [1] * 5, 2, 4, 128, 16, BF),
    ([127, 128, 129, 500], [1] * 4, 2, 7, 128, 32, HF),
    ([777], [1], 8, 4, 128, 16, BF),
    ([5000, 3, 900], [1] * 3, 1, 16, 128, 64, BF),
    ([1500, 40], [1, 1], 1, 64, 64, 256, BF),
    ([300, 17], [1, 1], 2, 5, 256, 16, HF),
    ([100, 64, 9], [5, 1, 9], 4, 7, 64, 32, HF),
    ([64, 65, 200], [64, 65, 3], 2, 2, 128, 16, BF),
    ([333, 130], [333, 7], 1, 8, 128, 64, BF),
    ([97], [97], 2, 3, 256, 128, BF),
    ([260, 1], [129, 1], 1, 4, 256, 16, HF),
    ([700], [257], 2, 1, 64, 64, HF),
    # many rows of few slots, shared between workgroups for the weights' sums
    ([900], [900], 1, 4, 128, 32, BF),
    ([600, 513], [600, 200], 1, 8, 64, 64, HF),
    ([520], [300], 1, 2, 256, 16, HF),
    ([1300, 200], [33, 40], 2, 2, 128, 64, BF),
]


@pytest.mark.parametrize("lens,new,kv,group,dim,page,dtype", SMALL)
def test_attention_against_64_bits(lens, new, kv, group, dim, page, dtype):
    print(f"case attention {lens} {new} kv={kv} g={group} dim={dim} page={page} {dtype}", flush=True)
    _attend_case(lens, new, kv, group, dim, page, dtype, 31)


@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, HF), (128, BF), (256, BF)])
def test_attention_rows_that_see_nothing(dim, dtype):
    # empty sequences, rows before the first slot, sequences without rows
    _attend_case([0, 3, 40, 0, 16], [2, 7, 0, 0, 17], 2, 3, dim, 16, dtype, 41)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_with_strides_large_logits_and_own_scale(dim, new):
    _attend_case([200, 90], [new, new], 2, 2, dim, 32, BF, 51, scale=0.7, q_gain=3.0, strided=True)
    _attend_case([200, 90], [new, new], 2, 2, dim, 32, HF, 52, scale=1e-3, mass=False)


@pytest.mark.parametrize("new", [1, 3, 33])
def test_attention_bounds_on_the_host_do_not_change_results(new):
    """Looser max_len / max_new only change the launch: with one split instead of several the sums may differ in order."""
    lens, kv, group, dim, page = [900, 411], 2, 4, 128, 16
    _attend_case(lens, [new, new], kv, group, dim, page, BF, 61, max_len=900)
    _attend_case(lens, [new, new], kv, group, dim, page, BF, 61, max_len=None)


def test_attention_shares_pages_and_repeats_bit_for_bit():
    pages, table, ln = _filled([600], 2, 128, 16, 71)
    q = _rows(4, 8, 128, BF, 72).to(DEV)
    tb = table.to(DEV).expand(4, -1).contiguous()
    lens = torch.tensor([600, 600, 37, 512], dtype=torch.int32, device=DEV)
    outs = [sz.kv4_attention(q, pages, tb, lens, return_lse=True) for _ in range(4)]
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
    ro, rl, _, big, mag = R.attention(q.cpu(), pages.cpu(), tb.cpu(), lens.cpu(), torch.arange(5), 128, 128 ** -0.5)
    tol, _ = R.attention_bounds(q, 128, [600], ro, big, mag)
    assert bool(((outs[0][0].cpu().double() - ro).abs() <= tol).all())


def test_attention_without_rows_copies_the_weights():
    pages, table, ln = _filled([90, 5], 2, 64, 16, 85)
    n = pages.shape[0]
    mass, out = torch.rand(n, 2, 16, device=DEV), torch.full((n, 2, 16), -1.0, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    o = sz.kv4_attention(torch.zeros(0, 4, 64, dtype=BF, device=DEV), pages, table.to(DEV), ln.to(DEV), cu=cu, mass=mass,
                         mass_out=out)
    assert tuple(o.shape) == (0, 4, 64)
    live = torch.zeros(n, 16, dtype=torch.bool)
    for b, m in enumerate([90, 5]):
        pg, t = R.slots_of(table, b, m, 16)
        live[pg, t] = True
    live = live[:, None].expand(-1, 2, -1).to(DEV)
    assert torch.equal(out[live], mass[live]) and bool((out[~live] == -1).all())


def test_arguments_that_do_not_fit_are_refused():
    pages, table, ln = _filled([20, 30], 2, 64, 16, 86)
    tb, ls = table.to(DEV), ln.to(DEV)
    q, k = torch.zeros(2, 4, 64, dtype=BF, device=DEV), torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    n = pages.shape[0]
    mass, pos = torch.zeros(n, 2, 16, device=DEV), torch.zeros(n, 2, 16, dtype=torch.int32, device=DEV)
    bad = [
        lambda: sz.kv4_attention(q.float(), pages, tb, ls),
        lambda: sz.kv4_attention(q[:, :3], pages, tb, ls),                       # heads of no group
        lambda: sz.kv4_attention(q[:1], pages, tb, ls),                          # one row for two sequences
        lambda: sz.kv4_attention(q[..., :32], pages, tb, ls),
        lambda: sz.kv4_attention(q, pages[:, :, :-16], tb, ls),
        lambda: sz.kv4_attention(q, pages, tb.long(), ls),
        lambda: sz.kv4_attention(q, pages, tb, ls[:1]),
        lambda: sz.kv4_attention(q, pages, tb, ls, max_len=10 ** 6),
        lambda: sz.kv4_attention(q, pages, tb, ls, mass=mass[:1]),
        lambda: sz.kv4_attention(q, pages, tb, ls, mass_out=mass),
        lambda: sz.kv4_attention(q, pages, tb, ls, out=q[:, :2]),
        lambda: sz.kv4_attention(q, pages, tb, ls, scale=0.0),
        lambda: sz.kv4_attention(q, pages, tb, ls, work=torch.zeros(8, dtype=torch.uint8, device=DEV)),
        lambda: sz.kv4_attention(q.transpose(0, 2), pages, tb, ls),
        lambda: sz.kv4_attention(torch.zeros(2, 4, 65, dtype=BF, device=DEV)[..., 1:], pages, tb, ls),
        lambda: sz.kv4_attention(q, pages, tb, ls, cu=torch.zeros(3, dtype=torch.int32, device=DEV), max_new=0),
        lambda: sz.kv4_append(pages, k, k[:1], tb, ls),
        lambda: sz.kv4_append(pages, k, k.half(), tb, ls),
        lambda: sz.kv4_append(pages, k[:, :1], k[:, :1], tb, ls),
        lambda: sz.kv4_append(pages, k, k, tb, ls, positions=torch.zeros(3, dtype=torch.int32, device=DEV)),
        lambda: sz.kv4_append(pages, k, k, tb, ls, status=torch.zeros(1, device=DEV)),
        lambda: sz.kv4_read(pages, tb, ls, 128),
        lambda: sz.kv4_read(pages, tb, ls, 64, dtype=torch.float32),
        lambda: sz.kv4_read(pages, tb, ls, 64, cu=torch.zeros(3, dtype=torch.int32, device=DEV)),
        lambda: sz.kv4_evict(pages, tb, ls, mass, pos, ls, 64, 0),
        lambda: sz.kv4_evict(pages, tb, ls, mass, pos, ls, 64, 8, sinks=5, recent=4),
        lambda: sz.kv4_evict(pages, tb, ls, mass, pos, ls, 64, -1),
        lambda: sz.kv4_evict(pages, tb, ls, mass[: n - 1], pos, ls, 64, 8),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, sz.SplitZipError)):
            call()
            print("accepted", i, flush=True)
    torch.cuda.synchronize()


def test_attention_mass_accumulates_in_place():
    pages, table, ln = _filled([90, 200], 2, 64, 16, 81)
    q = _rows(2, 4, 64, BF, 82).to(DEV)
    mass = torch.zeros(pages.shape[0], 2, 16, device=DEV)
    args = (pages, table.to(DEV), ln.to(DEV))
    for _ in range(3):
        sz.kv4_attention(q, *args, mass=mass)
    # every row's weights sum to 1: 2 heads of a group and 3 calls a sequence
    per_head = mass.double().sum((0, 2)).cpu()
    assert torch.allclose(per_head, torch.full((2,), 2.0 * 2 * 3, dtype=torch.float64), rtol=1e-5)


def test_pools_beyond_4_gib():
    dim, page, kv = 256, 256, 8
    n_pages = (5 << 30) // (kv * R.page_bytes(dim, page))
    pages = torch.empty(n_pages, kv, R.page_bytes(dim, page), dtype=torch.uint8, device=DEV)
    lens = torch.tensor([300, 40], dtype=torch.int32, device=DEV)
    table = torch.tensor([[n_pages - 1, n_pages - 3], [n_pages - 2, 0]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 300, 340], dtype=torch.int32, device=DEV)
    k, v = _rows(340, kv, dim, BF, 91, 0.3), _rows(340, kv, dim, BF, 92, 0.3)
    mass = torch.zeros(n_pages, kv, page, device=DEV)
    pos = torch.zeros(n_pages, kv, page, dtype=torch.int32, device=DEV)
    sz.kv4_append(pages, k.to(DEV), v.to(DEV), table, lens, cu=cu, mass=mass, pos=pos)
    gk, gv = sz.kv4_read(pages, table, lens, dim, cu=cu, n_tokens=340)
    assert torch.equal(gk.cpu().double(), R.quantize(k.float())[0])
    assert torch.equal(gv.cpu().double(), R.quantize(v.float())[0])
    small = pages[-3:].contiguous().cpu()
    q = _rows(2, kv, dim, BF, 93).to(DEV)
    out = sz.kv4_attention(q, pages, table, lens, mass=mass)
    tb = torch.tensor([[2, 0], [1, 0]], dtype=torch.int32)
    ro, _, rm, big, mag = R.attention(q.cpu(), small, tb, lens.cpu(), torch.arange(3), dim, dim ** -0.5, torch.zeros(3, kv, page))
    tol, d = R.attention_bounds(q, dim, [300], ro, big, mag)
    assert bool(((out.cpu().double() - ro).abs() <= tol).all())
    before = mass[-3:].cpu(), pos[-3:].cpu()
    next_pos = lens.clone()
    sz.kv4_evict(pages, table, lens, mass, pos, next_pos, dim, 100, recent=8)
    wl, wpages, wm, wp = R.evict(small, tb, torch.tensor([300, 40]), *before, torch.tensor([300, 40]), 100, 0, 8, dim)
    assert torch.equal(lens.cpu().long(), wl)
    assert torch.equal(pages[-3:].cpu(), wpages) and torch.equal(mass[-3:].cpu(), wm) and torch.equal(pos[-3:].cpu(), wp)


# -------------------------------------------------------------------- eviction
def _evict_case(lens, budget, sinks, recent, kv, dim, page, seed, in_place, special=True):
    n_pages = sum(-(-n // page) for n in lens) + 2
    g = torch.Generator().manual_seed(seed)
    table = R.table_of(lens, page, n_pages, seed)
    pages = torch.randint(0, 256, (n_pages, kv, R.page_bytes(dim, page)), generator=g, dtype=torch.uint8)
    mass = torch.randn(n_pages, kv, page, generator=g).exp()
    mass = torch.where(torch.rand(mass.shape, generator=g) < 0.3, torch.tensor(0.25), mass)  # ties
    if special:
        r = torch.rand(mass.shape, generator=g)
        for lo, x in ((0.02, math.nan), (0.04, math.inf), (0.06, -math.inf), (0.08, -0.0), (0.10, 0.0), (0.12, -1.5),
                      (0.13, torch.finfo(torch.float32).min), (0.14, 1e-42)):
            mass = torch.where((r < lo) & (r >= lo - 0.02), torch.tensor(x), mass)
    pos = torch.randint(0, 3 * max(lens) + 1, mass.shape, generator=g, dtype=torch.int32)
    next_pos = torch.tensor([3 * n for n in lens], dtype=torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32)
    want = R.evict(pages, table, ln, mass, pos, next_pos, budget, sinks, recent, dim)
    d = [t.to(DEV) for t in (pages, table, ln, mass, pos, next_pos)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = {} if in_place else {"lens_out": torch.full_like(d[2], -5), "mass_out": torch.full_like(d[3], -5.0),
                              "pos_out": torch.full_like(d[4], -5)}
    lo, mo, po = sz.kv4_evict(*d, dim, budget, sinks=sinks, recent=recent, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(lo.cpu(), want[0])
    assert torch.equal(d[0].cpu(), want[1]), "pages"
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))  # noqa: E731  NaN included
    if in_place:
        assert same(mo.cpu(), want[2]) and torch.equal(po.cpu(), want[3])
        return
    assert same(d[3].cpu(), mass) and torch.equal(d[4].cpu(), pos) and torch.equal(d[2].cpu(), ln)
    live = torch.zeros(n_pages, page, dtype=torch.bool)
    for b in range(len(lens)):
        pg, t = R.slots_of(table, b, int(want[0][b]), page)
        live[pg, t] = True
    sel = live[:, None].expand_as(mass)
    assert same(mo.cpu()[sel], want[2][sel]) and torch.equal(po.cpu()[sel], want[3][sel])
    assert bool((mo.cpu()[~sel] == -5).all()) and bool((po.cpu()[~sel] == -5).all())


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,budget,sinks,recent,kv,dim,page", [
    ([1], 1, 0, 0, 1, 64, 16),
    ([2, 0, 1], 1, 0, 1, 2, 128, 16),
    ([65, 64, 63], 64, 4, 8, 3, 128, 16),
    ([1025, 2000, 7], 1000, 1, 100, 2, 64, 32),
    ([300, 180], 7, 0, 0, 2, 256, 64),
    ([4097], 4096, 4, 64, 2, 128, 256),
    ([2500], 2000, 0, 2000, 1, 64, 16),
    ([4096, 4095, 1100], 1024, 0, 4, 2, 64, 16),       # one round of slots, moves within the listed ones
    ([8192, 5000], 2500, 4, 100, 1, 64, 32),           # two rounds, moves listed in memory
    ([16384, 12289, 700], 16000, 4, 100, 1, 64, 128),  # four rounds
    ([16385, 3], 300, 0, 10, 1, 64, 64),               # several workgroups a head
    ([20000, 16400, 40000], 16390, 2, 50, 1, 64, 256),
])
def test_evict_is_exact(lens, budget, sinks, recent, kv, dim, page, in_place):
    print(f"case evict {lens}->{budget} sinks={sinks} recent={recent} kv={kv} dim={dim} page={page}", flush=True)
    _evict_case(lens, budget, sinks, recent, kv, dim, page, 101, in_place)


@pytest.mark.parametrize("n,budget", [(300, 100), (9000, 4500), (50000, 17), (50000, 30000)])
@pytest.mark.parametrize("kind", ["equal", "two", "close", "one magnitude"])
def test_evict_with_few_distinct_weights(n, budget, kind):
    # ties over whole chunks, keys that differ in their last bits only
    g = torch.Generator().manual_seed(n + budget)
    n_pages = -(-n // 256)
    table = torch.randperm(n_pages, generator=g).to(torch.int32)[None]
    bits = {"equal": torch.zeros(n_pages, 1, 256, dtype=torch.int32),
            "two": torch.randint(0, 2, (n_pages, 1, 256), generator=g, dtype=torch.int32) << 20,
            "close": torch.randint(0, 50, (n_pages, 1, 256), generator=g, dtype=torch.int32),
            "one magnitude": torch.randint(0, 1 << 23, (n_pages, 1, 256), generator=g, dtype=torch.int32)}[kind]
    mass = (bits + 0x3F800000).view(torch.float32)
    pos = torch.full((n_pages, 1, 256), 100, dtype=torch.int32)
    pages = torch.randint(0, 256, (n_pages, 1, R.page_bytes(64, 256)), generator=g, dtype=torch.uint8)
    ln, nxt = torch.tensor([n], dtype=torch.int32), torch.tensor([1000000], dtype=torch.int32)
    want = R.evict(pages, table, ln, mass, pos, nxt, budget, 0, 5, 64)
    d = [t.to(DEV) for t in (pages, table, ln, mass, pos, nxt)]
    sz.kv4_evict(*d, 64, budget, recent=5)
    assert torch.equal(d[2].cpu(), want[0]) and torch.equal(d[0].cpu(), want[1]) and torch.equal(d[3].cpu(), want[2])


def test_evict_where_all_weights_are_equal_keeps_the_lowest_slots():
    lens = torch.tensor([50], dtype=torch.int32, device=DEV)
    pages = _pool(4, 1, 64, 16)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    mass = torch.zeros(4, 1, 16, device=DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV).view(4, 1, 16)
    sz.kv4_evict(pages, table, lens, mass, pos, torch.tensor([50], dtype=torch.int32, device=DEV), 64, 20, recent=5)
    p = pos.flatten()[:20].cpu()
    # 15 lowest slots and the 5 newest, which fill the holes in order
    assert int(lens.item()) == 20 and torch.equal(p, torch.cat([torch.arange(15), torch.arange(45, 50)]).int())


# ------------------------------------------------------------ bad device inputs
def test_bad_batches_are_reported_and_stay_in_bounds():
    """Lengths, row offsets and page numbers that point outside are refused by
    the kernels' own checks; the other sequences' results are right."""
    pages, table, ln = _filled([40, 40, 40], 2, 64, 16, 111, extra=4)
    n = pages.shape[0]
    q = _rows(3, 4, 64, BF, 112).to(DEV)
    good = sz.kv4_attention(q, pages, table.to(DEV), ln.to(DEV))
    keep = pages.clone()
    k = _rows(3, 2, 64, BF, 113).to(DEV)
    side = torch.zeros(n, 2, 16, device=DEV)
    posn = torch.zeros(n, 2, 16, dtype=torch.int32, device=DEV)
    cases = []
    for bad_len in (-1, 49, 2 ** 31 - 1):
        x = ln.clone(); x[1] = bad_len
        cases.append(("len", table, x, torch.arange(4, dtype=torch.int32)))
    for bad in (-1, n, 2 ** 31 - 1):
        x = table.clone(); x[1] = bad
        cases.append(("page", x, ln, torch.arange(4, dtype=torch.int32)))
    for cu in ([0, 1, 4, 3], [0, 1, 0, 1], [0, 1, -2, 3]):
        cases.append(("cu", table, ln, torch.tensor(cu, dtype=torch.int32)))
    for what, tb, ls, cu in cases:
        print(f"case bad {what} {ls.tolist()} {cu.tolist()}", flush=True)
        tb, ls, cu = tb.to(DEV), ls.to(DEV), cu.to(DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = sz.kv4_attention(q, pages, tb, ls, cu=cu, max_new=2, status=st, mass=side)
        torch.cuda.synchronize()
        assert int(st.item()) == sz.E_CORRUPT
        # [0, 1, 0, 1] names row 0 for the first and the last sequence: it is either's
        alt = sz.kv4_attention(q[:1], pages, tb[2:], ls[2:]) if cu.tolist() == [0, 1, 0, 1] else good
        assert torch.equal(out[0], good[0]) or torch.equal(out[0], alt[0])
        if what != "cu":
            assert torch.equal(out[2], good[2])
        st.zero_()
        sz.kv4_read(pages, tb, ls, 64, cu=cu, n_tokens=3, max_new=2, status=st)
        assert int(st.item()) == sz.E_CORRUPT
        st.zero_()
        sz.kv4_append(pages, k, k, tb, ls, cu=cu, max_new=2, mass=side, pos=posn, status=st)
        assert int(st.item()) == sz.E_CORRUPT
        pages.copy_(keep)
        if what != "cu":
            st.zero_()
            m2, p2 = side.clone(), posn.clone()
            sz.kv4_evict(pages, tb, ls.clone(), m2, p2, ls, 64, 20, status=st)
            assert int(st.item()) == sz.E_CORRUPT
            # a page of no sequence is never written
            used = torch.unique(table.long()).tolist()
            for x in set(range(n)) - set(used):
                assert torch.equal(m2[x], side[x]) and torch.equal(pages[x], keep[x])
            pages.copy_(keep)
    # more rows than slots: an error for append and read, empty rows for attention
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    two = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    one = torch.tensor([2], dtype=torch.int32, device=DEV)
    sz.kv4_append(pages, k, k, table[:1].to(DEV), one, cu=two, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == sz.E_CORRUPT and torch.equal(pages, keep)


# ------------------------------------------------------- streams, graphs, chains
def _decode_state(seed, lens, kv=2, group=4, dim=128, page=16, room=64):
    cap = [n + room for n in lens]
    n_pages = sum(-(-n // page) for n in cap) + 1
    table = R.table_of(cap, page, n_pages, seed).to(DEV)
    pages = _pool(n_pages, kv, dim, page)
    mass = torch.zeros(n_pages, kv, page, device=DEV)
    pos = torch.zeros(n_pages, kv, page, dtype=torch.int32, device=DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    total = sum(lens)
    k, v = _rows(total, kv, dim, BF, seed + 1, 0.3).to(DEV), _rows(total, kv, dim, BF, seed + 2, 0.3).to(DEV)
    sz.kv4_append(pages, k, v, table, ln, cu=_cu(lens).to(DEV), mass=mass, pos=pos)
    return {"pages": pages, "table": table, "lens": ln, "mass": mass, "pos": pos, "next": ln.clone(), "kv": kv,
            "group": group, "dim": dim, "page": page}


def _step(s, q, k, v, budget, stream=None):
    """One decoding step: the new token in, attention with its weights, the budget kept."""
    s["lens"] += 1
    sz.kv4_append(s["pages"], k, v, s["table"], s["lens"], positions=s["next"], mass=s["mass"], pos=s["pos"], stream=stream)
    out = sz.kv4_attention(q, s["pages"], s["table"], s["lens"], mass=s["mass"], stream=stream)
    s["next"] += 1
    sz.kv4_evict(s["pages"], s["table"], s["lens"], s["mass"], s["pos"], s["next"], s["dim"], budget, sinks=2, recent=8,
                 stream=stream)
    return out


def test_decoding_with_a_budget_end_to_end():
    """Append, attention, accumulation and eviction over many steps, each step
    checked against the plain forms from the state before it."""
    s = _decode_state(121, [30, 45, 3])
    budget = 40
    for step in range(12):
        q = _rows(3, 8, 128, BF, 200 + step).to(DEV)
        k, v = _rows(3, 2, 128, BF, 300 + step, 0.3).to(DEV), _rows(3, 2, 128, BF, 400 + step, 0.3).to(DEV)
        pages, mass, pos = s["pages"].cpu(), s["mass"].cpu(), s["pos"].cpu()
        lens, nxt, table = s["lens"].cpu() + 1, s["next"].cpu(), s["table"].cpu()
        out = _step(s, q, k, v, budget)
        torch.cuda.synchronize()
        for b in range(3):
            slot = int(lens[b]) - 1
            pg, t = int(table[b, slot // 16]), slot % 16
            for h in range(2):
                R.write(pages, 128, pg, t, h, k[b, h].cpu().float(), v[b, h].cpu().float())
            mass[pg, :, t], pos[pg, :, t] = 0.0, nxt[b]
        ro, _, rm, big, mag = R.attention(q.cpu(), pages, table, lens, torch.arange(4), 128, 128 ** -0.5, mass)
        tol, d = R.attention_bounds(q, 128, lens, ro, big, mag)
        assert bool(((out.cpu().double() - ro).abs() <= tol).all()), step
        # the eviction from the weights that the kernel itself accumulated, as far as the slots kept their place
        assert torch.equal(s["lens"].cpu(), lens.clamp(max=budget))
        for b in range(3):
            n = int(s["lens"][b])
            pg, t = R.slots_of(table, b, n, 16)
            for h in range(2):
                p = s["pos"].cpu()[pg, h, t].tolist()
                assert len(set(p)) == n and {0, 1} <= set(p)
                assert set(range(int(nxt[b]) + 1 - min(8, n), int(nxt[b]) + 1)) <= set(p)
                # a kept token's bytes are those appended for its position
                at = {int(x): i for i, x in enumerate(pos[R.slots_of(table, b, int(lens[b]), 16)[0], h,
                                                          R.slots_of(table, b, int(lens[b]), 16)[1]].tolist())}
                old_pg, old_t = R.slots_of(table, b, int(lens[b]), 16)
                kept = [float(rm[old_pg[at[x]], h, old_t[at[x]]]) for x in p]
                gone = [float(rm[old_pg[i], h, old_t[i]]) for x, i in at.items() if x not in set(p)]
                free = [w for w, x in zip(kept, p) if 2 <= x < int(nxt[b]) + 1 - 8]
                if gone and free:
                    assert max(gone) <= min(free) * (1 + 1e-4) + 1e-6
                for i, x in enumerate(p):
                    for a, c in zip(R.places(128, 16, int(t[i])), R.places(128, 16, int(old_t[at[x]]))):
                        assert torch.equal(s["pages"].cpu()[pg[i], h, a], pages[old_pg[at[x]], h, c])


def test_a_step_captured_in_a_graph_replays():
    s = _decode_state(131, [100, 61], room=80)
    e = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    q, k, v = (torch.zeros(2, h, 128, dtype=BF, device=DEV) for h in (8, 2, 2))
    out = torch.zeros(2, 8, 128, dtype=BF, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = {k2: v2.clone() if isinstance(v2, torch.Tensor) else v2 for k2, v2 in s.items()}
    with torch.cuda.stream(side):
        _step(warm, q, k, v, 90)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.copy_(_step(s, q, k, v, 90))
    for step in range(5):
        for x, h, seed in ((q, 8, 500), (k, 2, 600), (v, 2, 700)):
            x.copy_(_rows(2, h, 128, BF, seed + step, 0.3))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = _step(e, q, k, v, 90)
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
        for name in ("pages", "lens", "mass", "pos", "next"):
            assert torch.equal(s[name], e[name]), (step, name)


def test_two_streams_at_once():
    a, b = _decode_state(141, [900, 30], room=64), _decode_state(151, [333], room=64)
    ea = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    eb = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    ins = [[_rows(n, h, 128, BF, 800 + i * 3 + n, 0.3).to(DEV) for h in (8, 2, 2)] for i in range(6) for n in (2, 1)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for i in range(6):
        with torch.cuda.stream(s1):
            got.append(_step(a, *ins[2 * i], 300))
        with torch.cuda.stream(s2):
            got.append(_step(b, *ins[2 * i + 1], 300))
    torch.cuda.synchronize()
    for i in range(6):
        assert torch.equal(_step(ea, *ins[2 * i], 300), got[2 * i])
        assert torch.equal(_step(eb, *ins[2 * i + 1], 300), got[2 * i + 1])
    torch.cuda.synchronize()
    for x, y in ((a, ea), (b, eb)):
        for name in ("pages", "lens", "mass", "pos"):
            assert torch.equal(x[name], y[name])


def test_a_stream_given_by_argument():
    s = _decode_state(161, [64, 200])
    e = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    q, k, v = (_rows(2, h, 128, BF, 900 + h, 0.3).to(DEV) for h in (8, 2, 2))
    st = torch.cuda.Stream()
    s["lens"] += 1
    st.wait_stream(torch.cuda.current_stream())
    sz.kv4_append(s["pages"], k, v, s["table"], s["lens"], mass=s["mass"], pos=s["pos"], stream=st)
    out = sz.kv4_attention(q, s["pages"], s["table"], s["lens"], mass=s["mass"], stream=st)
    gk, gv = sz.kv4_read(s["pages"], s["table"], s["lens"], 128, stream=st)
    torch.cuda.synchronize()
    e["lens"] += 1
    sz.kv4_append(e["pages"], k, v, e["table"], e["lens"], mass=e["mass"], pos=e["pos"])
    assert torch.equal(sz.kv4_attention(q, e["pages"], e["table"], e["lens"], mass=e["mass"]), out)
    wk, wv = sz.kv4_read(e["pages"], e["table"], e["lens"], 128)
    assert torch.equal(gk, wk) and torch.equal(gv, wv) and torch.equal(s["mass"], e["mass"])


def test_a_sequence_handed_on_through_the_codec():
    """Out of the 4-bit cache as BF16, through the lossless codec, into another
    node's 4-bit cache: the bytes are the same there."""
    s = _decode_state(171, [513], room=0)
    lens, cu = s["lens"], torch.tensor([0, 513], dtype=torch.int32, device=DEV)
    k, v = sz.kv4_read(s["pages"], s["table"], lens, 128, cu=cu, n_tokens=513)
    kv = torch.stack([k, v])
    cb = sz.splitzip_calibrate(sz.BF16, kv.view(torch.int16).cpu())
    stream, nbytes = sz.compress(kv.view(torch.int16), cb)
    back, status = sz.decompress(stream, kv.numel(), sz.BF16, in_bytes=int(nbytes.item()))
    assert int(status.item()) == 0
    k2, v2 = back.view(BF).view_as(kv)
    pages = _pool(*s["pages"].shape[:2], 128, 16)
    sz.kv4_append(pages, k2.contiguous(), v2.contiguous(), s["table"], lens, cu=cu)
    a = sz.kv4_read(pages, s["table"], lens, 128, cu=cu, n_tokens=513)
    assert torch.equal(a[0], k) and torch.equal(a[1], v)
    assert int(nbytes.item()) < kv.numel() * 2
    q = _rows(1, 8, 128, HF, 172).to(DEV)
    x = [sz.kv4_attention(q, p, s["table"], lens) for p in (pages, s["pages"])]
    # the second encoding may choose a smaller scale for the same values; the values, and so the results, are equal
    assert torch.equal(x[0], x[1])
