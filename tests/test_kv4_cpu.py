"""The 4-bit KV cache's calls without a GPU: every refusal returns before any
GPU work (fake addresses, never dereferenced), the size queries, and the plain
forms that the GPU tests compare with."""
import ctypes

import pytest
import torch

import kv4lib as R

sz = pytest.importorskip("lossless_kv_cache_splitzip_amd")
N = sz._native
P = 1 << 20  # 256-byte aligned


def cache(**kw):
    return N.KV4CacheDesc(**{**dict(d_pages=P, n_pages=10, n_heads=2, head_dim=128, page_tokens=16), **kw})


def batch(**kw):
    return N.KV4BatchDesc(**{**dict(d_table=P, table_stride=4, d_lens=P, d_cu=P, n_seqs=3, max_len=64, max_new=5,
                                    n_rows=7), **kw})


BAD_CACHES = [dict(d_pages=None), dict(d_pages=P + 8), dict(n_pages=0), dict(n_pages=1 << 31), dict(n_heads=0),
              dict(n_heads=1025), dict(head_dim=0), dict(head_dim=96), dict(head_dim=512), dict(page_tokens=8),
              dict(page_tokens=24), dict(page_tokens=512)]
BAD_BATCHES = [dict(d_table=None), dict(d_lens=None), dict(d_lens=P + 2), dict(d_table=P + 1), dict(table_stride=3),
               dict(n_seqs=65536), dict(max_len=(1 << 23) + 1, table_stride=1 << 30)]
BAD_ROWS = [dict(d_cu=P + 2), dict(max_new=8), dict(n_rows=(1 << 30) + 1), dict(d_cu=None),
            dict(d_cu=None, n_rows=3, max_new=0), dict(max_new=0)]


def append(c, b, **kw):
    a = {**dict(dtype=sz.BF16, k=P, ks=256, kh=128, v=P, vs=256, vh=128, positions=None, mass=None, pos=None,
                status=None), **kw}
    return N.load().splitzip_kv4_append(ctypes.byref(c), ctypes.byref(b), a["dtype"], a["k"], a["ks"], a["kh"], a["v"],
                                        a["vs"], a["vh"], a["positions"], a["mass"], a["pos"], a["status"], None)


def read(c, b, **kw):
    a = {**dict(dtype=sz.BF16, k=P, v=P, status=None), **kw}
    return N.load().splitzip_kv4_read(ctypes.byref(c), ctypes.byref(b), a["dtype"], a["k"], a["v"], a["status"], None)


def attention(c, b, **kw):
    a = {**dict(dtype=sz.BF16, q=P, qs=512, qh=128, heads=4, scale=0.1, out=P, lse=None, mass=None, mass_out=None,
                work=P, bytes=1 << 40, status=None), **kw}
    return N.load().splitzip_kv4_attention(ctypes.byref(c), ctypes.byref(b), a["dtype"], a["q"], a["qs"], a["qh"],
                                           a["heads"], a["scale"], a["out"], a["lse"], a["mass"], a["mass_out"],
                                           a["work"], a["bytes"], a["status"], None)


def evict(c, b, **kw):
    a = {**dict(budget=32, sinks=2, recent=8, next=P, mass=P, pos=P, lens_out=P, mass_out=P, pos_out=P, work=P,
                bytes=1 << 40, status=None), **kw}
    return N.load().splitzip_kv4_evict(ctypes.byref(c), ctypes.byref(b), a["budget"], a["sinks"], a["recent"],
                                       a["next"], a["mass"], a["pos"], a["lens_out"], a["mass_out"], a["pos_out"],
                                       a["work"], a["bytes"], a["status"], None)


@pytest.mark.parametrize("call", [append, read, attention, evict])
def test_bad_caches_and_batches_are_refused(call):
    for kw in BAD_CACHES:
        assert call(cache(**kw), batch()) == sz.E_INVALID, kw
    for kw in BAD_BATCHES + ([] if call is evict else BAD_ROWS):
        assert call(cache(), batch(**kw)) == sz.E_INVALID, kw


def test_append_refusals():
    for kw in (dict(dtype=0), dict(dtype=4), dict(k=None), dict(v=None), dict(k=P + 8), dict(ks=257), dict(kh=4),
               dict(vs=2), dict(vh=12), dict(positions=P + 2), dict(mass=P + 1), dict(pos=P + 2), dict(status=P + 2),
               dict(dtype=sz.FP8_E5M2, k=P + 4)):
        assert append(cache(), batch(), **kw) == sz.E_INVALID, kw
    assert append(cache(), batch(n_seqs=0, max_new=0, n_rows=0)) == sz.OK  # nothing to do
    assert append(cache(), batch(max_new=0, n_rows=0), k=None, v=None) == sz.OK


def test_read_refusals():
    for kw in (dict(dtype=sz.FP8_E5M2), dict(k=P + 8), dict(v=P + 2), dict(status=P + 1)):
        assert read(cache(), batch(), **kw) == sz.E_INVALID, kw
    assert read(cache(), batch(), k=None, v=None) == sz.OK
    assert read(cache(), batch(max_new=0, n_rows=0)) == sz.OK


def test_attention_refusals():
    for kw in (dict(dtype=sz.FP8_E5M2), dict(q=None), dict(out=None), dict(q=P + 8), dict(out=P + 8), dict(qs=4),
               dict(qh=20), dict(heads=0), dict(heads=3), dict(heads=2 * 65), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(lse=P + 2), dict(mass=P), dict(mass_out=P),
               dict(mass=P + 2, mass_out=P), dict(work=P + 64), dict(work=None), dict(status=P + 2)):
        assert attention(cache(), batch(), **kw) == sz.E_INVALID, kw
    b = batch(max_len=10_000, table_stride=1000)
    need = N.load().splitzip_kv4_attention_work_bytes(ctypes.byref(cache()), ctypes.byref(b), 4, 1)
    assert need > 256 and need % 256 == 0
    assert attention(cache(), b, mass=P, mass_out=P, bytes=need - 1) == sz.E_CAPACITY
    assert attention(cache(), batch(n_seqs=0)) == sz.OK
    # the largest batches have a plan, with a workspace that fits the card
    for kw in (dict(n_seqs=65535, n_rows=65535, max_new=1, d_cu=None, max_len=1 << 23, table_stride=1 << 19),
               dict(n_seqs=60000, n_rows=1 << 20, max_new=40, max_len=4096, table_stride=256),
               dict(n_seqs=1, n_rows=1 << 17, max_new=1 << 17, max_len=1 << 17, table_stride=1 << 13)):
        need = N.load().splitzip_kv4_attention_work_bytes(ctypes.byref(cache()), ctypes.byref(batch(**kw)), 8, 1)
        assert 0 < need < 64 << 30, (kw, need)
    assert attention(cache(), batch(max_new=0, n_rows=0)) == sz.OK


def test_evict_refusals():
    for kw in (dict(budget=0), dict(budget=9), dict(sinks=1 << 31, recent=1 << 31), dict(next=None), dict(mass=None),
               dict(pos=None), dict(lens_out=None), dict(mass_out=None), dict(pos_out=None), dict(work=None),
               dict(work=P + 128), dict(mass=P + 2), dict(next=P + 1), dict(status=P + 3)):
        assert evict(cache(), batch(), **kw) == sz.E_INVALID, kw
    need = N.load().splitzip_kv4_evict_work_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 32)
    assert need >= 256 and evict(cache(), batch(), bytes=need - 1) == sz.E_CAPACITY
    assert evict(cache(), batch(n_seqs=0)) == sz.OK


def test_sizes():
    lib = N.load()
    for dim in (64, 128, 256):
        for page in (16, 32, 64, 128, 256):
            assert sz.kv4_page_bytes(dim, page) == R.page_bytes(dim, page)
    for dim, page in ((0, 16), (32, 16), (128, 0), (128, 48), (128, 512)):
        assert lib.splitzip_kv4_page_bytes(dim, page) == 0
        with pytest.raises(sz.SplitZipError):
            sz.kv4_page_bytes(dim, page)
    # arguments that the calls refuse have no workspace
    c, b = cache(), batch()
    for kw in BAD_CACHES:
        assert lib.splitzip_kv4_attention_work_bytes(ctypes.byref(cache(**kw)), ctypes.byref(b), 4, 0) == 0
        assert lib.splitzip_kv4_evict_work_bytes(ctypes.byref(cache(**kw)), ctypes.byref(b), 4) == 0
    for kw in BAD_BATCHES + BAD_ROWS:
        assert lib.splitzip_kv4_attention_work_bytes(ctypes.byref(c), ctypes.byref(batch(**kw)), 4, 0) == 0
    assert lib.splitzip_kv4_attention_work_bytes(ctypes.byref(c), ctypes.byref(b), 5, 0) == 0
    assert lib.splitzip_kv4_evict_work_bytes(ctypes.byref(c), ctypes.byref(b), 0) == 0
    assert lib.splitzip_kv4_attention_work_bytes(None, ctypes.byref(b), 4, 0) == 0
    assert sz.status_string(sz.E_NONFINITE) == "NaN or infinity in K or V"


def test_wrappers_refuse_host_tensors():
    pages = torch.zeros(4, 2, R.page_bytes(64, 16), dtype=torch.uint8)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    side = torch.zeros(4, 2, 16)
    with pytest.raises(ValueError):
        sz.kv4_append(pages, k, k, table, lens)
    with pytest.raises(ValueError):
        sz.kv4_read(pages, table, lens, 64)
    with pytest.raises(ValueError):
        sz.kv4_attention(k, pages, table, lens)
    with pytest.raises(ValueError):
        sz.kv4_evict(pages, table, lens, side, side.int(), lens, 64, 8)


# ------------------------------------------------------------- the plain forms
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_the_layout_uses_every_byte_once(dim, page):
    seen = torch.cat([torch.cat(R.places(dim, page, t)) for t in range(page)])
    assert torch.equal(seen.sort().values, torch.arange(R.page_bytes(dim, page)))


def test_quantizing_twice_changes_nothing_and_is_never_far():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(400, 64, generator=g, dtype=R.F64) * torch.exp(20 * torch.randn(400, 1, generator=g, dtype=R.F64))
    y, codes, scales = R.quantize(x)
    assert torch.equal(R.quantize(y)[0], y)
    e = scales.double().sub(127).exp2().repeat_interleave(32, -1)
    inside = (scales > 1).repeat_interleave(32, -1) & (scales < 252).repeat_interleave(32, -1)
    assert bool(((x - y).abs() <= e)[inside].all())
    top = x.abs().unflatten(-1, (-1, 32)).amax(-1)
    s = scales.double().sub(127).exp2()
    ok = (scales > 1) & (scales < 252)
    assert bool(((top < 7 * s) & (top >= 3.5 * s))[ok].all())  # the least such exponent
    assert int(codes.max()) <= 15


def test_pool_values_and_attention_of_the_plain_form():
    g = torch.Generator().manual_seed(4)
    pages = torch.full((3, 2, R.page_bytes(64, 16)), 255, dtype=torch.uint8)
    table = torch.tensor([[2, 0]], dtype=torch.int32)
    k, v = torch.randn(20, 2, 64, generator=g), torch.randn(20, 2, 64, generator=g)
    for i in range(20):
        for h in range(2):
            R.write(pages, 64, int(table[0, i // 16]), i % 16, h, k[i, h], v[i, h])
    kk, vv = R.values(pages, 64)
    pg, t = R.slots_of(table, 0, 20, 16)
    assert torch.equal(kk[pg, :, t], R.quantize(k)[0]) and torch.equal(vv[pg, :, t], R.quantize(v)[0])
    q = torch.randn(3, 4, 64, generator=g)
    mass = torch.zeros(3, 2, 16)
    out, lse, m, _, _ = R.attention(q, pages, table, [20], [0, 3], 64, 0.125, mass)
    x = (q[1, 3].double() @ R.quantize(k)[0][:19, 1].T) * 0.125
    assert torch.allclose(out[1, 3], torch.softmax(x, 0) @ R.quantize(v)[0][:19, 1], atol=1e-12)
    assert torch.allclose(lse[1, 3], torch.logsumexp(x, 0))
    assert torch.allclose(m.sum((0, 2)), torch.tensor([6.0, 6.0], dtype=R.F64))
