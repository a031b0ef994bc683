"""4-bit caches written and read on the GPU, against the 64-bit definition: bit for bit where the
vectors are stored as they are; after norms and rotations every code is the one next to the
FP32 channel over the stored step."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import serving_reference as ref
from . import window_reference as wref

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def cache(g, rows, tokens, hkv, d, layout, paged):
    """Codes and steps of one cache on the host, random, as [rows or pages, tokens, Hkv, ..]; and their device views in the call's order."""
    def make(last, dt):
        shape = (rows, tokens, hkv, last) if layout == "NHD" else (rows, hkv, tokens, last)
        x = torch.randint(0, 120, shape, generator=g, dtype=torch.uint8)
        host = x if layout == "NHD" else x.transpose(1, 2)
        dev = x.cuda() if layout == "NHD" else x.cuda().transpose(1, 2)
        return host.clone(), (dev if paged else dev.transpose(1, 2)).view(dt)
    return make(d // 2, torch.uint8), make(d // 16, FP8)


def bytes_of(x, paged):
    x = x.view(torch.uint8).cpu()
    return x if paged else x.transpose(1, 2)


def lists(g, B, S, T):
    """Distinct places of T tokens, and padding among them."""
    place = torch.randperm(B * S, generator=g)[:T]
    rows, pos = (place // S).to(torch.int32), (place % S).to(torch.int32)
    pad = torch.rand(T, generator=g) < 0.15
    if T < 4:
        pad[:] = False
    pos[pad] = -3
    return rows, pos


def heads(g, T, h, d, dt, mul):
    return (torch.randn(T, h, d, generator=g) * mul).to(dt)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("page,layout", [(0, "HND"), (0, "NHD"), (16, "NHD"), (64, "HND")])
@pytest.mark.parametrize("T,hkv,d,scaled", [(1, 1, 128, 0), (5, 3, 64, 1), (37, 8, 128, 1), (300, 2, 64, 0), (4096, 5, 128, 1), (9000, 1, 64, 0)])
def test_write_and_read_are_the_definition(T, hkv, d, scaled, page, layout, dt):
    g = torch.Generator().manual_seed(T + hkv + page)
    B, S = 7, max(16, T)
    per = -(-S // page) if page else 0
    places = (B * per + 1, page) if page else (B, S)
    caches = [cache(g, *places, hkv, d, layout, page) for _ in range(2)]
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32) if page else None
    rows, pos = lists(g, B, S, T)
    x = [heads(g, T, hkv, d, dt, mul) for mul in (1.0, 30.0)]
    x[0][0, 0, :16] = 0                                        # a group of zeros
    x[1][-1, -1, -16:] = 2.0 ** -20                              # below the smallest step
    x[1][0, 0, 16:32] *= 1e6                                     # beyond the largest
    sc = [torch.rand(hkv, generator=g) + 0.5 for _ in range(2)] if scaled else [None, None]
    (kc, dkc), (kst, dkst) = caches[0]
    (vc, dvc), (vst, dvst) = caches[1]
    kw = dict(rows=rows.cuda(), block_table=None if table is None else table.cuda(), k_scale=None if not scaled else sc[0].cuda(),
              v_scale=None if not scaled else sc[1].cuda(), max_seqlen=S)
    ta.tree_attn_cache_write_int4(x[0].cuda(), x[1].cuda(), dkc, dvc, dkst, dvst, pos.cuda(), **kw)
    out = {odt: ta.tree_attn_cache_read_int4(dkc, dvc, dkst, dvst, pos.cuda(), dtype=odt, **kw) for odt in (BF16, F32)}
    live = torch.nonzero(pos >= 0).squeeze(1)
    r, p = rows[live].long(), pos[live].long()
    at = (table[r, p // page].long(), p % page) if page else (r, p)
    for i, (codes, steps, dc, ds) in enumerate(((kc, kst, dkc, dkst), (vc, vst, dvc, dvst))):
        n, st = wref.quantize(x[i][live], sc[i])
        codes[at] = wref.pack(n)
        steps[at] = st.view(torch.uint8)
        assert torch.equal(bytes_of(dc, page), codes) and torch.equal(bytes_of(ds, page), steps)   # other places among them
        y = wref.dequantize(codes[at], steps[at].view(FP8), sc[i])
        for odt in (BF16, F32):
            got = out[odt][i].cpu()
            assert torch.equal(got[live], y.float().to(odt)) and not bool(got[pos < 0].any())
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("dt", [BF16, F32])
def test_ties_halves_and_neighbours(dt):
    """Channels in the middle of two codes, and the FP32 numbers next to it, for every E4M3 step."""
    steps = torch.arange(1, 0x7f, dtype=torch.uint8).view(FP8).float()             # 2^-9 .. 448
    d = 64
    k = torch.zeros(steps.numel() * 8, 1, d)
    t = 0
    for s in steps.tolist():
        for j in range(7):
            mid = torch.tensor((j + 0.5) * s)
            up, dn = torch.nextafter(mid, torch.tensor(math.inf)), torch.nextafter(mid, torch.tensor(0.0))
            row = torch.stack([torch.tensor(7.0 * s), mid, -mid, up, -up, dn, -dn, torch.tensor(j * s), torch.tensor(-float(j) * s)])
            k[t, 0, 0:9] = row
            k[t, 0, 16:25] = row.flip(0)
            k[t, 0, 39:48] = row
            t += 1
    k = k.to(dt)
    T = k.shape[0]
    kc = torch.zeros(1, 1, T, d // 2, dtype=torch.uint8).cuda()
    st = torch.zeros(1, 1, T, d // 16, dtype=torch.uint8).cuda().view(FP8)
    vc, vst = kc.clone(), st.clone()
    pos = torch.arange(T, dtype=torch.int32).cuda()
    ta.tree_attn_cache_write_int4(k.cuda(), k.cuda(), kc, vc, st, vst, pos, rows=torch.zeros_like(pos))
    n, s = wref.quantize(k)
    for c, x in ((kc, st), (vc, vst)):
        assert torch.equal(x.view(torch.uint8).cpu()[0, 0], s.view(torch.uint8)[:, 0])
        assert torch.equal(c.cpu()[0, 0], wref.pack(n)[:, 0])


@pytest.mark.parametrize("m", range(8))
def test_every_number_over_a_step(m):
    """All FP32 numbers z of 2^-2 .. 7.5 steps, for a step of each mantissa (1 + m / 8): in the middle of two codes, next to it and
    elsewhere.  The first channel of each 16 sets the step."""
    c = 1 + m / 8
    first = torch.tensor(c / 4).view(torch.int32).item()
    last = torch.tensor(7.5 * c).view(torch.int32).item()
    at, n = first, 15 * 4 * 65536                                 # 65536 tokens of 64 channels
    codes = torch.zeros(1, 1, 65536, 32, dtype=torch.uint8, device="cuda")
    steps = torch.zeros(1, 1, 65536, 4, dtype=torch.uint8, device="cuda").view(FP8)
    vc, vs = codes.clone(), steps.clone()
    pos = torch.arange(65536, dtype=torch.int32, device="cuda")
    rows = torch.zeros_like(pos)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    while at <= last:
        z = torch.arange(at, at + n, dtype=torch.int32, device="cuda").clamp(max=last).view(torch.float32).view(65536, 4, 15)
        sign = torch.where(torch.arange(15, device="cuda") % 2 == 0, 1.0, -1.0)
        x = torch.cat([torch.full((65536, 4, 1), 7 * c, device="cuda"), torch.where(z > 7 * c, 7 * c, z) * sign], 2)
        ta.tree_attn_cache_write_int4(x.view(65536, 1, 64), x.view(65536, 1, 64), codes, vc, steps, vs, pos, rows=rows)
        # (a quotient in 64 bits lies in the middle of two whole numbers only if the true one does)
        want = (torch.round(x.double() / c).clamp(-7, 7) + 8).to(torch.uint8).view(65536, 64)
        got = torch.stack([codes[0, 0] & 15, codes[0, 0] >> 4], -1).view(65536, 64)
        wrong += (got != want).sum() + (steps.float() != c).sum() + (codes != vc).sum()
        at += n
    assert int(wrong) == 0


@pytest.mark.parametrize("d,rot,inter", [(128, 128, 0), (128, 128, 1), (64, 64, 0), (128, 16, 0), (128, 48, 0), (64, 16, 0), (64, 48, 0), (128, 96, 1),
                                         (128, 80, 0), (64, 0, 0), (128, 112, 0), (64, 32, 1)])
@pytest.mark.parametrize("T", [1, 33, 4100])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_write_with_norm_and_rotation(T, d, rot, inter, dt):
    g = torch.Generator().manual_seed(rot + T)
    hq, hkv, S = 6, 3, 1 << 20
    q, k, v = (heads(g, T, h, d, dt, 2.0) for h in (hq, hkv, hkv))
    pos = torch.randint(0, S, (T,), generator=g).to(torch.int32)
    slots = torch.arange(T, dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(max(1, rot // 2)) / max(1, rot // 2))).float() if rot else None
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(dt) for _ in range(2))
    page = 16
    # position p of row t lies on page t (the block table sends every page of a row there)
    kc, vc = (torch.zeros(T, page, hkv, d // 2, dtype=torch.uint8).cuda() for _ in range(2))
    kst, vst = (torch.zeros(T, page, hkv, d // 16, dtype=torch.uint8).cuda().view(FP8) for _ in range(2))
    table = slots.view(T, 1).expand(T, S // page).contiguous() if T < 100 else None
    if table is None:                                             # many tokens: positions below the page's size
        pos = pos % page
        table = slots.view(T, 1).contiguous()
    qo = ta.tree_attn_cache_write_int4(k.cuda(), v.cuda(), kc, vc, kst, vst, pos.cuda(), block_table=table.cuda(), q=q.cuda(),
                                       inv_freq=None if f is None else f.cuda(), q_weight=qw.cuda(), k_weight=kw.cuda(), norm=True, interleaved=bool(inter))
    same, _ = ta.tree_attn_norm_rope(q.cuda(), None, pos.cuda(), None if f is None else f.cuda(), q_weight=qw.cuda(), norm=True, interleaved=bool(inter))
    assert torch.equal(qo, same)
    want, mag = ref.norm_rotate(k, pos, f, kw, True, 1e-6, bool(inter))
    at = (slots.long(), (pos % page).long())
    codes, steps = wref.unpack(kc.cpu()[at]), kst.view(torch.uint8).cpu()[at].view(FP8)
    # FP32 channels: the norm's sum of d squares (d + 4 roundings, half of them count under the root), the weight, and the
    # rotation with angles 9.4e-8 rad off, of numbers up to |a| + |b|
    off = (d + 16) * 2.0 ** -24 * mag + 1.3e-7 * mag
    top = want.abs().unflatten(-1, (-1, 16)).amax(-1)
    room = off.unflatten(-1, (-1, 16)).amax(-1)
    s = ref.values(steps)
    assert bool((( s - top / 7).abs() <= 2.0 ** -4 * top / 7 * (1 + 2.0 ** -20) + room / 7 + 2.0 ** -10).all())   # E4M3: half a step is 2^-4, 2^-10 at the bottom
    n = codes.double() - 8
    ss = s.repeat_interleave(16, -1)
    err = (n * ss - want).abs()
    inside = want.abs() <= 7 * ss
    assert bool((err <= ss / 2 + off)[inside].all()) and bool((n.abs() == 7)[want.abs() > 7.5 * ss + off].all())
    nv, sv = wref.quantize(v)
    assert torch.equal(wref.pack(nv), vc.cpu()[at]) and torch.equal(sv.view(torch.uint8), vst.view(torch.uint8).cpu()[at])
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("dt,d,hkv", [(BF16, 128, 2), (F32, 64, 3), (BF16, 64, 1)])
def test_views_of_one_tensor_and_repeated_reads(dt, d, hkv):
    """Queries, keys and values as views of one product, queries turned in place; outputs as views of one tensor; places read twice."""
    g = torch.Generator().manual_seed(3)
    T, hq = 75, 2 * hkv
    x = heads(g, T, hq + 2 * hkv, d, dt, 1.5).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    f = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()
    rows, pos = torch.randint(0, 4, (T,), generator=g, dtype=torch.int32).cuda(), torch.arange(T, dtype=torch.int32).cuda()
    caches = []
    for dense in (True, False):
        y = x.clone()
        a, b, c = (y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:]) if not dense else (q.contiguous(), k.contiguous(), v.contiguous())
        kc, vc = (torch.zeros(4, hkv, 80, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(4, hkv, 80, d // 16, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2))
        qo = ta.tree_attn_cache_write_int4(b, c, kc, vc, ks, vs, pos, rows=rows, q=a, q_out=a, inv_freq=f)
        assert qo is a
        caches.append([a.clone(), kc, vc, ks.view(torch.uint8), vs.view(torch.uint8)])
        if not dense:
            assert torch.equal(y[:, hq:], x[:, hq:])
    assert all(torch.equal(m, n) for m, n in zip(*caches))
    _, kc, vc, ks, vs = caches[0]
    ks, vs = ks.view(FP8), vs.view(FP8)
    k1, v1 = ta.tree_attn_cache_read_int4(kc, vc, ks, vs, pos, rows=rows, dtype=dt)
    twice = torch.arange(T).repeat_interleave(2).flip(0).cuda()
    both = torch.full((2 * T, 2 * hkv + 1, d), 5.0, dtype=dt, device="cuda")
    ta.tree_attn_cache_read_int4(kc, vc, ks, vs, pos[twice].contiguous(), rows=rows[twice].contiguous(), k_out=both[:, :hkv], v_out=both[:, hkv + 1:])
    assert torch.equal(both[:, :hkv], k1[twice]) and torch.equal(both[:, hkv + 1:], v1[twice]) and bool((both[:, hkv] == 5).all())
    assert ta.tree_attn_get_device_error() == 0


def test_values_not_finite():
    d, hkv = 128, 2
    k = torch.ones(4, hkv, d)
    k[0, 0, 5] = math.nan
    k[1, 1, 20] = math.inf
    k[2, 0, 127] = -math.inf
    k[3, 1, 64:66] = torch.tensor([math.nan, math.inf])
    kc, vc = (torch.zeros(4, hkv, 8, d // 2, dtype=torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.zeros(4, hkv, 8, d // 16, dtype=torch.uint8).cuda().view(FP8) for _ in range(2))
    pos = torch.tensor([0, 3, 7, 1], dtype=torch.int32).cuda()
    ta.tree_attn_cache_write_int4(k.cuda(), k.cuda(), kc, vc, ks, vs, pos)
    for out in ta.tree_attn_cache_read_int4(kc, vc, ks, vs, pos, dtype=F32):
        o = out.cpu()
        assert bool(torch.isnan(o[0, 0, :16]).all()) and bool(torch.isnan(o[3, 1, 64:80]).all()) and int(torch.isnan(o).sum()) == 32
        assert float(o[1, 1, 20]) == 7 * 448 and float(o[2, 0, 127]) == -7 * 448
        assert not bool(o[1, 1, 16:20].any())                     # 1 is less than half of a step of 448
        assert bool(((o[0, 1] - 1).abs() <= 2.0 ** -4 + 1 / 14).all())  # ones: the step within 2^-4 of 1/7, and half of one


def test_bad_places_and_padding():
    g = torch.Generator().manual_seed(0)
    d, hkv, page = 64, 1, 16
    k = heads(g, 6, hkv, d, BF16, 1.0).cuda()
    kc, vc = (torch.full((3, page, hkv, d // 2), 0x5A, dtype=torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.full((3, page, hkv, d // 16), 0x30, dtype=torch.uint8).cuda().view(FP8) for _ in range(2))
    table = torch.tensor([[0, 7], [2, -1]], dtype=torch.int32).cuda()
    rows = torch.tensor([0, 0, 1, 1, 2, -1], dtype=torch.int32).cuda()
    pos = torch.tensor([3, 17, 4, 20, 0, 1], dtype=torch.int32).cuda()
    ta.tree_attn_cache_write_int4(k, k, kc, vc, ks, vs, pos, rows=rows, block_table=table)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    changed = (kc.cpu() != 0x5A).any(-1).any(-1).nonzero().tolist()
    assert changed == [[0, 3], [2, 4]]
    a, b = (torch.full((6, hkv, d), 9.0, dtype=BF16).cuda() for _ in range(2))
    ta.tree_attn_cache_read_int4(kc, vc, ks, vs, pos, rows=rows, block_table=table, k_out=a, v_out=b)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    assert bool(torch.isnan(a[[1, 3, 4]]).all()) and bool((a[5] == 9).all()) and bool(torch.isfinite(a[[0, 2]]).all())
    ta.tree_attn_cache_write_int4(k[:2], k[:2], kc, vc, ks, vs, torch.tensor([32, 0], dtype=torch.int32).cuda(), block_table=table)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA       # behind the last page
