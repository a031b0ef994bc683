"""Page bounds, page selection and decode attention over selected pages on the
GPU, against plain 64-bit implementations.

Bounds and selections are compared exactly.  Attention: logits are sums of 128
products at most, |q . k| / sqrt(d) over their absolute values is under 12
for these inputs, so a logit is off by at most 128 * 2^-24 * 12 < 1e-4 and an
output by twice that times |v| < 5: 1e-3 with BF16 operands (the weights' two
parts keep 2^-16 more: 8e-5); FP32 caches sum 20 terms deep: 2e-4."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import serving_reference as ref

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
TOL = {torch.bfloat16: (1e-3, 2e-4), FP8: (1e-3, 2e-4), torch.float32: (2e-4, 1e-4)}


def pool(g, kv, pages, page, hkv, d, layout, mul=1.0):
    x = torch.randn(pages, page, hkv, d, generator=g) * (mul * (60.0 if kv == FP8 else 1.0))
    x = x.to(kv)
    if layout == "HND":
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    return x


def table(g, B, per, pages):
    return torch.randperm(pages, generator=g)[: B * per].view(B, per).to(torch.int32)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("kv,d,hkv,page", [(torch.bfloat16, 128, 3, 64), (torch.bfloat16, 64, 1, 16), (FP8, 128, 2, 32), (FP8, 64, 5, 128),
                                           (torch.float32, 128, 2, 16), (torch.float32, 64, 1, 64)])
def test_page_bounds(kv, d, hkv, page, layout):
    g = torch.Generator().manual_seed(d + page)
    lens = torch.tensor([0, 1, page - 1, page, page + 1, 5 * page, 5 * page + 7], dtype=torch.int32)
    B, per = len(lens), 7
    pages = B * per + 2
    k = pool(g, kv, pages, page, hkv, d, layout)
    bt = table(g, B, per, pages)
    bdt = torch.float32 if kv == torch.float32 else torch.bfloat16
    start = torch.randn(pages, hkv, 2, d, generator=g).to(bdt)
    for new in (0, 1, 2, page, page + 1, 3 * page + 5, 10 ** 6):
        b = start.clone().cuda()
        out = ta.tree_attn_page_bounds(k.cuda(), bt.cuda(), lens.cuda(), b, new_tokens=new)
        want = ref.page_bounds(k, bt, lens, start.double().clone(), new)
        assert out is b and torch.equal(b.cpu().double(), want), new
    assert ta.tree_attn_get_device_error() == 0
    fresh = ta.tree_attn_page_bounds(k.cuda(), bt.cuda(), lens.cuda())
    assert torch.equal(fresh.cpu().double(), ref.page_bounds(k, bt, lens, torch.zeros(pages, hkv, 2, d, dtype=torch.float64)))


def test_page_bounds_nan_inf_junk_and_bad_data():
    g = torch.Generator().manual_seed(0)
    for kv in (torch.bfloat16, torch.float32, FP8):
        k = pool(g, kv, 6, 16, 2, 64, "NHD")
        k = k.float()
        k[1, 3, 0, 5] = float("nan")
        if kv != FP8:
            k[1, 4, 1, 6], k[1, 5, 1, 7] = float("inf"), -float("inf")
        k[2, 9:] = float("nan")                              # behind the row's end
        k = k.to(kv)
        bt = torch.tensor([[1, 2, 9], [4, -2, 0]], dtype=torch.int32)
        lens = torch.tensor([25, 20], dtype=torch.int32)
        b = torch.full((6, 2, 2, 64), 3.0, dtype=torch.float32 if kv == torch.float32 else torch.bfloat16).cuda()
        ta.tree_attn_page_bounds(k.cuda(), bt.cuda(), lens.cuda(), b)
        assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA     # row 1's second page
        bt2 = torch.tensor([[1, 2, 9], [4, 0, 0]], dtype=torch.int32)
        want = ref.page_bounds(k, bt2[:1], lens[:1], torch.full((6, 2, 2, 64), 3.0, dtype=torch.float64))
        want = ref.page_bounds(k, bt2[1:], torch.tensor([16]), want)
        got = b.cpu().double()
        assert torch.isnan(got[1, 0, :, 5]).all()
        assert torch.equal(torch.nan_to_num(got, nan=1e9, posinf=1e8, neginf=-1e8), torch.nan_to_num(want, nan=1e9, posinf=1e8, neginf=-1e8))
        b0 = b.clone()
        ta.tree_attn_page_bounds(k.cuda(), bt2.cuda(), torch.tensor([-1, 49], dtype=torch.int32).cuda(), b)
        assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
        assert torch.equal(torch.nan_to_num(b, nan=7.0), torch.nan_to_num(b0, nan=7.0))


def page_ranges(g, pages, hkv, d, dt):
    mid = 0.6 * torch.randn(pages, hkv, 1, d, generator=g)
    return torch.cat([mid - 1 - torch.rand(pages, hkv, 1, d, generator=g), mid + 1 + torch.rand(pages, hkv, 1, d, generator=g)], 2).to(dt)


@pytest.mark.parametrize("qdt,bdt,d,hkv,G,page", [(torch.bfloat16, torch.bfloat16, 128, 2, 4, 64), (torch.bfloat16, torch.bfloat16, 64, 1, 16, 16),
                                                  (torch.float32, torch.float32, 128, 3, 1, 16), (torch.float32, torch.float32, 64, 2, 8, 32),
                                                  (torch.float32, torch.bfloat16, 128, 1, 5, 16), (torch.bfloat16, torch.float32, 64, 2, 2, 16)])
@pytest.mark.parametrize("nsel,first,last", [(1, 0, 0), (1, 1, 0), (7, 1, 2), (64, 0, 0), (64, 3, 61), (700, 2, 2)])
def test_select_pages(qdt, bdt, d, hkv, G, page, nsel, first, last):
    g = torch.Generator().manual_seed(nsel + d + G)
    lens = torch.tensor([0, 1, page * nsel, page * nsel + 1, page * 611 + 3, page * 612], dtype=torch.int32).clamp(max=page * 800)
    B, per = len(lens), 800
    pages = 1500
    bt = torch.randint(0, pages, (B, per), generator=g).to(torch.int32)      # rows may share pages: equal scores
    bounds = page_ranges(g, pages, hkv, d, bdt)
    q = torch.randn(B, hkv * G, d, generator=g).to(qdt)
    sel = ta.tree_attn_select_pages(q.cuda(), bounds.cuda(), bt.cuda(), lens.cuda(), page, nsel, first, last)
    assert torch.equal(sel.cpu(), ref.select_pages(q, bounds, bt, lens, page, nsel, first, last))
    assert ta.tree_attn_get_device_error() == 0


def test_select_pages_near_ties_ties_and_values_not_finite():
    """Scores that differ by one part in 2^30, equal ones, zeros of both signs, infinities, NaN and
    pages outside the pool; 20000 pages, so that a thread's run and a radix pass are long."""
    d, page, n = 64, 16, 20000
    g = torch.Generator().manual_seed(9)
    bounds = torch.zeros(n, 1, 2, d)
    bounds[:, 0, 1, 0] = 1.0
    step = torch.randint(0, 50, (n,), generator=g)           # score 1 + step * 2^-30 (exact in two FP32 numbers)
    bounds[:, 0, 1, 1] = step.float() * 2.0 ** -30
    bt = torch.randperm(n, generator=g).view(1, n).to(torch.int32)
    q = torch.ones(1, 2, d)
    lens = torch.tensor([n * page], dtype=torch.int32)
    for bdt in (torch.float32, torch.bfloat16):              # 2^-30 * (0..49) and 1 are exact in BF16
        b = bounds.to(bdt)
        for nsel in (5, 1000, 13000, 19999):
            sel = ta.tree_attn_select_pages(q.cuda(), b.cuda(), bt.cuda(), lens.cuda(), page, nsel)
            assert torch.equal(sel.cpu(), ref.select_pages(q, b, bt, lens, page, nsel, 1, 1)), nsel
    flat = torch.zeros(n, 1, 2, d)
    flat[::3] = -0.0
    sel = ta.tree_attn_select_pages(q.cuda(), flat.cuda(), bt.cuda(), lens.cuda(), page, 77, 0, 0)
    assert sel.cpu()[0, 0].tolist() == list(range(77))
    odd = page_ranges(g, n, 1, d, torch.float32)
    odd[5, 0, 1, 3], odd[77, 0, 0, 2], odd[400, 0, 1, 9] = float("inf"), -float("inf"), float("nan")
    sel = ta.tree_attn_select_pages(q.cuda(), odd.cuda(), bt.cuda(), lens.cuda(), page, 40, 0, 0)
    assert torch.equal(sel.cpu(), ref.select_pages(q, odd, bt, lens, page, 40, 0, 0))
    assert all((bt[0, sel.cpu()[0, 0].long()] == p).any() for p in (5, 77, 400))
    assert ta.tree_attn_get_device_error() == 0
    out = bt.clone()
    out[0, 123], out[0, 19000] = -1, n
    sel = ta.tree_attn_select_pages(q.cuda(), odd.cuda(), out.cuda(), lens.cuda(), page, 40, 0, 0)
    assert {123, 19000} <= set(sel.cpu()[0, 0].tolist())     # decoding them reports them
    sel = ta.tree_attn_select_pages(q.cuda(), odd.cuda(), bt.cuda(), torch.tensor([n * page + 1], dtype=torch.int32).cuda(), page, 40)
    assert (sel == -1).all() and ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA


def lists(g, B, hkv, nsel, pages_of_row, order, fill=1.0):
    sel = torch.full((B, hkv, nsel), -1, dtype=torch.int32)
    for b in range(B):
        for h in range(hkv):
            n = min(int(nsel * fill), int(pages_of_row[b]))
            pick = torch.randperm(int(pages_of_row[b]), generator=g)[:n] if n else torch.zeros(0, dtype=torch.int64)
            if order == "up":
                sel[b, h, :n] = pick.sort()[0].to(torch.int32)
            else:
                at = torch.randperm(nsel, generator=g)[:n]
                sel[b, h, at] = pick.to(torch.int32)
    return sel


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("nsel,order,fill", [(1, "up", 1.0), (3, "mixed", 0.7), (40, "up", 1.0), (65, "mixed", 0.5), (200, "up", 1.0)])
@pytest.mark.parametrize("kv,d,hkv,G,page", [(torch.bfloat16, 128, 2, 4, 64), (torch.bfloat16, 128, 1, 12, 16), (torch.bfloat16, 64, 3, 1, 32),
                                             (torch.bfloat16, 64, 1, 40, 16), (FP8, 128, 2, 8, 16), (FP8, 128, 1, 20, 128),
                                             (torch.float32, 128, 2, 1, 16), (torch.float32, 64, 2, 8, 64), (torch.float32, 128, 1, 6, 32),
                                             (torch.float32, 128, 1, 2, 64), (torch.float32, 64, 2, 3, 16), (torch.float32, 64, 1, 11, 32), (torch.float32, 128, 1, 16, 128)])
def test_decode_selected(kv, d, hkv, G, page, nsel, order, fill, layout):
    g = torch.Generator().manual_seed(d + G + nsel)
    lens = torch.tensor([0, 1, 17, page * 40 + 5, page * 60], dtype=torch.int32)
    B, per = len(lens), 60
    pages = B * per + 1
    k, v = pool(g, kv, pages, page, hkv, d, layout), pool(g, kv, pages, page, hkv, d, layout)
    bt = table(g, B, per, pages)
    qdt = torch.float32 if kv == torch.float32 else torch.bfloat16
    q = torch.randn(B, hkv * G, d, generator=g).to(qdt)
    sel = lists(g, B, hkv, nsel, -(-lens // page), order, fill)
    ks, vs = (((torch.rand(hkv, generator=g) * 0.01 + 0.01) if kv == FP8 else None) for _ in range(2))
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    out, lse = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda(), sel.cuda(), k_scale=cu(ks), v_scale=cu(vs))
    want, wl = ref.decode_selected(q, k, v, bt, lens, sel, k_scale=ks, v_scale=vs)
    to, tl = TOL[kv]
    assert (out.cpu().double() - want).abs().max() <= to
    fin = torch.isfinite(wl)
    assert torch.equal(torch.isfinite(lse.cpu()), fin) and (lse.cpu()[~fin] == -math.inf).all()
    assert not fin.any() or (lse.cpu().double() - wl)[fin].abs().max() <= tl
    again, none = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda(), sel.cuda(), k_scale=cu(ks), v_scale=cu(vs),
                                               want_lse=False)
    assert none is None and torch.equal(again, out)          # bitwise reproducible
    assert ta.tree_attn_get_device_error() == 0


def test_decode_selected_every_page_is_the_paged_decode_and_scale():
    g = torch.Generator().manual_seed(2)
    page, hkv, G, d = 32, 2, 4, 128
    lens = torch.tensor([1000, 333], dtype=torch.int32)
    k, v = pool(g, torch.bfloat16, 70, page, hkv, d, "NHD"), pool(g, torch.bfloat16, 70, page, hkv, d, "NHD")
    bt = table(g, 2, 32, 70)
    q = torch.randn(2, hkv * G, d, generator=g).to(torch.bfloat16)
    sel = torch.arange(32, dtype=torch.int32).expand(2, hkv, 32).contiguous()      # row 1: pages past its end hold no token
    args = (q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda())
    for scale in (None, 0.02):
        a, al = ta.tree_attn_decode_selected(*args, sel.cuda(), scale=scale)
        b, bl = ta.tree_attn_decode_paged(*args, scale=scale)
        assert (a - b).abs().max() <= 2e-3 and (al - bl).abs().max() <= 4e-4       # each within its own bound of the exact result
    # a page listed twice counts twice
    one = torch.tensor([[[3], [4]], [[1], [2]]], dtype=torch.int32)
    twice = torch.cat([one, one], 2).contiguous()
    a, al = ta.tree_attn_decode_selected(*args, one.cuda())
    b, bl = ta.tree_attn_decode_selected(*args, twice.cuda())
    assert (a - b).abs().max() <= 2e-3 and (bl - al - math.log(2)).abs().max() <= 4e-4


def test_decode_selected_junk_and_bad_data():
    """NaN behind a row's end and in unlisted pages is never read into a result; bad entries make
    their own (row, KV head) NaN and are reported."""
    g = torch.Generator().manual_seed(4)
    for kv, G in ((torch.bfloat16, 4), (FP8, 4), (torch.float32, 2)):
        page, hkv, d, B, per = 16, 2, 128, 3, 20
        pages = B * per
        lens = torch.tensor([300, 41, 5], dtype=torch.int32)
        bt = table(g, B, per, pages)
        k, v = (pool(g, kv, pages, page, hkv, d, "NHD").float() for _ in range(2))
        sel = torch.tensor([[[18, 2, 7, -5], [0, 1, -1, 9]], [[2, 0, 19, -1], [1, 2, 3, -2 ** 31]], [[0, 5, -1, -1], [-1, -1, 3, 7]]], dtype=torch.int32)
        keep = torch.zeros(pages, page, hkv, dtype=torch.bool)
        for b in range(B):
            for h in range(hkv):
                for s in sel[b, h].tolist():
                    if 0 <= s and s * page < int(lens[b]):
                        keep[int(bt[b, s]), : int(lens[b]) - s * page, h] = True
        k[~keep], v[~keep] = float("nan"), float("nan")
        k, v = k.to(kv), v.to(kv)
        qdt = torch.float32 if kv == torch.float32 else torch.bfloat16
        q = torch.randn(B, hkv * G, d, generator=g).to(qdt)
        sc = torch.full((hkv,), 0.015) if kv == FP8 else None
        kw = dict(k_scale=sc.cuda(), v_scale=sc.cuda()) if kv == FP8 else {}
        out, lse = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda(), sel.cuda(), **kw)
        want, wl = ref.decode_selected(q, k, v, bt, lens, sel, k_scale=sc, v_scale=sc)
        to, tl = TOL[kv]
        assert (out.cpu().double() - want).abs().max() <= to
        assert (lse.cpu()[2, G:] == -math.inf).all() and (out[2, G:] == 0).all()
        assert ta.tree_attn_get_device_error() == 0
        bad_sel, bad_bt = sel.clone(), bt.clone()
        bad_sel[1, 1, 3] = per                        # not below max_pages
        bad_bt[0, 18] = pages                         # a valid page outside the pool: row 0, head 0
        bad_bt[2, 7] = -9                             # behind row 2's end: never looked at
        o2, l2 = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bad_bt.cuda(), lens.cuda(), bad_sel.cuda(), **kw)
        assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
        bad = torch.zeros(B, hkv * G, dtype=torch.bool)
        bad[0, :G], bad[1, G:] = True, True
        assert torch.isnan(o2.cpu()[bad]).all() and torch.isnan(l2.cpu()[bad]).all()
        assert torch.equal(o2.cpu()[~bad], out.cpu()[~bad])
        o3, _ = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), torch.tensor([321, -1, 5], dtype=torch.int32).cuda(), sel.cuda(), **kw)
        assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
        assert torch.isnan(o3[:2]).all() and torch.equal(o3[2], out[2])


def test_many_lists_and_long_lists():
    """More lists than fit on the device at once (no clusters), and lists long enough that every
    warp looks several windows of slabs up."""
    g = torch.Generator().manual_seed(6)
    page, hkv, G, d = 16, 4, 2, 128
    for B, per, nsel in ((70, 12, 9), (1, 9000, 8990), (5, 2100, 2050)):
        lens = torch.randint(per * page // 2, per * page + 1, (B,), generator=g).to(torch.int32)
        pages = B * per
        kk = torch.randn(pages, page, hkv, d, generator=g).to(torch.bfloat16)
        bt = table(g, B, per, pages)
        q = torch.randn(B, hkv * G, d, generator=g).to(torch.bfloat16)
        sel = lists(g, B, hkv, nsel, -(-lens // page), "mixed")
        out, lse = ta.tree_attn_decode_selected(q.cuda(), kk.cuda(), kk.cuda(), bt.cuda(), lens.cuda(), sel.cuda())
        want, wl = ref.decode_selected(q, kk, kk, bt, lens, sel)
        assert (out.cpu().double() - want).abs().max() <= 1e-3 and (lse.cpu().double() - wl).abs().max() <= 2e-4
    assert ta.tree_attn_get_device_error() == 0


def test_decode_loop_with_selected_pages():
    """The calls as a serving loop uses them: a prompt written (normed, rotated, E4M3 or BF16),
    its bounds, then steps of write -> bounds -> select -> decode, one of them replayed from a
    graph; every stage checked against the 64-bit reference on what the stage before it left."""
    g = torch.Generator().manual_seed(8)
    page, hkv, G, d, B = 16, 2, 4, 128, 3
    hq, per = hkv * G, 40
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    for kv in (torch.bfloat16, FP8):
        pages = B * per
        kc, vc = torch.zeros(pages, page, hkv, d).to(kv).cuda(), torch.zeros(pages, page, hkv, d).to(kv).cuda()
        bt = table(g, B, per, pages)
        btd = bt.cuda()
        sc = dict(k_scale=torch.full((hkv,), 0.02).cuda(), v_scale=torch.full((hkv,), 0.02).cuda()) if kv == FP8 else {}
        lens = torch.tensor([500, 37, 260], dtype=torch.int32)
        rows = torch.repeat_interleave(torch.arange(B), lens.long()).to(torch.int32).cuda()
        pos = torch.cat([torch.arange(int(n)) for n in lens]).to(torch.int32).cuda()
        x = torch.randn(int(lens.sum()), hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
        ta.tree_attn_cache_write(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, pos, rows=rows, block_table=btd, inv_freq=f, norm=True, **sc)
        bounds = ta.tree_attn_page_bounds(kc, btd, lens.cuda())
        step_x = torch.zeros(B, hq + 2 * hkv, d, dtype=torch.bfloat16).cuda()
        step_pos, step_len = lens.cuda() - 1, lens.cuda().clone()
        qo, sel = torch.zeros(B, hq, d, dtype=torch.bfloat16).cuda(), torch.zeros(B, hkv, 8, dtype=torch.int32).cuda()
        out, lse = torch.zeros(B, hq, d).cuda(), torch.zeros(B, hq).cuda()
        ws = torch.empty(ta.tree_attn_select_workspace_bytes(B, hkv, per), dtype=torch.uint8).cuda()

        def step():
            step_pos.add_(1)
            step_len.add_(1)
            ta.tree_attn_cache_write(step_x[:, hq:hq + hkv], step_x[:, hq + hkv:], kc, vc, step_pos, block_table=btd, q=step_x[:, :hq], q_out=qo,
                                     inv_freq=f, norm=True, **sc)
            ta.tree_attn_page_bounds(kc, btd, step_len, bounds, new_tokens=1)
            ta.tree_attn_select_pages(qo, bounds, btd, step_len, page, 8, 1, 2, selected=sel, workspace=ws)
            ta.tree_attn_decode_selected(qo, kc, vc, btd, step_len, sel, out=out, lse=lse, **sc)

        graph = None
        for i in range(20):
            step_x.copy_(torch.randn(B, hq + 2 * hkv, d, generator=g).to(torch.bfloat16))
            if i == 3:
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    step()
            if graph is not None:
                graph.replay()
            else:
                step()
            n = step_len.cpu()
            assert torch.equal(n, lens + i + 1)
            assert torch.equal(bounds.cpu().double()[bt[0, 0]], ref.page_bounds(kc, bt, n, torch.zeros(pages, hkv, 2, d, dtype=torch.float64))[bt[0, 0]])
            full = ref.page_bounds(kc, bt, n, bounds.cpu().double().clone())
            assert torch.equal(bounds.cpu().double(), full)              # kept up to date for every page in use
            assert torch.equal(sel.cpu(), ref.select_pages(qo, bounds, bt, n, page, 8, 1, 2))
            s = sc.get("k_scale")
            want, wl = ref.decode_selected(qo, kc, vc, bt, n, sel.cpu(), k_scale=s.cpu() if s is not None else None,
                                           v_scale=s.cpu() if s is not None else None)
            # (normed queries and keys: |q . k| / sqrt(d) can reach sqrt(128) = 11.4, as above)
            assert (out.cpu().double() - want).abs().max() <= 1e-3 and (lse.cpu().double() - wl).abs().max() <= 2e-4
    assert ta.tree_attn_get_device_error() == 0


def test_two_streams_do_not_share_anything():
    """Two selections and decodes at once on two streams give what each gives alone."""
    g = torch.Generator().manual_seed(12)
    page, hkv, G, d, B, per = 16, 2, 4, 128, 2, 600
    pages = B * per
    kk = torch.randn(pages, page, hkv, d, generator=g).to(torch.bfloat16).cuda()
    bt = table(g, B, per, pages).cuda()
    lens = torch.tensor([9000, 9600], dtype=torch.int32).cuda()
    bounds = ta.tree_attn_page_bounds(kk, bt, lens)
    qs = [torch.randn(B, hkv * G, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]

    def both(q, stream=None):
        s = ta.tree_attn_select_pages(q, bounds, bt, lens, page, 100, stream=stream)
        return (s, *ta.tree_attn_decode_selected(q, kk, kk, bt, lens, s, stream=stream))
    alone = [both(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [both(q, st) for q, st in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("distinct", [True, False])
def test_select_pages_of_very_long_rows(distinct):
    """More pages than the selection keeps in shared memory; with few physical pages behind a
    long table most scores are equal, so ties decide."""
    d, page, n = 64, 16, 40003
    g = torch.Generator().manual_seed(21)
    pages = n if distinct else 60
    bounds = page_ranges(g, pages, 1, d, torch.bfloat16)
    bt = (torch.randperm(n, generator=g) if distinct else torch.randint(0, pages, (n,), generator=g)).view(1, n).to(torch.int32)
    q = torch.randn(1, 3, d, generator=g).to(torch.bfloat16)
    lens = torch.tensor([n * page - 5], dtype=torch.int32)
    for nsel, first, last in ((1, 0, 0), (700, 3, 5), (30000, 0, 1)):
        sel = ta.tree_attn_select_pages(q.cuda(), bounds.cuda(), bt.cuda(), lens.cuda(), page, nsel, first, last)
        assert torch.equal(sel.cpu(), ref.select_pages(q, bounds, bt, lens, page, nsel, first, last)), nsel
    assert ta.tree_attn_get_device_error() == 0


def test_pools_past_32_bit_offsets():
    """Bounds, selection and decode on pages whose element and byte offsets pass 2^32 (one 4.4 GB
    E4M3 pool for keys and values)."""
    page, hkv, d = 64, 8, 128
    pages = (2 ** 32) // (page * hkv * d) + 600
    k = torch.zeros(pages, page, hkv, d, dtype=torch.uint8, device="cuda")
    far = torch.tensor([0, 1, 65535, 65536, pages - 1, pages - 2, pages - 300], dtype=torch.int64)
    g = torch.Generator().manual_seed(1)
    for p in far.tolist():
        k[p] = (torch.randn(page, hkv, d, generator=g) * 50).to(FP8).view(torch.uint8).cuda()
    k = k.view(FP8)
    bt = far.view(1, 7).to(torch.int32)
    lens = torch.tensor([7 * page - 9], dtype=torch.int32)
    bounds = ta.tree_attn_page_bounds(k, bt.cuda(), lens.cuda())
    small = k.view(torch.uint8)[far.cuda()].cpu().view(FP8)
    near = torch.arange(7, dtype=torch.int32).view(1, 7)
    want = ref.page_bounds(small, near, lens, torch.zeros(7, hkv, 2, d, dtype=torch.float64))
    assert torch.equal(bounds[far.cuda()].cpu().double(), want)
    q = torch.randn(1, 32, d, generator=g).to(torch.bfloat16)
    sel = ta.tree_attn_select_pages(q.cuda(), bounds, bt.cuda(), lens.cuda(), page, 4, 1, 1)
    assert torch.equal(sel.cpu(), ref.select_pages(q, want.to(torch.bfloat16), near, lens, page, 4, 1, 1))
    sc = torch.full((hkv,), 0.02)
    out, lse = ta.tree_attn_decode_selected(q.cuda(), k, k, bt.cuda(), lens.cuda(), sel, k_scale=sc.cuda(), v_scale=sc.cuda())
    w, wl = ref.decode_selected(q, small, small, near, lens, sel.cpu(), k_scale=sc, v_scale=sc)
    assert (out.cpu().double() - w).abs().max() <= 1e-3 and (lse.cpu().double() - wl).abs().max() <= 2e-4
    assert ta.tree_attn_get_device_error() == 0


def test_stream_handles_and_empty_rows():
    g = torch.Generator().manual_seed(3)
    page, hkv, d, B = 16, 1, 64, 3
    k = pool(g, torch.bfloat16, 9, page, hkv, d, "NHD").cuda()
    bt = table(g, B, 3, 9).cuda()
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    q = torch.randn(B, 2, d, generator=g).to(torch.bfloat16).cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (None, 0, st, st.cuda_stream):
        b = ta.tree_attn_page_bounds(k, bt, lens, stream=stream)
        sel = ta.tree_attn_select_pages(q, b, bt, lens, page, 2, stream=stream)
        out, lse = ta.tree_attn_decode_selected(q, k, k, bt, lens, sel, stream=stream)
        torch.cuda.synchronize()
        assert (b == 0).all() and (sel == -1).all() and (out == 0).all() and (lse == -math.inf).all()
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kv,d,G", [(torch.bfloat16, 64, 3), (torch.bfloat16, 64, 16), (torch.bfloat16, 128, 9), (FP8, 128, 4), (torch.float32, 64, 2)])
def test_decode_selected_much_work(kv, d, G):
    """Enough tokens for the wide blocks (BF16), a page size of four slabs, lists in any order."""
    g = torch.Generator().manual_seed(d + G)
    page, hkv, B, per, nsel = 64, 2, 4, 520, 500
    lens = torch.tensor([page * per, page * 400 + 9, page * per - 1, 17], dtype=torch.int32)
    pages = B * per
    k, v = (pool(g, kv, pages, page, hkv, d, "HND") for _ in range(2))
    bt = table(g, B, per, pages)
    q = torch.randn(B, hkv * G, d, generator=g).to(torch.float32 if kv == torch.float32 else torch.bfloat16)
    sel = lists(g, B, hkv, nsel, -(-lens // page), "mixed")
    sc = torch.full((hkv,), 0.015) if kv == FP8 else None
    kw = dict(k_scale=sc.cuda(), v_scale=sc.cuda()) if kv == FP8 else {}
    out, lse = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda(), sel.cuda(), **kw)
    want, wl = ref.decode_selected(q, k, v, bt, lens, sel, k_scale=sc, v_scale=sc)
    to, tl = TOL[kv]
    assert (out.cpu().double() - want).abs().max() <= to and (lse.cpu().double() - wl).abs().max() <= tl
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("bdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("alike", [1, 2, 31, 32, 33, 200])
def test_select_pages_outliers_and_pages_alike(bdt, alike):
    """The last places fall among `alike` equal pages, at the numbers where the ways of telling
    pages apart change over; pages far above the others, forced or not, stretch the range."""
    d, page, n, nsel = 128, 16, 2011, 300
    g = torch.Generator().manual_seed(alike)
    q = torch.randn(1, 4, d, generator=g).to(bdt)
    lens = torch.tensor([n * page - 3], dtype=torch.int32)
    base = page_ranges(g, n, 1, d, bdt)
    for scaled, by in (([], 1.0), ([0, n - 1], 3.0e4), ([0, 700, n - 1], 3.0e4), ([700], 1.0e34), ([3, 1500], 1.0e37), (list(range(n)), 1.0e-30)):
        bounds = base.clone()
        bounds[scaled] = (bounds[scaled].float() * by).to(bdt)
        bt = torch.arange(n).view(1, n)
        scores = ref.page_scores(q[0], bounds, bt[0], 0, 4)
        edge = scores.argsort(descending=True)[nsel - 20]    # one of the last to be listed
        same = torch.randperm(n - 1000, generator=g)[:alike - 1] + 900    # pages that repeat one of the listed
        bt[0, same] = edge
        bt = bt.to(torch.int32)
        for first, last in ((1, 1), (0, 0), (2, 40), (150, 150)):
            sel = ta.tree_attn_select_pages(q.cuda(), bounds.cuda(), bt.cuda(), lens.cuda(), page, nsel, first, last)
            assert torch.equal(sel.cpu(), ref.select_pages(q, bounds, bt, lens, page, nsel, first, last)), (scaled, first, last)
    assert ta.tree_attn_get_device_error() == 0
