"""The calls around the decode step on the bounds-checking build, and guard regions around
what they write and read: as for the decode kernels, stand-ins for a memory checker.

Guards of 4096 bytes lie on both sides of every output, cache and workspace.  Behind outputs
they hold a pattern that must come back untouched; around inputs they hold NaN (all bits set),
which would show in a result that a read outside took part in."""
import os
import subprocess
import sys

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GUARD = 4096
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def test_serving_suites_run_clean_on_the_bounds_checking_build():
    from softmax_tree_reduction_gb300 import build
    lib = build.build(debug=True)
    env = dict(os.environ, TREE_ATTN_LIBRARY=lib, TREE_ATTN_CHECK_ERRORS="1")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_tokens_gpu.py",
           "tests/test_selected_pages_gpu.py", "tests/test_serving_limits_gpu.py", "tests/test_serving_bounds_gpu.py", "-k", "not checking_build"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in tail and "failed" not in tail, tail


class Guarded:
    """Device memory of one tensor between two guards."""

    def __init__(self, shape, dtype, init=None, pattern=0xA5):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        self.pattern = pattern
        self.raw = torch.full((n + 2 * GUARD,), pattern, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)
        if init is not None:
            self.t.copy_(init) if dtype != FP8 else self.t.view(torch.uint8).copy_(init.view(torch.uint8))

    def whole(self):
        return bool((self.raw[:GUARD] == self.pattern).all()) and bool((self.raw[self.raw.numel() - GUARD:] == self.pattern).all())


def source(x):
    """A copy of x on the device between guards of NaN."""
    return Guarded(x.shape, x.dtype, x.cuda(), 0xFF).t


def same(a, b):
    a, b = (x.view(torch.uint8) if x.dtype == FP8 else x for x in (a, b))
    return torch.equal(a, b) or torch.equal(torch.nan_to_num(a.float(), nan=3e33), torch.nan_to_num(b.float(), nan=3e33))


@pytest.mark.parametrize("T,hq,hkv,d,dt", [(1, 3, 1, 128, BF16), (5, 1, 1, 64, F32), (333, 7, 2, 64, BF16), (20000, 2, 1, 64, F32), (20001, 1, 1, 128, BF16)])
def test_norm_rope_guards(T, hq, hkv, d, dt):
    g = torch.Generator().manual_seed(T)
    q, k = (torch.randn(T, h, d, generator=g).to(dt) for h in (hq, hkv))
    pos = torch.arange(T, dtype=torch.int32)
    f = torch.rand(d // 2, generator=g)
    w = torch.rand(d, generator=g).to(dt)
    qo, ko = Guarded(q.shape, dt), Guarded(k.shape, dt)
    ta.tree_attn_norm_rope(source(q), source(k), source(pos), source(f), q_weight=source(w), k_weight=source(w), q_out=qo.t, k_out=ko.t)
    a, b = ta.tree_attn_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), q_weight=w.cuda(), k_weight=w.cuda())
    assert torch.equal(qo.t, a) and torch.equal(ko.t, b) and qo.whole() and ko.whole()
    assert bool(torch.isfinite(a).all()) and bool(torch.isfinite(b).all()) and ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kv,page,layout", [(BF16, 0, "HND"), (F32, 0, "NHD"), (FP8, 0, "HND"), (BF16, 16, "NHD"), (FP8, 32, "HND"), (F32, 16, "HND")])
@pytest.mark.parametrize("B,S,hkv,d", [(1, 1, 1, 64), (3, 37, 3, 128), (2, 1601, 1, 64)])
def test_cache_write_and_read_guards(kv, page, layout, B, S, hkv, d):
    """Every place of the cache written and read back, the first and the last among them."""
    g = torch.Generator().manual_seed(S + d)
    per = -(-S // page) if page else 0
    shape = (B * per, page, hkv, d) if page else (B, S, hkv, d)

    def cache(pattern):
        order = (0, 2, 1, 3)
        c = Guarded(tuple(shape[i] for i in order) if layout == "HND" else shape, kv, pattern=pattern)
        if page:                                            # [pages, page, heads, d]
            return c, (c.t.transpose(1, 2) if layout == "HND" else c.t)
        return c, (c.t if layout == "HND" else c.t.transpose(1, 2))
    gk, kc = cache(0xA5)
    gv, vc = cache(0xA5)
    T = B * S
    k, v = (torch.randn(T, hkv, d, generator=g).to(F32 if kv == F32 else BF16) for _ in range(2))
    place = torch.randperm(T, generator=g)
    rows, pos = source((place // S).to(torch.int32)), source((place % S).to(torch.int32))
    bt = source(torch.randperm(B * per, generator=g).view(B, per).to(torch.int32)) if page else None
    sc = dict(k_scale=source(torch.full((hkv,), 0.01)), v_scale=source(torch.full((hkv,), 0.02))) if kv == FP8 else {}
    ta.tree_attn_cache_write(source(k), source(v), kc, vc, pos, rows=rows, block_table=bt, max_seqlen=S, **sc)
    assert gk.whole() and gv.whole() and ta.tree_attn_get_device_error() == 0
    for odt in (BF16, F32):
        ko, vo = Guarded(k.shape, odt), Guarded(k.shape, odt)
        ta.tree_attn_cache_read(kc, vc, pos, rows=rows, block_table=bt, k_out=ko.t, v_out=vo.t, max_seqlen=S, **sc)
        assert ko.whole() and vo.whole() and ta.tree_attn_get_device_error() == 0
        for o, x, s in ((ko.t, k, 0.01), (vo.t, v, 0.02)):
            if kv == FP8:                                    # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale below its normal range
                lim = x.float().abs().clamp(max=448 * s)
                near = (o.cpu().float() - x.float().clamp(-448 * s, 448 * s)).abs() <= (2.0 ** -4 + 2.0 ** -7) * lim + 2.0 ** -10 * s * 1.01
                assert bool(near.all())
            else:
                assert torch.equal(o.cpu(), x.to(odt))


@pytest.mark.parametrize("kv,d,hkv,page", [(BF16, 128, 3, 16), (BF16, 64, 1, 64), (FP8, 128, 5, 32), (FP8, 64, 2, 16), (F32, 128, 1, 128), (F32, 64, 7, 16)])
def test_page_bounds_guards(kv, d, hkv, page):
    g = torch.Generator().manual_seed(page + d)
    lens = torch.tensor([page * 3 - 1, 1, page * 7, 0], dtype=torch.int32)
    per = 7
    k = torch.randn(4 * per, page, hkv, d, generator=g).to(kv)
    bt = torch.randperm(4 * per, generator=g).view(4, per).to(torch.int32)
    b = Guarded((4 * per, hkv, 2, d), F32 if kv == F32 else BF16)
    b.t.zero_()
    for new in (0, 1, page + 1):
        ta.tree_attn_page_bounds(source(k), source(bt), source(lens), b.t, new_tokens=new)
        assert b.whole()
    assert torch.equal(b.t, ta.tree_attn_page_bounds(k.cuda(), bt.cuda(), lens.cuda())) and bool(torch.isfinite(b.t).all())
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("hkv,d,bdt", [(1, 64, BF16), (3, 128, BF16), (5, 64, F32), (9, 128, F32)])
@pytest.mark.parametrize("n", [2, 5, 33, 251, 1031, 2047, 24577])
def test_select_pages_guards(n, hkv, d, bdt):
    """Odd page counts; all but one listed, one listed, and every page alike, which takes the exact
    sums and all of their workspace."""
    page, B, G = 16, 2, 2
    if n > 20000 and hkv > 3:
        hkv = 1
    g = torch.Generator().manual_seed(n)
    mid = torch.randn(n, hkv, 1, d, generator=g)
    bounds = torch.cat([mid - 1, mid + 1], 2).to(bdt)
    q = torch.randn(B, hkv * G, d, generator=g).to(bdt)
    bt = torch.stack([torch.randperm(n, generator=g) for _ in range(B)]).to(torch.int32)
    lens = torch.tensor([n * page, n * page - page + 1], dtype=torch.int32)
    nbytes = ta.tree_attn_select_workspace_bytes(B, hkv, n)
    ins = [source(x) for x in (q, bounds, bt, lens)]
    alike = source(bounds[:1].expand(n, hkv, 2, d).contiguous())
    for nsel in sorted({1, n // 2 or 1, n - 1}):
        for bnd in (ins[1], alike):
            sel, ws = Guarded((B, hkv, nsel), torch.int32), Guarded((nbytes,), torch.uint8)
            ta.tree_attn_select_pages(ins[0], bnd, ins[2], ins[3], page, nsel, 0, 1 if nsel > 1 else 0, selected=sel.t, workspace=ws.t, max_seqlen=n * page)
            assert sel.whole() and ws.whole() and ta.tree_attn_get_device_error() == 0
            got = sel.t.cpu()
            assert bool((got[..., 1:] > got[..., :-1]).all()) and int(got.min()) >= 0 and int(got.max()) < n
            if bnd is alike:                                 # the lowest pages, and the forced last one
                want = list(range(nsel)) if nsel == 1 else list(range(nsel - 1)) + [n - 1]
                assert got.tolist() == [[want] * hkv] * B


@pytest.mark.parametrize("kv,d,hkv,G,page", [(BF16, 128, 2, 4, 16), (BF16, 64, 1, 9, 64), (BF16, 128, 1, 33, 32), (FP8, 128, 2, 7, 16), (FP8, 128, 1, 17, 64),
                                             (F32, 128, 2, 3, 16), (F32, 64, 1, 1, 32), (F32, 64, 2, 9, 16)])
@pytest.mark.parametrize("nsel", [1, 5, 61, 700])
def test_decode_selected_guards(kv, d, hkv, G, page, nsel):
    g = torch.Generator().manual_seed(nsel + G)
    B, per = 3, max(5, nsel)
    lens = torch.tensor([page * per, page * (per - 1) + 1, 1], dtype=torch.int32)
    k, v = (torch.randn(B * per, page, hkv, d, generator=g).to(kv) for _ in range(2))
    bt = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32)
    q = torch.randn(B, hkv * G, d, generator=g).to(F32 if kv == F32 else BF16)
    sel = torch.randperm(per, generator=g)[:nsel].to(torch.int32).expand(B, hkv, nsel).contiguous()
    sc = dict(k_scale=source(torch.full((hkv,), 0.5)), v_scale=source(torch.full((hkv,), 0.5))) if kv == FP8 else {}
    out, lse = Guarded(q.shape, F32), Guarded(q.shape[:2], F32)
    ta.tree_attn_decode_selected(source(q), source(k), source(v), source(bt), source(lens), source(sel), out=out.t, lse=lse.t, **sc)
    a, b = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda(), sel.cuda(), **sc)
    assert torch.equal(out.t, a) and same(lse.t, b) and out.whole() and lse.whole()
    assert bool(torch.isfinite(a).all()) and not bool(torch.isnan(b).any()) and ta.tree_attn_get_device_error() == 0
