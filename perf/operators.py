"""Measured cases of the library's serving operators around the decode step.

Six calls, each in a plain form (elementary torch operations) and as the
library's own entry point:

  norm_rope   per-head RMS norms of queries and keys with the position rotation
  write       new keys and values into a dense or paged cache (BF16, FP32 or E4M3
              with a scale per KV head), optionally with the norms and the rotation
  read        tokens of a cache back as BF16 or FP32 vectors
  bounds      per-page channel minima and maxima of the cached keys
  select      the pages each KV head's query group should attend to, by those bounds
  attend      decode attention over the selected pages

A case is a dict of plain values; ``op`` names the call.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
ES = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a batch of 16 rows: 32/8 heads, one token a row (latency)
        dict(name="rope-step", op="norm_rope", tokens=16, hq=32, hkv=8, d=128, dt="bf16", rot=128, norm=1, inter=0, pad=0, maxpos=65536),
        # FP32 vectors of an odd number of tokens, half the channels rotated in adjacent pairs, no norm, some padding tokens
        dict(name="rope-f32-partial", op="norm_rope", tokens=5003, hq=12, hkv=4, d=64, dt="f32", rot=32, norm=0, inter=1, pad=1, maxpos=1048576),
        # a decode step of 64 rows straight into an E4M3 cache of 16-token pages, norms and rotation in the same call
        dict(name="write-step-fp8", op="write", tokens=64, rows=64, hq=32, hkv=8, d=128, dt="bf16", kv="e4m3", page=16, layout="NHD",
             rope=1, pad=0, maxpos=8192),
        # a 32768-token batch of prompts into a BF16 cache of 64-token pages (head-major pool), norms and rotation in the same call
        dict(name="write-prompt-bf16", op="write", tokens=32768, rows=5, hq=32, hkv=8, d=128, dt="bf16", kv="bf16", page=64, layout="HND",
             rope=1, pad=0, maxpos=0),
        # a shared prefix of 65536 tokens read back from an E4M3 cache as BF16
        dict(name="read-prefix-fp8", op="read", tokens=65536, rows=3, hkv=8, d=128, dt="bf16", kv="e4m3", page=16, layout="NHD", pad=0, maxpos=0),
        # a few single tokens of a dense FP32 cache
        dict(name="read-few-f32", op="read", tokens=37, rows=37, hkv=2, d=64, dt="f32", kv="f32", page=0, layout="HND", pad=1, maxpos=4096),
        # key bounds of the whole 131072-token cache of one 8-head layer, after its prompt
        dict(name="bounds-prompt", op="bounds", rows=1, hkv=8, d=128, kv="bf16", page=64, layout="NHD", lo=131072, hi=131072, new=0),
        # key bounds after one decode step of 16 ragged rows: the last page of each
        dict(name="bounds-step-fp8", op="bounds", rows=16, hkv=8, d=128, kv="e4m3", page=64, layout="NHD", lo=512, hi=4096, new=1),
        # 64 of the 2048 pages of a 131072-token row, 32/8 heads (latency)
        dict(name="select-8b", op="select", rows=1, hq=32, hkv=8, d=128, q="bf16", kv="bf16", page=64, lo=131072, hi=131072, nsel=64, first=1, last=2),
        # 256 of the 4096 pages of each of four 262144-token rows, 64/8 heads
        dict(name="select-70b", op="select", rows=4, hq=64, hkv=8, d=128, q="bf16", kv="bf16", page=64, lo=262144, hi=262144, nsel=256, first=1, last=2),
        # a decode step over 64 pages of a 131072-token E4M3 cache, 32/8 heads (latency)
        dict(name="attend-8b-fp8", op="attend", rows=1, hq=32, hkv=8, d=128, q="bf16", kv="e4m3", page=64, layout="NHD", lo=131071, hi=131071,
             nsel=64, fill=1.0, order="up"),
        # a decode step over 256 pages of each of four 262144-token rows, 64/8 heads: 268 MB of keys and values
        dict(name="attend-70b-bf16", op="attend", rows=4, hq=64, hkv=8, d=128, q="bf16", kv="bf16", page=64, layout="HND", lo=262100, hi=262144,
             nsel=256, fill=1.0, order="up"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    return hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), hkv


def draw(rng):
    op = rng.choice(["norm_rope", "write", "read", "bounds", "select", "attend"])
    hq, hkv = _heads(rng)
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["NHD", "HND"])
    if op == "norm_rope":
        rot = rng.choice([0, 16, 32, 48, 64]) if d == 64 else rng.choice([0, 16, 64, 96, 128])
        dt = rng.choice(["bf16", "f32"])
        return dict(op=op, tokens=_log(rng, 1, min(16384, (1 << 28) // ((hq + hkv) * d * ES[dt]))), hq=hq, hkv=hkv, d=d, dt=dt, rot=rot,
                    norm=1 if rot == 0 else rng.choice([0, 1]), inter=rng.choice([0, 1]), pad=rng.choice([0, 1]), maxpos=_log(rng, 64, 1 << 21))
    if op in ("write", "read"):
        kv = rng.choice(["bf16", "f32", "e4m3"])
        rows, tokens = rng.randint(1, 24), _log(rng, 1, min(16384, (1 << 28) // ((hq + 2 * hkv) * d * 4)))
        c = dict(op=op, tokens=tokens, rows=min(rows, tokens), hkv=hkv, d=d, dt="f32" if kv == "f32" else rng.choice(["bf16", "f32"]), kv=kv,
                 page=rng.choice([0, page]), layout=layout, pad=rng.choice([0, 1]), maxpos=rng.choice([0, 0, _log(rng, 1, 2048)]))
        if op == "write":
            c.update(hq=hq, rope=rng.choice([0, 1]))
        return c
    # keys of one pool: at most 2^27 elements
    most = max(256, min(262144, (1 << 27) // (hkv * d)))
    rows = _log(rng, 1, 16)
    hi = _log(rng, 1, max(1, most // rows))
    lo = rng.choice([0, 1, hi // 2, hi])
    c = dict(op=op, rows=rows, hkv=hkv, d=d, page=page, lo=min(lo, hi), hi=hi)
    kv = rng.choice(["bf16", "bf16", "f32", "e4m3"])
    if op == "bounds":
        c.update(kv=kv, layout=layout, new=rng.choice([0, 0, 1, _log(rng, 1, hi)]))
        return c
    if kv == "e4m3":
        c.update(d=128)
    if kv == "f32":
        hq = hkv * rng.choice([1, 2, 4, 8])
    pages = -(-hi // page)
    nsel = _log(rng, 4, max(4, min(1024, pages + 3)))
    c.update(hq=hq, q="f32" if kv == "f32" else "bf16", kv=kv, nsel=nsel)
    if op == "select":
        c.update(first=rng.choice([0, 1, 2]), last=rng.choice([0, 1, 2]))
    else:
        c.update(layout=layout, fill=rng.choice([1.0, 0.5, 0.0]), order=rng.choice(["up", "mixed"]))
    return c


# --------------------------------------------------------------- their inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dt=torch.float32, mul=1.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dt == torch.float8_e4m3fn else dt)
    return (x * mul).to(dt) if mul != 1.0 else x.to(dt)


def _pool(g, case, pages, page):
    """One cache pool viewed as [pages, page, Hkv, d]; E4M3: codes of values of a few scales' size."""
    hkv, d, kv = case["hkv"], case["d"], DT[case["kv"]]
    mul = 60.0 if case["kv"] == "e4m3" else 1.0
    if case.get("layout", "NHD") == "NHD":
        return _randn(g, pages, page, hkv, d, dt=kv, mul=mul)
    return _randn(g, pages, hkv, page, d, dt=kv, mul=mul).permute(0, 2, 1, 3)


def _scales(g, hkv):
    return (torch.rand(hkv, generator=g, device="cuda") * 0.02 + 0.005).float()


def _lengths(g, case):
    lo, hi = int(case["lo"]), int(case["hi"])
    n = torch.randint(lo, hi + 1, (case["rows"],), generator=g, device="cuda").to(torch.int32)
    if lo == 0:
        n[0] = 0
    return n


def _table(g, rows, per_row, pages):
    """Block table [rows, per_row] of distinct physical pages in random order."""
    return torch.randperm(pages, generator=g, device="cuda")[: rows * per_row].to(torch.int32).view(rows, per_row)


def _inv_freq(rot, scaled):
    f = 500000.0 ** (-torch.arange(0, rot // 2, device="cuda", dtype=torch.float64) / max(1, rot // 2))
    return (f / 8 if scaled else f).float()


def _token_lists(g, case):
    """rows, positions int32 [tokens]: with maxpos, one random position per token in a row of its own turn
    (all distinct); without, the tokens of `rows` prompts of unequal lengths, packed."""
    T, R = case["tokens"], case["rows"]
    if case["maxpos"]:
        per = -(-T // R)
        cap = max(case["maxpos"], per)
        rows = torch.arange(T, device="cuda", dtype=torch.int32) % R
        turn = torch.arange(T, device="cuda", dtype=torch.int64) // R
        off = torch.randint(0, cap // per, (T,), generator=g, device="cuda")
        pos = (turn * (cap // per) + off).to(torch.int32)
    else:
        cut = [T * r * (r + 1) // (R * (R + 1)) for r in range(R + 1)]   # row r holds a share of r + 1 parts
        start = torch.tensor(cut, device="cuda")
        t = torch.arange(T, device="cuda")
        rows = (torch.searchsorted(start, t, right=True) - 1).to(torch.int32)
        pos = (t - start[rows.long()]).to(torch.int32)
        cap = max(b - a for a, b in zip(cut, cut[1:]))
    if case["pad"]:
        pos[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    return rows, pos, cap


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case=dict(c))
    op, d = c["op"], c["d"]
    if op == "norm_rope":
        T, hq, hkv, dt = c["tokens"], c["hq"], c["hkv"], DT[c["dt"]]
        qkv = _randn(g, T, hq + 2 * hkv, d, dt=dt, mul=1.5)      # the packed projection's output
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], q_out=torch.zeros(T, hq, d, device="cuda", dtype=dt),
                 k_out=torch.zeros(T, hkv, d, device="cuda", dtype=dt))
        pos = torch.randint(0, c["maxpos"], (T,), generator=g, device="cuda").to(torch.int32)
        if c["pad"]:
            pos[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
        s.update(pos=pos, freq=_inv_freq(c["rot"], seed & 1) if c["rot"] else None)
        if c["norm"]:
            s.update(qw=(1 + 0.2 * _randn(g, d)).to(dt), kw=(1 + 0.2 * _randn(g, d)).to(dt))
        return s
    if op in ("write", "read"):
        T, R, hkv, dt = c["tokens"], c["rows"], c["hkv"], DT[c["dt"]]
        rows, pos, cap = _token_lists(g, c)
        s.update(rows=rows, pos=pos, keep=torch.nonzero(pos >= 0).squeeze(1), table=None)
        if c["page"]:
            per = -(-cap // c["page"])
            pages = R * per + 2
            s.update(table=_table(g, R, per, pages), kc=_pool(g, c, pages, c["page"]), vc=_pool(g, c, pages, c["page"]))
        else:                                                     # dense [rows, Hkv, cap, d]
            s.update(kc=_pool(g, c, R, cap).permute(0, 2, 1, 3), vc=_pool(g, c, R, cap).permute(0, 2, 1, 3))
        if c["kv"] == "e4m3":
            s.update(ks=_scales(g, hkv), vs=_scales(g, hkv))
        if op == "write":
            hq = c["hq"]
            qkv = _randn(g, T, hq + 2 * hkv, d, dt=dt, mul=1.5)
            s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], q_out=torch.zeros(T, hq, d, device="cuda", dtype=dt))
            if c["rope"]:
                s.update(freq=_inv_freq(d, seed & 1), qw=(1 + 0.2 * _randn(g, d)).to(dt), kw=(1 + 0.2 * _randn(g, d)).to(dt))
        else:
            s.update(k_out=torch.zeros(T, hkv, d, device="cuda", dtype=dt), v_out=torch.zeros(T, hkv, d, device="cuda", dtype=dt))
        return s
    R, hkv, ps = c["rows"], c["hkv"], c["page"]
    per = max(1, -(-c["hi"] // ps))
    pages = R * per + 2
    s.update(len=_lengths(g, c), table=_table(g, R, per, pages))
    if op == "bounds":
        bt = torch.float32 if c["kv"] == "f32" else torch.bfloat16
        s.update(kc=_pool(g, c, pages, ps), bounds=_randn(g, pages, hkv, 2, d, dt=bt))
    elif op == "select":
        bt = torch.float32 if c["kv"] == "f32" else torch.bfloat16
        # pages of keys around a centre of their own, a few standard deviations wide
        mid = _randn(g, pages, hkv, 1, d, mul=0.6)
        b = torch.cat([mid - 1 - 0.4 * _randn(g, pages, hkv, 1, d).abs(), mid + 1 + 0.4 * _randn(g, pages, hkv, 1, d).abs()], 2)
        s.update(bounds=b.to(bt), q=_randn(g, R, c["hq"], d, dt=DT[c["q"]]),
                 sel=torch.empty(R, hkv, c["nsel"], device="cuda", dtype=torch.int32))
    else:
        s.update(kc=_pool(g, c, pages, ps), vc=_pool(g, c, pages, ps), q=_randn(g, R, c["hq"], d, dt=DT[c["q"]]),
                 out=torch.empty(R, c["hq"], d, device="cuda"), lse=torch.empty(R, c["hq"], device="cuda"))
        if c["kv"] == "e4m3":
            s.update(ks=_scales(g, hkv), vs=_scales(g, hkv))
        # a selection of each row's pages, `fill` of the list used, ascending or in any order, -1 elsewhere
        n = -(-s["len"].long() // ps)
        score = torch.rand(R, hkv, per, generator=g, device="cuda")
        score = torch.where(torch.arange(per, device="cuda") < n[:, None, None], score, -1.0)
        top, idx = torch.sort(score, dim=2, descending=True)
        idx = torch.where(top >= 0, idx, per)[:, :, : c["nsel"]]
        if idx.shape[2] < c["nsel"]:
            idx = torch.nn.functional.pad(idx, (0, c["nsel"] - idx.shape[2]), value=per)
        used = max(0, int(c["nsel"] * c["fill"]))
        idx[:, :, used:] = per
        if c["order"] == "up":
            idx = torch.sort(idx, dim=2)[0]
        s.update(sel=torch.where(idx >= per, -1, idx).to(torch.int32).contiguous())
    return s


# ------------------------------------------------------------ the plain forms
def _codes(x, scale):
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _bytes_of(x):
    """One-byte types through indexing as bytes."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _norm_rope_plain(x, pos, freq, w, norm, inter):
    y = x.float()
    if norm:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        if w is not None:
            y = y * w.float()
    if freq is None:
        return y
    a = pos.double()[:, None, None] * freq.double()
    cos, sin = a.cos().float(), a.sin().float()
    half = freq.numel()
    r, rest = y[..., : 2 * half], y[..., 2 * half:]
    if inter:
        y1, y2 = r[..., 0::2], r[..., 1::2]
        r = torch.stack([y1 * cos - y2 * sin, y2 * cos + y1 * sin], -1).flatten(-2)
    else:
        y1, y2 = r[..., :half], r[..., half:]
        r = torch.cat([y1 * cos - y2 * sin, y2 * cos + y1 * sin], -1)
    return torch.cat([r, rest], -1)


def _place(s, rows, pos):
    """Index tuple of (row, position) in the cache's [page, slot] or [row, position] axes."""
    rows, pos = rows.long(), pos.long()
    ps = s["case"]["page"]
    if ps:
        return s["table"][rows, pos // ps].long(), pos % ps
    return rows, pos


def _cache_view(s, name):
    """[page or row, slot, Hkv, d] view of a cache."""
    x = s[name]
    return _bytes_of(x if s["case"]["page"] else x.permute(0, 2, 1, 3))


def _run_norm_rope(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        return ta.tree_attn_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s.get("qw"), k_weight=s.get("kw"), norm=bool(c["norm"]),
                                      eps=EPS, interleaved=bool(c["inter"]), q_out=s["q_out"], k_out=s["k_out"])
    live = (s["pos"] >= 0)[:, None, None]
    for x, w, o in (("q", "qw", "q_out"), ("k", "kw", "k_out")):
        y = _norm_rope_plain(s[x], s["pos"], s["freq"], s.get(w), c["norm"], c["inter"])
        s[o].copy_(torch.where(live, y.to(s[o].dtype), s[o]))
    return s["q_out"], s["k_out"]


def _run_write(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        rope = dict(q=s["q"], q_out=s["q_out"], inv_freq=s["freq"], q_weight=s["qw"], k_weight=s["kw"], norm=True, eps=EPS) if c["rope"] else {}
        ta.tree_attn_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["pos"], rows=s["rows"], block_table=s["table"], k_scale=s.get("ks"),
                                 v_scale=s.get("vs"), **rope)
        return s["q_out"], s["kc"], s["vc"]
    k, v = s["k"].float(), s["v"].float()
    if c["rope"]:
        k = _norm_rope_plain(s["k"], s["pos"], s["freq"], s["kw"], 1, 0)
        q = _norm_rope_plain(s["q"], s["pos"], s["freq"], s["qw"], 1, 0)
        s["q_out"].copy_(torch.where((s["pos"] >= 0)[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    keep = s["keep"]
    at = _place(s, s["rows"][keep], s["pos"][keep])
    for x, name, sc in ((k, "kc", "ks"), (v, "vc", "vs")):
        y = _codes(x, s[sc]) if c["kv"] == "e4m3" else x.to(DT[c["kv"]])
        _cache_view(s, name)[at] = _bytes_of(y)[keep]
    return s["q_out"], s["kc"], s["vc"]


def _run_read(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        return ta.tree_attn_cache_read(s["kc"], s["vc"], s["pos"], rows=s["rows"], block_table=s["table"], k_scale=s.get("ks"), v_scale=s.get("vs"),
                                       k_out=s["k_out"], v_out=s["v_out"])
    keep = s["keep"]
    at = _place(s, s["rows"][keep], s["pos"][keep])
    for name, o, sc in (("kc", "k_out", "ks"), ("vc", "v_out", "vs")):
        y = _cache_view(s, name)[at]
        if c["kv"] == "e4m3":
            y = y.view(torch.float8_e4m3fn).float() * s[sc][:, None]
        s[o][keep] = y.to(s[o].dtype)
    return s["k_out"], s["v_out"]


def _run_bounds(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        return ta.tree_attn_page_bounds(s["kc"], s["table"], s["len"], s["bounds"], new_tokens=c["new"], max_seqlen=max(1, c["hi"]))
    ps, n, b = c["page"], s["len"].long(), s["bounds"]
    per = s["table"].shape[1]
    count = min(per, -(-c["new"] // ps) + 1) if c["new"] else per
    first = (n - c["new"]).clamp(min=0) // ps if c["new"] else torch.zeros_like(n)
    page = first[:, None] + torch.arange(count, device=n.device)                    # logical pages [R, count]
    live = page * ps < n[:, None]
    phys = torch.where(live, s["table"].long().gather(1, page.clamp(max=per - 1)), b.shape[0])
    k = s["kc"][:, :, :, :] if c["kv"] != "e4m3" else s["kc"].view(torch.uint8)
    k = k[phys.clamp(max=b.shape[0] - 1)]                                            # [R, count, ps, Hkv, d]
    k = (k.view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else k).float()
    tok = page[:, :, None] * ps + torch.arange(ps, device=n.device)
    valid = (tok < n[:, None, None])[..., None, None]
    lo = torch.where(valid, k, math.inf).amin(2)
    hi = torch.where(valid, k, -math.inf).amax(2)
    wide = torch.cat([b, b[:1]])                                                     # one more page takes what is not live
    wide[phys] = torch.stack([lo, hi], 3).to(b.dtype)
    b.copy_(wide[:-1])
    return b


def _chosen(score, n, nsel, first, last):
    """Ascending list [R, Hkv, nsel] of the chosen pages (-1 behind them) from scores [R, Hkv, pages]."""
    pages = score.shape[2]
    at = torch.arange(pages, device=score.device).expand_as(score)
    n = n[:, None, None]
    score = torch.where(torch.isfinite(score), score, math.inf)
    order = torch.sort(torch.where(at < n, score, -math.inf), dim=2, descending=True, stable=True)[1]
    must = ((at < first) | (at >= n - last)) & (at < n)
    cls = torch.where(must, 2, torch.where(at < n, 1, 0)).gather(2, order)
    order = order.gather(2, torch.sort(cls, dim=2, descending=True, stable=True)[1])
    keep = order[:, :, :nsel]
    keep = torch.sort(torch.where(keep < n, keep, pages), dim=2)[0]
    keep = torch.where(keep < pages, keep, -1)
    return torch.nn.functional.pad(keep, (0, nsel - keep.shape[2]), value=-1).to(torch.int32)


def _run_select(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        return ta.tree_attn_select_pages(s["q"], s["bounds"], s["table"], s["len"], c["page"], c["nsel"], first_pages=c["first"],
                                         last_pages=c["last"], selected=s["sel"])
    R, hq, d = s["q"].shape
    hkv = c["hkv"]
    q = s["q"].double().view(R, hkv, hq // hkv, d)          # 64 bits: pages next to the last place differ by little
    up, dn = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)    # [R, Hkv, d]
    b = s["bounds"][s["table"].long()].double()              # [R, pages, Hkv, 2, d]
    score = (b[:, :, :, 1] * up[:, None]).sum(-1) + (b[:, :, :, 0] * dn[:, None]).sum(-1)
    s["sel"].copy_(_chosen(score.permute(0, 2, 1), -(-s["len"].long() // c["page"]), c["nsel"], c["first"], c["last"]))
    return s["sel"]


def _listed_tokens(s, name, scale):
    """The listed pages' vectors [R, Hkv, nsel * page, d] and which of them count."""
    c, sel = s["case"], s["sel"].long()
    ps = c["page"]
    R, hkv, nsel = sel.shape
    phys = s["table"].long().gather(1, sel.clamp(min=0).view(R, -1)).view(R, hkv, nsel)
    x = _bytes_of(s[name])[phys[..., None], torch.arange(ps, device=sel.device), torch.arange(hkv, device=sel.device)[:, None, None]]
    x = x.view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else x
    tok = sel[..., None] * ps + torch.arange(ps, device=sel.device)
    valid = (sel[..., None] >= 0) & (tok < s["len"].long()[:, None, None, None])
    return x.flatten(2, 3), valid.flatten(2, 3), None if scale is None else s[scale][None, :, None, None]


def _run_attend(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        return ta.tree_attn_decode_selected(s["q"], s["kc"], s["vc"], s["table"], s["len"], s["sel"], out=s["out"], lse=s["lse"],
                                            max_seqlen=max(1, c["hi"]), k_scale=s.get("ks"), v_scale=s.get("vs"))
    R, hq, d = s["q"].shape
    hkv = c["hkv"]
    fp8 = c["kv"] == "e4m3"
    k, valid, ks = _listed_tokens(s, "kc", "ks" if fp8 else None)
    v, _, vs = _listed_tokens(s, "vc", "vs" if fp8 else None)
    k, v = k.float(), v.float()
    if fp8:
        k, v = k * ks, v * vs
    q = s["q"].float().view(R, hkv, hq // hkv, d)
    z = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    z = torch.where(valid[:, :, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(valid[..., None], v, 0.0)) / torch.where(l > 0, l, 1.0)
    s["out"].copy_(o.reshape(R, hq, d))
    s["lse"].copy_((m + torch.log(l)).reshape(R, hq))
    return s["out"], s["lse"]


_RUN = dict(norm_rope=_run_norm_rope, write=_run_write, read=_run_read, bounds=_run_bounds, select=_run_select, attend=_run_attend)


def run(state):
    return _RUN[state["case"]["op"]](state)


# ------------------------------------------------------------------ their work
def work(case):
    c = case
    op, d = c["op"], c["d"]
    if op == "norm_rope":
        v = c["tokens"] * (c["hq"] + c["hkv"]) * d
        return {"bytes": 2 * v * ES[c["dt"]] + 4 * c["tokens"], "flops": v * (3 * c["norm"] + 3 * c["rot"] / d)}
    if op == "write":
        q, kv = c["tokens"] * c["hq"] * d * c["rope"], 2 * c["tokens"] * c["hkv"] * d
        return {"bytes": (2 * q + kv) * ES[c["dt"]] + kv * ES[c["kv"]] + 8 * c["tokens"], "flops": (q + kv / 2) * 6 * c["rope"] + kv}
    if op == "read":
        kv = 2 * c["tokens"] * c["hkv"] * d
        return {"bytes": kv * (ES[c["kv"]] + ES[c["dt"]]) + 8 * c["tokens"], "flops": kv}
    mean = (c["lo"] + c["hi"]) / 2
    ps, hkv, R = c["page"], c["hkv"], c["rows"]
    if op == "bounds":
        tokens = mean if not c["new"] else min(mean, c["new"] + ps / 2)
        pages = max(1, math.ceil(tokens / ps))
        es = 4 if c["kv"] == "f32" else 2
        return {"bytes": R * hkv * d * (tokens * ES[c["kv"]] + pages * 2 * es), "flops": 2 * R * hkv * d * tokens}
    pages = max(1, math.ceil(mean / ps))
    if op == "select":
        es = 4 if c["kv"] == "f32" else 2
        return {"bytes": R * (hkv * pages * 2 * d * es + c["hq"] * d * ES[c["q"]] + 4 * pages + 4 * hkv * c["nsel"]), "flops": 4 * R * hkv * pages * d}
    tokens = min(mean, max(1, int(c["nsel"] * c["fill"])) * ps)
    return {"bytes": R * (2 * hkv * tokens * d * ES[c["kv"]] + c["hq"] * (d * ES[c["q"]] + 4 * d + 4) + 4 * hkv * c["nsel"]),
            "flops": 4 * R * c["hq"] * tokens * d}


# ------------------------------------------- the same from the definitions, in 64 bits
def _norm_rope_exact(x, pos, freq, w, norm, inter):
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS)
        if w is not None:
            y = y * w.double()
    if freq is None:
        return y
    n = freq.numel()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), pos.double()[:, None] * freq.double()[None])[:, None]
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + n)
    z = torch.complex(y[..., a], y[..., b]) * turn
    out = y.clone()
    out[..., a], out[..., b] = z.real, z.imag
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "norm_rope":
        res = []
        for x, w, o in (("q", "qw", "q_out"), ("k", "kw", "k_out")):
            y = _norm_rope_exact(s[x], s["pos"], s["freq"], s.get(w), c["norm"], c["inter"])
            y[s["pos"] < 0] = s[o].double()[s["pos"] < 0]
            res.append(y)
        return tuple(res)
    if op in ("write", "read"):
        live = torch.nonzero(s["pos"] >= 0).squeeze(1)
        rows, pos = s["rows"][live].long(), s["pos"][live].long()
        caches = []
        for name in ("kc", "vc"):                                   # the cache in its own layout, in 64 bits
            caches.append(s[name].double())
        if c["page"]:
            spot = (s["table"].long()[rows, torch.div(pos, c["page"], rounding_mode="floor")], torch.remainder(pos, c["page"]))
            seen = caches
        else:
            spot, seen = (rows, pos), [x.transpose(1, 2) for x in caches]
        if op == "read":
            res = []
            for x, o, sc in ((seen[0], "k_out", "ks"), (seen[1], "v_out", "vs")):
                y = s[o].double()
                got = x[spot]
                y[live] = got * s[sc].double().view(1, -1, 1) if sc in s else got
                res.append(y)
            return tuple(res)
        q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        if c["rope"]:
            k = _norm_rope_exact(s["k"], s["pos"], s["freq"], s["kw"], 1, 0)
            q[live] = _norm_rope_exact(s["q"], s["pos"], s["freq"], s["qw"], 1, 0)[live]
        for x, y, sc in ((seen[0], k, "ks"), (seen[1], v, "vs")):
            if sc in s:
                y = (y / s[sc].double().view(1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX)
            x[spot] = y[live]
        return q, caches[0], caches[1]
    if op == "bounds":
        b = s["bounds"].double()
        ps, n = c["page"], s["len"].tolist()
        for r in range(c["rows"]):
            if n[r] <= 0:
                continue
            low = max(0, n[r] - c["new"]) // ps if c["new"] else 0
            full = n[r] // ps
            for part, count in ((s["table"][r, low:full].long(), ps), (s["table"][r, max(low, full):-(-n[r] // ps)].long(), n[r] % ps)):
                if part.numel() and count:
                    k = s["kc"].view(torch.uint8)[part].view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else s["kc"][part]
                    k = k[:, :count].double()
                    b[part] = torch.stack([-((-k).max(1)[0]), k.max(1)[0]], 2)
        return b
    if op == "select":
        R, hq, d = s["q"].shape
        q = s["q"].double().view(R, c["hkv"], -1, 1, d)
        res = torch.full_like(s["sel"], -1)
        n = (-(-s["len"].long() // c["page"])).tolist()
        for r in range(R):
            if n[r] <= c["nsel"]:
                res[r, :, : n[r]] = torch.arange(n[r], device="cuda", dtype=torch.int32)
                continue
            b = s["bounds"][s["table"][r, : n[r]].long()].double().permute(1, 2, 0, 3)          # [Hkv, 2, pages, d]
            score = torch.maximum(q[r] * b[:, None, 0], q[r] * b[:, None, 1]).sum((1, 3))       # [Hkv, pages]
            for h in range(c["hkv"]):
                mid = list(range(c["first"], n[r] - c["last"]))
                val = score[h].tolist()
                mid.sort(key=lambda p: (-val[p], p))
                take = list(range(c["first"])) + mid[: c["nsel"] - c["first"] - c["last"]] + list(range(n[r] - c["last"], n[r]))
                res[r, h] = torch.tensor(sorted(take), dtype=torch.int32, device="cuda")
        return res
    out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.full_like(s["lse"], -math.inf, dtype=torch.float64)
    G = c["hq"] // c["hkv"]
    k, valid, ks = _listed_tokens(s, "kc", "ks" if c["kv"] == "e4m3" else None)
    v, _, vs = _listed_tokens(s, "vc", "vs" if c["kv"] == "e4m3" else None)
    for r in range(c["rows"]):
        for h in range(c["hkv"]):
            at = torch.nonzero(valid[r, h]).squeeze(1)
            if not at.numel():
                continue
            kk = (k[r, h].view(torch.uint8)[at].view(torch.float8_e4m3fn) if ks is not None else k[r, h][at]).double()
            vv = (v[r, h].view(torch.uint8)[at].view(torch.float8_e4m3fn) if vs is not None else v[r, h][at]).double()
            if ks is not None:
                kk, vv = kk * s["ks"][h].double(), vv * s["vs"][h].double()
            z = (s["q"][r, h * G:(h + 1) * G].double() @ kk.T) * (c["d"] ** -0.5)
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
            out[r, h * G:(h + 1) * G] = torch.softmax(z, 1) @ vv
    return out, lse
