"""Measured cases of the library's 4-bit caches and of its attention to a window of the cache.

Four calls, each in a plain form (elementary torch operations) and as the
library's own entry point:

  append  new keys and values into a 4-bit cache, optionally with the norms and the rotation
          in the same call, and the rounded vectors taken back (what a prompt's own attention
          uses, so that it sees the keys and values that later steps see)
  read    tokens of a 4-bit cache back as BF16 or FP32 vectors
  int4    decode attention over a 4-bit cache, one or several queries a row, with or without
          a window
  window  decode attention to the first tokens of a row (sinks) and its last ones (window),
          over BF16, FP32 and E4M3 caches

A 4-bit cache holds, for each token and KV head, head_dim codes of 4 bits (two channels a
byte, the even one in the low half) and an E4M3 step for each 16 channels; a channel's value
is scale * step * (code - 8), with one FP32 scale a KV head (1 where none is given).

A case is a dict of plain values; ``op`` names the call.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
ES = {"bf16": 2, "f32": 4, "e4m3": 1}
FP8 = torch.float8_e4m3fn
E4M3_MAX, E4M3_MIN = 448.0, 2.0 ** -9
EPS = 1e-6
GROUP = 16           # channels of one step


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 rows into pages of 16 tokens: norms, rotation, 4-bit rounding (latency)
        dict(name="append-step", op="append", tokens=64, rows=64, hq=32, hkv=8, d=128, dt="bf16", page=16, layout="NHD", rope=1, scaled=1,
             pad=0, maxpos=8192),
        # a 16384-token batch of prompts into pages of 64 tokens (head-major pool), norms and rotation in the same call
        dict(name="append-prompt", op="append", tokens=16384, rows=5, hq=32, hkv=8, d=128, dt="bf16", page=64, layout="HND", rope=1, scaled=0,
             pad=0, maxpos=0),
        # FP32 vectors of an odd number of tokens and heads into a dense cache, some padding tokens, nothing rotated
        dict(name="append-f32-odd", op="append", tokens=1237, rows=7, hq=3, hkv=3, d=64, dt="f32", page=0, layout="NHD", rope=0, scaled=1,
             pad=1, maxpos=0),
        # a shared prefix of 65536 tokens read back as BF16
        dict(name="read-prefix", op="read", tokens=65536, rows=3, hkv=8, d=128, dt="bf16", page=64, layout="HND", scaled=1, pad=0, maxpos=0),
        # a few single tokens of a dense cache as FP32
        dict(name="read-few-f32", op="read", tokens=37, rows=37, hkv=2, d=64, dt="f32", page=0, layout="HND", scaled=0, pad=1, maxpos=4096),
        # a decode step over a whole 131072-token row, 32/8 heads: 151 MB of codes and steps
        dict(name="int4-8b-131k", op="int4", rows=1, hq=32, hkv=8, d=128, page=64, layout="HND", lo=131072, hi=131072, nq=1, window=0, sinks=0,
             scaled=1),
        # 16 rows of very different lengths, 64/8 heads, token-major pages of 16: a serving batch
        dict(name="int4-batch-ragged", op="int4", rows=16, hq=64, hkv=8, d=128, page=16, layout="NHD", lo=4096, hi=32768, nq=1, window=0, sinks=0,
             scaled=0),
        # four rows at the start of their answers (latency)
        dict(name="int4-short", op="int4", rows=4, hq=32, hkv=8, d=128, page=16, layout="NHD", lo=37, hi=700, nq=1, window=0, sinks=0, scaled=1),
        # four draft tokens a row checked at once, a window of 4096 tokens behind 4 sinks
        dict(name="int4-drafts-window", op="int4", rows=8, hq=32, hkv=8, d=128, page=64, layout="HND", lo=20000, hi=65536, nq=4, window=4096,
             sinks=4, scaled=1),
        # a decode step of 16 rows with a window of 4096 tokens behind 4 sinks, far into their answers: 269 MB
        dict(name="window-8b-bf16", op="window", rows=16, hq=32, hkv=8, d=128, q="bf16", kv="bf16", page=64, layout="HND", lo=60000, hi=131072,
             nq=1, window=4096, sinks=4),
        # one row of an E4M3 cache, a window of 1024 tokens behind 4 sinks (latency)
        dict(name="window-1k-fp8", op="window", rows=1, hq=32, hkv=8, d=128, q="bf16", kv="e4m3", page=16, layout="NHD", lo=8191, hi=8191,
             nq=1, window=1024, sinks=4),
        # drafts over a dense cache of 64 channels, odd sizes everywhere, some rows shorter than the window
        dict(name="window-odd-drafts", op="window", rows=11, hq=9, hkv=3, d=64, q="bf16", kv="bf16", page=0, layout="NHD", lo=0, hi=2500,
             nq=5, window=1001, sinks=17),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "int4", "window"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    d = rng.choice([64, 128])
    page = rng.choice([0, 16, 32, 64, 128])
    layout = rng.choice(["NHD", "HND"])
    if op in ("append", "read"):
        dt = rng.choice(["bf16", "f32"])
        rows, tokens = rng.randint(1, 24), _log(rng, 1, min(16384, (1 << 27) // ((hkv * G + 2 * hkv) * d * ES[dt])))
        c = dict(op=op, tokens=tokens, rows=min(rows, tokens), hkv=hkv, d=d, dt=dt, page=page, layout=layout, scaled=rng.choice([0, 1]),
                 pad=rng.choice([0, 1]) if tokens > 4 else 0, maxpos=rng.choice([0, 0, _log(rng, 1, 2048)]))
        if op == "append":   # (a rotated FP32 vector that lies next to the middle of two codes has no one rounding: BF16 results only)
            c.update(hq=hkv * G, rope=rng.choice([0, 1]) if dt == "bf16" else 0)
        return c
    rows = _log(rng, 1, 24)
    nq = rng.choice([1, 1, 1, 2, 3, 4, 7])
    hi = _log(rng, 1, max(1, min(131072, (1 << 27) // (hkv * d * rows))))
    c = dict(op=op, rows=rows, hkv=hkv, d=d, page=page, layout=layout, lo=min(hi, max(int(rows == 1), rng.choice([0, 1, hi // 2, hi]))), hi=hi, nq=nq,
             sinks=rng.choice([0, 0, 1, 4, rng.randint(1, 80)]))
    if op == "int4":
        c.update(hq=hkv * G, scaled=rng.choice([0, 1]), window=rng.choice([0, 0, _log(rng, 1, hi)]))
        return c
    kv = rng.choice(["bf16", "bf16", "e4m3", "f32"])
    if kv == "e4m3":
        c.update(d=128)
    if kv != "bf16":
        G = rng.choice([1, 2, 4, 8])
    c.update(hq=hkv * G, q="f32" if kv == "f32" else "bf16", kv=kv, window=_log(rng, 1, max(1, min(hi, 8192))))
    return c


# --------------------------------------------------------------- their inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dt=torch.float32, mul=1.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if dt == FP8 else dt)
    return (x * mul).to(dt) if mul != 1.0 else x.to(dt)


def _laid(case, make, rows, tokens, last):
    """A cache's memory made by make(shape), viewed as [rows or pages, tokens, Hkv, last]."""
    if case["layout"] == "NHD":
        return make((rows, tokens, case["hkv"], last))
    return make((rows, case["hkv"], tokens, last)).permute(0, 2, 1, 3)


def _int4_cache(g, case, rows, tokens):
    """Codes [.., d / 2] and steps [.., d / 16] of one cache: every code, steps between 0.05 and 0.35."""
    d = case["d"]
    codes = _laid(case, lambda s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8), rows, tokens, d // 2)
    steps = _laid(case, lambda s: (torch.rand(s, generator=g, device="cuda") * 0.3 + 0.05).to(FP8), rows, tokens, d // GROUP)
    return codes, steps


def _call_view(case, x):
    """The axes' order that the library takes: [pages, page, Hkv, ..] pools, [B, Hkv, S, ..] dense caches."""
    return x if case["page"] else x.permute(0, 2, 1, 3)


def _scales(g, hkv, lo=0.5, hi=1.5):
    return (torch.rand(hkv, generator=g, device="cuda") * (hi - lo) + lo).float()


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
        cap = max(1, max(b - a for a, b in zip(cut, cut[1:])))
    if case["pad"]:
        pos[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    return rows, pos, cap


def _first_seen(case, n):
    """The first token of the window of a row's first query (n: lengths)."""
    if not case["window"]:
        return torch.zeros_like(n)
    return (n - case["nq"] + 1 - case["window"]).clamp(min=0)


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case=dict(c))
    op, d, hkv, ps = c["op"], c["d"], c["hkv"], c["page"]
    if op in ("append", "read"):
        T, R, dt = c["tokens"], c["rows"], DT[c["dt"]]
        rows, pos, cap = _token_lists(g, c)
        per = -(-cap // ps) if ps else 0
        pages, room = (R * per + 2, ps) if ps else (R, cap)
        s.update(rows=rows, pos=pos, keep=torch.nonzero(pos >= 0).squeeze(1),
                 table=torch.randperm(pages, generator=g, device="cuda")[: R * per].to(torch.int32).view(R, per) if ps else None,
                 k_out=torch.zeros(T, hkv, d, device="cuda", dtype=dt), v_out=torch.zeros(T, hkv, d, device="cuda", dtype=dt))
        for x in ("k", "v"):
            s[x + "c"], s[x + "s"] = _int4_cache(g, c, pages, room)
            s[x + "g"] = _scales(g, hkv) if c["scaled"] else None
        if op == "append":
            hq = c["hq"]
            qkv = _randn(g, T, hq + 2 * hkv, d, dt=dt, mul=1.5)      # the packed projection's output
            s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], q_out=torch.zeros(T, hq, d, device="cuda", dtype=dt))
            if c["rope"]:
                f = 500000.0 ** (-torch.arange(0, d // 2, device="cuda", dtype=torch.float64) / (d // 2))
                s.update(freq=(f / 8 if seed & 1 else f).float(), qw=(1 + 0.2 * _randn(g, d)).to(dt), kw=(1 + 0.2 * _randn(g, d)).to(dt))
        return s
    R = c["rows"]
    lo, hi = int(c["lo"]), int(c["hi"])
    n = torch.randint(lo, hi + 1, (R,), generator=g, device="cuda")
    if lo == 0:
        n[0] = 0
    if ps:
        # a pool that holds the pages some query can see; the others' table entries are stale (-1)
        per = max(1, -(-hi // ps))
        seen = min(per, -(-c["sinks"] // ps) + -(-(c["window"] + c["nq"]) // ps) + 1) if c["window"] else per
        pages = R * seen + 2
        at = torch.arange(per, device="cuda")[None]
        need = (at * ps < n[:, None]) & ((at * ps < c["sinks"]) | ((at + 1) * ps > _first_seen(c, n)[:, None]))
        order = torch.randperm(pages, generator=g, device="cuda")
        place = (torch.cumsum(need.flatten().long(), 0) - 1).view(R, per).clamp(min=0)
        s.update(table=torch.where(need, order[place], -1).to(torch.int32))
    else:
        pages, ps = R, max(1, hi)
        s.update(table=None)
    s.update(len=n.to(torch.int32), out=torch.empty(R, c["hq"], c["nq"], d, device="cuda"), lse=torch.empty(R, c["hq"], c["nq"], device="cuda"))
    if op == "int4":
        s.update(q=_randn(g, R, c["hq"], c["nq"], d, dt=torch.bfloat16))
        for x in ("k", "v"):
            s[x + "c"], s[x + "s"] = _int4_cache(g, c, pages, ps)
            s[x + "g"] = _scales(g, hkv) if c["scaled"] else None
    else:
        s.update(q=_randn(g, R, c["hq"], c["nq"], d, dt=DT[c["q"]]))
        for x in ("k", "v"):
            s[x + "c"] = _laid(c, lambda sh: _randn(g, *sh, dt=DT[c["kv"]], mul=60.0 if c["kv"] == "e4m3" else 1.0), pages, ps, d)
            s[x + "g"] = _scales(g, hkv, 0.005, 0.025) if c["kv"] == "e4m3" else None
    return s


# ------------------------------------------------------------ the plain forms
def _norm_rope_plain(x, pos, freq, w):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    a = pos.double()[:, None, None] * freq.double()
    cos, sin = a.cos().float(), a.sin().float()
    y1, y2 = y.chunk(2, -1)
    return torch.cat([y1 * cos - y2 * sin, y2 * cos + y1 * sin], -1)


def _place(s, rows, pos):
    """Index tuple of (row, position) in the cache's [page, slot] or [row, position] axes."""
    rows, pos = rows.long(), pos.long()
    ps = s["case"]["page"]
    if ps:
        return s["table"][rows, pos // ps].long(), pos % ps
    return rows, pos


def _to_int4(y, scale):
    """Codes [.., d / 2] and steps [.., d / 16] of FP32 vectors [.., Hkv, d]: the step is the E4M3 number next to a seventh of the
    largest of its 16 channels, the codes the whole numbers next to the channel over the step."""
    if scale is not None:
        y = y / scale[:, None]
    y = y.unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1)
    step = (top / torch.full_like(top, 7)).clamp(E4M3_MIN, E4M3_MAX).to(FP8)      # (a division: by a number it would be a product)
    code = (torch.round(y / step.float()[..., None]).clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), step


def _from_int4(codes, steps, scale):
    """FP32 values [.., Hkv, d] of codes and steps."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    y = (code.unflatten(-1, (-1, GROUP)) * steps.float()[..., None]).flatten(-2)
    return y if scale is None else y * scale[:, None]


def _read_plain(s):
    keep = s["keep"]
    at = _place(s, s["rows"][keep], s["pos"][keep])
    for x in ("k", "v"):
        y = _from_int4(s[x + "c"][at], s[x + "s"].view(torch.uint8)[at].view(FP8), s[x + "g"])
        s[x + "_out"][keep] = y.to(s[x + "_out"].dtype)
    return s["k_out"], s["v_out"]


def _read_own(s):
    import softmax_tree_reduction_gb300 as ta
    c = s["case"]
    cache = [_call_view(c, s[x]) for x in ("kc", "vc", "ks", "vs")]
    return ta.tree_attn_cache_read_int4(*cache, s["pos"], rows=s["rows"], block_table=s["table"], k_scale=s["kg"], v_scale=s["vg"], k_out=s["k_out"],
                                        v_out=s["v_out"])


def _run_append(s):
    c = s["case"]
    if own:
        import softmax_tree_reduction_gb300 as ta
        cache = [_call_view(c, s[x]) for x in ("kc", "vc", "ks", "vs")]
        rope = dict(q=s["q"], q_out=s["q_out"], inv_freq=s["freq"], q_weight=s["qw"], k_weight=s["kw"], norm=True, eps=EPS) if c["rope"] else {}
        ta.tree_attn_cache_write_int4(s["k"], s["v"], *cache, s["pos"], rows=s["rows"], block_table=s["table"], k_scale=s["kg"], v_scale=s["vg"], **rope)
        return (*(s["q_out"],) * c["rope"], *_read_own(s))
    k, v = s["k"].float(), s["v"].float()
    if c["rope"]:
        k = _norm_rope_plain(s["k"], s["pos"], s["freq"], s["kw"])
        q = _norm_rope_plain(s["q"], s["pos"], s["freq"], s["qw"])
        s["q_out"].copy_(torch.where((s["pos"] >= 0)[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    keep = s["keep"]
    at = _place(s, s["rows"][keep], s["pos"][keep])
    for x, y in (("k", k), ("v", v)):
        codes, steps = _to_int4(y[keep], s[x + "g"])
        s[x + "c"][at] = codes
        s[x + "s"].view(torch.uint8)[at] = steps.view(torch.uint8)
    return (*(s["q_out"],) * c["rope"], *_read_plain(s))


def _run_read(s):
    return _read_own(s) if own else _read_plain(s)


def _seen_tokens(s):
    """Tokens that some query of a row may see, int64 [R, L] (sinks, then the rest), and which queries see them, bool [R, nq, L]."""
    c, n = s["case"], s["len"].long()
    nq, W, dev = c["nq"], c["window"], n.device
    if not W:
        tok = torch.arange(max(1, c["hi"]), device=dev)[None].expand(n.numel(), -1)
        last = n[:, None] - nq + torch.arange(nq, device=dev)
        return tok, tok[:, None] <= last[:, :, None]
    first = _first_seen(c, n)
    sinks = torch.arange(c["sinks"], device=dev)[None].expand(n.numel(), -1)
    rest = first[:, None] + torch.arange(min(W + nq - 1, max(1, c["hi"])), device=dev)
    tok = torch.cat([sinks, rest], 1)
    last = (n[:, None] - nq + torch.arange(nq, device=dev))[:, :, None]
    t = tok[:, None]
    see = (t <= last) & ((t > last - W) | (t < c["sinks"]))
    see[:, :, c["sinks"]:] &= rest[:, None] >= c["sinks"]                  # a sink inside the window counts once
    return tok, see


def _gather(s, name, tok):
    """A cache's entries [R, L, Hkv, ..] of the tokens."""
    x, ps = s[name], s["case"]["page"]
    x = x.view(torch.uint8) if x.dtype == FP8 else x
    if ps:
        tok = tok.clamp(max=s["table"].shape[1] * ps - 1)
        page = s["table"].long().gather(1, tok // ps).clamp(min=0)
        x = x[page, tok % ps]
    else:
        x = x[torch.arange(tok.shape[0], device=tok.device)[:, None], tok.clamp(max=x.shape[1] - 1)]
    return x.view(FP8) if s[name].dtype == FP8 else x


def _run_attend(s):
    c = s["case"]
    q4 = c["op"] == "int4"
    if own:
        import softmax_tree_reduction_gb300 as ta
        kw = dict(block_table=s["table"], out=s["out"], lse=s["lse"], max_seqlen=max(1, c["hi"]), sinks=c["sinks"])
        if q4:
            cache = [_call_view(c, s[x]) for x in ("kc", "vc", "ks", "vs")]
            return ta.tree_attn_decode_int4(s["q"], *cache, s["len"], window=c["window"] or None, k_scale=s["kg"], v_scale=s["vg"], **kw)
        return ta.tree_attn_decode_window(s["q"], _call_view(c, s["kc"]), _call_view(c, s["vc"]), s["len"], c["window"], k_scale=s["kg"],
                                          v_scale=s["vg"], **kw)
    R, hq, nq, d = s["q"].shape
    hkv = c["hkv"]
    tok, see = _seen_tokens(s)
    if q4:
        k, v = (_from_int4(_gather(s, x + "c", tok), _gather(s, x + "s", tok), s[x + "g"]) for x in ("k", "v"))
    else:
        k, v = (_gather(s, x + "c", tok).float() for x in ("k", "v"))
        if s["kg"] is not None:
            k, v = k * s["kg"][:, None], v * s["vg"][:, None]
    k, v = k.transpose(1, 2), v.transpose(1, 2)                             # [R, Hkv, L, d]
    q = s["q"].float().reshape(R, hkv, -1, d)                               # (head, query) pairs
    z = (torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)).view(R, hkv, -1, nq, tok.shape[1])
    z = torch.where(see[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    v = torch.where(see.any(1)[:, None, :, None], v, 0.0)
    o = torch.matmul(p.flatten(2, 3), v).view(R, hkv, -1, nq, d) / torch.where(l > 0, l, 1.0)
    s["out"].copy_(o.reshape(R, hq, nq, d))
    s["lse"].copy_((m + torch.log(l)).reshape(R, hq, nq))
    return s["out"], s["lse"]


_RUN = dict(append=_run_append, read=_run_read, int4=_run_attend, window=_run_attend)


def run(state):
    return _RUN[state["case"]["op"]](state)


# ------------------------------------------------------------------ their work
def work(case):
    c = case
    op, d, hkv = c["op"], c["d"], c["hkv"]
    vec4 = d / 2 + d / GROUP                                                # bytes of a 4-bit vector
    if op in ("append", "read"):
        n = 2 * c["tokens"] * hkv                                           # key and value vectors
        if op == "read":
            return {"bytes": n * (vec4 + d * ES[c["dt"]]) + 8 * c["tokens"], "flops": 2 * n * d}
        q = c["tokens"] * c["hq"] * d * c["rope"]
        return {"bytes": (2 * q + 2 * n * d) * ES[c["dt"]] + n * vec4 + 8 * c["tokens"], "flops": 6 * n * d + 6 * c["rope"] * (q + n * d / 2)}
    tokens = (c["lo"] + c["hi"]) / 2
    if c["window"]:
        tokens = min(tokens, c["sinks"] + c["window"] + c["nq"] - 1)
    es = vec4 if op == "int4" else d * ES[c["kv"]]
    qb = 2 if op == "int4" else ES[c["q"]]
    cols = c["hq"] * c["nq"]
    return {"bytes": c["rows"] * (2 * hkv * tokens * es + cols * (d * (qb + 4) + 4)), "flops": 4 * c["rows"] * cols * tokens * d}


# ------------------------------------------- the same from the definitions, in 64 bits
def _norm_rope_exact(x, pos, freq, w):
    y = x.double()
    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS) * w.double()
    n = freq.numel()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), pos.double()[:, None] * freq.double()[None])[:, None]
    z = torch.complex(y[..., :n], y[..., n:]) * turn
    return torch.cat([z.real, z.imag], -1)


def _value_exact(code, step, scale):
    """float64 values of unpacked codes [.., Hkv, d]."""
    y = (code.double() - 8) * step.double().repeat_interleave(GROUP, -1)
    return y if scale is None else y * scale.double().view(-1, 1)


def _unpacked(codes):
    d2 = codes.shape[-1]
    out = torch.empty(*codes.shape[:-1], 2 * d2, dtype=torch.int16, device=codes.device)
    out[..., 0::2] = codes.to(torch.int16) % 16
    out[..., 1::2] = torch.div(codes.to(torch.int16), 16, rounding_mode="floor")
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    op, d = c["op"], c["d"]
    ps = c["page"]
    if op in ("append", "read"):
        live = torch.nonzero(s["pos"] >= 0).squeeze(1)
        rows, pos = s["rows"][live].long(), s["pos"][live].long()
        spot = (s["table"].long()[rows, torch.div(pos, ps, rounding_mode="floor")], torch.remainder(pos, ps)) if ps else (rows, pos)
        res = []
        if op == "append":
            q = s["q_out"].double()
            vec = {"k": s["k"].double(), "v": s["v"].double()}
            if c["rope"]:
                vec["k"] = _norm_rope_exact(s["k"], s["pos"], s["freq"], s["kw"])
                q[live] = _norm_rope_exact(s["q"], s["pos"], s["freq"], s["qw"])[live]
                res.append(q)
        for x in ("k", "v"):
            if op == "append":
                y = vec[x][live].float()                                    # a channel is an FP32 number, and so is its quotient by the scale
                if s[x + "g"] is not None:
                    y = (y.double() / s[x + "g"].double()[:, None]).float()
                y = y.double().unflatten(-1, (d // GROUP, GROUP))
                step = torch.div(y.abs().max(-1)[0], torch.tensor(7.0, dtype=torch.float64, device="cuda")).float()
                step = torch.where(step > E4M3_MAX, E4M3_MAX, torch.where(step < E4M3_MIN, E4M3_MIN, step)).to(FP8)
                code = (torch.round(y / step.double().unsqueeze(-1)).clamp(-7, 7) + 8).flatten(-2)
            else:
                code, step = _unpacked(s[x + "c"][spot]), s[x + "s"].view(torch.uint8)[spot].view(FP8)
            out = s[x + "_out"].double()
            out[live] = _value_exact(code, step, s[x + "g"])
            res.append(out)
        return tuple(res)
    R, hq, nq = c["rows"], c["hq"], c["nq"]
    G = hq // c["hkv"]
    out = torch.zeros(R, hq, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((R, hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    lengths = s["len"].tolist()
    for r in range(R):
        n = lengths[r]
        low = max(0, n - nq + 1 - c["window"]) if c["window"] else 0
        tok = torch.arange(n, device="cuda")
        tok = tok[(tok >= low) | (tok < c["sinks"])]
        if not tok.numel():
            continue
        spot = (s["table"][r, torch.div(tok, ps, rounding_mode="floor")].long(), tok % ps) if ps else (torch.full_like(tok, r), tok)
        vec = []
        for x in ("k", "v"):
            if op == "int4":
                vec.append(_value_exact(_unpacked(s[x + "c"][spot]), s[x + "s"].view(torch.uint8)[spot].view(FP8), s[x + "g"]))
            elif c["kv"] == "e4m3":
                vec.append(s[x + "c"].view(torch.uint8)[spot].view(FP8).double() * s[x + "g"].double()[:, None])
            else:
                vec.append(s[x + "c"][spot].double())
        for i in range(nq):
            at = n - nq + i
            see = (tok <= at) & ((tok < c["sinks"]) | (tok >= at + 1 - c["window"])) if c["window"] else tok <= at
            if not bool(see.any()):
                continue
            for h in range(c["hkv"]):
                z = (s["q"][r, h * G:(h + 1) * G, i].double() @ vec[0][see, h].T) * (d ** -0.5)
                lse[r, h * G:(h + 1) * G, i] = torch.logsumexp(z, 1)
                out[r, h * G:(h + 1) * G, i] = torch.softmax(z, 1) @ vec[1][see, h]
    return out, lse
