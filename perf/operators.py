"""The quantised K^F/V^F cache: what is measured of it.

Four operators over a key/value cache held in 4 bits (per row a scale and a
zero point) or in 8 bits (e4m3 with a scale per row):

  store   hs_kv_quant_write + hs_kv_quant_read: rows are quantised as they are
          written, then read back as bf16
  full    hs_decode_step_quant, full step: one new token per sequence attends
          to its whole cache and selects its index set
  sparse  hs_decode_step_quant, sparse step: one new token per sequence over
          the rows of an index set
  reuse   hs_sparse_attn_reuse_quant: a prefill chunk's queries, each over the
          rows of its own index set (tokens, or blocks of keys)

A stored row of head_dim values has codes, and a scale and a zero point in bf16:
a code stands for scale * code + zero. In 4 bits, scale = bf16((max - min) / 15),
zero = bf16(min), code = rint((x - zero) / scale) in 0..15; in 8 bits, scale =
bf16(max|x| / 448), zero = 0, code = e4m3(x / scale).
"""
import math

import torch

own = False
DEV = "cuda"

#: head layouts: (query heads, kv heads, head_dim)
LAYOUTS = ((64, 4, 128), (32, 8, 128), (16, 1, 128), (32, 8, 64), (10, 2, 128), (7, 7, 64))


def listed():
    return [
        # a chunked prefill stores its 8192 new rows behind a long prefix and hands them on in bf16
        dict(name="store int4 chunk", op="store", fmt="int4", batch=1, hq=64, hkv=4, d=128, t_q=8192, t_kv=65536, page=0, ragged=False),
        # a serving batch appends prompts of different lengths to a paged cache
        dict(name="store fp8 paged prompts", op="store", fmt="fp8", batch=7, hq=32, hkv=8, d=128, t_q=509, t_kv=4096, page=64, ragged=True),
        # a decode step appends one row per sequence: latency
        dict(name="store int4 token", op="store", fmt="int4", batch=32, hq=64, hkv=4, d=128, t_q=1, t_kv=4096, page=64, ragged=True),
        # the full layer's decode step of 32 sequences with long caches, the serving load of the 64/4 configuration
        dict(name="full int4 32x128k", op="full", fmt="int4", batch=32, hq=64, hkv=4, d=128, t_kv=131072, k=1024, window=128, page=0, ragged=False),
        # the same step at the end of one 2^20-token context
        dict(name="full int4 1x1m", op="full", fmt="int4", batch=1, hq=64, hkv=4, d=128, t_kv=1 << 20, k=1024, window=128, page=0, ragged=False),
        # a ragged paged batch in 8 bits, 32/8 heads
        dict(name="full fp8 paged ragged", op="full", fmt="fp8", batch=9, hq=32, hkv=8, d=128, t_kv=20032, k=512, window=64, page=64, ragged=True),
        # short caches, smaller heads: latency
        dict(name="full int4 short", op="full", fmt="int4", batch=3, hq=32, hkv=8, d=64, t_kv=1500, k=256, window=32, page=0, ragged=True),
        # the sparse layers' decode step, 11 of them behind each full one
        dict(name="sparse int4 32x1024", op="sparse", fmt="int4", batch=32, hq=64, hkv=4, d=128, t_kv=131072, k=1024, window=128, page=0, ragged=True),
        # one sequence, paged, 8 bits
        dict(name="sparse fp8 paged 1x1152", op="sparse", fmt="fp8", batch=1, hq=32, hkv=8, d=128, t_kv=32768, k=1152, window=128, page=64, ragged=False),
        # a prefill chunk's sparse layer in token mode
        dict(name="reuse int4 tokens", op="reuse", fmt="int4", batch=1, hq=64, hkv=4, d=128, t_q=2048, t_kv=65536, k=1024, window=128, block=1, page=0),
        # a prefill chunk's sparse layer over 64-key blocks, 32/8 heads
        dict(name="reuse fp8 blocks", op="reuse", fmt="fp8", batch=2, hq=32, hkv=8, d=128, t_q=500, t_kv=16384, k=1024, window=0, block=64, page=0),
        # a short prompt, odd sizes, paged
        dict(name="reuse int4 paged short", op="reuse", fmt="int4", batch=2, hq=10, hkv=2, d=128, t_q=33, t_kv=1008, k=200, window=24, block=1, page=48),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("store", "full", "sparse", "reuse"))
    hq, hkv, d = rng.choice(LAYOUTS)
    c = dict(op=op, fmt=rng.choice(("int4", "fp8")), hq=hq, hkv=hkv, d=d)
    page = rng.choice((0, 0, 16, 48, 64, 256))
    if op == "store":
        t_q = _log(rng, 1, 4000)
        c |= dict(batch=_log(rng, 1, max(1, min(64, 8000 // t_q))), t_q=t_q, t_kv=t_q + _log(rng, 1, 30000), ragged=rng.random() < 0.6)
    else:
        window = rng.choice((0, 16, 64, 128))
        k = window + _log(rng, 32, 1024)
        if op == "reuse":
            batch = rng.choice((1, 1, 2, 3))
            t_q = _log(rng, 1, 900 // batch)
            c |= dict(batch=batch, t_q=t_q, t_kv=t_q + _log(rng, 1, 30000), k=k, window=window, block=1)
            if rng.random() < 0.4:
                c["block"] = rng.choice((16, 32, 64, 128))
                c["k"], c["window"] = c["block"] * rng.randint(1, max(1, min(64, 1024 // c["block"]))), 0
        else:
            t_kv = _log(rng, 300, 200000)
            c |= dict(batch=_log(rng, 1, max(1, min(48, 2000000 // (t_kv * hkv)))), t_kv=t_kv, k=k, window=window, ragged=rng.random() < 0.6)
    c["page"] = page
    if page:
        c["t_kv"] = -(-c["t_kv"] // page) * page
    return c


# ------------------------------------------------------------------ inputs
def _row_bytes(c):
    return c["d"] // 2 if c["fmt"] == "int4" else c["d"]


def _quantise(x, fmt):
    """Codes (uint8) and scales of the rows of x, in 32 bits."""
    x = x.float()
    if fmt == "fp8":
        s = (x.abs().amax(-1, keepdim=True) / 448.0).bfloat16().float()
        y = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
        y = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return y, torch.cat([s, torch.zeros_like(s)], -1).bfloat16()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).bfloat16().float()
    z = lo.bfloat16().float()
    y = torch.where(s > 0, (x - z) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    y = y.round().clamp(0, 15).to(torch.uint8)
    return y[..., 0::2] | (y[..., 1::2] << 4), torch.cat([s, z], -1).bfloat16()


def _values(codes, scale, fmt):
    """The values that rows of codes stand for, in 32 bits."""
    if fmt == "fp8":
        x = codes.view(torch.float8_e4m3fn).float()
    else:
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return x * scale[..., :1].float() + scale[..., 1:].float()


def _empty_cache(c):
    rows = (c["n_pages"], c["hkv"], c["page"]) if c["page"] else (c["batch"], c["hkv"], c["t_kv"])
    return torch.zeros(*rows, _row_bytes(c), dtype=torch.uint8, device=DEV), torch.zeros(*rows, 2, dtype=torch.bfloat16, device=DEV)


def _flat_rows(c, table, pos):
    """Rows of the cache, flattened, that hold positions pos [batch, hkv, ...] of each sequence and group."""
    shape = (1,) * (pos.dim() - 2)
    b = torch.arange(pos.shape[0], device=pos.device).view(-1, 1, *shape)
    u = torch.arange(c["hkv"], device=pos.device).view(1, -1, *shape)
    if not c["page"]:
        return (b * c["hkv"] + u) * c["t_kv"] + pos
    page = table.long()[b, pos // c["page"]]
    return (page * c["hkv"] + u) * c["page"] + pos % c["page"]


def _lengths(c, gen):
    if not c.get("ragged"):
        return torch.full((c["batch"],), c["t_kv"], dtype=torch.int32, device=DEV)
    n = torch.randint(max(1, c["t_kv"] // 3), c["t_kv"] + 1, (c["batch"],), generator=gen, device=DEV, dtype=torch.int32)
    n[0] = c["t_kv"]
    if c["batch"] > 2:
        n[1] = 1 if c["op"] != "store" else c["t_q"]
    return n


def _fill(c, s, gen, q=None):
    """Fills the cache of state s, one sequence at a time, with Gaussian rows. For a full step, k - window keys of each
    group are strongly relevant to one of its heads, so that no rounding decides which keys are selected."""
    std = lambda *n: torch.randn(*n, generator=gen, device=DEV)  # noqa: E731
    hkv, d, T = c["hkv"], c["d"], c["t_kv"]
    g = c["hq"] // hkv
    pos = torch.arange(T, device=DEV).expand(1, hkv, T)
    for b in range(c["batch"]):
        k, v = std(hkv, T, d), std(hkv, T, d)
        if q is not None:
            L, n = int(s["lens"][b]), c["k"] - c["window"]
            n = min(n, max(0, L - c["window"]))
            for u in range(hkv):
                at = torch.randperm(max(L - c["window"], 0), generator=gen, device=DEV)[:n]
                qh = q[b, u * g + torch.arange(n, device=DEV) % g, 0].float()
                sq = qh.square().sum(-1, keepdim=True)
                want = (10.0 + 3.0 * torch.rand(n, 1, generator=gen, device=DEV)) * math.sqrt(d)
                k[u, at] += (want - (k[u, at] * qh).sum(-1, keepdim=True)) / sq * qh
        rows = _flat_rows(c, s["table"][b:b + 1] if c["page"] else None, pos)[0]
        if not c["page"]:
            rows = rows + b * hkv * T
        for name, x in (("k", k), ("v", v)):
            codes, scale = _quantise(x.bfloat16(), c["fmt"])
            s[name + "_codes"].view(-1, codes.shape[-1])[rows] = codes
            s[name + "_scale"].view(-1, 2)[rows] = scale


def _strata(lo, n, gen, shape):
    """n distinct ascending ids of 0..lo-1 for each row; lo [*shape] >= n."""
    u = torch.rand(*shape, n, generator=gen, device=DEV, dtype=torch.float64)
    j = torch.arange(n, device=DEV, dtype=torch.float64)
    a, b = torch.floor(j * lo[..., None] / n), torch.floor((j + 1) * lo[..., None] / n)
    return torch.minimum(a + torch.floor(u * (b - a)), b - 1).long()


def _index(c, last, gen):
    """Index sets [batch, hkv, (rows,) ksel] and counts of queries at positions last [batch, (rows)]."""
    block = c.get("block", 1)
    ksel = c["k"] // block
    last = last.long()[:, None].expand(-1, c["hkv"], *last.shape[1:])
    seen, w = last // block + 1, c["window"] if block == 1 else 0
    n = ksel - w
    lo = (seen - w).clamp(min=max(n, 1))
    ids = torch.cat([_strata(lo.double(), n, gen, lo.shape), (seen - w)[..., None] + torch.arange(w, device=DEV)], -1)
    every = torch.arange(ksel, device=DEV).expand_as(ids)
    ids = torch.where((seen <= ksel)[..., None], torch.where(every < seen[..., None], every, -1), ids)
    return ids.int().contiguous(), seen.clamp(max=ksel).int().contiguous()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if c["page"]:
        c["max_pages"] = c["t_kv"] // c["page"]
        c["n_pages"] = c["batch"] * c["max_pages"] + 3
    s = {"c": c, "table": None}
    if c["page"]:
        s["table"] = torch.randperm(c["n_pages"], generator=gen, device=DEV)[:c["batch"] * c["max_pages"]].view(c["batch"], -1).int()
    for name in "kv":
        s[name + "_codes"], s[name + "_scale"] = _empty_cache(c)
    s["lens"] = _lengths(c, gen)
    if c["op"] == "store":
        shape = (c["batch"], c["hkv"], c["t_q"], c["d"])
        s["k"], s["v"] = (torch.randn(*shape, generator=gen, device=DEV).bfloat16() for _ in "kv")
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
        n = torch.full((c["batch"],), c["t_q"], dtype=torch.int32, device=DEV)
        if c["ragged"] and c["t_q"] > 1:
            n = torch.randint(0, c["t_q"] + 1, (c["batch"],), generator=gen, device=DEV, dtype=torch.int32)
            n[0] = c["t_q"]
        s["n_new"] = torch.minimum(n, s["lens"])
        return s
    t_q = c.get("t_q", 1)
    s["q"] = torch.randn(c["batch"], c["hq"], t_q, c["d"], generator=gen, device=DEV).bfloat16()
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(c["batch"], c["hq"], t_q, dtype=torch.float32, device=DEV)
    _fill(c, s, gen, s["q"] if c["op"] == "full" else None)
    if c["op"] == "full":
        s["idx"] = torch.empty(c["batch"], c["hkv"], c["k"], dtype=torch.int32, device=DEV)
        s["cnt"] = torch.empty(c["batch"], c["hkv"], dtype=torch.int32, device=DEV)
    elif c["op"] == "sparse":
        s["idx"], s["cnt"] = _index(c, s["lens"] - 1, gen)
    else:
        last = (c["t_kv"] - t_q + torch.arange(t_q, device=DEV)).expand(c["batch"], -1)
        s["idx"], s["cnt"] = _index(c, last, gen)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    c = s["c"]
    return {"store": _store, "full": _full, "sparse": _selected, "reuse": _selected}[c["op"]](s, c)


def _run_own(s):
    from oracle_top_kv_b200 import hs
    c = s["c"]
    if "plan" not in s:
        t_q = c.get("t_q", 1)
        block = c.get("block", 1)
        p = hs.make_params(c["batch"], c["hq"], c["hkv"], c["d"], t_q, c["t_kv"], c["t_kv"] - t_q if c["op"] == "reuse" else 0, "bf16",
                           "token" if block == 1 else "block", block, c.get("k", 1), c.get("window", 0))
        kv = hs.make_kv_quant(c["fmt"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])
        pages = hs.make_pages(s["table"], c["page"], c["n_pages"]) if c["page"] else None
        s["plan"] = p, kv, pages, hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT) if c["op"] == "full" else None
    p, kv, pages, ws = s["plan"]
    if c["op"] == "store":
        hs.hs_kv_quant_write(p, kv, pages, s["k"], s["v"], s["lens"], s["n_new"])
        hs.hs_kv_quant_read(p, kv, pages, s["k_out"], s["v_out"], s["lens"], s["n_new"])
        return s["k_out"], s["v_out"]
    if c["op"] == "full":
        hs.hs_decode_step_quant(p, kv, pages, hs.HS_DECODE_FULL_INDEX, s["q"], s["lens"], s["idx"], s["cnt"], s["o"], s["lse"], workspace=ws)
        return s["o"], s["lse"], s["idx"], s["cnt"]
    if c["op"] == "sparse":
        hs.hs_decode_step_quant(p, kv, pages, hs.HS_DECODE_SPARSE, s["q"], s["lens"], s["idx"], s["cnt"], s["o"], s["lse"])
    else:
        hs.hs_sparse_attn_reuse_quant(p, kv, pages, s["q"], s["idx"], s["cnt"], s["o"], s["lse"])
    return s["o"], s["lse"]


def _new_rows(s, c):
    """Cache rows of the new rows j < n_new, and which rows j are new."""
    j = torch.arange(c["t_q"], device=DEV)
    n = s["n_new"].long()[:, None]
    new = (j < n)[:, None].expand(-1, c["hkv"], -1)
    pos = (s["lens"].long()[:, None] - n + j).clamp(0, c["t_kv"] - 1)[:, None].expand(-1, c["hkv"], -1)
    return _flat_rows(c, s["table"], pos), new


def _store(s, c):
    rows, new = _new_rows(s, c)

    def one(x, codes, scale, out):
        flat, flat_s = codes.view(-1, codes.shape[-1]), scale.view(-1, 2)
        new_codes, new_scale = _quantise(x, c["fmt"])
        flat[rows[new]] = new_codes[new]
        flat_s[rows[new]] = new_scale[new]
        back = _values(flat[rows], flat_s[rows], c["fmt"]).to(out.dtype)
        out.copy_(torch.where(new[..., None], back, out))
        return out

    return one(s["k"], s["k_codes"], s["k_scale"], s["k_out"]), one(s["v"], s["v_codes"], s["v_scale"], s["v_out"])


def _attend(q, k, v, keep):
    """Softmax attention of q [..., g, d] over k, v [..., n, d] where keep [..., n]; natural-log lse, and the scaled logits."""
    a = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    a = torch.where(keep[..., None, :], a, torch.full_like(a, -math.inf))
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - m)
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / total, (m + torch.log(total)).squeeze(-1), a


def _full(s, c):
    B, hkv, T, k, w = c["batch"], c["hkv"], c["t_kv"], c["k"], c["window"]
    g = c["hq"] // hkv
    if c["page"]:
        rows = _flat_rows(c, s["table"], torch.arange(T, device=DEV).expand(B, hkv, T))
        at = lambda x: x.view(-1, *x.shape[3:])[rows]  # noqa: E731
    else:
        at = lambda x: x  # noqa: E731
    key = torch.arange(T, device=DEV)
    L = s["lens"].long()[:, None, None]
    q = s["q"].float().view(B, hkv, g, -1)
    keys = _values(at(s["k_codes"]), at(s["k_scale"]), c["fmt"])
    values = _values(at(s["v_codes"]), at(s["v_scale"]), c["fmt"])
    o, lse, a = _attend(q, keys, values, (key < L).expand(B, hkv, T))
    score = (a - lse[..., None]).amax(-2)
    score = torch.where((key >= L - w) & (key < L), torch.full_like(score, math.inf), score)
    top = torch.topk(score, min(k, T), dim=-1)
    ids = torch.where(top.values > -math.inf, top.indices, T).sort(-1).values
    ids = torch.where(ids < T, ids, -1).int()
    ids = torch.cat([ids, torch.full((B, hkv, k - ids.shape[-1]), -1, dtype=torch.int32, device=DEV)], -1)
    cnt = s["lens"].clamp(max=k)[:, None].expand(B, hkv).contiguous()
    return o.to(torch.bfloat16).view_as(s["o"]), lse.view_as(s["lse"]), ids, cnt


def _tokens(s, c):
    """Selected positions [batch, hkv, rows, n] of each query row, and which of them count."""
    B, hkv = c["batch"], c["hkv"]
    ids, cnt = s["idx"].long().view(B, hkv, -1, s["idx"].shape[-1]), s["cnt"].long().view(B, hkv, -1, 1)
    keep = torch.arange(ids.shape[-1], device=DEV) < cnt
    block = c.get("block", 1)
    if block > 1:
        ids = (ids[..., None] * block + torch.arange(block, device=DEV)).flatten(-2)
        last = c["t_kv"] - c["t_q"] + torch.arange(c["t_q"], device=DEV)
        keep = keep.repeat_interleave(block, -1) & (ids <= last[None, None, :, None])
    return torch.where(keep, ids, 0), keep


def _selected(s, c):
    B, hkv, d = c["batch"], c["hkv"], c["d"]
    g = c["hq"] // hkv
    ids, keep = _tokens(s, c)
    rows = _flat_rows(c, s["table"], ids)
    at = lambda x: x.view(-1, *x.shape[3:])[rows]  # noqa: E731
    keys = _values(at(s["k_codes"]), at(s["k_scale"]), c["fmt"])
    values = _values(at(s["v_codes"]), at(s["v_scale"]), c["fmt"])
    q = s["q"].float().view(B, hkv, g, -1, d).transpose(2, 3)
    o, lse, _ = _attend(q, keys, values, keep)
    return o.transpose(2, 3).reshape(s["o"].shape).to(torch.bfloat16), lse.transpose(2, 3).reshape(s["lse"].shape)


# ------------------------------------------------------------------ work, and the definition in 64 bits
def work(case):
    c = case
    row = _row_bytes(c) + 4
    d, hq, hkv, B = c["d"], c["hq"], c["hkv"], c["batch"]
    mean = 2 / 3 if c.get("ragged") and B > 1 else 1.0
    if c["op"] == "store":
        n = 2 * B * hkv * c["t_q"] * (0.5 if c["ragged"] and c["t_q"] > 1 and B > 1 else 1.0)
        return {"bytes": n * (2 * d + row + 2 * d), "flops": n * d * 8}
    t_q = c.get("t_q", 1)
    io = B * hq * t_q * (4 * d + 4)
    if c["op"] == "full":
        keys = B * c["t_kv"] * mean
        return {"bytes": keys * hkv * 2 * row + io + B * hkv * 4 * c["k"], "flops": 4.0 * d * hq * keys}
    picked = min(c["k"], c["t_kv"])
    keys = B * hkv * t_q * picked
    return {"bytes": min(keys, B * hkv * c["t_kv"]) * 2 * row + io + B * hkv * t_q * 4 * (c["k"] // c.get("block", 1)),
            "flops": 4.0 * d * keys * (hq // hkv)}


def _decode64(codes, scale, fmt):
    if fmt == "fp8":
        bits = torch.arange(256, device=DEV)
        e, m = (bits >> 3) & 15, bits & 7
        mag = torch.where(e > 0, (8 + m).double() * 2.0 ** (e - 10).double(), m.double() * 2.0 ** -9)
        return torch.where(bits > 127, -mag, mag)[codes.long()] * scale[..., :1].double() + scale[..., 1:].double()
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=DEV)
    out[..., 0::2] = (codes % 16).double()
    out[..., 1::2] = (codes // 16).double()
    return out.mul_(scale[..., 0:1].double()).add_(scale[..., 1:2].double())


def _stored64(x, fmt):
    """What row values x, in 64 bits, are stored as."""
    if fmt == "fp8":
        s = (x.abs().amax(-1, keepdim=True) / 448).bfloat16().double()
        y = x / s.clamp(min=1e-300)
        step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(y / step) * step).clamp(-448, 448) * s
    s = ((x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15).bfloat16().double()
    z = x.amin(-1, keepdim=True)
    return torch.round((x - z) / s.clamp(min=1e-300)).clamp(0, 15) * s + z


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "store":
        n = s["n_new"].tolist()
        outs = [s["k_out"].double(), s["v_out"].double()]
        for out, x in zip(outs, (s["k"], s["v"])):
            for b in range(c["batch"]):
                if n[b]:
                    out[b, :, :n[b]] = _stored64(x[b, :, :n[b]].double(), c["fmt"])
        return tuple(outs)
    g, d = c["hq"] // c["hkv"], c["d"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    block = c.get("block", 1)
    for b in range(c["batch"]):
        for u in range(c["hkv"]):
            heads = slice(u * g, (u + 1) * g)

            def rows_at(pos):
                if c["page"]:
                    pos = (s["table"][b].long()[pos // c["page"]] * c["hkv"] + u) * c["page"] + pos % c["page"]
                else:
                    pos = pos + (b * c["hkv"] + u) * c["t_kv"]
                flat = [s[n].view(-1, *s[n].shape[3:])[pos] for n in ("k_codes", "k_scale", "v_codes", "v_scale")]
                return _decode64(*flat[:2], c["fmt"]), _decode64(*flat[2:], c["fmt"])

            if c["op"] == "full":
                k, v = rows_at(torch.arange(int(s["lens"][b]), device=DEV))
                a = s["q"][b, heads, 0].double() @ k.T * d ** -0.5
                l = torch.logsumexp(a, -1)
                o[b, heads, 0], lse[b, heads, 0] = torch.exp(a - l[:, None]) @ v, l
                continue
            t_q = s["q"].shape[2]
            ids = s["idx"][b, u].long().view(t_q, -1)
            cnt = s["cnt"][b, u].view(t_q, 1)
            keep = torch.arange(ids.shape[1], device=DEV)[None] < cnt
            last = (s["lens"][b].long() - 1).expand(t_q) if c["op"] == "sparse" else c["t_kv"] - t_q + torch.arange(t_q, device=DEV)
            if block > 1:
                ids = torch.cat([ids[:, :, None] * block + i for i in range(block)], -1).reshape(t_q, -1)
                keep = keep[:, :, None].expand(-1, -1, block).reshape(t_q, -1) & (ids <= last[:, None])
            for t in range(0, t_q, 256):
                part = slice(t, min(t_q, t + 256))
                k, v = rows_at(ids[part].clamp(min=0))
                a = torch.einsum("htd,tnd->htn", s["q"][b, heads, part].double(), k) * d ** -0.5
                a = a.masked_fill(~keep[part][None], -math.inf)
                l = torch.logsumexp(a, -1)
                o[b, heads, part] = torch.einsum("htn,tnd->htd", torch.exp(a - l[..., None]), v)
                lse[b, heads, part] = l
    return (o, lse, None, None) if c["op"] == "full" else (o, lse)
