"""The quantised K^F/V^F cache at its edges: rows past 4 GB, the largest budget,
page and block sizes around a step of the kernels, calls that run at once,
repeated index entries, numbers near the ends of their range.

Bars: those of tests/parity.py where the fp64 oracle is the reference; equal bits
where two calls do the same arithmetic on the same codes.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle_top_kv_b200 import hs
from tests import parity as P
from tests.test_gpu_quant import (DEV, FMTS, Cache, _decode_outputs, _filled, _params, _randn)

pytestmark = pytest.mark.gpu


def _full(p, c, q, seq, ws=None):
    ws = hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT) if ws is None else ws
    idx, cnt, o, lse, sel = _decode_outputs(p)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse,
                            sel, ws)
    return o, lse, idx, cnt, sel


def _check_decode(p, c, q, qs, lens):
    """A full and a sparse step against the oracle."""
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, lse, idx, cnt, _ = _full(p, c, q, seq)
    os_, ls = torch.empty_like(o), torch.empty_like(lse)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_SPARSE, qs, seq, idx, cnt, os_, ls)
    assert hs.hs_device_status() == 0
    kd, vd = c.values()
    rows = np.array([[i, u, 0] for i in range(p.batch) for u in range(p.hkv)], np.int32)
    pos = np.array(lens)[rows[:, 0]] - 1
    g = p.hq // p.hkv
    orc = oracle.full_attn_rows(q.double().cpu().numpy(), kd, vd, rows, pos, "token", 1, p.k, p.window)
    P.check_o(P.gpu_rows(P.f64(o), rows, True, g), orc["o"], "bf16", "full o")
    P.check_lse(P.gpu_rows(lse.cpu().double().numpy(), rows, True, g), orc["lse"], "bf16", "lse")
    g_idx, g_cnt = idx.cpu().numpy()[rows[:, 0], rows[:, 1]], cnt.cpu().numpy()[rows[:, 0], rows[:, 1]]
    P.check_index(g_idx, g_cnt, orc, "token", p.window, p.k, "index")
    sp = oracle.sparse_attn_rows(qs.double().cpu().numpy(), kd, vd, g_idx, g_cnt, rows, pos,
                                 "token", 1, p.k, p.window)
    P.check_o(P.gpu_rows(P.f64(os_), rows, True, g), sp["o_g"], "bf16", "sparse o")
    P.check_lse(P.gpu_rows(ls.cpu().double().numpy(), rows, True, g), sp["lse_g"], "bf16", "sparse lse")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", [
    # batch, hq, hkv, d, t_kv, k, window, page, lengths
    (1, 9, 1, 128, 9000, 4096, 0, 0, [9000]),          # the largest budget, nine heads
    (2, 20, 2, 128, 4000, 3000, 200, 16, [4000, 3500]),  # a budget that leaves little room
    (2, 12, 1, 128, 4096, 100, 4, 32, [4096, 1000]),   # pages of a step
    (2, 2, 2, 64, 4160, 100, 4, 1, [4160, 2001]),      # pages of one row, groups of one
    (3, 14, 2, 64, 2000, 64, 0, 40, [2000, 65, 64]),
    (1, 8, 1, 128, 1, 1, 0, 0, [1]),                   # one row
    (1, 16, 1, 128, 33, 16, 15, 0, [17]),              # one ranked key of two
    (2, 8, 1, 128, 50000, 900, 0, 0, [14400, 14416]),  # as many tiles of 16 as ranked keys, one more
])
def test_decode_sizes(fmt, case):
    b, hq, hkv, d, T, k, w, page, lens = case
    p = _params(b, hq, hkv, d, 1, T, k=k, window=w)
    q, qs = _randn(b, hq, 1, d, seed=81), _randn(b, hq, 1, d, seed=82)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c = _filled(p, fmt, page, 83, q, needles=min(12, T), lens=seq)
    _check_decode(p, c, q, qs, lens)


@pytest.mark.parametrize("fmt", FMTS)
def test_bounds_past_what_a_cta_holds(fmt):
    """One sequence of a batch so wide that a CTA selects alone has more tiles than fit on chip."""
    b, hq, hkv, d, T, L, k, w = 80, 2, 1, 64, 290000, 280005, 100, 10
    p = _params(b, hq, hkv, d, 1, T, k=k, window=w)
    c = Cache(p, fmt, seed=1)
    n = 20000
    pw = _params(b, hq, hkv, d, n, T, q_offset=0)
    lens = torch.full((b,), 50, dtype=torch.int32, device=DEV)
    g = torch.Generator(DEV).manual_seed(5)
    b_long = 37
    for at in range(0, L, n):
        m = min(n, L - at)
        x = torch.zeros(b, hkv, n, d, dtype=torch.bfloat16, device=DEV)
        x[b_long] = torch.randn(hkv, n, d, generator=g, device=DEV).bfloat16()
        new = torch.zeros_like(lens)
        new[b_long] = m
        lens[b_long] = at + m
        hs.hs_kv_quant_write(pw, c.kv, None, x, x, lens, new)
    q = _randn(b, hq, 1, d, seed=84)
    o, lse, idx, cnt, sel = _full(p, c, q, lens)
    assert hs.hs_device_status() == 0
    codes, entry = c.t[0][b_long, 0, :L], c.t[1][b_long, 0, :L].double()
    if fmt == "int4":
        cv = torch.stack([codes & 15, codes >> 4], -1).flatten(1).double()
    else:
        cv = codes.view(torch.float8_e4m3fn).double()
    kd = cv * entry[:, :1] + entry[:, 1:]
    a = q[b_long, :, 0].double() @ kd.T / d ** 0.5
    want = torch.logsumexp(a, -1)
    assert (lse[b_long, :, 0].double() - want).abs().max() < P.LSE_TOL["bf16"]
    score = (a - want[:, None]).amax(0)
    got = idx[b_long, 0].long()
    assert int(cnt[b_long, 0]) == k and (got[1:] > got[:-1]).all()
    assert torch.equal(got[k - w:], torch.arange(L - w, L, device=DEV))
    kth = score[:L - w].topk(k - w).values[-1]
    # the exponent of a near-tie: the bar of the index sets
    assert (score[got[:k - w]] >= kth - P.INDEX_REL).all()
    assert ((sel[b_long, 0].double() / score[got].exp()) - 1).abs().max() < 2e-4
    # the short ones select all of their 50 rows
    rest = torch.arange(b, device=DEV) != b_long
    assert (cnt[rest] == 50).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_past_4_gb(fmt):
    """Rows whose byte offsets pass 2^32, contiguous and in a pool, against the same rows in a
    small cache: equal bits."""
    hq, hkv, d, page, T = 8, 1, 128, 16, 512
    width = d // 2 if fmt == "int4" else d
    rows = (1 << 32) // width + 4096
    p = _params(1, hq, hkv, d, 1, T, k=64, window=8)
    pw = _params(1, hq, hkv, d, T, T)
    k, v = _randn(1, hkv, T, d, seed=85), _randn(1, hkv, T, d, seed=86)
    q = _randn(1, hq, 1, d, seed=87)
    seq = torch.tensor([T], dtype=torch.int32, device=DEV)
    small = Cache(p, fmt)
    small.write(k, v, p=pw)
    want = _full(p, small, q, seq)
    ws_, wl_ = torch.empty_like(want[0]), torch.empty_like(want[1])
    hs.hs_decode_step_quant(p, small.kv, None, hs.HS_DECODE_SPARSE, q, seq, want[2], want[3], ws_, wl_)
    big = hs.kv_quant_cache(_params(1, hq, hkv, d, 1, rows), fmt, DEV)
    kv = hs.make_kv_quant(fmt, *big)
    # a pool: the last pages, in turn
    n_pages = rows // page
    table = (n_pages - 1 - torch.arange(T // page, device=DEV)).int()[None].contiguous()
    pages = hs.make_pages(table, page, n_pages)
    hs.hs_kv_quant_write(pw, kv, pages, k, v)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    hs.hs_kv_quant_read(pw, kv, pages, ko, vo)
    ks, vs = torch.empty_like(k), torch.empty_like(v)
    hs.hs_kv_quant_read(pw, small.kv, None, ks, vs)
    assert torch.equal(ko, ks) and torch.equal(vo, vs)
    idx, cnt, o, lse, _ = _decode_outputs(p)
    ws = hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT)
    hs.hs_decode_step_quant(p, kv, pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse, None, ws)
    assert torch.equal(idx, want[2]) and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    os_, ls = torch.empty_like(o), torch.empty_like(lse)
    hs.hs_decode_step_quant(p, kv, pages, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, os_, ls)
    assert torch.equal(os_, ws_) and torch.equal(ls, wl_)
    # contiguous: the last T rows of one long sequence, by their index
    pb = _params(1, hq, hkv, d, 1, rows, k=64, window=8)
    first = rows - T
    hs.hs_kv_quant_write(_params(1, hq, hkv, d, T, rows, q_offset=first), kv, None, k, v)
    far = torch.where(want[2] >= 0, want[2] + first, want[2]).int()
    seq.fill_(rows)
    hs.hs_decode_step_quant(pb, kv, None, hs.HS_DECODE_SPARSE, q, seq, far, cnt, os_, ls)
    assert torch.equal(os_, ws_) and torch.equal(ls, wl_)
    # a prefill row at the same position
    pr = _params(1, hq, hkv, d, 1, rows, k=64, window=8, q_offset=rows - 1)
    hs.hs_sparse_attn_reuse_quant(pr, kv, None, q, far[:, :, None], cnt[:, :, None], os_, ls)
    assert hs.hs_device_status() == 0
    P.check_o(P.f64(os_), P.f64(ws_), "bf16", "prefill row")
    assert (ls - wl_).abs().max() < 1e-5  # the same sums in another order
    # the full step over all of it (zero rows before the last T): finite, and it finds them
    torch.cuda.empty_cache()
    idx, cnt, o, lse, _ = _decode_outputs(pb)
    hs.hs_decode_step_quant(pb, kv, None, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse, None,
                            hs.workspace(pb, hs.HS_WS_DECODE_FULL_QUANT))
    assert hs.hs_device_status() == 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all() and int(cnt[0, 0]) == 64
    assert set(idx[0, 0].tolist()) <= set(range(first - 65536, rows))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", [
    # hq, hkv, d, t_q, q_offset, t_kv, mode, block, k, page
    (32, 2, 128, 17, 980, 1000, "block", 16, 256, 8),
    (18, 2, 64, 17, 1200, 1217, "block", 32, 512, 0),
    (4, 2, 64, 40, 2000, 2048, "block", 128, 1024, 32),
    (4, 4, 128, 3, 5000, 5008, "token", 1, 4096, 16),
    (8, 1, 128, 1, 0, 1, "token", 1, 1, 0),
    (22, 2, 128, 5, 100, 105, "token", 1, 64, 1),
])
def test_prefill_sizes(fmt, case):
    """Ragged index sets of every size, some empty, some with the block that the query cuts."""
    hq, hkv, d, t_q, off, T, mode, B, k, page = case
    T = -(-T // page) * page if page else T
    p = _params(2, hq, hkv, d, t_q, T, k=k, window=0, mode=mode, block_size=B, q_offset=off)
    c = _filled(p, fmt, page, 91)
    q = _randn(2, hq, t_q, d, seed=92)
    gen = np.random.default_rng(7)
    ksel = p.ksel
    idx = np.full((2, hkv, t_q, ksel), -1, np.int32)
    cnt = np.zeros((2, hkv, t_q), np.int32)
    for i in np.ndindex(2, hkv, t_q):
        seen = (off + i[2]) // B + 1
        n = min(seen, int(gen.integers(0, ksel + 1)))
        ids = gen.choice(seen - 1, max(n - 1, 0), replace=False) if n else []
        idx[i][:n] = np.sort(np.append(ids, seen - 1))[:n] if n else 0
        cnt[i] = n
    o, lse = torch.empty_like(q), torch.empty(2, hq, t_q, dtype=torch.float32, device=DEV)
    hs.hs_sparse_attn_reuse_quant(p, c.kv, c.pages, q, torch.tensor(idx, device=DEV),
                                  torch.tensor(cnt, device=DEV), o, lse)
    assert hs.hs_device_status() == 0
    kd, vd = c.values()
    rows = np.array(list(np.ndindex(2, hkv, t_q)), np.int32)
    sp = oracle.sparse_attn_rows(q.double().cpu().numpy(), kd, vd, idx.reshape(-1, ksel),
                                 cnt.reshape(-1), rows, off + rows[:, 2], mode, B, k, 0)
    g = hq // hkv
    P.check_o(P.gpu_rows(P.f64(o), rows, True, g), sp["o_g"], "bf16", "o")
    P.check_lse(P.gpu_rows(lse.cpu().double().numpy(), rows, True, g), sp["lse_g"], "bf16", "lse")


@pytest.mark.parametrize("fmt", FMTS)
def test_repeated_entries_of_a_decode_step_count_each_time(fmt):
    p = _params(1, 8, 1, 128, 1, 300, k=64, window=0)
    c = _filled(p, fmt, 0, 95)
    q = _randn(1, 8, 1, 128, seed=96)
    seq = torch.tensor([300], dtype=torch.int32, device=DEV)
    idx = torch.full((1, 1, 64), 5, dtype=torch.int32, device=DEV)
    idx[0, 0, 0] = 2
    cnt = torch.full((1, 1), 64, dtype=torch.int32, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(1, 8, 1, device=DEV)
    hs.hs_decode_step_quant(p, c.kv, None, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, o, lse)
    kd, vd = (x[0, 0] for x in c.values())
    a = q[0, :, 0].double().cpu().numpy() @ kd[[2] + [5] * 63].T / 128 ** 0.5
    w = np.exp(a - a.max(1, keepdims=True))
    want = (w / w.sum(1, keepdims=True)) @ vd[[2] + [5] * 63]
    P.check_o(P.f64(o)[0, :, 0], want, "bf16", "o")
    P.check_lse(lse.cpu().double().numpy()[0, :, 0], np.log(np.exp(a).sum(1)), "bf16", "lse")


@pytest.mark.parametrize("fmt", FMTS)
def test_calls_at_once(fmt):
    """Two batches on two streams with a workspace each, again and again: the bits of each alone."""
    ps = [_params(6, 16, 2, 128, 1, 9000, k=256, window=32), _params(1, 16, 1, 128, 1, 60000, k=512, window=0)]
    cs = [_filled(p, fmt, 0, 97 + i) for i, p in enumerate(ps)]
    qs = [_randn(p.batch, p.hq, 1, 128, seed=99) for p in ps]
    seqs = [torch.full((p.batch,), p.t_kv - 3, dtype=torch.int32, device=DEV) for p in ps]
    alone = [_full(p, c, q, s) for p, c, q, s in zip(ps, cs, qs, seqs)]
    streams = [torch.cuda.Stream() for _ in ps]
    wss = [hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT) for p in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i, p in enumerate(ps):
            with torch.cuda.stream(streams[i]):
                got.append((i, _full(p, cs[i], qs[i], seqs[i], wss[i])))
    torch.cuda.synchronize()
    assert hs.hs_device_status() == 0
    for i, g in got:
        for x, y in zip(g, alone[i]):
            assert torch.equal(x, y)


def test_two_graphs_share_a_workspace():
    """Replayed in turn, with other work between them: the bits of eager calls."""
    ps = [_params(2, 16, 2, 128, 1, 5000, k=64, window=8), _params(1, 8, 2, 64, 1, 700, k=32, window=0)]
    need = max(hs.hs_workspace_size(p, hs.HS_WS_DECODE_FULL_QUANT) for p in ps)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    cs = [_filled(p, "int4", 0, 100 + i) for i, p in enumerate(ps)]
    qs = [_randn(p.batch, p.hq, 1, p.head_dim, seed=102) for p in ps]
    seqs = [torch.full((p.batch,), p.t_kv, dtype=torch.int32, device=DEV) for p in ps]
    want = [_full(p, c, q, s) for p, c, q, s in zip(ps, cs, qs, seqs)]
    outs, graphs = [_decode_outputs(p) for p in ps], []
    torch.cuda.synchronize()
    for i, p in enumerate(ps):
        idx, cnt, o, lse, sel = outs[i]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hs.hs_decode_step_quant(p, cs[i].kv, None, hs.HS_DECODE_FULL_INDEX, qs[i], seqs[i], idx,
                                    cnt, o, lse, sel, ws)
        graphs.append(g)
    for _ in range(3):
        for i, g in enumerate(graphs):
            ws.fill_(0xFF)
            g.replay()
            idx, cnt, o, lse, sel = outs[i]
            for x, y in zip((o, lse, idx, cnt, sel), want[i]):
                assert torch.equal(x, y)
            for x in outs[i]:
                x.zero_()
    assert hs.hs_device_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq", [8, 16])
@pytest.mark.parametrize("up", [60, -60])
def test_powers_of_two_cancel(fmt, hq, up):
    """q 2^s against K 2^-s, and V 2^s: scales and codes are the same but for the exponent, so o
    is too, exactly, and lse and the index set are unchanged."""
    p = _params(1, hq, 1, 128, 1, 2000, k=64, window=8)
    pw = _params(1, hq, 1, 128, 2000, 2000)
    k, v = _randn(1, 1, 2000, 128, seed=110), _randn(1, 1, 2000, 128, seed=111)
    q = _randn(1, hq, 1, 128, seed=112, std=2.0)
    seq = torch.tensor([2000], dtype=torch.int32, device=DEV)
    outs = []
    for s in (0, up):
        c = Cache(p, fmt)
        c.write((k.float() * 2.0 ** -s).bfloat16(),
                (v.float() * 2.0 ** s).bfloat16(), p=pw)
        qs = (q.float() * 2.0 ** s).bfloat16()
        o, lse, idx, cnt, sel = _full(p, c, qs, seq)
        os_, ls = torch.empty_like(o), torch.empty_like(lse)
        hs.hs_decode_step_quant(p, c.kv, None, hs.HS_DECODE_SPARSE, qs, seq, idx, cnt, os_, ls)
        outs.append([o.float() * 2.0 ** -s, os_.float() * 2.0 ** -s, lse, ls, idx, sel])
    assert hs.hs_device_status() == 0
    assert torch.isfinite(outs[0][0]).all() and (outs[0][0] != 0).any()
    for x, y in zip(*outs):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", FMTS)
def test_extreme_logits(fmt):
    """Logits of thousands of both signs: one key takes all of the weight."""
    p = _params(1, 16, 1, 128, 1, 3000, k=64, window=0)
    c = _filled(p, fmt, 0, 115)
    q = _randn(1, 16, 1, 128, seed=116, std=300.0)
    seq = torch.tensor([3000], dtype=torch.int32, device=DEV)
    o, lse, idx, _, _ = _full(p, c, q, seq)
    kd, vd = (x[0, 0] for x in c.values())
    a = q[0, :, 0].double().cpu().numpy() @ kd.T / 128 ** 0.5
    assert np.abs(a).max() > 1000
    want = np.logaddexp.reduce(a, 1)
    # lse in fp32 from logits that are sums of 128 fp32 terms of up to |q||k| each
    tol = 128 * 2.0 ** -23 * np.abs(q[0, :, 0].double().cpu().numpy()) @ np.abs(kd).max(0) / 128 ** 0.5
    assert (np.abs(lse.cpu().double().numpy()[0, :, 0] - want) <= tol + 1e-3).all()
    best = a.argmax(1)
    assert set(best.tolist()) <= set(idx[0, 0].tolist())
    gap = np.sort(a, 1)
    for h in np.nonzero(gap[:, -1] - gap[:, -2] > 30)[0]:  # e^-30: no other key shows
        got = P.f64(o)[0, h, 0]
        assert (np.abs(got - vd[best[h]]) <= 2.0 ** -7 * np.abs(vd[best[h]]) + 2.0 ** -10).all()


def test_tensors_that_the_binding_refuses(monkeypatch):
    p = _params(1, 8, 1, 64, 4, 16)
    c = Cache(p, "int4")
    k = _randn(1, 1, 4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        hs.hs_kv_quant_write(p, c.kv, None, k.cpu(), k)
    with pytest.raises(ValueError, match="contiguous"):
        hs.hs_kv_quant_write(p, c.kv, None, k.transpose(2, 3), k)
    monkeypatch.setattr(hs, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_kv_quant_write(p, c.kv, None, k, k, stream=0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq", [5, 16])
def test_any_codes_and_entries(fmt, hq):
    """Caches that hs_kv_quant_write would not write: every code, scales of both signs and zero,
    zero points in both formats; and a scale argument of the caller's."""
    p = _params(2, hq, 1, 128, 1, 1500, k=80, window=16, scale=0.03)
    c = Cache(p, fmt)
    g = torch.Generator().manual_seed(120)
    for codes, entry in (c.t[:2], c.t[2:]):
        x = torch.randint(0, 256, codes.shape, generator=g)
        if fmt == "fp8":
            x = torch.where(x % 128 == 127, x - 1, x)  # not NaN
        codes.copy_(x.to(torch.uint8))
        e = torch.randn(entry.shape, generator=g) * torch.tensor([0.2 if fmt == "int4" else 0.005, 0.5])
        e[:, :, ::7, 0] = 0
        entry.copy_(e.bfloat16())
    q = _randn(2, hq, 1, 128, seed=121)
    seq = torch.tensor([1500, 700], dtype=torch.int32, device=DEV)
    o, lse, idx, cnt, _ = _full(p, c, q, seq)
    os_, ls = torch.empty_like(o), torch.empty_like(lse)
    hs.hs_decode_step_quant(p, c.kv, None, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, os_, ls)
    assert hs.hs_device_status() == 0
    kd, vd = c.values()
    for b, L in enumerate(seq.tolist()):
        a = 0.03 * (q[b, :, 0].double().cpu().numpy() @ kd[b, 0, :L].T)
        l = np.logaddexp.reduce(a, 1)
        w = np.exp(a - l[:, None])
        P.check_lse(lse.cpu().double().numpy()[b, :, 0], l, "bf16", "lse")
        # p scale is rounded to fp16, 2^-12 of each term p scale c; the output to bf16
        z = c.t[3][b, 0, :, 1].double().cpu().numpy()[:, None]
        size = np.abs(vd[b, 0] - z) + np.abs(z)
        mag = w @ size[:L]
        want = w @ vd[b, 0, :L]
        err = np.abs(P.f64(o)[b, :, 0] - want)
        assert (err <= 2.0 ** -11 * mag + 2.0 ** -8 * np.abs(want) + 1e-6).all()
        got = idx[b, 0].cpu().numpy()
        score = (a - l[:, None]).max(0)
        kth = np.sort(score[:L - 16])[-64]
        assert int(cnt[b, 0]) == 80 and (score[got[:64]] >= kth - P.INDEX_REL).all()
        at = a[:, got]
        P.check_lse(ls.cpu().double().numpy()[b, :, 0], np.logaddexp.reduce(at, 1), "bf16", "sparse lse")
        w = np.exp(at - np.logaddexp.reduce(at, 1)[:, None])
        err = np.abs(P.f64(os_)[b, :, 0] - w @ vd[b, 0, got])
        assert (err <= 2.0 ** -11 * (w @ size[got]) + 2.0 ** -8 * np.abs(w @ vd[b, 0, got]) + 1e-6).all()


def test_long_diffuse_attention_in_4_bits():
    """131072 keys of nearly equal weight, many to a warp: what is left of the codes' mean once
    the zero points are in is a 900th of it, and is held to the usual bar."""
    b, hq, hkv, d, T = 32, 64, 4, 128, 131072
    p = _params(b, hq, hkv, d, 1, T, k=64, window=8)
    gen = torch.Generator(DEV).manual_seed(130)
    t = hs.kv_quant_cache(p, "int4", DEV)
    for codes, entry in (t[:2], t[2:]):
        codes.random_(0, 256, generator=gen)
        entry[..., 0], entry[..., 1] = 0.3125, -0.3125 * 7.5
    q = _randn(b, hq, 1, d, seed=131, std=0.3)
    seq = torch.full((b,), T, dtype=torch.int32, device=DEV)
    idx, cnt, o, lse, _ = _decode_outputs(p)
    hs.hs_decode_step_quant(p, hs.make_kv_quant("int4", *t), None, hs.HS_DECODE_FULL_INDEX, q, seq,
                            idx, cnt, o, lse, None, hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT))
    assert hs.hs_device_status() == 0
    for i, u in ((0, 0), (13, 2), (31, 3)):
        k, v = ((torch.stack([c[i, u] & 15, c[i, u] >> 4], -1).flatten(1).double() - 7.5) * 0.3125
                for c in (t[0], t[2]))
        heads = slice(u * 16, (u + 1) * 16)
        a = q[i, heads, 0].double() @ k.T / d ** 0.5
        l = torch.logsumexp(a, -1)
        want = torch.exp(a - l[:, None]) @ v
        P.check_o(P.f64(o[i, heads, 0]), P.f64(want), "bf16", "o")
        P.check_lse(P.f64(lse[i, heads, 0]), P.f64(l), "bf16", "lse")
