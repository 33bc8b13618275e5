"""GPU parity of the quantised K^F/V^F cache: rows written and read back, the
decode steps and the sparse prefill layer over them.

Rows are compared with quant_ref (equal codes, scales and zeros); attention is
compared with the fp64 oracle on the values that the stored codes stand for,
under the bars of tests/parity.py.  These cover what the kernels round: q and
the codes enter the products exactly, p_i scale_i is rounded to fp16 (2^-12 of
each term: against an output of independent terms at most a few 2^-12 of its
RMS, below 1.5e-2), the output once more (the half ulp).
"""
import numpy as np
import pytest
import torch

import oracle
from oracle_top_kv_b200 import hs
from oracle_top_kv_b200 import workloads as wl
from tests import parity as P
from tests import quant_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = ["int4", "fp8"]


class Cache:
    """A quantised cache, contiguous (page = 0) or paged with a shuffled table."""

    def __init__(self, p, fmt, page=0, seed=0, junk=False):
        self.p, self.fmt, self.page = p, fmt, page
        gen = torch.Generator().manual_seed(seed)
        self.table = self.pages = None
        n_pages = 0
        if page:
            mp = p.t_kv // page
            n_pages = p.batch * mp + 2
            self.table = torch.randperm(n_pages, generator=gen)[:p.batch * mp].view(
                p.batch, mp).int().to(DEV)
            self.pages = hs.make_pages(self.table, page, n_pages)
        self.t = hs.kv_quant_cache(p, fmt, DEV, page, n_pages)
        if junk:  # NaN entries and any codes in rows that nobody wrote
            for codes, entry in (self.t[:2], self.t[2:]):
                codes.copy_(torch.randint(0, 256, codes.shape, generator=gen).to(torch.uint8))
                entry.fill_(float("nan"))
        self.kv = hs.make_kv_quant(fmt, *self.t)

    def write(self, k, v, seq=None, n_new=None, p=None):
        hs.hs_kv_quant_write(p or self.p, self.kv, self.pages, k, v, seq, n_new)

    def values(self):
        """Logical K and V [b, hkv, t_kv, d], float64."""
        out = []
        for codes, entry in (self.t[:2], self.t[2:]):
            x = R.values(codes, entry, self.fmt)
            out.append(oracle.gather_pages(x, self.table, self.page) if self.page else x)
        return out


def _randn(*shape, seed=0, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def _params(batch, hq, hkv, d, t_q, t_kv, k=64, window=8, **kw):
    kw.setdefault("mode", "token")
    kw.setdefault("block_size", 1)
    return hs.make_params(batch, hq, hkv, d, t_q, t_kv, k=k, window=window, **kw)


# ------------------------------------------------------------------- rows
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 24])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_written_and_read_back(fmt, d, page, dtype):
    b, hkv, t_q, T = 3, 2, 21, 96
    p = _params(b, 4, hkv, d, t_q, T, dtype="bf16" if dtype == torch.bfloat16 else "fp32")
    c = Cache(p, fmt, page, seed=d)
    before = [x.clone() for x in c.t]
    k, v = (_randn(b, hkv, t_q, d, seed=s, dtype=torch.bfloat16).to(dtype) for s in (1, 2))
    seq = torch.tensor([96, 21, 30], dtype=torch.int32, device=DEV)
    n_new = torch.tensor([5, 21, 0], dtype=torch.int32, device=DEV)  # padded batch
    c.write(k, v, seq, n_new)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    hs.hs_kv_quant_read(p, c.kv, c.pages, ko, vo, seq, n_new)
    assert hs.hs_device_status() == 0
    back = c.values()
    old = Cache(p, fmt, page, seed=d).values()
    for x, out, logical, was in ((k, ko, back[0], old[0]), (v, vo, back[1], old[1])):
        for i in range(b):
            n, L = int(n_new[i]), int(seq[i])
            cw, s, z = R.encode(x[i, :, :n].double().cpu().numpy(), fmt)
            want = cw * s[..., None] + z[..., None]
            assert np.array_equal(logical[i, :, L - n:L], want)
            # read back: one rounding of scale * c + zero (after fp32: 2^-24 more)
            got = out[i, :, :n].double().cpu().numpy()
            eps = (2.0 ** -8 if dtype == torch.bfloat16 else 0) + 2.0 ** -23
            # |scale c| + |zero| bounds what fp32 rounded
            mag = np.abs(cw * s[..., None]) + np.abs(z[..., None])
            assert (np.abs(got - want) <= (eps - 2.0 ** -23) * np.abs(want) + 2.0 ** -23 * mag).all()
            assert (out[i, :, n:] == 7).all()           # padding rows stay
            keep = np.ones(T, bool)
            keep[L - n:L] = False
            assert np.array_equal(logical[i, :, keep], was[i, :, keep])  # so do other rows
    if page:  # pages that no sequence owns
        free = np.setdiff1d(np.arange(c.t[0].shape[0]), c.table.cpu().numpy().ravel())
        for now, was in zip(c.t, before):
            assert torch.equal(now[free], was[free])


@pytest.mark.parametrize("fmt", FMTS)
def test_fp32_rows_follow_ieee_fp32(fmt):
    """fp32 rows: the codes of the stated fp32 arithmetic, replayed by torch on the CPU."""
    p = _params(1, 2, 1, 128, 300, 300, dtype="fp32")
    c = Cache(p, fmt)
    k, v = (_randn(1, 1, 300, 128, seed=s, dtype=torch.float32, std=10.0 ** (s - 3)) for s in (3, 9))
    c.write(k, v)
    for x, codes, entry in ((k, *c.t[:2]), (v, *c.t[2:])):
        x = x.cpu()
        if fmt == "int4":
            lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            s, z = ((hi - lo) / 15).bfloat16().float(), lo.bfloat16().float()
            want = ((x - z) / s).round().clamp(0, 15)
        else:
            s = (x.abs().amax(-1, keepdim=True) / 448).bfloat16().float()
            z = torch.zeros_like(s)
            want = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(entry.float().cpu(), torch.cat([s, z], -1))
        assert np.array_equal(R.codes_of(codes, fmt), want.double().numpy())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_special_rows(fmt, d):
    rows = [torch.zeros(d), torch.full((d,), -2.5), torch.ones(d), torch.ones(d), torch.ones(d),
            torch.linspace(-1, 1, d) * 1e-38, torch.linspace(-1, 1, d) * 3e38,
            torch.linspace(100, 101, d)]
    rows[2][5] = float("nan")
    rows[3][d - 1] = float("inf")
    rows[4][0] = float("-inf")
    x = torch.stack(rows)[None, None].bfloat16().to(DEV)
    p = _params(1, 2, 1, d, len(rows), len(rows))
    c = Cache(p, fmt)
    c.write(x, x.flip(2).contiguous())
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    hs.hs_kv_quant_read(p, c.kv, None, ko, vo)
    assert hs.hs_device_status() == 0
    ref = x[0, 0].double().cpu().numpy()
    for out in (ko, vo.flip(2)):
        got = out[0, 0].double().cpu().numpy()
        assert (got[0] == 0).all()
        if fmt == "int4":
            assert (got[1] == -2.5).all()
        assert np.isnan(got[2:5]).all()
        if fmt == "int4":
            assert np.isnan(got[6]).all()  # max - min overflows fp32
            live = [5, 7]
        else:
            live = [1, 5, 6, 7]
        cw, s, z = R.encode(ref, fmt)
        want = cw * s[:, None] + z[:, None]
        for i in live:
            # row 5: scale and products are subnormal, steps of 2^-133 in bf16
            tol = 2.0 ** -8 * np.abs(want[i]) + 2.0 ** -130
            assert (np.abs(got[i] - want[i]) <= tol).all(), i


@pytest.mark.parametrize("fmt", FMTS)
def test_write_with_defaults_appends_a_chunk(fmt):
    p = _params(2, 4, 2, 128, 7, 40, q_offset=11)
    c = Cache(p, fmt)
    k, v = _randn(2, 2, 7, 128, seed=4), _randn(2, 2, 7, 128, seed=5)
    c.write(k, v)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    hs.hs_kv_quant_read(p, c.kv, None, ko, vo)
    cw, s, z = R.encode(k.double().cpu().numpy(), fmt)
    want = cw * s[..., None] + z[..., None]
    assert np.array_equal(c.values()[0][:, :, 11:18], want)
    assert (c.t[1][:, :, :11] == 0).all() and (c.t[1][:, :, 18:] == 0).all()


def test_bad_lengths_and_pages_are_skipped():
    p = _params(4, 4, 2, 64, 3, 32)
    k, v = _randn(4, 2, 3, 64, seed=6), _randn(4, 2, 3, 64, seed=7)
    seq = torch.tensor([33, 2, 10, 12], dtype=torch.int32, device=DEV)
    n_new = torch.tensor([3, 3, 4, 3], dtype=torch.int32, device=DEV)
    c = Cache(p, "int4")
    c.write(k, v, seq, n_new)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert (c.t[0][:3] == 0).all() and (c.t[1][3, :, 9:12] != 0).any(-1).all()
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    hs.hs_kv_quant_read(p, c.kv, None, ko, vo, seq, n_new)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert (ko[:3] == 7).all() and (vo[:3] == 7).all() and (ko[3] != 7).any()
    c = Cache(p, "fp8", page=8)
    c.table[3, 1] = 1 << 20
    c.write(k, v, torch.full_like(seq, 12), torch.full_like(seq, 3))
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert hs.hs_device_status() == 0


# ----------------------------------------------------------------- attention
def _filled(p, fmt, page, seed, q=None, needles=0, lens=None):
    """A cache of t_kv Gaussian rows, some of them needles of the queries q; what lies behind
    lens[b] is junk."""
    c = Cache(p, fmt, page, seed=seed, junk=True)
    w = wl.Workload("quant", p.batch, p.hq, p.hkv, p.head_dim, p.t_kv, "bf16", "token", 1, p.k,
                    p.window, 1, False, 1.0, 1.0, "decode:1")
    k = _randn(w.batch, w.hkv, w.t, w.head_dim, seed=seed + 1)
    v = _randn(w.batch, w.hkv, w.t, w.head_dim, seed=seed + 2)
    if q is not None:
        g = torch.Generator().manual_seed(seed)
        for b in range(p.batch):
            for u in range(p.hkv):
                for i in torch.randperm(p.t_kv, generator=g)[:needles].tolist():
                    h = u * w.group + int(torch.randint(0, w.group, (1,), generator=g))
                    k[b, u, i] = (q[b, h, 0].float() * (10 / p.head_dim ** 0.5)).bfloat16()
    pw = _params(p.batch, p.hq, p.hkv, p.head_dim, p.t_kv, p.t_kv)
    if lens is None:
        c.write(k, v, p=pw)
    else:
        c.write(k, v, lens, lens.clone(), p=pw)
    return c


def _decode_outputs(p):
    return (torch.full((p.batch, p.hkv, p.ksel), -7, dtype=torch.int32, device=DEV),
            torch.empty(p.batch, p.hkv, dtype=torch.int32, device=DEV),
            torch.empty(p.batch, p.hq, 1, p.head_dim, dtype=torch.bfloat16, device=DEV),
            torch.empty(p.batch, p.hq, 1, dtype=torch.float32, device=DEV),
            torch.full((p.batch, p.hkv, p.ksel), -7.0, dtype=torch.float32, device=DEV))


DECODE = [
    # batch, hq, hkv, d, t_kv, k, window, page, lengths
    (4, 32, 2, 128, 3008, 256, 64, 0, [3008, 1, 777, 2049]),
    (4, 32, 2, 128, 3000, 256, 64, 24, [3000, 1, 777, 2049]),
    (3, 8, 2, 64, 700, 40, 0, 0, [700, 41, 40]),          # no window; one past the budget
    (2, 6, 2, 64, 512, 33, 33, 16, [512, 100]),           # window only
    (2, 15, 1, 128, 1111, 17, 16, 0, [1111, 18]),         # odd group, one ranked key
    (1, 16, 1, 128, 40000, 1024, 128, 0, [39999]),        # many slices
    (1, 4, 1, 128, 20000, 1500, 100, 0, [20000]),         # k - w > 1024
    (5, 7, 7, 128, 100, 300, 10, 0, [1, 31, 32, 33, 100]),  # everything selected, groups of one
    (1, 16, 1, 64, 9000, 4096, 0, 0, [9000]),               # the largest budget, no window
    (2, 3, 1, 128, 70000, 64, 16, 16, [70000, 66001]),      # units on clusters, small group
    (40, 4, 2, 64, 96, 16, 4, 16, [(7 * i) % 96 + 1 for i in range(40)]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", DECODE)
def test_decode_steps(fmt, case):
    b, hq, hkv, d, T, k, w, page, lens = case
    p = _params(b, hq, hkv, d, 1, T, k=k, window=w)
    q, qs = _randn(b, hq, 1, d, seed=11), _randn(b, hq, 1, d, seed=12)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c = _filled(p, fmt, page, 20, q, needles=12, lens=seq)
    ws = hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT)
    ws.fill_(0xFF)  # nothing may rest on what the workspace held
    idx, cnt, o, lse, sel = _decode_outputs(p)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse,
                            sel, ws)
    os_, ls = torch.empty_like(o), torch.empty_like(lse)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_SPARSE, qs, seq, idx, cnt, os_, ls)
    assert hs.hs_device_status() == 0
    kd, vd = c.values()
    rows = np.array([[i, u, 0] for i in range(b) for u in range(hkv)], np.int32)
    pos = np.array(lens)[rows[:, 0]] - 1
    g = hq // hkv
    orc = oracle.full_attn_rows(q.double().cpu().numpy(), kd, vd, rows, pos, "token", 1, k, w)
    P.check_o(P.gpu_rows(P.f64(o), rows, True, g), orc["o"], "bf16", "full o")
    P.check_lse(P.gpu_rows(lse.cpu().double().numpy(), rows, True, g), orc["lse"], "bf16", "lse")
    g_idx, g_cnt = idx.cpu().numpy()[rows[:, 0], rows[:, 1]], cnt.cpu().numpy()[rows[:, 0], rows[:, 1]]
    P.check_index(g_idx, g_cnt, orc, "token", w, k, "index")
    got = sel.cpu().double().numpy()[rows[:, 0], rows[:, 1]]
    for n in range(len(rows)):
        want = orc["scores"][n][g_idx[n, :g_cnt[n]]]
        # p = 2^(a - lse): an error of 1e-4 in the exponent's natural log
        assert np.abs(got[n, :g_cnt[n]] / want - 1).max() < 2e-4
        assert (got[n, g_cnt[n]:] == 0).all()
    sp = oracle.sparse_attn_rows(qs.double().cpu().numpy(), kd, vd, g_idx, g_cnt, rows, pos,
                                 "token", 1, k, w)
    P.check_o(P.gpu_rows(P.f64(os_), rows, True, g), sp["o_g"], "bf16", "sparse o")
    P.check_lse(P.gpu_rows(ls.cpu().double().numpy(), rows, True, g), sp["lse_g"], "bf16", "sparse lse")


REUSE = [
    # batch, hq, hkv, d, t_q, q_offset, t_kv, mode, block, k, window, page
    (1, 32, 2, 128, 70, 630, 700, "token", 1, 96, 32, 0),
    (2, 8, 2, 64, 33, 0, 48, "token", 1, 20, 5, 16),
    (2, 8, 2, 128, 40, 600, 640, "block", 64, 256, 0, 0),
    (1, 12, 1, 128, 25, 500, 576, "block", 16, 128, 0, 48),
    (1, 5, 5, 64, 9, 1, 10, "token", 1, 300, 0, 0),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", REUSE)
def test_sparse_prefill(fmt, case):
    b, hq, hkv, d, t_q, off, T, mode, B, k, w, page = case
    p = _params(b, hq, hkv, d, t_q, T, k=k, window=w, mode=mode, block_size=B, q_offset=off)
    c = _filled(p, fmt, page, 30)
    q = _randn(b, hq, t_q, d, seed=31)
    gen = np.random.default_rng(5)
    ksel = p.ksel
    idx = np.full((b, hkv, t_q, ksel), -1, np.int32)
    cnt = np.zeros((b, hkv, t_q), np.int32)
    for i in np.ndindex(b, hkv, t_q):
        seen = (off + i[2]) // B + 1
        n = min(seen, ksel, int(gen.integers(0, ksel + 1)))
        idx[i][:n] = np.sort(gen.choice(seen, n, replace=False))
        cnt[i] = n
    cnt[0, 0, 0] = 0  # an empty set: o = 0, lse = -inf
    o, lse = torch.empty_like(q), torch.empty(b, hq, t_q, dtype=torch.float32, device=DEV)
    hs.hs_sparse_attn_reuse_quant(p, c.kv, c.pages, q, torch.tensor(idx, device=DEV),
                                  torch.tensor(cnt, device=DEV), o, lse)
    assert hs.hs_device_status() == 0
    kd, vd = c.values()
    rows = np.array(list(np.ndindex(b, hkv, t_q)), np.int32)
    sp = oracle.sparse_attn_rows(q.double().cpu().numpy(), kd, vd, idx.reshape(-1, ksel),
                                 cnt.reshape(-1), rows, off + rows[:, 2], mode, B, k, w)
    g = hq // hkv
    P.check_o(P.gpu_rows(P.f64(o), rows, True, g), sp["o_g"], "bf16", "o")
    P.check_lse(P.gpu_rows(lse.cpu().double().numpy(), rows, True, g), sp["lse_g"], "bf16", "lse")


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_sequences_pages_and_indices(fmt):
    p = _params(3, 8, 2, 64, 1, 64, k=16, window=4)
    q = _randn(3, 8, 1, 64, seed=41)
    c = _filled(p, fmt, 16, 40)
    ws = hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT)
    idx, cnt, o, lse, sel = _decode_outputs(p)
    seq = torch.tensor([0, 65, 64], dtype=torch.int32, device=DEV)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse,
                            sel, ws)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert (o[:2] == 0).all() and torch.isneginf(lse[:2]).all() and (cnt[:2] == 0).all()
    assert (idx[:2] == -1).all() and (sel[:2] == 0).all() and (cnt[2] == 16).all()
    os_, ls = torch.empty_like(o), torch.empty_like(lse)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, os_, ls)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert (os_[:2] == 0).all() and torch.isneginf(ls[:2]).all() and torch.isfinite(ls[2]).all()
    # a key past the sequence, and a page outside the pool: those rows are left out
    seq = torch.tensor([20, 20, 20], dtype=torch.int32, device=DEV)
    idx.copy_(torch.arange(16, device=DEV).expand_as(idx))
    cnt.fill_(16)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, os_, ls)
    assert hs.hs_device_status() == 0
    idx[0, 0, 3], idx[0, 1, 5] = 20, -4
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, o, lse)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert (lse[0] < ls[0]).all() and torch.equal(lse[1:], ls[1:])
    c.table[1, 0] = -1
    idx.copy_(torch.arange(4, 20, device=DEV).expand_as(idx))
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, o, lse)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse,
                            None, ws)
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_nan_row_shows_and_only_where_it_is_read(fmt):
    p = _params(2, 8, 2, 128, 1, 128, k=16, window=4)
    q = _randn(2, 8, 1, 128, seed=51)
    c = _filled(p, fmt, 0, 50)
    c.t[1][0, 1, 77] = float("nan")  # one K entry of sequence 0, kv head 1
    seq = torch.tensor([128, 77], dtype=torch.int32, device=DEV)
    c.t[1][1, :, 77:] = float("nan")
    c.t[3][1, :, 77:] = float("nan")  # behind the end of sequence 1
    ws = hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT)
    idx, cnt, o, lse, _ = _decode_outputs(p)
    hs.hs_decode_step_quant(p, c.kv, None, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse, None, ws)
    assert torch.isnan(o[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(o[0, :4]).all() and torch.isfinite(o[1]).all()


# ------------------------------------------------------------- as it is used
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [0, 16])
def test_a_generation_on_a_side_stream_and_in_a_graph(fmt, page):
    """A prompt is stored, then per token: append, full step, two sparse steps; the same steps
    captured once and replayed give the same bits, on a stream of their own."""
    b, hq, hkv, d, T, k, w = 3, 16, 2, 128, 192, 32, 8
    p = _params(b, hq, hkv, d, 1, T, k=k, window=w)
    n0 = torch.tensor([100, 37, 64], dtype=torch.int32, device=DEV)
    pp = _params(b, hq, hkv, d, 100, T)
    kp, vp = _randn(b, hkv, 100, d, seed=60), _randn(b, hkv, 100, d, seed=61)
    steps = 4
    new = [[_randn(b, hkv, 1, d, seed=70 + 10 * s + i) for i in range(2)] +
           [_randn(b, hq, 1, d, seed=75 + 10 * s + i) for i in range(3)] for s in range(steps)]
    st = torch.cuda.Stream()
    results = []
    for mode in ("eager", "graph"):
        c = Cache(p, fmt, page, seed=3, junk=True)
        ws = hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT)
        buf = [x.clone() for x in new[0]]
        seq = n0.clone()
        idx, cnt, o, lse, _ = _decode_outputs(p)
        outs = [o, lse, idx, cnt] + [torch.empty_like(o) for _ in range(2)]

        def token():
            c_kv = c.kv
            hs.hs_kv_quant_write(p, c_kv, c.pages, buf[0], buf[1], seq)
            hs.hs_decode_step_quant(p, c_kv, c.pages, hs.HS_DECODE_FULL_INDEX, buf[2], seq, idx,
                                    cnt, o, lse, None, ws)
            for i in range(2):
                hs.hs_decode_step_quant(p, c_kv, c.pages, hs.HS_DECODE_SPARSE, buf[3 + i], seq,
                                        idx, cnt, outs[4 + i])

        graph = None
        seen = []
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            c.write(kp, vp, n0, n0.clone(), p=pp)
            if mode == "graph":
                seq.copy_(n0 + 1)
                graph = torch.cuda.CUDAGraph()
                st.synchronize()
                with torch.cuda.graph(graph, stream=st):
                    token()
            for s in range(steps):
                for dst, src in zip(buf, new[s]):
                    dst.copy_(src)
                seq.copy_(n0 + 1 + s)
                if graph is None:
                    token()
                else:
                    graph.replay()
                seen.append([x.clone() for x in outs])
        st.synchronize()
        assert hs.hs_device_status() == 0
        results.append(seen)
        del graph
    for a, g in zip(*results):
        for x, y in zip(a, g):
            assert torch.equal(x, y)
    # the last token against the oracle
    kd, vd = c.values()
    o, lse, idx, cnt, o1, _ = results[1][-1]
    rows = np.array([[i, u, 0] for i in range(b) for u in range(hkv)], np.int32)
    pos = (n0.cpu().numpy() + steps - 1)[rows[:, 0]]
    g = hq // hkv
    orc = oracle.full_attn_rows(new[-1][2].double().cpu().numpy(), kd, vd, rows, pos, "token", 1, k, w)
    P.check_o(P.gpu_rows(P.f64(o), rows, True, g), orc["o"], "bf16", "o")
    g_idx, g_cnt = idx.cpu().numpy()[rows[:, 0], rows[:, 1]], cnt.cpu().numpy()[rows[:, 0], rows[:, 1]]
    P.check_index(g_idx, g_cnt, orc, "token", w, k, "index")
    sp = oracle.sparse_attn_rows(new[-1][3].double().cpu().numpy(), kd, vd, g_idx, g_cnt, rows,
                                 pos, "token", 1, k, w)
    P.check_o(P.gpu_rows(P.f64(o1), rows, True, g), sp["o_g"], "bf16", "sparse o")


@pytest.mark.parametrize("fmt", FMTS)
def test_chunked_prefill_on_rows_read_back(fmt):
    """A chunk is stored, the prefix read back in bf16 and the full layer run on it; its sparse
    layer reads the codes."""
    w = wl.scaled(wl.WORKLOADS["hysparse2_prefill"], name="quant_chunk", hq=32, hkv=2, t=400,
                  k=64, window=16)
    q, k, v, _ = wl.full_layer_inputs(w)
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    p = P.abi_params(w)
    c = Cache(p, fmt)
    c.write(k, v)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    hs.hs_kv_quant_read(p, c.kv, None, kb, vb)
    o, lse, idx, cnt, _ = hs.full_outputs(p)
    hs.hs_full_attn_index(p, q, kb, vb, o, lse, idx, cnt)
    qs = wl.sparse_layer_query(w, 0).to(DEV)
    og, lg = torch.empty_like(qs), torch.empty_like(lse)
    hs.hs_sparse_attn_reuse_quant(p, c.kv, None, qs, idx, cnt, og, lg)
    assert hs.hs_device_status() == 0
    kd, vd = c.values()
    rows = P.all_rows(w)[::3]
    g_idx = P.gpu_rows(idx.cpu().numpy(), rows, False)
    g_cnt = P.gpu_rows(cnt.cpu().numpy(), rows, False)
    sp = oracle.sparse_attn_rows(qs.double().cpu().numpy(), kd, vd, g_idx, g_cnt, rows,
                                 rows[:, 2], "token", 1, w.k, w.window)
    P.check_o(P.gpu_rows(P.f64(og), rows, True, w.group), sp["o_g"], "bf16", "o")
    P.check_lse(P.gpu_rows(lg.cpu().double().numpy(), rows, True, w.group), sp["lse_g"], "bf16", "lse")
