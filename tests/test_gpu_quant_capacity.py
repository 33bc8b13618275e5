"""The quantised full step where a sequence ends in the last rows of its capacity
and that is no whole number of the kernels' 32-key steps: index sets against the
fp64 oracle with the best keys among each unit's first 16, and what lies behind
the workspace.  Bars: those of tests/parity.py.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle_top_kv_b200 import build as hsbuild
from oracle_top_kv_b200 import hs
from tests import parity as P

DEV = "cuda"
FMTS = ["int4", "fp8"]


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("hkv", [1, 4, 8, 12])
@pytest.mark.parametrize("t_kv", [1, 16, 33, 2000, 9000, 20016, 100016, 131056, 270001])
def test_workspace_holds_whole_steps(head_dim, hkv, t_kv):
    """A step of 32 keys writes the maxima of both its tiles: a capacity that ends in the first
    of them takes the workspace of one that ends in the second."""
    hsbuild.build()

    def need(t):
        p = hs.make_params(1, 4 * hkv, hkv, head_dim, 1, t, mode="token", block_size=1, k=1, window=0)
        return hs.hs_workspace_size(p, hs.HS_WS_DECODE_FULL_QUANT)

    assert need(t_kv) == need(-(-t_kv // 32) * 32)


def _cache_with_first_keys_best(p, fmt, page, lens, q, seed):
    """Gaussian rows; in every unit keys 0, 5 and 15 are strongly relevant to three of its heads,
    and so is one of its last."""
    from tests.test_gpu_quant import _filled, _randn  # noqa: PLC0415 (their module needs a GPU)
    c = _filled(p, fmt, page, seed, lens=lens)
    g = p.hq // p.hkv
    k, v = (_randn(p.batch, p.hkv, 16, p.head_dim, seed=seed + s) for s in (7, 8))
    for at, h in ((0, 0), (5, g // 2), (15, g - 1)):
        k[:, :, at] = (q[:, h::g, 0].float() * (12 / p.head_dim ** 0.5)).bfloat16()
    first = torch.full_like(lens, 16)
    pw = hs.make_params(p.batch, p.hq, p.hkv, p.head_dim, 16, p.t_kv, mode="token", block_size=1,
                        k=p.k, window=p.window)
    c.write(k, v, first, first.clone(), p=pw)
    return c


def _check(p, c, q, lens, outs):
    o, lse, idx, cnt = outs
    kd, vd = c.values()
    rows = np.array([[i, u, 0] for i in range(p.batch) for u in range(p.hkv)], np.int32)
    pos = lens.cpu().numpy()[rows[:, 0]] - 1
    orc = oracle.full_attn_rows(q.double().cpu().numpy(), kd, vd, rows, pos, "token", 1, p.k, p.window)
    g = p.hq // p.hkv
    P.check_o(P.gpu_rows(P.f64(o), rows, True, g), orc["o"], "bf16", "o")
    P.check_lse(P.gpu_rows(lse.cpu().double().numpy(), rows, True, g), orc["lse"], "bf16", "lse")
    g_idx, g_cnt = idx.cpu().numpy()[rows[:, 0], rows[:, 1]], cnt.cpu().numpy()[rows[:, 0], rows[:, 1]]
    for row in g_idx:
        assert {0, 5, 15} <= set(row.tolist())
    P.check_index(g_idx, g_cnt, orc, "token", p.window, p.k, "index")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", [
    # batch, hq, hkv, d, t_kv, k, window, page, lengths
    (1, 16, 1, 128, 20016, 64, 8, 0, [20016]),
    (1, 64, 4, 128, 20016, 128, 16, 0, [20016]),
    (1, 64, 4, 64, 40016, 128, 0, 0, [40011]),
    (1, 32, 8, 64, 20016, 64, 8, 0, [20016]),
    (1, 32, 8, 128, 20016, 64, 8, 16, [20016]),        # an odd number of pages
    (2, 32, 4, 128, 20016, 64, 8, 48, [20016, 20001]),
    (6, 32, 2, 128, 9000, 256, 32, 0, [8997] * 6),
    (3, 8, 4, 64, 2000, 40, 0, 16, [2000, 1999, 1985]),
])
def test_first_keys_are_selected_at_the_end_of_the_capacity(fmt, case):
    from tests.test_gpu_quant import _decode_outputs, _params, _randn  # noqa: PLC0415
    b, hq, hkv, d, T, k, w, page, lens = case
    p = _params(b, hq, hkv, d, 1, T, k=k, window=w)
    q = _randn(b, hq, 1, d, seed=201)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c = _cache_with_first_keys_best(p, fmt, page, seq, q, 202)
    need = hs.hs_workspace_size(p, hs.HS_WS_DECODE_FULL_QUANT)
    # the workspace is the front of a larger buffer, of which the rest stays as it was
    buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(3):
        idx, cnt, o, lse, sel = _decode_outputs(p)
        hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse,
                                sel, (buf.data_ptr(), need))
        assert hs.hs_device_status() == 0
        assert (buf[need:] == 0xA5).all()
        _check(p, c, q, seq, (o, lse, idx, cnt))
        got = (o, lse, idx, cnt, sel)
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first))
