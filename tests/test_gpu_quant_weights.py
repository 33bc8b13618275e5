"""Attention over 4-bit rows where many keys have equal weights that fp16 rounds:
what the codes' mean and the zero points cancel to is held to the usual bar.

The kernels round p_i scale_i to fp16, to at most 2^-12 of itself.  With that
error common to the keys of one scale, the outputs may be off by 2^-12 of what
the values' own sum is, however large the codes' and the zero points' sums are
beside it; the bar (1.5e-2 of the output's RMS and half its ulp, tests/parity.py)
leaves room for the sums' order.
"""
import numpy as np
import pytest
import torch

from oracle_top_kv_b200 import hs
from tests import parity as P
from tests.test_gpu_quant import DEV, _decode_outputs, _params

pytestmark = pytest.mark.gpu

HEADS = 16


def _equal_keys(T, skew, seed):
    """A 4-bit cache of one unit whose keys have one of two logits each, every 32nd the larger;
    Gaussian or one-sided values of mean 0.  The larger logit over the others' is 2.8 to 3.8 in
    the log2 domain, by head."""
    gen = torch.Generator(DEV).manual_seed(seed)
    p = _params(1, HEADS, 1, 128, 1, T, k=64, window=0)
    t = hs.kv_quant_cache(p, "int4", DEV)
    kv = hs.make_kv_quant("int4", *t)
    v = torch.randn(1, 1, T, 128, generator=gen, device=DEV)
    if skew:
        v.exponential_(generator=gen).sub_(1)
    hs.hs_kv_quant_write(_params(1, HEADS, 1, 128, T, T), kv, None, torch.zeros_like(v).bfloat16(),
                         v.bfloat16())
    del v
    t[1][0, 0, ::32, 1] = 0.25
    gap = 2.8 + torch.arange(HEADS, device=DEV) / (HEADS - 1)
    q = (gap * np.log(2) * 128 ** 0.5 / (128 * 0.25)).bfloat16()[None, :, None, None]
    return p, kv, t, q.expand(1, HEADS, 1, 128).contiguous()


def _want(t, q, rows):
    """o [heads, d] and lse [heads] over the rows, in 64 bits."""
    c, e = t[2][0, 0, rows], t[3][0, 0, rows].double()
    v = torch.stack([c & 15, c >> 4], -1).flatten(1).double() * e[:, :1] + e[:, 1:]
    a = q[0, :, 0].double().sum(-1, keepdim=True) * t[1][0, 0, rows, 1].double() / 128 ** 0.5
    l = torch.logsumexp(a, -1)
    return torch.exp(a - l[:, None]) @ v, l


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("T", [16384, 131072, 1 << 20])
def test_full_step_over_equal_keys(T, skew):
    p, kv, t, q = _equal_keys(T, skew, 301)
    seq = torch.tensor([T], dtype=torch.int32, device=DEV)
    idx, cnt, o, lse, _ = _decode_outputs(p)
    hs.hs_decode_step_quant(p, kv, None, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse, None,
                            hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT))
    assert hs.hs_device_status() == 0
    want, l = _want(t, q, slice(0, T))
    P.check_lse(P.f64(lse)[0, :, 0], P.f64(l), "bf16", "lse")
    P.check_o(P.f64(o)[0, :, 0], P.f64(want), "bf16", "o")
    assert torch.equal(idx[0, 0].long(), torch.arange(64, device=DEV) * 32)


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("decode", [False, True])
def test_sparse_layers_over_equal_keys(decode, skew):
    T, k = 131072, 4096
    _, kv, t, q = _equal_keys(T, skew, 302)
    first = T - 32 * 40
    rows = torch.arange(0, k, device=DEV) * (first // k)
    rows[::32] = rows[::32] // 32 * 32  # the larger ones
    rows = rows.unique()
    idx = torch.full((1, 1, k), -1, dtype=torch.int32, device=DEV)
    idx[0, 0, :len(rows)] = rows.int()
    cnt = torch.full((1, 1), len(rows), dtype=torch.int32, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(1, HEADS, 1, device=DEV)
    if decode:
        p = _params(1, HEADS, 1, 128, 1, T, k=k, window=0)
        seq = torch.tensor([T], dtype=torch.int32, device=DEV)
        hs.hs_decode_step_quant(p, kv, None, hs.HS_DECODE_SPARSE, q, seq, idx, cnt, o, lse)
    else:
        p = _params(1, HEADS, 1, 128, 1, T, k=k, window=0, q_offset=T - 1)
        hs.hs_sparse_attn_reuse_quant(p, kv, None, q, idx[:, :, None], cnt[:, :, None], o, lse)
    assert hs.hs_device_status() == 0
    want, l = _want(t, q, rows)
    P.check_lse(P.f64(lse)[0, :, 0], P.f64(l), "bf16", "lse")
    P.check_o(P.f64(o)[0, :, 0], P.f64(want), "bf16", "o")


def test_zero_points_of_8_bit_rows_over_equal_keys():
    """e4m3 rows of codes of one sign whose zero points take their mean away: held to what
    include/hs.h states, 2^-12 of each key's weight on scale c (and as much again for the
    sums), not to what is left of it."""
    T = 131072
    gen = torch.Generator(DEV).manual_seed(303)
    p = _params(1, HEADS, 1, 128, 1, T, k=64, window=0)
    t = hs.kv_quant_cache(p, "fp8", DEV)
    t[2].random_(0x70, 0x7f, generator=gen)  # 128 .. 448
    t[3][..., 0], t[3][..., 1] = 0.01, -2.5
    t[1][0, 0, ::32, 1] = 0.25
    gap = 2.8 + torch.arange(HEADS, device=DEV) / (HEADS - 1)
    q = (gap * np.log(2) * 128 ** 0.5 / (128 * 0.25)).bfloat16()[None, :, None, None].expand(
        1, HEADS, 1, 128).contiguous()
    seq = torch.tensor([T], dtype=torch.int32, device=DEV)
    idx, cnt, o, lse, _ = _decode_outputs(p)
    hs.hs_decode_step_quant(p, hs.make_kv_quant("fp8", *t), None, hs.HS_DECODE_FULL_INDEX, q, seq,
                            idx, cnt, o, lse, None, hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT))
    assert hs.hs_device_status() == 0
    c = t[2][0, 0].view(torch.float8_e4m3fn).double()
    e = t[3][0, 0].double()
    a = q[0, :, 0].double().sum(-1, keepdim=True) * t[1][0, 0, :, 1].double() / 128 ** 0.5
    l = torch.logsumexp(a, -1)
    P.check_lse(P.f64(lse)[0, :, 0], P.f64(l), "bf16", "lse")
    w = torch.exp(a - l[:, None])
    want = w @ (c * e[:, :1] + e[:, 1:])
    bound = 2.0 ** -11 * (w @ (c * e[:, :1]).abs()) + 2.0 ** -8 * want.abs() + 1e-6
    assert ((o[0, :, 0].double() - want).abs() <= bound).all()
