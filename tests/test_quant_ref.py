"""Pins of the tests' own reference of the quantised rows, and the host-side
checks of the quantised-cache entry points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle_top_kv_b200 import build as hsbuild
from oracle_top_kv_b200 import hs
from tests import quant_ref as R

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails first


def test_e4m3_is_torchs():
    x = torch.linspace(-460, 460, 40001, dtype=torch.float32)
    x = torch.cat([x, x / 448, x * 1e-5])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3(x.double().numpy()), want)


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_reference_is_near_its_input(fmt):
    x = torch.randn(200, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    c, s, z = R.encode(x.double().numpy(), fmt)
    back = c * s[:, None] + z[:, None]
    err = np.abs(back - x.double().numpy())
    if fmt == "int4":
        # half a step, and at the top what rounding scale and zero (2^-9 each) cut off
        span = 15 * s + np.abs(z)
        assert (err <= 0.5 * s[:, None] * (1 + 1e-9) + (span * 2.0 ** -8)[:, None]).all()
    else:
        # half a step of e4m3: 2^-4 of the value, or half the smallest subnormal; and at the
        # top the scale's own rounding
        assert (err <= np.maximum(np.abs(x.double().numpy()) * (2.0 ** -4 + 2.0 ** -9),
                                  s[:, None] * 2.0 ** -10)).all()


def test_reference_special_rows():
    rows = np.stack([np.zeros(8), np.full(8, 3.5), np.r_[np.nan, np.ones(7)],
                     np.r_[np.inf, np.zeros(7)], np.r_[-3e38, 3e38, np.zeros(6)]])
    for fmt in ("int4", "fp8"):
        c, s, z = R.encode(rows, fmt)
        back = c * s[:, None] + z[:, None]
        assert (back[0] == 0).all()
        assert np.isnan(back[2:4]).all()
        if fmt == "int4":
            assert (back[1] == 3.5).all()


@pytest.fixture(scope="module")
def lib():
    hsbuild.build()
    return hs.load()


def _p(**kw):
    base = dict(batch=2, hq=32, hkv=8, head_dim=128, t_q=1, t_kv=1024, dtype="bf16",
                mode="token", block_size=1, k=256, window=32)
    base.update(kw)
    return hs.make_params(**base)


def _kv(fmt=0, **kw):
    a = dict(k_codes=FAKE, k_scale=FAKE, v_codes=FAKE, v_scale=FAKE)
    a.update(kw)
    return hs.hs_kv_quant(fmt, a["k_codes"], a["k_scale"], a["v_codes"], a["v_scale"])


def _calls(lib, p, kv, pages=None, ptr=FAKE, ws=None, ws_bytes=0):
    """The status of every entry point with these arguments."""
    r = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return dict(
        write=lib.hs_kv_quant_write(r(p), r(kv), r(pages), ptr, FAKE, None, None, None),
        read=lib.hs_kv_quant_read(r(p), r(kv), r(pages), ptr, FAKE, None, None, None),
        reuse=lib.hs_sparse_attn_reuse_quant(r(p), r(kv), r(pages), ptr, FAKE, FAKE, FAKE, FAKE,
                                             None),
        full=lib.hs_decode_step_quant(r(p), r(kv), r(pages), 0, ptr, FAKE, FAKE, FAKE, FAKE, FAKE,
                                      None, ws, ws_bytes, None),
        sparse=lib.hs_decode_step_quant(r(p), r(kv), r(pages), 1, ptr, FAKE, FAKE, FAKE, FAKE,
                                        FAKE, None, None, 0, None))


INV, UNS = hs.HS_ERR_INVALID_ARG, hs.HS_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(p=None), dict(kv=None), dict(kv=_kv(2)), dict(kv=_kv(-1)), dict(kv=_kv(k_codes=None)),
    dict(kv=_kv(k_scale=FAKE + 4)), dict(kv=_kv(v_codes=FAKE + 8)), dict(kv=_kv(v_scale=None)),
    dict(ptr=None), dict(ptr=FAKE + 2), dict(p=_p(hq=30)), dict(p=_p(batch=0)),
    dict(p=_p(batch=1 << 20, hq=4096, hkv=4096, t_kv=1)),
    dict(pages=hs.hs_pages(None, 16, 64, 10)), dict(pages=hs.hs_pages(FAKE, 0, 64, 10)),
    dict(pages=hs.hs_pages(FAKE, 16, 63, 10)), dict(pages=hs.hs_pages(FAKE, 16, 64, 1 << 27)),
])
def test_every_entry_point_refuses(lib, bad):
    args = dict(p=_p(), kv=_kv())
    args.update(bad)
    assert set(_calls(lib, **args).values()) == {INV}


@pytest.mark.parametrize("p", [_p(head_dim=256), _p(hq=64, hkv=2), _p(hq=17, hkv=1)])
def test_every_entry_point_names_what_is_not_built(lib, p):
    assert set(_calls(lib, p, _kv()).values()) == {UNS}


def test_attention_takes_bf16_and_decode_token_mode(lib):
    got = _calls(lib, _p(dtype="fp32"), _kv())
    assert {got[k] for k in ("reuse", "full", "sparse")} == {UNS}
    p = _p(mode="block", block_size=64, k=256, window=0)
    got = _calls(lib, p, _kv())
    assert {got[k] for k in ("full", "sparse")} == {UNS}
    p = _p()
    assert lib.hs_decode_step_quant(ctypes.byref(p), ctypes.byref(_kv()), None, 2, FAKE, FAKE,
                                    FAKE, FAKE, FAKE, FAKE, None, None, 0, None) == INV
    # more than one query per sequence is a prefill, not a decode step
    got = _calls(lib, _p(t_q=2), _kv())
    assert {got[k] for k in ("full", "sparse")} == {INV}


def test_rows_beyond_the_capacity_are_refused(lib):
    p = _p(t_q=8, q_offset=1020)
    assert lib.hs_kv_quant_write(ctypes.byref(p), ctypes.byref(_kv()), None, FAKE, FAKE, None,
                                 None, None) == INV
    assert lib.hs_kv_quant_write(ctypes.byref(_p(t_q=0)), ctypes.byref(_kv()), None, FAKE, FAKE,
                                 None, None, None) == hs.HS_OK  # nothing to do


def test_full_step_workspace(lib):
    p = _p()
    need = hs.hs_workspace_size(p, hs.HS_WS_DECODE_FULL_QUANT)
    assert need > 0
    # no logit is kept: far below the bf16 step's workspace on a long cache
    long = _p(t_kv=1 << 17)
    assert hs.hs_workspace_size(long, hs.HS_WS_DECODE_FULL_QUANT) < \
        hs.hs_workspace_size(long, hs.HS_WS_DECODE_FULL) // 2
    for ws, n in ((None, need), (FAKE, need - 1), (FAKE + 8, need)):
        assert _calls(lib, p, _kv(), ws=ws, ws_bytes=n)["full"] == hs.HS_ERR_WORKSPACE
    assert hs.hs_workspace_size(_p(head_dim=256), hs.HS_WS_DECODE_FULL_QUANT) == 0
    with pytest.raises(hs.HsError):
        hs.hs_workspace_size(p, 5)


def test_binding_refuses_unknown_formats():
    with pytest.raises(KeyError):
        hs.make_kv_quant("int3", None, None, None, None)


def test_lengths_that_a_step_could_pass_are_refused(lib):
    p = _p(batch=1, hq=1, hkv=1, head_dim=64, t_kv=2 ** 31 - 4096)
    assert set(_calls(lib, p, _kv()).values()) == {INV}
