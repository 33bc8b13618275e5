"""The quantised full step over a pool where a selected key lies on a bad page."""
import pytest
import torch

from oracle_top_kv_b200 import hs
from tests.test_gpu_quant import DEV, FMTS, _decode_outputs, _filled, _params, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("length", [30, 64])  # below the budget: every key is selected; above it
def test_scores_of_selected_keys_on_bad_pages_are_zero(fmt, length):
    """As over bf16 pages (hs_decode_step_paged): a masked key has p = 0, and the window's keys
    are selected all the same."""
    p = _params(2, 8, 2, 128, 1, 64, k=40, window=20)
    q = _randn(2, 8, 1, 128, seed=401)
    c = _filled(p, fmt, 8, 400)
    c.table[1, length // 8 - 1] = -1
    seq = torch.full((2,), length, dtype=torch.int32, device=DEV)
    idx, cnt, o, lse, sel = _decode_outputs(p)
    hs.hs_decode_step_quant(p, c.kv, c.pages, hs.HS_DECODE_FULL_INDEX, q, seq, idx, cnt, o, lse, sel,
                            hs.workspace(p, hs.HS_WS_DECODE_FULL_QUANT))
    assert hs.hs_device_status() == hs.HS_ERR_BOUNDS
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    bad = (length // 8 - 1) * 8
    masked = (idx[1] >= bad) & (idx[1] < bad + 8)
    assert masked.sum() == 2 * 8 and (sel[1][masked] == 0).all()
    n = min(length, p.k)
    assert (cnt == n).all() and (sel[0, :, :n] > 0).all() and (sel[1][~masked][idx[1][~masked] >= 0] > 0).all()
    assert (sel[:, :, n:] == 0).all()
