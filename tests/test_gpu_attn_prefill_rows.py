"""Prompt attention beside rows that are not finite: what a tile of queries holds of other
sequences, or of a query that turned NaN, changes neither results nor time."""
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_attn_prefill, gdn_stream_status
from tests.attention_util import offsets
from tests.test_gpu_attn_prefill import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(3, 1), (8, 1), (14, 2)])
def test_rows_of_others_do_nothing(h_q, h_kv, D):
    """A few queries on many keys, next to a sequence whose q and k are NaN: the rows of a
    tile that are no queries of the sequence hold that, and change nothing, bit for bit."""
    q_len, k_len = [2, 60], [1500, 60]
    q, k, v = (x.cuda() for x in inputs(q_len, k_len, h_q, h_kv, D, 96))
    cq, ck = offsets(q_len), offsets(k_len)
    ref = gdn_attn_prefill(q, k, v, cq, ck)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[2:] = bad
        got = gdn_attn_prefill(q2, k, v, cq, ck)
        assert gdn_stream_status() == "GDN_OK"
        assert torch.equal(got[:2], ref[:2]) and not torch.isfinite(got[2:]).any()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("h_q", [3, 8])
def test_rows_that_are_nan_cost_no_time(h_q, D):
    """Two queries on 16,000 keys, one after the other through the key tiles.  Where rows of
    NaN moved the references, O was rescaled in each of them: 1.4 to 2 times the time.  The
    shortest of several calls, in turn, may differ by an eighth."""
    q_len, k_len = [2, 30], [16000, 30]
    q, k, v = (x.cuda() for x in inputs(q_len, k_len, h_q, 1, D, 97))
    cq, ck = offsets(q_len), offsets(k_len)
    others, own = q.clone(), q.clone()
    others[2:], own[0] = float("nan"), float("nan")
    sides = {"finite": q, "others": others, "own": own}
    best = dict.fromkeys(sides, float("inf"))
    for _ in range(12):
        for name, x in sides.items():
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            gdn_attn_prefill(x, k, v, cq, ck)
            start.record()
            for _ in range(5):
                gdn_attn_prefill(x, k, v, cq, ck)
            end.record()
            torch.cuda.synchronize()
            best[name] = min(best[name], start.elapsed_time(end))
    assert gdn_stream_status() == "GDN_OK"
    assert max(best["others"], best["own"]) <= 1.125 * best["finite"], best
