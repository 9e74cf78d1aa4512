"""Prompt attention with scale 0, whatever the products of queries and keys are."""
import pytest

from gated_deltanet_linear_recurrence_gb300 import gdn_attn_prefill, gdn_stream_status
from oracle.paged_attention import prompt
from tests.attention_util import BF16, check, offsets
from tests.test_gpu_attn_prefill import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("power", [20, 50, 58])
def test_scale_zero_with_large_products(power, D):
    """All scores are 0 whatever q and k are: o is the mean of the visible values."""
    q, k, v = inputs([300], [300], 8, 1, D, 95)
    q, k = ((x.double() * 2.0 ** power).to(x.dtype) for x in (q, k))
    cu = offsets([300])
    o = gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu, scale=0.0)
    assert gdn_stream_status() == "GDN_OK"
    check(o, prompt(q, k, v, cu, cu, 0.0), prompt(q, k, v.abs(), cu, cu, 0.0), BF16)
