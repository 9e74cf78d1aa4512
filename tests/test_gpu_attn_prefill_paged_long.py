"""Attention of new tokens over long caches against the fp64 oracle, with a bound that holds at
these lengths (attention_util's counts a sum of L weights as L 2^-24, which ends at L = 2^13).

With A = sum_j w_j |v_j| and n = L / 128 key tiles, from how the kernel sums:

* a thread adds the weights of at most 128 columns of a key tile in four chains, joins those,
  adds the tile's sum to a running one and the parts of at most 80 pairs after that: at most
  32 + 3 + n + 80 additions of positive numbers, each off by 2^-24: under 2^-15 for n <= 400;
* each product adds 16 keys to O in fp32, off by at most 2^-23 of what is added and there
  before: 8 n + 80 of them, under 2^-11.3 A for n <= 400;
* scores of at most 8 in size (asserted) are off by D 2^-24 8 <= 2^-13, their weights and the
  sum of these by that share each, 2^-12 A together, with the exponential's 2^-22;
* weights are rounded to bf16 before the product with V, 2^-8 A, and o at the end, 2^-8 |o|.

Together (2^-8 + 2^-10) A + 2^-8 |o|, where 2^-10.5 covers the first three.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_stream_status
from tests.attention_util import BF16, check
from tests.test_gpu_attn_prefill_paged import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,h_q,new,length", [(128, 8, 1, 30011), (256, 4, 5, 50000), (128, 2, 150, 20001)])
def test_long_caches(D, h_q, new, length, fp8):
    b = Batch([new], [length], h_q, 1, D, 64, fp8, 31)
    top = torch.einsum("ahd,nd->ahn", b.q.double(), b.k[0][0].double()).abs().max() * D ** -0.5
    assert top <= 8
    for kw in (dict(), dict(window=length - 4000, sinks=4)):
        got = b.run(**kw)
        assert gdn_stream_status() == "GDN_OK"
        check(got, *b.want(window=kw.get("window", 0), sinks=kw.get("sinks", 0)), BF16)
        assert np.isfinite(got.double().cpu().numpy()).all()
        assert torch.equal(b.run(**kw), got)
