"""Prompt attention where earlier tests do not reach: several tiles of queries a pair of
CTAs with values that are not finite, both orders of the tiles at either head dimension,
offsets past 32 bits, sound sequences beside one with bad offsets."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_attn_prefill, gdn_stream_status
from tests.attention_util import gen, normal, offsets
from tests.test_gpu_attn_prefill import agrees, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n,length", [(40, 160), (30, 224)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_in_later_tiles(bad, n, length, D):
    """Five tiles or more a pair, in both orders of the tiles (up to 32 sequences and more):
    in two sequences of three a value of V is not finite.  Queries before it are unchanged
    bit for bit, those from it on in every other channel."""
    lens = [length] * n
    q, k, v = (x.cuda() for x in inputs(lens, lens, 16, 2, D, 90))
    cu = offsets(lens)
    ref = gdn_attn_prefill(q, k, v, cu)
    r = np.random.default_rng(n)
    v2, want = v.clone(), torch.zeros(ref.shape, dtype=torch.bool)
    for i in range(n):
        if i % 3 == 2:
            continue
        t, h, d = int(r.integers(0, length)), int(r.integers(0, 2)), int(r.integers(0, D))
        v2[i * length + t, h, d] = bad
        want[i * length + t:(i + 1) * length, 8 * h:8 * h + 8, d] = True
    want = want.cuda()
    for _ in range(3):
        got = gdn_attn_prefill(q, k, v2, cu)
        assert gdn_stream_status() == "GDN_OK"
        assert torch.equal(torch.isfinite(got), ~want)
        assert torch.equal(torch.where(want, ref, got), ref)


@pytest.mark.parametrize("D,k_len", [(128, 900), (256, 700)])
def test_sequence_by_sequence_order_of_the_tiles(D, k_len):
    """Few sequences whose keys and values exceed 64 MB (40 KV heads), several tiles a pair."""
    q_len = [257, 1, 256, 255]
    assert len(q_len) * k_len * 40 * D * 4 > 64 << 20
    agrees(q_len, [k_len] * 4, h_q=40, h_kv=40, D=D, seed=91)


@pytest.mark.parametrize("D", [128, 256])
def test_sound_sequences_beside_one_that_decreases(D):
    """Offsets of four sequences of which the second's decrease: the other three are computed,
    and rows of o that belong to none of them stay as they were."""
    q, k, v = (x.cuda() for x in inputs([120], [120], 4, 1, D, 92))
    cq = torch.tensor([0, 50, 40, 70, 120], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, 50, 50, 80, 120], dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 3.0)
    # rows 40 .. 49 belong to the first and the third sequence: not compared
    gdn_attn_prefill(q, k, v, cq, ck, o=o)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS" and gdn_stream_status() == "GDN_OK"
    one = lambda a, b, c, d: gdn_attn_prefill(q[a:b], k[c:d], v[c:d], offsets([b - a]), offsets([d - c]))  # noqa: E731
    assert torch.equal(o[:40], one(0, 50, 0, 50)[:40])
    assert torch.equal(o[50:70], one(40, 70, 50, 80)[10:])
    assert torch.equal(o[70:], one(70, 120, 80, 120))
    # a range past the end: its rows stay
    cq = torch.tensor([0, 50, 130, 120], dtype=torch.int32, device="cuda")
    o.fill_(3.0)
    gdn_attn_prefill(q, k, v, cq, torch.tensor([0, 50, 100, 120], dtype=torch.int32, device="cuda"), o=o)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
    assert torch.equal(o[:50], one(0, 50, 0, 50)) and (o[50:] == 3).all()


def test_inputs_past_32_bits():
    """Slices of a fused tensor of 2.6e9 values, with a NaN that the queries see; and the same
    from copies."""
    T, D = 20000, 256
    x = torch.zeros((T, 512, D), dtype=torch.bfloat16, device="cuda")
    g = gen(93)
    for at, heads in ((0, 4), (300, 1), (511, 1)):
        x[:, at:at + heads] = normal(g, T, heads, D).cuda()
    x[T - 20, 511, 7] = float("nan")
    q, k, v = x[T - 64:, :4], x[:, 300:301], x[:, 511:512]
    cq, ck = offsets([64]), offsets([T])
    a = gdn_attn_prefill(q, k, v, cq, ck)
    b = gdn_attn_prefill(q.contiguous(), k.contiguous(), v.contiguous(), cq, ck)
    assert gdn_stream_status() == "GDN_OK"
    assert torch.equal(torch.nan_to_num(a, nan=-99.0), torch.nan_to_num(b, nan=-99.0))
    want = torch.zeros_like(a, dtype=torch.bool)
    want[44:, :, 7] = True
    assert torch.equal(torch.isnan(a), want)


def test_output_past_32_bits():
    """2.3e9 values of o from sequences of 128 tokens: the last ones as alone."""
    n, h_q, D = 550, 128, 256
    T = 128 * n
    q = torch.zeros((T, h_q, D), dtype=torch.bfloat16, device="cuda")
    g = gen(94)
    q[-256:] = normal(g, 256, h_q, D).cuda()
    k, v = (torch.zeros((T, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[-256:], v[-256:] = normal(g, 256, 16, D).cuda(), normal(g, 256, 16, D).cuda()
    o = gdn_attn_prefill(q, k, v, offsets([128] * n))
    alone = gdn_attn_prefill(q[-256:], k[-256:], v[-256:], offsets([128] * 2))
    assert gdn_stream_status() == "GDN_OK" and o.numel() > 2 ** 31
    assert torch.equal(o[-256:], alone)
