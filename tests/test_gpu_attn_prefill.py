"""Packed causal prompt attention on the GPU against the fp64 oracle (bounds:
tests/attention_util.py): group sizes, head dimensions, lengths from none to several
tiles, prefixes, queries without a key, strided inputs, non-finite values where a query
does not see them, and the call's ways of failing."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_attn_prefill, gdn_stream_status
from oracle.paged_attention import prompt
from tests.attention_util import BF16, check, gen, normal, offsets

pytestmark = pytest.mark.gpu


def inputs(q_len, k_len, h_q, h_kv, D, seed):
    g = gen(seed)
    return (normal(g, sum(q_len), h_q, D), normal(g, sum(k_len), h_kv, D),
            normal(g, sum(k_len), h_kv, D))


def run(q_len, k_len=None, h_q=8, h_kv=1, D=256, seed=0, scale=None, tweak=None):
    k_len = q_len if k_len is None else k_len
    q, k, v = inputs(q_len, k_len, h_q, h_kv, D, seed)
    if tweak:
        tweak(q, k, v)
    scale = D ** -0.5 if scale is None else scale
    cq, ck = offsets(q_len), offsets(k_len)
    o = gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cq, ck, scale=scale)
    assert gdn_stream_status() == "GDN_OK"
    ref = prompt(q, k, v, cq, ck, scale)
    wabs = prompt(q, k, v.abs(), cq, ck, scale)
    return o, ref, wabs


def agrees(*args, **kw):
    o, ref, wabs = run(*args, **kw)
    check(o, ref, wabs, BF16)
    return o, ref


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (2, 1), (6, 2), (4, 1), (5, 1), (12, 2), (7, 1), (16, 2)])
def test_group_sizes(h_q, h_kv, D):
    """One to eight query heads on a KV head; a tile's rows end inside a token's heads for
    those that do not divide 128."""
    agrees([200, 1, 37], h_q=h_q, h_kv=h_kv, D=D, seed=h_q)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [32], [33], [127], [128], [129],
                                  [255], [257], [0, 5, 0, 0, 64, 0], [500, 3, 260]])
def test_lengths(lens, D):
    """Around the edges of a token tile (16 tokens a CTA, 32 a pair) and of a key tile."""
    agrees(lens, D=D, seed=len(lens) + lens[0])


@pytest.mark.parametrize("D,h_kv", [(128, 40), (256, 40)])
@pytest.mark.parametrize("q_len,k_len", [([150, 0, 7], [150, 30, 200]), ([300, 20], [1300, 900]),
                                         ([257, 1, 256, 255], [700, 700, 700, 700])])
def test_orders_of_the_tiles(q_len, k_len, D, h_kv):
    """More tiles than pairs of CTAs: with keys and values on either side of 64 MB, which
    choose the order of the tiles."""
    agrees(q_len, k_len, h_q=h_kv, h_kv=h_kv, D=D, seed=50)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("q_len,k_len", [([1], [300]), ([40, 1, 3], [41, 129, 1000]),
                                         ([130], [900]), ([33, 64], [161, 64])])
def test_pieces_over_earlier_rows(q_len, k_len, D):
    agrees(q_len, k_len, D=D, seed=sum(q_len))


@pytest.mark.parametrize("D", [128, 256])
def test_queries_without_a_key(D):
    """More queries than keys: the first ones see nothing and get zeros, also a whole
    tile of them, and a sequence without any key."""
    o, ref = agrees([100, 40, 300], [60, 0, 10], D=D, seed=3)
    assert (o[:40] == 0).all() and (o[100:140] == 0).all() and (o[140:430] == 0).all()
    assert (o[40:100] != 0).any()
    o, _ = agrees([5, 9], [0, 0], D=D, seed=4)
    assert (o == 0).all()


@pytest.mark.parametrize("n", [31, 32, 33, 70])
def test_many_sequences(n):
    """Up to 32 sequences are scheduled by what their tiles see, more of them in order."""
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.integers(0, 90, n)]
    agrees(lens, h_q=4, h_kv=2, D=128, seed=n)
    agrees(lens, [x + int(e) for x, e in zip(lens, r.integers(0, 40, n))], h_q=4, h_kv=2, D=128, seed=n)


@pytest.mark.parametrize("D", [128, 256])
def test_several_passes(D):
    """More tiles than pairs of CTAs: a pair goes through several (100 sequences on
    4 KV heads), with long and short ones next to each other."""
    lens = [700] + [1, 40, 130] * 33
    agrees(lens, h_q=4, h_kv=4, D=D, seed=11)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(scale, D):
    """No scale, a negative one, and one that leaves a few keys with the whole weight and
    moves the reference often (keys grow along the sequence)."""
    def grow(q, k, v):
        if scale == 1.0:
            k *= (torch.linspace(0.05, 0.3, len(k))[:, None, None]).to(k.dtype)
            q *= 0.5
    agrees([300], scale=scale, D=D, seed=5, tweak=grow)


def test_growing_scores_rescale():
    """Each key tile's scores exceed the one before's by far more than the slack."""
    def tweak(q, k, v):
        q.fill_(1.0)
        k.copy_((torch.arange(len(k)) // 64 * 0.125)[:, None, None].expand_as(k))
    for D in (128, 256):
        agrees([640], D=D, scale=2.0 ** -2, seed=6, tweak=tweak)


@pytest.mark.parametrize("D", [128, 256])
def test_strided_inputs(D):
    """Slices of one fused projection give the same bits as their copies."""
    h_q, h_kv = 6, 2
    x = normal(gen(7), 300, h_q + 2 * h_kv, D).cuda()
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    cu = offsets([100, 0, 200])
    a = gdn_attn_prefill(q, k, v, cu)
    b = gdn_attn_prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert gdn_stream_status() == "GDN_OK" and torch.equal(a, b)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unseen_values_do_nothing(bad, D):
    """Keys and values of later tokens and of the next sequence, not finite: the queries
    that do not see them are unchanged, bit for bit."""
    lens = [150, 70, 90]
    q, k, v = (x.cuda() for x in inputs(lens, lens, 4, 2, D, 8))
    cu = offsets(lens)
    ref = gdn_attn_prefill(q, k, v, cu)
    at = 137  # in the first sequence; then all of the second and the last token of the third
    k2, v2 = k.clone(), v.clone()
    k2[at], v2[at, :, 3:40] = bad, bad
    k2[150:220], v2[150:220] = bad, bad
    v2[309] = bad
    got = gdn_attn_prefill(q, k2, v2, cu)
    assert gdn_stream_status() == "GDN_OK"
    assert torch.equal(got[:at], ref[:at]) and torch.equal(got[220:309], ref[220:309])
    assert not torch.isfinite(got[150:220]).any()


@pytest.mark.parametrize("D", [128, 256])
def test_seen_values_that_are_not_finite(D):
    """A non-finite value reaches the queries that see it, in its own dimension only."""
    def tweak(q, k, v):
        v[5, 0, 7] = float("inf")
        v[130, 0, D - 1] = float("nan")
        v[131, 0, 0] = -float("inf")
        v[140, 0, 0] = float("inf")
    o, ref, wabs = run([150], h_q=4, D=D, seed=9, tweak=tweak)
    got = o.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref))
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    fine = np.isfinite(ref)
    err = np.abs(got[fine] - ref[fine])
    assert (err <= (BF16 + 2.0 ** -10) * wabs[fine] + BF16 * np.abs(ref[fine]) + 1e-6).all()


@pytest.mark.parametrize("D", [128, 256])
def test_writes_stay_inside_o(D):
    """Rows around o, and o at an address that is a multiple of 16 bytes only."""
    lens = [33, 0, 140]
    q, k, v = (x.cuda() for x in inputs(lens, lens, 6, 2, D, 10))
    cu, n = offsets(lens), sum(lens) * 6 * D
    ref = gdn_attn_prefill(q, k, v, cu)
    for shift in (0, 8, 16):
        buf = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        o = buf[256 + shift:256 + shift + n].view(-1, 6, D)
        gdn_attn_prefill(q, k, v, cu, o=o)
        assert gdn_stream_status() == "GDN_OK" and torch.equal(o, ref)
        assert (buf[:256 + shift] == 7).all() and (buf[256 + shift + n:] == 7).all()


def test_deterministic_and_on_another_stream():
    lens = [700, 1, 300]
    q, k, v = (x.cuda() for x in inputs(lens, lens, 16, 2, 256, 12))
    cu = offsets(lens)
    ref = gdn_attn_prefill(q, k, v, cu)
    assert all(torch.equal(gdn_attn_prefill(q, k, v, cu), ref) for _ in range(5))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = gdn_attn_prefill(q, k, v, cu, stream=s)
    assert gdn_stream_status(s) == "GDN_OK" and torch.equal(o, ref)


def test_captured_into_a_graph():
    lens = [65, 300]
    q, k, v = (x.cuda() for x in inputs(lens, lens, 8, 2, 128, 13))
    cu, o = offsets(lens), torch.empty((365, 8, 128), dtype=torch.bfloat16, device="cuda")
    ref = gdn_attn_prefill(q, k, v, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn_attn_prefill(q, k, v, cu, o=o)
    o.zero_()
    g.replay()
    assert gdn_stream_status() == "GDN_OK" and torch.equal(o, ref)


@pytest.mark.parametrize("cq,ck,keep", [
    ([1, 50, 90], [0, 50, 90], None),           # does not start at 0
    ([0, 50, 80], [0, 50, 90], None),           # does not end at the total
    ([0, 60, 50, 90], [0, 20, 50, 90], None),   # decreasing: that sequence is skipped
    ([0, 50, 1 << 30], [0, 50, 90], slice(0, 50)),   # past the end: skipped, the first is right
    ([0, 50, 90], [0, 50, -7], slice(0, 50)),
])
def test_bad_offsets_are_reported(cq, ck, keep):
    """Recorded in the error word, once; nothing outside the tensors is touched and the
    sequences with sound offsets are computed."""
    q, k, v = (x.cuda() for x in inputs([90], [90], 4, 1, 128, 14))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o = torch.full_like(q, 3.0)
    gdn_attn_prefill(q, k, v, i32(cq), i32(ck), o=o)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
    assert gdn_stream_status() == "GDN_OK"
    if keep is not None:
        ref = gdn_attn_prefill(q[keep], k[keep], v[keep], i32([0, 50]))
        assert torch.equal(o[keep], ref) and (o[50:] == 3).all()


def test_no_tokens():
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    assert gdn_attn_prefill(e, kv, kv, offsets([0, 0])).shape == (0, 4, 128)
    assert gdn_stream_status() == "GDN_OK"
