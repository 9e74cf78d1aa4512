"""Attention of new tokens over the paged cache against the fp64 oracle: lengths, heads,
pages and windows at their edges, keys split over many SMs, what must not be seen.

Bounds: attention_util's for prompt attention (weights rounded to bf16).  Joining parts adds a
base-2 exponential (2^-22) and a product a part: far inside the 2^-10 of the scores' term.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_attn_prefill_paged,
                                                    gdn_attn_prefill_paged_workspace_size,
                                                    gdn_kv_append, gdn_stream_status)
from oracle.paged_attention import dequantise, quantise
from oracle.window_attention import attend, seen
from tests.attention_util import BF16, check, gen, normal, offsets

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Sequences of `lengths` cached rows in pages handed out in no order, the last new[n] of
    each with queries.  Slots behind the lengths hold NaN (and NaN codes), table entries that
    no row needs name no page."""

    def __init__(self, new, lengths, h_q, h_kv, D, page, fp8, seed, extra_entries=1, loud=1.0):
        g = gen(seed)
        self.new, self.lengths, self.D, self.page, self.fp8 = new, lengths, D, page, fp8
        counts = [-(-x // page) for x in lengths]
        P = sum(counts) + 2
        total = sum(lengths)
        self.q = normal(g, sum(new), h_q, D)
        k, v = normal(g, total, h_kv, D), normal(g, total, h_kv, D)
        k[..., 0] *= loud
        v *= torch.exp2(torch.randint(-3, 4, (total, 1, 1), generator=g)).to(torch.bfloat16)
        shape = (P, h_kv, page, D)
        if fp8:
            self.kp = torch.full(shape, 0x7f, dtype=torch.uint8).cuda().view(E4M3)
            self.ke = torch.randint(0, 256, shape[:3], generator=g, dtype=torch.uint8).cuda()
            self.ve = self.ke.clone()
        else:
            self.kp = torch.full(shape, float("nan"), dtype=torch.bfloat16).cuda()
            self.ke = self.ve = None
        self.vp = self.kp.clone()
        order = torch.randperm(P, generator=g)
        self.table = torch.full((len(lengths), max(counts + [0]) + extra_entries), -1, dtype=torch.int32)
        at = 0
        for n, c in enumerate(counts):
            self.table[n, :c] = order[at:at + c]
            at += c
        self.table = self.table.cuda()
        gdn_kv_append(k.cuda(), v.cuda(), self.kp, self.vp, self.table, offsets(lengths), i32([0] * len(lengths)),
                      k_exp=self.ke, v_exp=self.ve)
        assert gdn_stream_status() == "GDN_OK"
        if fp8:
            k, v = (torch.from_numpy(dequantise(*quantise(x))) for x in (k, v))
        cut = np.cumsum([0] + list(lengths))
        self.k = [k[cut[n]:cut[n + 1]].transpose(0, 1) for n in range(len(lengths))]
        self.v = [v[cut[n]:cut[n + 1]].transpose(0, 1) for n in range(len(lengths))]

    def run(self, **kw):
        a = dict(kw)  # (what is not given is brought to the GPU, which a capture does not allow)
        for name, make in (("q", self.q.cuda), ("cu_seqlens_q", lambda: offsets(self.new)),
                           ("cache_len", lambda: i32(self.lengths))):
            if name not in a:
                a[name] = make()
        return gdn_attn_prefill_paged(a.pop("q"), self.kp, self.vp, self.table, a.pop("cu_seqlens_q"),
                                      a.pop("cache_len"), k_exp=self.ke, v_exp=self.ve, **a)

    def want(self, scale=None, window=0, sinks=0, gone=None):
        o, size, t = [], [], 0
        for n, a in enumerate(self.new):
            x, y = attend(self.q[t:t + a], self.k[n], self.v[n], self.D ** -0.5 if scale is None else scale, window,
                          sinks, None if gone is None else gone[n])
            o.append(x)
            size.append(y)
            t += a
        return np.concatenate(o), np.concatenate(size)

    def check(self, name="", window=None, sinks=0, gone=None, **kw):
        got = self.run(window=window, sinks=sinks, **kw)
        status = gdn_stream_status()
        assert status == ("GDN_OK" if gone is None else "GDN_ERR_BAD_PAGE"), status
        ref, size = self.want(kw.get("scale"), window or 0, sinks, gone)
        check(got, ref, size, BF16, name)
        return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("a,L", [(1, 1), (1, 7), (2, 128), (3, 129), (16, 16), (33, 33), (65, 300), (257, 257), (5, 640)])
def test_one_sequence(a, L, D, fp8):
    Batch([a], [L], 8, 1, D, 16, fp8, a + L).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("h_q,h_kv,D,page", [(1, 1, 256, 8), (2, 1, 128, 1024), (3, 1, 256, 16), (8, 2, 128, 8),
                                             (5, 1, 128, 32), (12, 2, 256, 64), (7, 1, 256, 128), (16, 2, 128, 64),
                                             (9, 9, 128, 16), (24, 8, 256, 32)])
def test_heads_and_pages(h_q, h_kv, D, page, fp8):
    Batch([70, 1, 9, 200], [333, 50, 9, 201], h_q, h_kv, D, page, fp8, h_q).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_mixed_batch(D, fp8):
    """A piece of a prompt, whole prompts, drafted tokens, single ones, sequences without new
    tokens, and queries that see nothing."""
    new = [150, 1, 0, 40, 4, 1, 1, 0, 3, 30, 2]
    lengths = [700, 260, 100, 40, 129, 1, 0, 0, 3, 20, 0]
    b = Batch(new, lengths, 8, 2, D, 16, fp8, 3)
    got = b.check()
    cut = np.cumsum([0] + new)
    assert not got[cut[6]:cut[7]].any() and not got[cut[10]:cut[11]].any()
    assert not got[cut[9]:cut[9] + 10].any() and got[cut[9] + 10:cut[10]].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (64, 0), (127, 130), (128, 128), (129, 4), (300, 257),
                                          (1000, 0), (256, 5000)])
def test_windows(window, sinks, D, fp8):
    b = Batch([70, 1, 5, 260], [700, 450, 129, 261], 8, 1, D, 32, fp8, window)
    b.check(window=window, sinks=sinks)


def test_a_window_that_holds_everything_is_none():
    b = Batch([20, 300], [90, 300], 4, 1, 128, 16, False, 4)
    want = b.run()
    for window, sinks in ((300, 0), (301, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 40, 0)):
        got = b.run(window=window, sinks=sinks).double()
        assert ((got - want.double()).abs() <= 4 * BF16 * (want.double().abs() + 1)).all()
    assert gdn_stream_status() == "GDN_OK"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,h_q,h_kv,new,lengths", [
    (256, 16, 2, [5], [20000]), (128, 8, 1, [1], [30011]), (256, 4, 1, [40, 3], [9000, 12345]),
    (128, 32, 8, [3, 1, 1, 2], [5000, 17, 4097, 2900]), (128, 6, 1, [300], [6000])])
def test_keys_split_over_many_pairs(D, h_q, h_kv, new, lengths, fp8):
    b = Batch(new, lengths, h_q, h_kv, D, 64, fp8, 5)
    got = b.check()
    for _ in range(3):
        assert torch.equal(b.run(), got)  # the same every time
    b.check(window=3333, sinks=4)


@pytest.mark.parametrize("D", [128, 256])
def test_widened_once_or_by_each_tile(D):
    """Over e4m3 rows: sequences with many tiles of queries have their rows widened into the
    workspace while there is room, with the same results; a mixture of both, with windows,
    missing pages, NaN codes and units above 2^7."""
    new, lengths = [300, 1, 140, 200, 3, 129], [500, 700, 140, 1001, 333, 129]
    b = Batch(new, lengths, 8, 1, D, 16, True, 20)
    least = gdn_attn_prefill_paged_workspace_size(8, 1, D)
    full = gdn_attn_prefill_paged_workspace_size(8, 1, D, E4M3, sum(new))
    assert full - least == 128 << 20 and least == gdn_attn_prefill_paged_workspace_size(8, 1, D, E4M3, 64)
    assert least == gdn_attn_prefill_paged_workspace_size(8, 1, D, torch.bfloat16, 10 ** 6)
    ws = torch.full((full,), 0xff, dtype=torch.uint8, device="cuda")
    row = 4 * D
    for kw in (dict(), dict(window=150, sinks=20)):
        want = b.check(**kw, workspace=ws[:least])
        # none fits, some do, the last one ends a row too late, all do
        for rows in (0, 400, 500, 639, 640, 1640, 1641, 1769, 1770, 5000):
            ws[least:] = 0xff
            assert torch.equal(b.run(**kw, workspace=ws[:least + rows * row]), want), rows
    b.table[3, 20] = 10 ** 6
    gone = [np.arange(x) // 16 == (20 if i == 3 else -1) for i, x in enumerate(lengths)]
    want = b.check(gone=gone, workspace=ws[:least])
    assert torch.equal(b.check(gone=gone, workspace=ws), want)
    b.table[3, 20] = 0  # (some page: its rows are other ones)
    b.kp.view(torch.uint8)[int(b.table[0, 25]), 0, 5, 9] = 0xff
    b.vp.view(torch.uint8)[int(b.table[2, 3]), 0, 7, D - 1] = 0x7f
    b.ve[int(b.table[0, 2]), 0, 3] = 200
    b.ke[int(b.table[5, 2]), 0, 3] = 140
    want = b.run(workspace=ws[:least])
    got = b.run(workspace=ws)
    assert gdn_stream_status() == "GDN_OK" and torch.isnan(want).any() and torch.isfinite(want).any()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("D,h_kv", [(128, 1), (256, 1), (128, 4)])
def test_pieces_widened_and_copied_in_turn(D, h_kv):
    """Over e4m3 rows a pair goes from a piece whose rows are copied (widened once) to one that it
    widens for itself and back, with more key tiles in each than there are slots for."""
    new, lengths = [], []
    for i in range(5):
        new += [5, 300, 1, 2, 0, 160]
        lengths += [5000 - 700 * i, 3000 + 111 * i, 1500, 2900 + i, 40, 2500]
    b = Batch(new, lengths, 8 * h_kv, h_kv, D, 32, True, D + h_kv)
    got = b.check()
    for _ in range(5):
        assert torch.equal(b.run(), got)
    b.check(window=1100, sinks=200)
    assert gdn_stream_status() == "GDN_OK"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_many_sequences(D, fp8):
    """More than 32: the block counts the sequences together; more than its threads."""
    rng = np.random.default_rng(6)
    for n, top in ((33, 300), (700, 40)):
        lengths = rng.integers(0, top, n).tolist()
        new = [int(rng.integers(0, x + 2)) if i % 3 else 1 for i, x in enumerate(lengths)]
        Batch(new, lengths, 4, 2, D, 16, fp8, n).check()


@pytest.mark.parametrize("n", [31, 32, 63, 64, 65, 255, 256, 257])
def test_sequences_counted_by_a_warp_or_the_block(n):
    """Up to 256 are counted by one warp, some a lane: empty ones in between and at both ends,
    long ones (whose e4m3 rows are widened once) at places that end a lane's."""
    new, lengths = [1] * n, [(7 * i) % 50 for i in range(n)]
    for i in range(0, n, 5):
        new[i] = 0
    for i in (1, n // 2, n - 2):
        new[i], lengths[i] = 150, 300 + i
    new[-1] = 0
    for fp8 in (False, True):
        b = Batch(new, lengths, 8, 1, 128, 16, fp8, n)
        b.check()
        b.check(window=40, sinks=3)


def test_weight_on_one_row():
    """Each query puts all its weight on one cached row, which its output has to be."""
    for fp8 in (False, True):
        L, a = 1500, 9
        b = Batch([a], [L], 4, 1, 128, 16, fp8, 7)
        for shift in (0, 131, 1000):
            target = torch.arange(a)[:, None].repeat(1, 4) * 50 + shift
            kk = b.k[0][0].double()
            q = (kk[target.flatten()].view(a, 4, 128) * 3).to(torch.bfloat16)
            b.q = q
            got = b.run(scale=1.0).double().cpu()
            want = b.v[0][0].double()[target.flatten()].view(a, 4, 128)
            assert ((got - want).abs() <= 2 * BF16 * want.abs() + 1e-6).all()


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-6, 0.5])
def test_scales(scale):
    for D in (128, 256):
        for fp8 in (False, True):
            Batch([40, 2], [300, 77], 8, 2, D, 16, fp8, 8).check(scale=scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_what_is_not_seen(D, fp8):
    """NaN and infinities in rows that a query does not see, ahead of it and behind its window,
    leave it as it was; where it sees them they spread over their dimension."""
    new, lengths, window, sinks = [100, 3], [600, 500], 200, 4
    b = Batch(new, lengths, 8, 2, D, 16, fp8, 9)
    for kw in (dict(), dict(window=window, sinks=sinks)):
        ref, size = b.want(window=kw.get("window", 0), sinks=kw.get("sinks", 0))
        clean = b.run(**kw)
        for pos, what in ((550, "v"), (4, "v"), (310, "v"), (599, "k"), (345, "v"), (2, "v")):
            page, slot = int(b.table[0, pos // 16]), pos % 16
            pool = b.vp if what == "v" else b.kp
            keep = pool[page, 1, slot].clone()
            if fp8:
                pool.view(torch.uint8)[page, 1, slot, 5:9] = 0x7f
            else:
                pool[page, 1, slot, 5:9] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")]).cuda()
            got = b.run(**kw)
            pool.view(torch.uint8)[page, 1, slot] = keep.view(torch.uint8)
            see = torch.from_numpy(seen(100, 600, kw.get("window", 0), kw.get("sinks", 0))[:, pos])
            touched = torch.zeros(got.shape, dtype=torch.bool)
            if what == "v":
                touched[:100, 4:, 5:9] = see[:, None, None]
            else:
                touched[:100, 4:] = see[:, None, None]
            touched = touched.cuda()
            assert not torch.isfinite(got[touched]).any(), (pos, what)
            # (a reference may move otherwise: within the rounding, not the bits)
            far = (got.double() - clean.double()).abs() > 4 * BF16 * (torch.from_numpy(size).cuda() + 1e-3)
            assert not (far | ~torch.isfinite(got))[~touched].any(), (pos, what)
    assert gdn_stream_status() == "GDN_OK"


@pytest.mark.parametrize("D", [128, 256])
def test_codes_whose_values_overflow(D):
    """A unit of 2^120 and a code of 448 read back as infinite: seen or not seen like one."""
    b = Batch([70], [300], 8, 1, D, 16, True, 19)
    clean = b.run()
    for pos in (295, 100):
        page, slot = int(b.table[0, pos // 16]), pos % 16
        b.vp.view(torch.uint8)[page, 0, slot] = 0
        b.vp.view(torch.uint8)[page, 0, slot, 3] = 0x7e
        b.ve[page, 0, slot] = 247
        got = b.run()
        see = torch.from_numpy(seen(70, 300, 0, 0)[:, pos]).cuda()
        assert torch.isinf(got[see][..., 3]).all() and torch.isfinite(got[~see]).all()
        rest = got.clone()
        rest[..., 3] = 0
        assert torch.isfinite(rest).all()
        assert not (~see).any() or ((got[~see] - clean[~see]).abs().max() < 0.1 * clean.abs().max())
        b.ve[page, 0, slot] = 127
    assert gdn_stream_status() == "GDN_OK"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_missing_pages(page, fp8):
    """Positions without a page take no part, wherever they are, and are reported."""
    for D in (128, 256):
        b = Batch([150, 4], [900, 777], 8, 1, D, page, fp8, 10)
        for n, entry, value in ((0, 0, -1), (0, 300 // page, 10 ** 6), (1, 770 // page, -5), (0, 899 // page, -1)):
            keep = int(b.table[n, entry])
            b.table[n, entry] = value
            gone = [np.arange(x) // page == (entry if i == n else -1) for i, x in enumerate(b.lengths)]
            b.check(gone=gone)
            if not gone[0].all():
                b.check(gone=gone, window=850, sinks=8)
            b.table[n, entry] = keep
        b.check()


def test_no_pages_at_all():
    for dtype in (torch.bfloat16, E4M3):
        q = normal(gen(11), 5, 4, 128).cuda()
        pool = torch.empty((0, 2, 16, 128), dtype=dtype, device="cuda")
        exps = dict(k_exp=torch.empty((0, 2, 16), dtype=torch.uint8, device="cuda"),
                    v_exp=torch.empty((0, 2, 16), dtype=torch.uint8, device="cuda")) if dtype == E4M3 else {}
        table = i32([[3, 1], [0, 0]])
        o = gdn_attn_prefill_paged(q, pool, pool, table, offsets([2, 3]), i32([20, 3]), **exps)
        assert gdn_stream_status() == "GDN_ERR_BAD_PAGE" and not o.any()
        o = gdn_attn_prefill_paged(q, pool, pool, table, offsets([2, 3]), i32([0, 0]), **exps)
        assert gdn_stream_status() == "GDN_OK" and not o.any()
        o = gdn_attn_prefill_paged(q, pool, pool, table[:, :0].contiguous(), offsets([2, 3]), i32([0, 0]), **exps)
        assert gdn_stream_status() == "GDN_OK" and not o.any()


def test_bad_lengths_and_offsets():
    b = Batch([20, 30, 10], [100, 200, 50], 4, 2, 128, 16, False, 12)
    want = b.run()
    o = torch.full_like(want, 7.0)
    for bad in (-1, 14 * 16 + 1, 2 ** 31 - 1):
        got = b.run(cache_len=i32([100, bad, 50]), o=o.clone())
        assert gdn_stream_status() == "GDN_ERR_BAD_CACHE_LEN"
        assert not got[20:50].any()
        for part in (slice(0, 20), slice(50, 60)):
            assert ((got[part].double() - want[part].double()).abs() <= 2 * BF16 * (want[part].double().abs() + 1)).all()
    for cu, kept in (([0, 20, 10, 60], slice(0, 20)), ([0, 20, 50, 61], slice(0, 50)), ([-4, 20, 50, 60], slice(20, 60))):
        got = b.run(cu_seqlens_q=i32(cu), o=o.clone())
        assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
        if cu[2] == 50:
            assert ((got[kept].double() - want[kept].double()).abs() <= 2 * BF16 * (want[kept].double().abs() + 1)).all()
    got = b.run(cu_seqlens_q=i32([5, 20, 50, 55]), o=o.clone())  # rows of no sequence stay
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
    assert (got[:5] == 7).all() and (got[55:] == 7).all() and (got[5:55] != 7).any()


def test_strided_q_given_outputs_and_workspace():
    b = Batch([50, 1, 7], [400, 300, 7], 8, 2, 256, 32, True, 13)
    want = b.run()
    wide = torch.zeros((58, 13, 256), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = b.q.cuda()
    o = torch.empty_like(want)
    ws = torch.full((gdn_attn_prefill_paged_workspace_size(8, 2, 256),), 0xff, dtype=torch.uint8, device="cuda")
    got = b.run(q=wide[:, 3:11], o=o, workspace=ws)
    assert got.data_ptr() == o.data_ptr() and torch.equal(o, want)
    canary = torch.full((58 + 2, 8, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    b.run(o=canary[1:59], workspace=ws)
    assert torch.equal(canary[1:59], want) and (canary[0] == 3).all() and (canary[59] == 3).all()


def test_captured_and_replayed():
    b = Batch([3, 1, 2], [3000, 1, 77], 8, 2, 128, 16, True, 14)
    q, cu, lens = b.q.cuda(), offsets(b.new), i32(b.lengths)
    call = lambda: b.run(q=q, cu_seqlens_q=cu, cache_len=lens, window=2000, sinks=4)  # noqa: E731
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for lengths in ([3000, 1, 77], [2500, 1, 70], [40, 1, 2]):
        lens.copy_(i32(lengths))
        q.mul_(0.9)
        g.replay()
        replayed = got.clone()
        assert torch.equal(replayed, call())
    assert gdn_stream_status() == "GDN_OK"


def test_on_another_stream_and_two_at_once():
    a = Batch([40, 2], [900, 5000], 8, 1, 256, 64, False, 15)
    b = Batch([40, 2], [900, 5000], 8, 1, 256, 64, True, 16)
    qa, qb, cu, lens = a.q.cuda(), b.q.cuda(), offsets(a.new), i32(a.lengths)
    want = [x.run(q=q, cu_seqlens_q=cu, cache_len=lens) for x, q in ((a, qa), (b, qb))]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [x.run(q=q, cu_seqlens_q=cu, cache_len=lens, stream=h)
               for x, q, h in ((a, qa, streams[0]), (b, qb, streams[1].cuda_stream))]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert gdn_stream_status(streams[0]) == "GDN_OK"


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, its last pages in use."""
    D, page, h_kv = 256, 1024, 8
    P = 1100  # 2.3e9 values, 4.6e9 bytes
    for dtype in (torch.bfloat16, E4M3):
        P = 1100 if dtype == torch.bfloat16 else 2200
        kp = torch.empty((P, h_kv, page, D), dtype=dtype, device="cuda")
        vp = torch.empty_like(kp)
        exps = dict(k_exp=torch.empty((P, h_kv, page), dtype=torch.uint8, device="cuda"),
                    v_exp=torch.empty((P, h_kv, page), dtype=torch.uint8, device="cuda")) if dtype == E4M3 else {}
        table = i32([[P - 1, 0, P - 2]])
        L = 2500
        g = gen(17)
        q, k, v = normal(g, 30, 16, D), normal(g, L, h_kv, D), normal(g, L, h_kv, D)
        gdn_kv_append(k.cuda(), v.cuda(), kp, vp, table, offsets([L]), i32([0]), **exps)
        got = gdn_attn_prefill_paged(q.cuda(), kp, vp, table, offsets([30]), i32([L]), **exps)
        assert gdn_stream_status() == "GDN_OK"
        if exps:
            k, v = (torch.from_numpy(dequantise(*quantise(x))) for x in (k, v))
        check(got, *attend(q, k.transpose(0, 1), v.transpose(0, 1), D ** -0.5), BF16)
        del kp, vp


def test_binding_refuses():
    b = Batch([4], [40], 4, 2, 128, 16, False, 18)
    for kw in (dict(window=0), dict(window=-1), dict(window=5, sinks=-1), dict(q=b.q.cuda().half()),
               dict(q=b.q.cuda()[:, :, :64]), dict(cu_seqlens_q=i32([0])), dict(cache_len=i32([40, 40])),
               dict(o=torch.empty((4, 4, 128), device="cuda")), dict(q=b.q)):
        with pytest.raises(ValueError):
            b.run(**kw)
    with pytest.raises(TypeError):
        b.run(window="x")
    for kw in (dict(q=torch.zeros((4, 3, 128), dtype=torch.bfloat16, device="cuda")),
               dict(q=torch.zeros((4, 18, 128), dtype=torch.bfloat16, device="cuda")),
               dict(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(RuntimeError):
            b.run(**kw)
    assert b.run(q=b.q.cuda()[:0], cu_seqlens_q=i32([0, 0])).shape == (0, 4, 128)
    torch.cuda.synchronize()
    assert gdn_stream_status() == "GDN_OK"
