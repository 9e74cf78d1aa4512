"""Norms and rotation of q's and k's heads, dense and on the way into the paged cache, against
the fp64 oracle.

Bound: the result is rounded to bf16 once (2^-8 of it); the norm's factor (a sum of up to 256
squares in fp32 by lanes and shuffles: 16 roundings in a row at most, 2^-20, and rsqrt 2^-22)
and the weights' product make 2^-19 of each value; an angle is right to 2^-25 of a turn, 2^-22
radians, sine and cosine to 2^-22, so that a turned value is off by 2^-19 of |y_a| + |y_b|, all
together.  2^-133 is the step of bf16's smallest numbers.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_kv_append, gdn_kv_append_rope,
                                                    gdn_qk_norm_rope, gdn_stream_status)
from oracle.rope import rotate
from tests.attention_util import BF16, gen, normal, offsets
from tests.test_gpu_kv_cache import Cache, i32

pytestmark = pytest.mark.gpu


def freqs(rotary, theta=1e6):
    n = rotary // 2
    return (theta ** (-torch.arange(n, dtype=torch.float64) / n)).float()


def check(got, ref, size, name=""):
    got = got.detach().double().cpu().numpy()
    bound = (BF16 + 2.0 ** -19) * np.abs(ref) + 2.0 ** -19 * size + 2.0 ** -133
    err = np.abs(got - ref)
    worst = np.unravel_index((err - bound).argmax(), err.shape)
    assert (err <= bound).all(), f"{name}: {got[worst]} for {ref[worst]} at {worst}"


def inputs(T, h_q, h_kv, D, seed, extra=1):
    x = normal(gen(seed), T, h_q + 2 * h_kv + extra, D)
    return x, x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:h_q + 2 * h_kv]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,h_q,h_kv,D,rotary,norm", [
    (1, 1, 1, 128, 8, True), (1, 16, 2, 256, 64, True), (3, 7, 3, 128, 128, False),
    (37, 5, 1, 256, 256, True), (9, 32, 8, 128, 72, True), (700, 3, 2, 128, 16, True),
    (2, 65, 9, 256, 8, False)])
def test_dense(T, h_q, h_kv, D, rotary, norm, interleaved):
    x, q, k, _ = inputs(T, h_q, h_kv, D, 1)
    g = gen(2)
    pos = torch.randint(-1000, 300000, (T,), generator=g, dtype=torch.int32)
    f, w = freqs(rotary), torch.randn((2, D), generator=g)
    kw = dict(q_weight=w[0], k_weight=w[1], norm_eps=1e-5) if norm else {}
    xd = x.cuda()
    before = xd.clone()
    qo, ko = gdn_qk_norm_rope(xd[:, :h_q], xd[:, h_q:h_q + h_kv], pos.cuda(), f.cuda(), interleaved=interleaved,
                              **{n: v.cuda() if torch.is_tensor(v) else v for n, v in kw.items()})
    assert torch.equal(xd, before) and qo.is_contiguous() and ko.is_contiguous()
    for got, src, i in ((qo, q, 0), (ko, k, 1)):
        ref, size = rotate(src, pos, f, interleaved=interleaved, weight=w[i] if norm else None,
                           eps=1e-5 if norm else None)
        check(got, ref, size, "qk"[i])
        if not norm:  # what does not turn is copied
            assert torch.equal(got[..., rotary:].cpu(), src[..., rotary:])


def test_far_positions_and_frequencies():
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937], dtype=torch.int32)
    f = torch.tensor([1.0, -0.7, 3e-9, 1e-30, 2.0 ** -149, 6.5, 1e6, 2.0 ** 39], dtype=torch.float32)
    _, q, k, _ = inputs(7, 2, 1, 128, 3)
    qo, ko = gdn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda())
    for got, src in ((qo, q), (ko, k)):
        check(got, *rotate(src, pos, f))


@pytest.mark.parametrize("A", [1, 2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(A, interleaved):
    T, rotary = 41, 96
    _, q, k, _ = inputs(T, 4, 2, 128, 4)
    g = gen(5)
    pos = torch.randint(0, 50000, (A, T), generator=g, dtype=torch.int32)
    axes = torch.randint(0, A, (rotary // 2,), generator=g).tolist()
    f = freqs(rotary)
    got = [gdn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), axes=a, interleaved=interleaved)
           for a in (axes, bytes(axes))]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for o, src in zip(got[0], (q, k)):
        check(o, *rotate(src, pos, f, axes=axes, interleaved=interleaved))


@pytest.mark.parametrize("D", [128, 256])
def test_norms_at_the_ends_of_the_range(D):
    """Squares that overflow or vanish in 32 bits, rows of zeros, one value alone."""
    big, small = 3.0e38, 2.0 ** -133
    row = normal(gen(6), 8, 1, D).double()
    row[0] = 0
    row[1] *= 1e37
    row[2] = big
    row[3] *= 1e-37
    row[4] = small
    row[5] = 0
    row[5, 0, 7] = big
    row[6] = 0
    row[6, 0, D - 1] = -small
    row[7] *= 2e19
    x = row.to(torch.bfloat16)
    pos, f = torch.arange(8, dtype=torch.int32) * 1000, freqs(32)
    for eps in (0.0, 1e-38, 1e-6, 10.0):
        qo, ko = gdn_qk_norm_rope(x.cuda(), x.cuda(), pos.cuda(), f.cuda(), norm_eps=eps)
        assert torch.equal(qo.view(torch.int16), ko.view(torch.int16))
        first = 1 if eps == 0 else 0
        if first:
            assert torch.isnan(qo[0]).all()  # 0 / 0, as the formula
        ref, size = rotate(x[first:], pos[first:], f, eps=eps)
        check(qo[first:], ref, size, f"eps {eps}")


def test_values_that_are_not_finite():
    """A NaN or an infinity reaches its pair, or with the norm its row, and nothing else."""
    inf, nan = float("inf"), float("nan")
    _, q, k, _ = inputs(4, 3, 1, 128, 7)
    pos, f = torch.tensor([5, 6, 7, 8], dtype=torch.int32), freqs(64)
    clean = gdn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda())[0].cpu()
    dirty = q.clone()
    dirty[1, 2, 3], dirty[2, 0, 100], dirty[3, 1, 63] = nan, -inf, inf
    got = gdn_qk_norm_rope(dirty.cuda(), k.cuda(), pos.cuda(), f.cuda())[0].cpu()
    touched = torch.zeros_like(got, dtype=torch.bool)
    for t, h, d in ((1, 2, 3), (1, 2, 35), (2, 0, 100), (3, 1, 63), (3, 1, 31)):
        touched[t, h, d] = True
    assert torch.equal(got[~touched], clean[~touched]) and not torch.isfinite(got[touched]).any()
    normed = gdn_qk_norm_rope(dirty.cuda(), k.cuda(), pos.cuda(), f.cuda(), norm_eps=1e-6)[0].cpu()
    clean = gdn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), norm_eps=1e-6)[0].cpu()
    rows = touched.any(-1)
    assert torch.equal(normed[~rows], clean[~rows])
    assert torch.isnan(normed[1, 2]).all() and torch.isnan(normed[2, 0, 100])
    assert (normed[2, 0, 64:100] == 0).all()
    f[3] = nan
    got = gdn_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda())[0]
    assert torch.isnan(got[..., [3, 35]]).all()
    got[..., [3, 35]] = 0
    assert torch.isfinite(got).all()


def test_in_place_and_given_outputs():
    x, *_ = inputs(50, 6, 2, 256, 8)
    x = x.cuda()
    pos, f = torch.arange(50, dtype=torch.int32, device="cuda"), freqs(64).cuda()
    q, k = x[:, :6], x[:, 6:8]
    want = gdn_qk_norm_rope(q, k, pos, f, norm_eps=1e-6)
    out = torch.zeros((50, 12, 256), dtype=torch.bfloat16, device="cuda")
    got = gdn_qk_norm_rope(q, k, pos, f, norm_eps=1e-6, q_out=out[:, 2:8], k_out=out[:, 9:11])
    assert got[0].data_ptr() == out[:, 2:8].data_ptr()
    assert torch.equal(out[:, 2:8], want[0]) and torch.equal(out[:, 9:11], want[1])
    assert not out[:, :2].any() and not out[:, 8].any() and not out[:, 11].any()
    rest = x[:, 8:].clone()
    gdn_qk_norm_rope(q, k, pos, f, norm_eps=1e-6, q_out=q, k_out=k)
    assert torch.equal(x[:, :6], want[0]) and torch.equal(x[:, 6:8], want[1]) and torch.equal(x[:, 8:], rest)


def test_offsets_past_32_bits():
    """A token stride that puts the last rows beyond 2^31 elements and 2^32 bytes."""
    T, stride = 3, 1 << 30
    buf = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((T, 2, 128), (stride, 128, 1))
    src = normal(gen(9), T, 2, 128).cuda()
    q.copy_(src)
    pos, f = torch.tensor([3, 40, 500], dtype=torch.int32).cuda(), freqs(128).cuda()
    want = gdn_qk_norm_rope(src, src, pos, f)
    got = gdn_qk_norm_rope(q, src, pos, f, q_out=q)
    assert torch.equal(got[0], want[0]) and torch.equal(q, want[0]) and torch.equal(got[1], want[1])


def test_many_tokens_and_no_tokens():
    """Every split of a token's rows over warps gives the same rows."""
    f, w = freqs(64).cuda(), torch.rand(256, device="cuda")
    T = 20000
    x = torch.randn((T, 20, 256), device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    q, k = gdn_qk_norm_rope(x[:, :16], x[:, 16:], pos, f, w, w, 1e-6)
    for n in (1, 60, 300, 1500, 7001):
        a, b = gdn_qk_norm_rope(x[T - n:, :16], x[T - n:, 16:], pos[T - n:].clone(), f, w, w, 1e-6)
        assert torch.equal(a, q[T - n:]) and torch.equal(b, k[T - n:])
    a, b = gdn_qk_norm_rope(x[:0, :16], x[:0, 16:], pos[:0], f)
    assert a.shape == (0, 16, 256) and b.shape == (0, 4, 256)


# ------------------------------------------------------------------ into the cache
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,page,h_q,h_kv,rotary,interleaved,norm", [
    (128, 8, 4, 1, 128, False, True), (128, 64, 9, 3, 32, True, False), (256, 16, 16, 2, 64, False, True),
    (256, 1024, 1, 1, 256, True, True), (128, 16, 0, 5, 64, False, True)])
def test_append_is_the_two_calls(D, page, h_q, h_kv, rotary, interleaved, norm, fp8):
    new, start = [1, 0, 37, 130, 5], [0, 9, 63, 1, 2000]
    counts = [-(-(s + n) // page) for s, n in zip(start, new)]
    T, g = sum(new), gen(10)
    x, *_ = inputs(T, max(h_q, 1), h_kv, D, 11)
    x = x.cuda()
    h = max(h_q, 1)
    q, k, v = x[:, :h], x[:, h:h + h_kv], x[:, h + h_kv:h + 2 * h_kv]
    f = freqs(rotary).cuda()
    kw = dict(interleaved=interleaved)
    if norm:
        kw.update(q_weight=torch.randn(D, generator=g).cuda(), k_weight=torch.randn(D, generator=g).cuda(),
                  norm_eps=1e-6)
    cu, st = offsets(new), i32(start)
    at = torch.cat([torch.arange(s, s + n, dtype=torch.int32) for s, n in zip(start, new)]).cuda()
    for given in (None, torch.randint(0, 10 ** 6, (T,), generator=g, dtype=torch.int32).cuda()):
        one = Cache(counts, h_kv, D, page, fp8, 12)
        two = Cache(counts, h_kv, D, page, fp8, 12)
        got = gdn_kv_append_rope(q if h_q else None, k, v, one.k, one.v, one.table, cu, st, f, positions=given,
                                 **kw, **one.args())
        qo, ko = gdn_qk_norm_rope(q, k, at if given is None else given, f, **kw)
        gdn_kv_append(ko, v, two.k, two.v, two.table, cu, st, **two.args())
        assert gdn_stream_status() == "GDN_OK"
        assert (got is None) if not h_q else torch.equal(got, qo)
        for a, b in zip(one.bytes(), two.bytes()):
            assert torch.equal(a, b)


def test_append_with_axes_and_given_output():
    D, page, new = 128, 16, [33, 4]
    x, *_ = inputs(37, 4, 2, D, 13)
    x = x.cuda()
    pos = torch.randint(0, 5000, (3, 37), generator=gen(14), dtype=torch.int32).cuda()
    f, axes = freqs(96).cuda(), bytes(i % 3 for i in range(48))
    c, c2 = Cache([4, 1], 2, D, page, True, 15), Cache([4, 1], 2, D, page, True, 15)
    cu, st = offsets(new), i32([20, 3])
    want = gdn_qk_norm_rope(x[:, :4], x[:, 4:6], pos, f, norm_eps=0.1, axes=axes)
    gdn_kv_append(want[1], x[:, 6:8], c2.k, c2.v, c2.table, cu, st, **c2.args())
    got = gdn_kv_append_rope(x[:, :4], x[:, 4:6], x[:, 6:8], c.k, c.v, c.table, cu, st, f, positions=pos,
                             norm_eps=0.1, axes=axes, q_out=x[:, :4], **c.args())
    assert gdn_stream_status() == "GDN_OK" and got.data_ptr() == x.data_ptr()
    assert torch.equal(x[:, :4], want[0])
    for a, b in zip(c.bytes(), c2.bytes()):
        assert torch.equal(a, b)


def test_append_reports_bad_pages_and_offsets():
    D, page = 128, 16
    x, *_ = inputs(40, 2, 2, D, 16)
    x = x.cuda()
    f = freqs(64).cuda()
    call = lambda c, cu, st, q_out: gdn_kv_append_rope(  # noqa: E731
        x[:, :2], x[:, 2:4], x[:, 4:6], c.k, c.v, c.table, cu, st, f, q_out=q_out)
    want, _ = gdn_qk_norm_rope(x[:, :2], x[:, 2:4], torch.arange(40, dtype=torch.int32).cuda(), f)
    # a page that is missing: its rows are not written, q is
    c, ref = Cache([3], 2, D, page, False, 17), Cache([3], 2, D, page, False, 17)
    c.table[0, 1] = -1
    q_out = torch.zeros_like(want)
    call(c, offsets([40]), i32([0]), q_out)
    assert gdn_stream_status() == "GDN_ERR_BAD_PAGE" and torch.equal(q_out, want)
    gdn_kv_append_rope(None, x[:16, 2:4], x[:16, 4:6], ref.k, ref.v, ref.table, offsets([16]), i32([0]), f)
    gdn_kv_append_rope(None, x[32:, 2:4], x[32:, 4:6], ref.k, ref.v, ref.table, offsets([8]), i32([32]), f)
    assert gdn_stream_status() == "GDN_OK"
    assert torch.equal(c.k, ref.k) and torch.equal(c.v, ref.v)
    # tokens that no sequence holds: nothing of theirs is written
    c = Cache([3], 2, D, page, False, 17)
    before, q_out = c.bytes(), torch.zeros_like(want)
    call(c, i32([30, 40]), i32([0]), q_out)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
    assert not q_out[:30].any() and torch.equal(q_out[30:], gdn_qk_norm_rope(
        x[30:, :2], x[30:, 2:4], torch.arange(10, dtype=torch.int32).cuda(), f)[0])
    changed = [(a != b).sum() for a, b in zip(before, c.bytes())]
    assert all(0 < int(n) <= 10 * 2 * D * 2 for n in changed)


def test_captured_and_replayed():
    """One graph of both calls, replayed over new inputs in place."""
    D, page, T = 256, 64, 6
    x, *_ = inputs(T, 4, 2, D, 18)
    x = x.cuda()
    f, pos = freqs(64).cuda(), torch.arange(T, dtype=torch.int32).cuda()
    c = Cache([1] * T, 2, D, page, True, 19)
    cu, st = offsets([1] * T), i32(list(range(T)))

    def step():
        a = gdn_qk_norm_rope(x[:, :4], x[:, 4:6], pos, f, norm_eps=1e-6)
        b = gdn_kv_append_rope(x[:, :4], x[:, 4:6], x[:, 6:8], c.k, c.v, c.table, cu, st, f, norm_eps=1e-6,
                               **c.args())
        return a[0], a[1], b

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (20, 21):
        x.copy_(inputs(T, 4, 2, D, seed)[0])
        st.add_(1)
        pos.add_(1)
        g.replay()
        replayed, pool = [t.clone() for t in got], c.bytes()
        want = step()
        assert gdn_stream_status() == "GDN_OK"
        for a, b in zip(replayed + pool, list(want) + c.bytes()):
            assert torch.equal(a, b)
        assert torch.equal(want[0], want[2])  # positions and places are the same here


@pytest.mark.parametrize("name", ["dense", "append"])
def test_on_another_stream(name):
    x, *_ = inputs(30, 4, 2, 128, 22)
    x = x.cuda()
    f, pos = freqs(64).cuda(), torch.arange(30, dtype=torch.int32).cuda()
    c = Cache([2], 2, 128, 16, False, 23)
    cu, st = offsets([30]), i32([0])

    def call(s):
        if name == "dense":
            return gdn_qk_norm_rope(x[:, :4], x[:, 4:6], pos, f, stream=s)
        return gdn_kv_append_rope(x[:, :4], x[:, 4:6], x[:, 6:8], c.k, c.v, c.table, cu, st, f, stream=s),

    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = call(stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gdn_stream_status(s) == "GDN_OK"


def test_binding_refuses():
    x = torch.zeros((4, 3, 128), dtype=torch.bfloat16, device="cuda")
    f, p = torch.ones(32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    call = lambda **kw: gdn_qk_norm_rope(**{**dict(q=x, k=x, positions=p, inv_freq=f), **kw})  # noqa: E731
    for kw in (dict(q=x.half()), dict(k=x[:3]), dict(positions=p.long()), dict(positions=p[:3]), dict(positions=None),
               dict(positions=p[None].repeat(3, 1)), dict(inv_freq=f.double()), dict(inv_freq=f[None]),
               dict(inv_freq=f[::2]), dict(q_weight=f), dict(norm_eps=1e-6, q_weight=f),
               dict(axes=[0] * 31), dict(axes=[0] * 31 + [1]), dict(axes=[0] * 32, positions=p[None].repeat(2, 2)),
               dict(axes=[0] * 31 + [256]), dict(q_out=x[:, :2]), dict(k_out=x.float()), dict(q_out=x.cpu()),
               dict(q=x.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(norm_eps="x")
    for kw in (dict(inv_freq=f[:30]), dict(inv_freq=torch.ones(68, device="cuda")), dict(inv_freq=f[:0]),
               dict(norm_eps=-1.0)):
        with pytest.raises(RuntimeError):
            call(**kw)
    with pytest.raises(ValueError):
        gdn_kv_append_rope(None, x[:, :1], x[:, :1], x[None, :1, :, :], x[None, :1, :, :], p[None, :1], p[:2], p[:1], f,
                           axes=[0] * 32)
    torch.cuda.synchronize()
    assert gdn_stream_status() == "GDN_OK"


def test_outputs_share_an_allocation_and_nothing_else():
    q, k = torch.randn(5, 3, 128).bfloat16().cuda(), torch.randn(5, 2, 128).bfloat16().cuda()
    pos, f = torch.zeros(5, dtype=torch.int32).cuda(), torch.ones(8).cuda()
    a, b = gdn_qk_norm_rope(q, k, pos, f)  # (position 0: as they were)
    assert a.shape == q.shape and b.shape == k.shape and a.is_contiguous() and b.is_contiguous()
    a.zero_()
    assert torch.equal(b, k) and a._version == 1 and b._version == 0
    b.fill_(2)
    assert not a.any()
    del a
    torch.full((5, 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert (b == 2).all()
    with torch.inference_mode():
        a, b = gdn_qk_norm_rope(q, k, pos, f)
        assert torch.equal(a, q) and torch.equal(b, k) and b.is_inference()
    a, b = gdn_qk_norm_rope(q[:0], k[:0], pos[:0], f)
    assert a.shape == (0, 3, 128) and b.shape == (0, 2, 128)
