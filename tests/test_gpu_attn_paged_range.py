"""Decode attention over the paged cache where sizes differ: rows of V next to rows of
zeros or to one very large channel, a long tail of small weights, values, and keys with
queries, at the ends of bf16's range, NaN codes.  Both cache types against the fp64 oracle over the cached values.

Bounds, by element, from the arithmetic (A = the oracle's attention over |v|, A >= |o|):
o is stored in bf16, 2^-8 |o|; the weights are bf16 pairs, 2^-16 A, or one fp16, 2^-11 A;
scores, exponentials and the sums of weights 2^-10 A together (a thread's sum has at most
L / (CTAs x 32) + 40 terms of one sign, each off by 2^-24 of the sum: below 2^-14 for the
lengths here).  No absolute term but bf16's smallest number: what a weight loses must be
small against its own product."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_stream_status
from tests.attention_util import BF16, F16, gen, normal
from tests.test_gpu_attn_paged import FORMS, build, call, reference

pytestmark = pytest.mark.gpu


def close(c, q, lens, page, scale):
    o = call(c, q.cuda(), scale)
    assert gdn_stream_status() == "GDN_OK"
    ref, wabs = reference(c, q, lens, page, scale)
    got = o.double().cpu().numpy()
    assert np.isfinite(got).all()
    bound = (F16 + 2.0 ** -10) * wabs + BF16 * np.abs(ref) + 2.0 ** -133
    err = np.abs(got - ref)
    at = np.unravel_index((err - bound).argmax(), err.shape)
    assert (err <= bound).all(), f"err {err[at]:.3e} > bound {bound[at]:.3e}, ref {ref[at]:.3e} at {at}"
    return got, ref


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("power", [20, 30, 100])
def test_one_large_channel_beside_ordinary_rows(power, D, fp8):
    """Every eighth row of V is 2^power in channel 5 and zero elsewhere: the other channels
    come from the other rows alone."""
    def rows(name, x, g):
        if name == "v":
            x[:, :, 3::8] = 0
            x[:, :, 3::8, 5] = 2.0 ** power
        return x
    lens = [2, 300, 40]
    close(build(lens, 2, D, 16, fp8, 60, rows), normal(gen(61), 3, 8, D), lens, 16, D ** -0.5)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("power", [-20, -40, -100])
def test_rows_of_zeros_among_small_values(power, D, fp8):
    """A row of zeros has the unit 1, far above that of small values."""
    def rows(name, x, g):
        if name == "v":
            x = (x.double() * 2.0 ** power).to(x.dtype)
            x[:, :, 2::5] = 0
        return x
    lens = [300, 1, 40]
    close(build(lens, 2, D, 16, fp8, 62, rows), normal(gen(63), 3, 8, D), lens, 16, D ** -0.5)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("down", [18.0, 21.0, 24.5])
def test_a_long_tail_of_small_weights(down, D, fp8):
    """One key with the largest weight and 131,071 others 2^-down of it, whose values are
    the only ones that are not zero: their shares have to count in full."""
    lens, page = [131072], 1024

    def rows(name, x, g):
        if name == "k":
            x[...] = 0
            x[..., 0] = -down  # a score of -down log(2), by the scale below
        return x
    c = build(lens, 1, D, page, fp8, 64, rows)
    first = int(c["table"][0, 0])
    for name, value in (("k", 0.0), ("v", 0.0)):  # the sequence's first row
        c[name + "_vals"][first, 0, 0] = value
        raw = c[name].view(torch.uint8) if fp8 else c[name]
        raw[first, 0, 0] = 0
    q = torch.zeros((1, 4, D), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    close(c, q, lens, page, float(np.log(2.0)))


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("power", [116, -118])
def test_keys_and_queries_at_the_ends_of_the_range(power, D, fp8):
    """Ordinary scores from keys of 2^power and queries of 2^-power."""
    def rows(name, x, g):
        return (x.double() * 2.0 ** power).to(x.dtype) if name == "k" else x
    lens = [200, 9]
    q = (normal(gen(66), 2, 8, D).double() * 2.0 ** -power).to(torch.bfloat16)
    close(build(lens, 1, D, 16, fp8, 65, rows), q, lens, 16, D ** -0.5)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_values_at_the_ends_of_the_range(D, fp8):
    """Values of 2^112 and of 2^-112 in one sequence, in channels of their own."""
    def rows(name, x, g):
        if name == "v":
            even = torch.zeros_like(x)
            even[:, :, 0::2, 0::2] = (x[:, :, 0::2, 0::2].double() * 2.0 ** 112).to(x.dtype)
            even[:, :, 1::2, 1::2] = (x[:, :, 1::2, 1::2].double() * 2.0 ** -112).to(x.dtype)
            return even
        return x
    lens = [150, 2]
    close(build(lens, 2, D, 16, fp8, 67, rows), normal(gen(68), 2, 8, D), lens, 16, D ** -0.5)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n", [1, 31, 33, 500])
def test_codes_that_are_nan(n, D):
    """NaN codes of either sign in V: in their own channels, for the heads that read them,
    wherever in a tile the row lies; in K: every channel of those heads."""
    lens = [n, 40]
    c = build(lens, 2, D, 16, True, 69)
    q = normal(gen(70), 2, 8, D).cuda()
    good = call(c, q)
    assert torch.isfinite(good).all()
    r = np.random.default_rng(n)
    for trial in range(6):
        p = [0, n - 1][trial] if trial < 2 else int(r.integers(0, n))
        d = int(r.integers(0, D))
        page, slot = int(c["table"][0, p // 16]), p % 16
        v = c["v"].view(torch.uint8)
        was = int(v[page, 1, slot, d])
        v[page, 1, slot, d] = 0x7f if trial % 2 else 0xff
        got = call(c, q)
        want = torch.zeros_like(got, dtype=torch.bool)
        want[0, 4:, d] = True
        assert torch.equal(torch.isnan(got), want)
        assert torch.equal(torch.where(want, good, got), good)
        v[page, 1, slot, d] = was
        k = c["k"].view(torch.uint8)
        was = int(k[page, 1, slot, d])
        k[page, 1, slot, d] = 0x7f
        got = call(c, q)
        assert torch.isnan(got[0, 4:]).all() and torch.equal(got[0, :4], good[0, :4])
        assert torch.equal(got[1], good[1])
        k[page, 1, slot, d] = was
    assert gdn_stream_status() == "GDN_OK"


def test_every_code_and_unit():
    """A sequence of one row gives the row back: each of the 254 finite codes with units
    between 2^-107 and the largest that the append writes."""
    D = 256
    codes = torch.arange(256, dtype=torch.uint8)
    codes[0x7f], codes[0xff] = 0, 0
    bytes_ = torch.tensor([20, 21, 60, 119, 126, 127, 128, 133, 134, 135, 136, 200, 240, 246], dtype=torch.uint8)
    n = len(bytes_)
    v = codes.repeat(n, 1, 8, 1).contiguous().view(torch.float8_e4m3fn).cuda()
    k = torch.zeros((n, 1, 8, D), dtype=torch.uint8).view(torch.float8_e4m3fn).cuda()
    c = dict(k=k, v=v, k_exp=torch.full((n, 1, 8), 127, dtype=torch.uint8).cuda(),
             v_exp=bytes_[:, None, None].expand(n, 1, 8).contiguous().cuda(),
             table=torch.arange(n, dtype=torch.int32).cuda()[:, None].contiguous(),
             lens=torch.ones(n, dtype=torch.int32).cuda())
    q = normal(gen(71), n, 3, D).cuda()
    o = call(c, q)
    assert gdn_stream_status() == "GDN_OK"
    want = codes.view(torch.float8_e4m3fn).double()[None] * torch.exp2(bytes_.double() - 127)[:, None]
    want = want.to(torch.bfloat16)[:, None].expand(n, 3, D)
    assert torch.equal(o.cpu(), want)
