"""Decode attention over the paged cache against the fp64 oracle (bounds:
tests/attention_util.py), bf16 and e4m3: lengths, pages, heads, units of every size,
slots and pages that must not be read, and the call's ways of failing."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_attn_decode_paged,
                                                    gdn_attn_decode_paged_workspace_size,
                                                    gdn_stream_status)
from oracle.paged_attention import cached_rows, decode, dequantise, quantise
from tests.attention_util import BF16, F16, check, gen, normal

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def build(lens, h_kv, D, page, fp8, seed, rows=None, extra=3):
    """Pools (values kept in fp64 beside them) and a table; slots past a sequence's
    length, unused pages and unused table entries poisoned."""
    g = gen(seed)
    counts = [-(-n // page) for n in lens]
    P = sum(counts) + extra
    order = torch.randperm(P, generator=g)
    table = torch.full((len(lens), max(counts + [0]) + 1), -1, dtype=torch.int32)
    used = torch.zeros((P, page), dtype=torch.bool)
    at = 0
    for n, c in enumerate(counts):
        table[n, :c] = order[at:at + c]
        for p in range(lens[n]):
            used[order[at + p // page], p % page] = True
        at += c
    out = dict(table=table.cuda(), lens=i32(lens))
    for name in ("k", "v"):
        x = normal(g, P, h_kv, page, D)
        if rows is not None:
            x = rows(name, x, g)
        mask = used[:, None, :, None].expand_as(x)
        if fp8:
            vals, e = quantise(x)
            codes = torch.tensor(vals).to(torch.float32).to(E4M3)
            exps = torch.tensor(e + 127).to(torch.uint8)
            out[name + "_vals"] = dequantise(vals, e)
            codes = torch.where(mask, codes.view(torch.uint8), torch.tensor(0x7f, dtype=torch.uint8))
            out[name] = codes.view(E4M3).cuda()
            out[name + "_exp"] = torch.where(mask[..., 0], exps, torch.tensor(255, dtype=torch.uint8)).cuda()
        else:
            out[name + "_vals"] = x.double().numpy()
            out[name] = torch.where(mask, x, torch.tensor(float("nan"), dtype=x.dtype)).cuda()
            out[name + "_exp"] = None
    return out


def reference(c, q, lens, page, scale):
    o, wabs = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        t = c["table"][b].cpu()
        k, v = cached_rows(c["k_vals"], t, n, page), cached_rows(c["v_vals"], t, n, page)
        o[b], wabs[b] = decode(q[b], k, v, scale), decode(q[b], k, np.abs(v), scale)
    return o, wabs


def call(c, q, scale=None, **kw):
    return gdn_attn_decode_paged(q, c["k"], c["v"], c["table"], c["lens"], k_exp=c["k_exp"],
                                 v_exp=c["v_exp"], scale=scale, **kw)


def agrees(lens, h_q=16, h_kv=2, D=256, page=64, fp8=False, seed=0, scale=None, rows=None, q_times=1.0):
    c = build(lens, h_kv, D, page, fp8, seed, rows)
    q = normal(gen(seed + 1000), len(lens), h_q, D) * q_times
    scale = D ** -0.5 if scale is None else scale
    o = call(c, q.cuda(), scale)
    assert gdn_stream_status() == "GDN_OK"
    ref, wabs = reference(c, q, lens, page, scale)
    check(o, ref, wabs, F16 if fp8 else 2.0 ** -16)
    return c, q, o


FORMS = [(128, False), (128, True), (256, False), (256, True)]


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (2, 1), (6, 2), (4, 1), (15, 3), (6, 1), (14, 2), (16, 2)])
def test_group_sizes(h_q, h_kv, D, fp8):
    agrees([200, 1, 77], h_q, h_kv, D, fp8=fp8, seed=h_q)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("page", [8, 16, 32, 128, 1024])
def test_pages(page, D, fp8):
    """Pages smaller and larger than a tile, lengths that end anywhere inside them."""
    agrees([1030, 333, 1, 0, 8, 64, 127], 8, 2, D, page, fp8, seed=page)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129, 257])
def test_lengths(n, D, fp8):
    agrees([n], 8, 1, D, 16, fp8, seed=n)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_long_and_ragged(D, fp8):
    """Several CTAs on one sequence, several sequences on one CTA, empty ones between."""
    agrees([5000, 0, 0, 3, 900, 1, 0, 2100], 8, 2, D, 32, fp8, seed=21)
    r = np.random.default_rng(2)
    agrees([int(x) for x in r.integers(0, 60, 700)], 4, 1, D, 8, fp8, seed=22)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_one_sequence_on_every_cta(D, fp8):
    agrees([40000], 2, 1, D, 256, fp8, seed=23)


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("h_q,h_kv", [(8, 8), (16, 2)])
def test_one_long_sequence_among_many(h_q, h_kv, D, fp8):
    """One sequence on many CTAs (more of them than query heads and parts of a row, and in
    other layouts fewer), every other one on a part of a CTA or empty; and a batch of more
    than 32 with less work than there are CTAs."""
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(0, 40, 150)]
    lens[70] = 12000
    lens[71] = lens[149] = 0
    agrees(lens, h_q, h_kv, D, 16, fp8, seed=42)
    agrees([0] * 20 + [1, 700, 0] + [2] * 15, h_q, h_kv, D, 16, fp8, seed=43)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_calls_one_after_the_other(D, fp8):
    """Calls that follow each other without a wait between, with very
    different shares, give what each gives alone."""
    cases = []
    for seed, lens in ((44, [3000, 50]), (45, [60] * 90), (46, [9000]), (47, [0, 1, 500] * 15)):
        c = build(lens, 2, D, 16, fp8, seed=seed)
        q = normal(gen(seed), len(lens), 8, D).cuda()
        cases.append((c, q, call(c, q)))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, q, alone in cases:
            assert torch.equal(call(c, q), alone)
    outs = [[call(c, q) for c, q, _ in cases] for _ in range(10)]
    for got in outs:
        for (_, _, alone), o in zip(cases, got):
            assert torch.equal(o, alone)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_all_empty(D, fp8):
    _, _, o = agrees([0, 0, 0], 8, 2, D, 16, fp8, seed=24)
    assert (o == 0).all()


@pytest.mark.parametrize("D,fp8", FORMS)
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.5])
def test_scales(scale, D, fp8):
    agrees([700, 30], 8, 1, D, 16, fp8, seed=25, scale=scale)


@pytest.mark.parametrize("D", [128, 256])
def test_units_of_every_size(D):
    """Rows of V whose units span 2^-100 .. 2^60 in one sequence, and rows of zeros: the
    weights of the small ones count in the sum whatever their values are."""
    def rows(name, x, g):
        if name == "v":
            e = torch.randint(-100, 60, x.shape[:3], generator=g).double()
            x = (x.double() * torch.exp2(e)[..., None]).to(torch.bfloat16)
            x[:, :, 3] = 0
        return x
    agrees([300, 40], 8, 2, D, 16, True, seed=26, rows=rows)

    def tiny(name, x, g):  # every value small: nothing may underflow on the way
        return (x.double() * 2.0 ** -110).to(torch.bfloat16) if name == "v" else x
    c, q, o = agrees([300], 8, 2, D, 16, True, seed=27, rows=tiny)
    ref, _ = reference(c, q, [300], 16, D ** -0.5)
    err = np.linalg.norm(o.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert err < BF16 + F16


@pytest.mark.parametrize("D", [128, 256])
def test_keys_and_queries_of_every_size(D):
    """Units of K and sizes of q that make the same scores from very different numbers."""
    for kx, qx in ((2.0 ** 40, 2.0 ** -40), (2.0 ** -60, 2.0 ** 60), (1.0, 1.0)):
        agrees([200], 8, 1, D, 16, True, seed=28, q_times=qx,
               rows=lambda name, x, g, s=kx: x * s if name == "k" else x)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_growing_scores_rescale(D, fp8):
    def rows(name, x, g):
        return x * 8 if name == "k" else x
    agrees([2000], 8, 1, D, 64, fp8, seed=29, scale=0.02, rows=rows)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_order_of_the_pages_changes_nothing(D, fp8):
    """The same rows on other pages: the same bits; and the same bits every time, whatever
    the workspace holds."""
    lens, page = [3000, 50], 16
    c = build(lens, 2, D, page, fp8, seed=30)
    q = normal(gen(31), 2, 12, D).cuda()
    o = call(c, q)
    ws = torch.empty(gdn_attn_decode_paged_workspace_size(12, 2, D), dtype=torch.uint8, device="cuda")
    for byte in (0, 0xff):
        ws.fill_(byte)
        assert torch.equal(call(c, q, workspace=ws), o)
    perm = torch.randperm(c["k"].shape[0], generator=gen(32)).cuda()
    inv = torch.argsort(perm)
    d = dict(c, table=torch.where(c["table"] >= 0, inv[c["table"].clamp(min=0).long()].int(), -1))
    for name in ("k", "v"):
        d[name] = c[name].view(torch.uint8)[perm].view(c[name].dtype)
        if fp8:
            d[name + "_exp"] = c[name + "_exp"][perm]
    assert torch.equal(call(d, q), o) and gdn_stream_status() == "GDN_OK"


@pytest.mark.parametrize("D,fp8", FORMS)
def test_pages_that_are_missing(D, fp8):
    """Rows without a page take no part; the error is reported."""
    lens, page = [100, 64], 16
    c = build(lens, 2, D, page, fp8, seed=33)
    q = normal(gen(34), 2, 8, D)
    ref1, wabs1 = reference(c, q, lens, page, D ** -0.5)
    good = c["table"].clone()
    for bad in (-1, c["k"].shape[0], 1 << 30):
        c["table"] = good.clone()
        c["table"][0, 2] = bad
        o = call(c, q.cuda())
        assert gdn_stream_status() == "GDN_ERR_BAD_PAGE" and gdn_stream_status() == "GDN_OK"
        keep = [i for i in range(100) if i // page != 2]
        k, v = (cached_rows(c[x + "_vals"], good[0], 100, page)[:, keep] for x in ("k", "v"))
        ref, wabs = decode(q[0], k, v, D ** -0.5), decode(q[0], k, np.abs(v), D ** -0.5)
        check(o[:1], ref[None], wabs[None], F16 if fp8 else 2.0 ** -16)
        check(o[1:], ref1[1:], wabs1[1:], F16 if fp8 else 2.0 ** -16)


def test_bad_lengths_are_reported():
    c = build([30, 30], 2, 128, 16, False, seed=35)
    q = normal(gen(36), 2, 8, 128).cuda()
    ref = call(c, q)
    for bad in (49, -1, 1 << 30):  # the table has three entries: 48 rows
        c["lens"] = i32([bad, 30])
        o = call(c, q)
        assert gdn_stream_status() == "GDN_ERR_BAD_CACHE_LEN" and gdn_stream_status() == "GDN_OK"
        assert (o[0] == 0).all() and torch.equal(o[1], ref[1])


@pytest.mark.parametrize("D,fp8", FORMS)
def test_strided_queries_and_a_given_output(D, fp8):
    c = build([300, 20], 2, D, 16, fp8, seed=37)
    x = normal(gen(38), 2, 12, D).cuda()
    ref = call(c, x[:, 2:10].contiguous())
    assert torch.equal(call(c, x[:, 2:10]), ref)
    n = 2 * 8 * D
    buf = torch.full((n + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    call(c, x[:, 2:10], o=buf[128:128 + n].view(2, 8, D))
    assert gdn_stream_status() == "GDN_OK"
    assert torch.equal(buf[128:128 + n].view(2, 8, D), ref)
    assert (buf[:128] == 7).all() and (buf[128 + n:] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_values_that_are_not_finite(fp8):
    """A cached NaN reaches the heads that read its row, in its own dimension only."""
    def rows(name, x, g):
        if name == "v":
            x[:, 1, :, 9] = float("nan")
        return x
    c = build([200], 2, 128, 16, fp8, seed=39, rows=rows)
    q = normal(gen(40), 1, 8, 128)
    o = call(c, q.cuda())
    assert gdn_stream_status() == "GDN_OK"
    bad = torch.zeros((1, 8, 128), dtype=torch.bool)
    bad[:, 4:, 9] = True
    assert torch.equal(torch.isnan(o.cpu()), bad)


def test_offsets_past_32_bits():
    """A pool of 9.7e6 rows of 256 values; the sequence's pages are its first and last."""
    page, P = 1024, 9500
    k = torch.empty((P, 1, page, 256), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    x = normal(gen(41), 2, 1, page, 256).cuda()
    k[[P - 1, 0]], v[[P - 1, 0]] = x, -x
    q = normal(gen(42), 1, 4, 256).cuda()
    o = gdn_attn_decode_paged(q, k, v, i32([[P - 1, 0]]), i32([1500]))
    small = gdn_attn_decode_paged(q, x, -x, i32([[0, 1]]), i32([1500]))
    assert gdn_stream_status() == "GDN_OK" and torch.equal(o, small)


@pytest.mark.parametrize("D,fp8", FORMS)
def test_on_another_stream_and_in_a_graph(D, fp8):
    c = build([900, 5, 64], 2, D, 16, fp8, seed=43)
    q = normal(gen(44), 3, 8, D).cuda()
    ref = call(c, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(c, q, stream=s)
    assert gdn_stream_status(s) == "GDN_OK" and torch.equal(got, ref)
    o = torch.empty_like(ref)
    ws = torch.empty(gdn_attn_decode_paged_workspace_size(8, 2, D), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, q, o=o, workspace=ws)
    for _ in range(3):
        o.zero_()
        g.replay()
        assert gdn_stream_status() == "GDN_OK" and torch.equal(o, ref)
