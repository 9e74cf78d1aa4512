"""The paged cache written and read back, against the fp64 oracle's rows (exact: the
codes, the exponent bytes and the values read back all follow from the definition)."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_kv_append, gdn_kv_gather, gdn_stream_status
from oracle.paged_attention import dequantise, quantise
from tests.attention_util import gen, normal, offsets

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


class Cache:
    """A pool of random content, and a table whose unused entries name no page."""

    def __init__(self, counts, h_kv, D, page, fp8, seed, extra=2, pad_entries=1):
        g = gen(seed)
        self.P = sum(counts) + extra
        shape = (self.P, h_kv, page, D)
        self.fp8, self.page = fp8, page
        rnd = lambda s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()  # noqa: E731
        if fp8:
            self.k, self.v = rnd(shape).view(E4M3), rnd(shape).view(E4M3)
            self.ke, self.ve = rnd(shape[:3]), rnd(shape[:3])
        else:
            self.k, self.v = normal(g, *shape).cuda(), normal(g, *shape).cuda()
            self.ke = self.ve = None
        order = torch.randperm(self.P, generator=g)
        self.table = torch.full((len(counts), max(counts + [0]) + pad_entries), -1, dtype=torch.int32)
        at = 0
        for n, c in enumerate(counts):
            self.table[n, :c] = order[at:at + c]
            at += c
        self.table = self.table.cuda()

    def bytes(self):
        return [t.view(torch.uint8).clone() for t in (self.k, self.v, self.ke, self.ve) if t is not None]

    def args(self):
        return dict(k_exp=self.ke, v_exp=self.ve)


def append(c, k, v, cu, start, **kw):
    gdn_kv_append(k, v, c.k, c.v, c.table, cu, start, **c.args(), **kw)


def gather(c, cu, start, total, **kw):
    return gdn_kv_gather(c.k, c.v, c.table, cu, start, total, **c.args(), **kw)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def expect(c, pages, exps, x, lens, start):
    """The pool after rows x were written: what the definition says, elsewhere unchanged."""
    want, want_e = pages.view(torch.uint8).clone().cpu(), None if exps is None else exps.clone().cpu()
    table, t = c.table.cpu(), 0
    if c.fp8:
        vals, e = quantise(x)
        codes = torch.tensor(vals).to(torch.float32).to(E4M3).view(torch.uint8)
    for n, (a, s) in enumerate(zip(lens, start)):
        for i in range(a):
            pg, slot = int(table[n, (s + i) // c.page]), (s + i) % c.page
            if c.fp8:
                want[pg, :, slot] = codes[t]
                want_e[pg, :, slot] = torch.tensor(e[t] + 127).to(torch.uint8)
            else:
                want[pg, :, slot] = x[t].contiguous().view(torch.uint8)
            t += 1
    return want, want_e


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("h_kv", [1, 2, 3, 8])
@pytest.mark.parametrize("page", [8, 64, 1024])
def test_rows_in_and_out(page, h_kv, D, fp8):
    """Sequences that start and end inside pages, an empty one, one token alone."""
    lens, start = [5, 0, 1, 40, 130], [3, 0, 63, 0, 7]
    counts = [-(-(s + a) // page) for s, a in zip(start, lens)]
    c = Cache(counts, h_kv, D, page, fp8, seed=page + h_kv)
    x = normal(gen(D), sum(lens), 2 * h_kv, D)
    x[3] *= 1000
    x[7] = 0
    k, v = x[:, :h_kv].cuda(), x[:, h_kv:].cuda()   # slices of one projection
    cu, st = offsets(lens), i32(start)
    kw, kwe = expect(c, c.k, c.ke, x[:, :h_kv], lens, start)
    vw, vwe = expect(c, c.v, c.ve, x[:, h_kv:], lens, start)
    append(c, k, v, cu, st)
    assert gdn_stream_status() == "GDN_OK"
    # NaN codes compare by value elsewhere in the file; here every code is a number
    assert torch.equal(c.k.view(torch.uint8).cpu(), kw) and torch.equal(c.v.view(torch.uint8).cpu(), vw)
    if fp8:
        assert torch.equal(c.ke.cpu(), kwe) and torch.equal(c.ve.cpu(), vwe)
    gk, gv = gather(c, cu, st, sum(lens))
    assert gdn_stream_status() == "GDN_OK"
    for got, rows in ((gk, x[:, :h_kv]), (gv, x[:, h_kv:])):
        want = rows.double().numpy() if not fp8 else dequantise(*quantise(rows))
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_values_of_every_size():
    """Rows around every edge of the format: largest value at and next to 448 units, ties,
    values below a unit's smallest step, the smallest and largest bf16, subnormals."""
    x = torch.zeros((40, 1, 128), dtype=torch.bfloat16)
    tops = [448.0, 450.0, 446.0, 1.75, 1.7578125, 3.0e38, 1.0, 2.0 ** -126, 2.0 ** -118, 1.75 * 2.0 ** -118,
            1.7656 * 2.0 ** -118, 9.2e-41, 1e-39]
    g = gen(1)
    for i, t in enumerate(tops):
        x[i, 0] = torch.rand(128, generator=g).to(torch.bfloat16) * t
        x[i, 0, 5] = t
        x[i, 0, 6] = -t
    x[20, 0, :8] = torch.tensor([448.0, 17.0, 19.0, 21.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11])
    x[21:40, 0] = normal(g, 19, 128) * (10.0 ** torch.linspace(-38, 38, 19))[:, None].to(torch.bfloat16)
    c = Cache([2], 1, 128, 32, True, seed=2)
    cu, st = offsets([40]), i32([0])
    append(c, x.cuda(), x.cuda(), cu, st)
    k, v = gather(c, cu, st, 40)
    assert gdn_stream_status() == "GDN_OK"
    want = torch.tensor(dequantise(*quantise(x))).to(torch.bfloat16)  # below 2^-133: bf16's own end
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


@pytest.mark.parametrize("D", [128, 256])
def test_values_that_are_not_finite(D):
    """Stored as NaN; the row's unit follows from its finite values alone."""
    x = normal(gen(3), 6, 2, D)
    x[0, 0, 3], x[1, 1, 0], x[2, 0, D - 1] = float("nan"), float("inf"), -float("inf")
    x[3, 0] = float("inf")
    c = Cache([1], 2, D, 8, True, seed=4)
    cu, st = offsets([6]), i32([1])
    append(c, x.cuda(), x.cuda(), cu, st)
    k, v = gather(c, cu, st, 6)
    assert gdn_stream_status() == "GDN_OK"
    want = dequantise(*quantise(x))
    for got in (k, v):
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_positions_without_a_page(fp8):
    """Past the table, at an entry that names no page, before the start: reported, not
    written, read back as zeros; the other rows are right."""
    c = Cache([2, 2], 2, 128, 8, fp8, seed=5, pad_entries=0)
    c.table[1, 1] = c.P
    x = normal(gen(6), 22, 2, 128).cuda()
    before = c.bytes()
    cu = offsets([6, 16])
    append(c, x, x, cu, i32([12, 0]))  # 0: positions 12 .. 17 of 16; 1: page 1 is missing
    assert gdn_stream_status() == "GDN_ERR_BAD_PAGE"
    k, v = gather(c, cu, i32([12, 0]), 22)
    assert gdn_stream_status() == "GDN_ERR_BAD_PAGE"
    sound = [0, 1, 2, 3] + list(range(6, 14))
    want = torch.zeros_like(x)
    rows = x.cpu()
    want[sound] = (rows if not fp8 else
                   torch.tensor(dequantise(*quantise(rows))).to(torch.bfloat16))[sound].cuda()
    assert torch.equal(k, want) and torch.equal(v, want)
    append(c, x[:3], x[:3], offsets([3, 0]), i32([-3, 0]))
    assert gdn_stream_status() == "GDN_ERR_BAD_PAGE" and gdn_stream_status() == "GDN_OK"
    kept = torch.ones(c.P, 8, dtype=torch.bool)
    table = c.table.cpu()
    kept[table[0, 1], 4:] = False
    kept[table[1, 0]] = False
    for now, was in zip(c.bytes(), before):
        assert torch.equal(now.transpose(1, 2)[kept.cuda()], was.transpose(1, 2)[kept.cuda()])


@pytest.mark.parametrize("cu", [[1, 4, 9], [0, 4, 8], [0, 7, 4, 9], [0, 4, 1 << 30], [-5, 4, 9], [0, -3, 9]])
def test_bad_offsets_are_reported(cu):
    c = Cache([2] * 3, 1, 128, 8, False, seed=7)
    n = len(cu) - 1
    c.table = c.table[:n].contiguous()
    x = normal(gen(8), 9, 1, 128).cuda()
    append(c, x, x, i32(cu), i32([0] * n))
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
    k, v = gather(c, i32(cu), i32([0] * n), 9)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS" and gdn_stream_status() == "GDN_OK"
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_more_sequences_than_a_warp_searches_at_once():
    r = np.random.default_rng(9)
    for n in (33, 1100):
        lens = [int(x) for x in r.integers(0, 3, n)]
        start = [int(x) for x in r.integers(0, 9, n)]
        c = Cache([2] * n, 1, 128, 8, True, seed=n)
        x = normal(gen(n), sum(lens), 1, 128)
        cu, st = offsets(lens), i32(start)
        append(c, x.cuda(), -x.cuda(), cu, st)
        k, v = gather(c, cu, st, sum(lens))
        assert gdn_stream_status() == "GDN_OK"
        want = torch.tensor(dequantise(*quantise(x))).to(torch.bfloat16)
        assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), -want)


def test_outputs_given_and_strided():
    c = Cache([3], 2, 256, 16, True, seed=10)
    x = normal(gen(11), 40, 2, 256).cuda()
    cu, st = offsets([40]), i32([2])
    append(c, x, x, cu, st)
    ref, _ = gather(c, cu, st, 40)
    buf = torch.full((40, 8, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    k, v = gather(c, cu, st, 40, k=buf[:, 1:3], v=buf[:, 5:7])
    assert gdn_stream_status() == "GDN_OK"
    assert torch.equal(buf[:, 1:3], ref) and torch.equal(buf[:, 5:7], ref)
    assert (buf[:, [0, 3, 4, 7]] == 5).all()


def test_offsets_past_32_bits():
    """A pool of 9.7e6 rows of 256 values: its last pages lie past 2^31 values and 2^32 bytes."""
    page, P = 1024, 9500
    k = torch.empty((P, 1, page, 256), dtype=torch.bfloat16, device="cuda")
    table = i32([[P - 1, 0, P - 2]])
    x = normal(gen(12), 3000, 1, 256).cuda()
    cu, st = offsets([3000]), i32([10])
    gdn_kv_append(x, -x, k, k.clone(), table, cu, st)
    v = torch.empty_like(k)
    gdn_kv_append(x, -x, k, v, table, cu, st)
    gk, gv = gdn_kv_gather(k, v, table, cu, st, 3000)
    assert gdn_stream_status() == "GDN_OK"
    assert torch.equal(gk, x) and torch.equal(gv, -x)
    assert torch.equal(k[P - 1, 0, 10:], x[:1014, 0])


def test_on_another_stream_and_in_a_graph():
    c = Cache([2], 2, 128, 64, True, seed=13)
    x = normal(gen(14), 100, 2, 128).cuda()
    cu, st = offsets([100]), i32([5])
    append(c, x, x, cu, st)
    ref, _ = gather(c, cu, st, 100)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    append(c, -x, -x, cu, st, stream=s)
    got, _ = gather(c, cu, st, 100, stream=s)
    assert gdn_stream_status(s) == "GDN_OK" and torch.equal(got, -ref)
    k, v = torch.empty_like(x), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        append(c, x, x, cu, st)
        gather(c, cu, st, 100, k=k, v=v)
    g.replay()
    assert gdn_stream_status() == "GDN_OK" and torch.equal(k, ref) and torch.equal(v, ref)
