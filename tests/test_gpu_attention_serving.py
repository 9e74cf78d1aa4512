"""Norms, rotation, the paged cache and attention over it together, as a server's step runs
them: against the operators that do the same in more calls, in a graph, on streams of their
own, and as examples/attention_serving.py runs them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_attn_decode_paged, gdn_attn_prefill,
                                                    gdn_attn_prefill_paged, gdn_kv_append,
                                                    gdn_kv_append_rope, gdn_kv_gather,
                                                    gdn_qk_norm_rope, gdn_stream_status)
from oracle.paged_attention import dequantise, quantise
from oracle.rope import rotate
from oracle.window_attention import attend
from tests.attention_util import BF16, check, gen, normal, offsets

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def freqs(rotary):
    n = rotary // 2
    return (1e6 ** (-torch.arange(n, dtype=torch.float64) / n)).float()


class Layer:
    def __init__(self, sequences, per_seq, h_kv, D, page, bits, seed):
        shape = (sequences * per_seq, h_kv, page, D)
        dtype = E4M3 if bits == 8 else torch.bfloat16
        self.k = torch.zeros(shape, dtype=torch.uint8 if bits == 8 else dtype, device="cuda").view(dtype)
        self.v = self.k.clone()
        self.exps = dict(k_exp=torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda"),
                         v_exp=torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda")) if bits == 8 else {}
        self.table = torch.randperm(shape[0], generator=gen(seed)).view(sequences, per_seq).int().cuda().contiguous()


STEPS = [([200, 0, 33], [0, 0, 0]), ([180, 70, 1], [200, 0, 33]), ([1, 5, 1], [380, 70, 34]), ([4, 1, 2], [381, 75, 35])]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D,h_q,h_kv,rotary,window,sinks", [(256, 8, 1, 64, 0, 0), (128, 6, 2, 128, 100, 3)])
def test_steps_against_the_formulas(D, h_q, h_kv, rotary, window, sinks, bits):
    """Four steps of three sequences (pieces of prompts, single and drafted tokens) against the
    oracles, whose q and k go through bf16 as the layer's do.  An element that rounds the other
    way moves a score by 2^-8 of one of its D products, below the scores' own term.  In the e4m3
    cache it may move a code by one step (an eighth), so there the rows read back are held
    against the oracle's, code by code, and are what the attention's oracle takes."""
    layer = Layer(3, 30, h_kv, D, 16, bits, 1)
    f, g = freqs(rotary), gen(2)
    wq, wk = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    past = [[], [], []]
    for new, start in STEPS:
        x = normal(g, sum(new), h_q + 2 * h_kv, D)
        xd, cu = x.cuda(), offsets(new)
        q = gdn_kv_append_rope(xd[:, :h_q], xd[:, h_q:h_q + h_kv], xd[:, h_q + h_kv:], layer.k, layer.v, layer.table, cu,
                               i32(start), f.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(), norm_eps=1e-6, **layer.exps)
        lengths = [s + a for s, a in zip(start, new)]
        o = gdn_attn_prefill_paged(q, layer.k, layer.v, layer.table, cu, i32(lengths), window=window or None,
                                   sinks=sinks, **layer.exps)
        assert gdn_stream_status() == "GDN_OK"
        at = np.concatenate([np.arange(s, s + a) for s, a in zip(start, new)])
        bf = lambda y: torch.from_numpy(y).to(torch.bfloat16)  # noqa: E731
        qr = bf(rotate(x[:, :h_q], at, f, weight=wq, eps=1e-6)[0])
        kr, v = bf(rotate(x[:, h_q:h_q + h_kv], at, f, weight=wk, eps=1e-6)[0]), x[:, h_q + h_kv:]
        if bits == 8:
            back = gdn_kv_gather(layer.k, layer.v, layer.table, cu, i32(start), sum(new), **layer.exps)
            kq, v = (torch.from_numpy(dequantise(*quantise(y))) for y in (kr, v))
            kr = back[0].double().cpu()
            assert torch.equal(back[1].double().cpu(), v)
            assert ((kr - kq).abs() <= kq.abs() / 8 + 2.0 ** -9 * kq.abs().amax(-1, keepdim=True) / 224).all()
            assert (kr != kq).double().mean() < 1e-3
        ref, size, t = [], [], 0
        for n, a in enumerate(new):
            past[n].append((kr[t:t + a], v[t:t + a]))
            rows = [torch.cat([y[i].double() for y in past[n]]).transpose(0, 1) for i in (0, 1)]
            r = attend(qr[t:t + a], *rows, D ** -0.5, window, sinks)
            ref.append(r[0])
            size.append(r[1])
            t += a
        check(o, np.concatenate(ref), np.concatenate(size), BF16, f"{new}")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D", [128, 256])
def test_against_the_calls_one_by_one(D, bits):
    """gdn_qk_norm_rope, gdn_kv_append, gdn_kv_gather and gdn_attn_prefill (for single tokens
    gdn_attn_decode_paged) give the same within the weights' rounding of both."""
    h_q, h_kv, page = 8, 2, 32
    new, start = [300, 1, 70, 1, 4], [0, 333, 65, 0, 500]
    lengths = [a + s for a, s in zip(new, start)]
    one, two = (Layer(5, 20, h_kv, D, page, bits, 3) for _ in range(2))
    f, cu, st = freqs(64).cuda(), offsets(new), i32(start)
    old = normal(gen(4), sum(start), 2 * h_kv, D).cuda()
    for layer in (one, two):
        gdn_kv_append(old[:, :h_kv], old[:, h_kv:], layer.k, layer.v, layer.table, offsets(start), i32([0] * 5), **layer.exps)
    x = normal(gen(5), sum(new), h_q + 2 * h_kv, D).cuda()
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    qo = gdn_kv_append_rope(q, k, v, one.k, one.v, one.table, cu, st, f, norm_eps=1e-6, **one.exps)
    got = gdn_attn_prefill_paged(qo, one.k, one.v, one.table, cu, i32(lengths), **one.exps)
    at = i32(np.concatenate([np.arange(s, s + a) for s, a in zip(start, new)]).tolist())
    q2, k2 = gdn_qk_norm_rope(q, k, at, f, norm_eps=1e-6)
    gdn_kv_append(k2, v, two.k, two.v, two.table, cu, st, **two.exps)
    assert torch.equal(qo, q2) and torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8))
    rk, rv = gdn_kv_gather(two.k, two.v, two.table, offsets(lengths), i32([0] * 5), sum(lengths), **two.exps)
    want = gdn_attn_prefill(q2, rk, rv, cu, offsets(lengths)).double()
    size = gdn_attn_prefill(q2, rk, rv.abs(), cu, offsets(lengths)).double() * (1 + BF16)
    single = [1, 3]
    rows = [int(cu[n]) for n in single]
    dec = gdn_attn_decode_paged(q2[rows].contiguous(), two.k, two.v, two.table[single].contiguous(),
                                i32([lengths[n] for n in single]), **two.exps).double()
    assert gdn_stream_status() == "GDN_OK"
    bound = 2 * ((BF16 + 2.0 ** -10) * size + BF16 * want.abs() + 1e-6)
    assert ((got.double() - want).abs() <= bound).all()
    assert ((got[rows].double() - dec).abs() <= bound[rows]).all()


def test_a_step_in_a_graph():
    """A server's step captured once and replayed with new tokens and lengths, its buffers kept."""
    D, h_q, h_kv, N = 128, 8, 2, 4
    layer, eager = (Layer(N, 40, h_kv, D, 16, 8, 6) for _ in range(2))
    f = freqs(128).cuda()
    x = normal(gen(7), N, h_q + 2 * h_kv, D).cuda()
    cu, start, length = offsets([1] * N), i32([0, 300, 17, 555]), i32([1, 301, 18, 556])
    old = normal(gen(8), 300 + 17 + 555, 2 * h_kv, D).cuda()
    for l in (layer, eager):
        gdn_kv_append(old[:, :h_kv], old[:, h_kv:], l.k, l.v, l.table, offsets([0, 300, 17, 555]), i32([0] * N), **l.exps)

    def step(l):
        q = gdn_kv_append_rope(x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], l.k, l.v, l.table, cu, start, f,
                               norm_eps=1e-6, **l.exps)
        o = gdn_attn_prefill_paged(q, l.k, l.v, l.table, cu, length, window=200, sinks=4, **l.exps)
        start.add_(1)
        length.add_(1)
        return o

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = start.clone(), length.clone()
    with torch.cuda.stream(s):
        step(layer)
    torch.cuda.current_stream().wait_stream(s)
    start.copy_(keep[0])
    length.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(layer)
    for i in range(20):
        x.copy_(normal(gen(100 + i), N, h_q + 2 * h_kv, D))
        at = start.clone(), length.clone()
        graph.replay()
        got = o.clone()
        start.copy_(at[0])
        length.copy_(at[1])
        assert torch.equal(got, step(eager))
    assert torch.equal(layer.k.view(torch.uint8), eager.k.view(torch.uint8))
    assert gdn_stream_status() == "GDN_OK"


def calls():
    D, h_q, h_kv = 128, 8, 2
    layer = Layer(3, 10, h_kv, D, 16, 16, 9)
    x = normal(gen(10), 236, h_q + 2 * h_kv, D).cuda()
    f, cu, st, lens = freqs(64).cuda(), offsets([150, 9, 77]), i32([0, 5, 20]), i32([150, 14, 97])
    pos = torch.arange(236, dtype=torch.int32, device="cuda")
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    cache = (layer.k, layer.v, layer.table)
    gdn_kv_append(k, v, *cache, cu, st)
    return {
        "rope": lambda s: gdn_qk_norm_rope(q, k, pos, f, norm_eps=1e-6, stream=s),
        "append": lambda s: (gdn_kv_append_rope(q, k, v, *cache, cu, st, f, stream=s),),
        "attend": lambda s: (gdn_attn_prefill_paged(q, *cache, cu, lens, stream=s),),
    }


def busy(ms=30):
    """Work that keeps the current stream for some tens of milliseconds."""
    x = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    for _ in range(8 * ms):
        x.fill_(1.0)


@pytest.mark.parametrize("name", ["rope", "append", "attend"])
def test_allocations_belong_to_the_given_stream(name):
    call = calls()[name]
    if name == "attend":
        calls()["append"](None)
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    busy()
    sizes = [n for w in want for n in [w.numel() * w.element_size()] * 4] + [1 << k for k in range(10, 26)] * 2
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    for t in held:
        t.fill_(0xff)
    del held, t
    got = call(s)
    s.synchronize()
    first = [t.clone() for t in got]
    torch.cuda.synchronize()
    assert gdn_stream_status(s) == "GDN_OK"
    for w, g, c in zip(want, got, first):
        assert torch.equal(g, w) and torch.equal(c, w)


@pytest.mark.parametrize("name", ["rope", "append", "attend"])
def test_outputs_are_kept_for_the_current_stream(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    for _ in range(2):
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
        busy(10)
        copies = [t.clone() for t in got]
        shapes = [(t.shape, t.dtype) for t in got]
        del got
        with torch.cuda.stream(s):
            for _ in range(4):
                for shape, dtype in shapes:
                    torch.empty(shape, dtype=dtype, device="cuda").fill_(float("nan"))
        torch.cuda.synchronize()
        for w, c in zip(want, copies):
            assert torch.equal(c, w)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "attention_serving", os.path.join(ROOT, "examples", "attention_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("window", [None, 300])
def test_example(example, bits, window):
    """Both attentions round o and their weights to bf16 (2^-8 each); random values: the
    outputs' size is near the largest weighted sum of |v| only up to a factor of about 4."""
    assert example.serve(5, 1100, 8, bits, window) <= 4 * 4 * BF16
