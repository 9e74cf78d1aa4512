"""The serving path together, key by key: queries that put all their weight on one cached
row get that row's value, from decoding over the cache and from prompt attention over the
gathered rows, whichever row it is.  A neighbouring row, page or sequence would show.

The target's score is above 8 sqrt(D) / 2 = 45 (D = 128) where the others stay below 30, so
the rest weighs under 2,048 e^-15 = 2^-10.6; the weights and o are rounded by 2^-8 each."""
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_attn_decode_paged, gdn_attn_prefill,
                                                    gdn_kv_append, gdn_kv_gather, gdn_stream_status)
from tests.attention_util import BF16, gen, normal, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D,page", [(128, 16), (256, 64), (256, 8)])
def test_each_query_finds_its_row(D, page, bits):
    h_kv, G, L = 2, 4, 2000
    targets = sorted({0, 1, 7, 8, page - 1, page, 15, 16, 31, 32, 63, 64, 127, 128, 129, 255, 256, 1023, 1024,
                      1500, L - 2 * page, L - page, L - 2, L - 1})
    B = len(targets)
    lens = [L - n % 3 * page // 2 if t < 1500 else L for n, t in enumerate(targets)]
    g = gen(110)
    T = sum(lens)
    k = normal(g, T, h_kv, D).cuda()
    # rows of one length, so that no other row scores near the target
    k = (k.float() * (D ** 0.5 / k.float().norm(dim=-1, keepdim=True))).to(torch.bfloat16)
    v = normal(g, T, h_kv, D).cuda()
    counts = [-(-n // page) for n in lens]
    order = torch.randperm(sum(counts), generator=g).int()
    table = torch.full((B, max(counts)), -1, dtype=torch.int32)
    at = 0
    for n, c in enumerate(counts):
        table[n, :c] = order[at:at + c]
        at += c
    table = table.cuda()
    shape = (sum(counts), h_kv, page, D)
    pages = [torch.zeros(shape, dtype=torch.float8_e4m3fn if bits == 8 else torch.bfloat16, device="cuda")
             for _ in range(2)]
    exps = {n: torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for n in ("k_exp", "v_exp")} if bits == 8 else {}
    cu, zero = offsets(lens), torch.zeros(B, dtype=torch.int32, device="cuda")
    # in two pieces, the second from the middle of a page
    cut = [n // 2 + 3 for n in lens]
    first = torch.cat([torch.arange(int(cu[n]), int(cu[n]) + c) for n, c in enumerate(cut)]).cuda()
    rest = torch.cat([torch.arange(int(cu[n]) + c, int(cu[n + 1])) for n, c in enumerate(cut)]).cuda()
    gdn_kv_append(k[first], v[first], *pages, table, offsets(cut), zero, **exps)
    gdn_kv_append(k[rest], v[rest], *pages, table, offsets([n - c for n, c in zip(lens, cut)]),
                  torch.tensor(cut, dtype=torch.int32, device="cuda"), **exps)
    rk, rv = gdn_kv_gather(*pages, table, cu, zero, T, **exps)
    if bits == 16:
        assert torch.equal(rk, k) and torch.equal(rv, v)
    rows = torch.tensor([int(cu[n]) + t for n, t in enumerate(targets)], device="cuda")
    q = (4 * k[rows].float()).to(torch.bfloat16).repeat_interleave(G, dim=1)
    want = rv[rows].double().repeat_interleave(G, dim=1)
    top = rv.double().abs().max()
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    decoded = gdn_attn_decode_paged(q, *pages, table, length, **exps)
    prompted = gdn_attn_prefill(q, rk, rv, offsets([1] * B), cu)
    assert gdn_stream_status() == "GDN_OK"
    for got in (decoded, prompted):
        assert ((got.double() - want).abs() <= 2 * BF16 * want.abs() + 2.0 ** -10.6 * top).all()
