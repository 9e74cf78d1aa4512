"""Offsets that break the packing rules are reported by the cache's calls, also where
every token still finds a sequence; rows of sound sequences are right."""
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_kv_append, gdn_kv_gather, gdn_stream_status
from tests.attention_util import gen, normal

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cu", [
    [0, 4, 9, 20, 9],             # a sequence past the end, and one that decreases
    [0, 4, 9, 4, 9],              # one that decreases among empty ones
    [0, 4, 4, -1, 9],             # a negative offset: the last sequence's range is bad too
    [0, 9, 1, 9, 1, 9],
    [0] + [4] * 300 + [3] + [9] * 40,
])
def test_bad_offsets_are_reported_wherever_they_are(cu):
    n, T = len(cu) - 1, 9
    x = normal(gen(80), T, 1, 128).cuda()
    k = torch.zeros((2 * n, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.arange(2 * n, dtype=torch.int32, device="cuda").view(n, 2).contiguous()
    start = i32([0] * n)
    gdn_kv_append(x, x, k, v, table, i32(cu), start)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS"
    gdn_kv_gather(k, v, table, i32(cu), start, T)
    assert gdn_stream_status() == "GDN_ERR_BAD_CU_SEQLENS" and gdn_stream_status() == "GDN_OK"
    if cu[1:2] == [4]:  # the first sequence is sound: its rows are in its first page
        assert torch.equal(k[0, 0, :3], x[:3, 0])


def test_sound_offsets_with_many_empty_sequences():
    for lens in ([0] * 2000 + [3] + [0] * 2000, [1] * 33 + [0] * 700, [0, 0, 5, 0]):
        n, T = len(lens), sum(lens)
        cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
        x = normal(gen(81), T, 1, 128).cuda()
        k = torch.zeros((n, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
        gdn_kv_append(x, -x, k, v, table, cu, i32([1] * n))
        gk, gv = gdn_kv_gather(k, v, table, cu, i32([1] * n), T)
        assert gdn_stream_status() == "GDN_OK"
        assert torch.equal(gk, x) and torch.equal(gv, -x)
