"""Outputs that a call makes are tensors of their own: one that grows, is written over or goes
takes nothing from another with it."""
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_qk_norm_rope, gdn_stream_status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("other_stream", [False, True])
def test_rotated_q_and_k_have_memory_of_their_own(other_stream):
    q, k = torch.randn(5, 3, 128).bfloat16().cuda(), torch.randn(5, 2, 128).bfloat16().cuda()
    pos, f = torch.zeros(5, dtype=torch.int32).cuda(), torch.ones(8).cuda()  # (position 0: as they were)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if other_stream else None
    a, b = gdn_qk_norm_rope(q, k, pos, f, stream=stream)
    torch.cuda.synchronize()
    assert a.untyped_storage().nbytes() == a.nbytes and b.untyped_storage().nbytes() == b.nbytes
    a.resize_(5, 5, 128)
    a.fill_(9)
    assert torch.equal(b, k)
    a, b = gdn_qk_norm_rope(q, k, pos, f, stream=stream)
    torch.cuda.synchronize()
    b.resize_(5, 5, 128)
    b.fill_(9)
    assert torch.equal(a, q)
    assert gdn_stream_status(stream) == "GDN_OK"
