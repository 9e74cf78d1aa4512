"""The attention layers' calls on a stream of their own beside a busy current stream: what
they allocate must not be memory that the current stream's queue still writes, nor go
back to the call's stream while the current one reads it."""
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_attn_decode_paged, gdn_attn_prefill,
                                                    gdn_kv_gather, gdn_stream_status)
from tests.attention_util import gen, normal, offsets

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    """name -> (call on a stream, shapes of what it allocates)."""
    B, h_q, h_kv, D, page = 3, 8, 2, 128, 16
    g = gen(100)
    k, v = (normal(g, 30, h_kv, page, D).cuda() for _ in range(2))
    table = torch.arange(30, dtype=torch.int32, device="cuda").view(3, 10).contiguous()
    q = normal(g, B, h_q, D).cuda()
    lens, start = i32([150, 9, 77]), i32([0, 5, 20])
    rows = normal(g, 236, h_q + 2 * h_kv, D).cuda()
    cu = offsets([150, 9, 77])
    return {
        "decode": lambda s: (gdn_attn_decode_paged(q, k, v, table, lens, stream=s),),
        "gather": lambda s: gdn_kv_gather(k, v, table, offsets_of, start, 90, stream=s),
        "prompt": lambda s: (gdn_attn_prefill(rows[:, :8], rows[:, 8:10], rows[:, 10:], cu, stream=s),),
    }


offsets_of = None


@pytest.fixture(scope="module", autouse=True)
def _offsets():
    global offsets_of
    offsets_of = offsets([50, 4, 36])
    yield


def busy(stream_ms=30):
    """Work that keeps the current stream for some tens of milliseconds."""
    x = torch.empty(1 << 28, dtype=torch.float32, device="cuda")  # 1 GB
    for _ in range(8 * stream_ms):
        x.fill_(1.0)


@pytest.mark.parametrize("name", ["decode", "gather", "prompt"])
def test_allocations_belong_to_the_given_stream(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    busy()
    # blocks of every size up to the workspace's, written by the current stream's queue
    # after it is through with the work above, and free for the allocator at once
    sizes = [n for w in want for n in [w.numel() * w.element_size()] * 4] + [1 << k for k in range(10, 24)] * 2
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    for t in held:
        t.fill_(0xff)
    del held, t
    got = call(s)
    s.synchronize()
    first = [t.clone() for t in got]  # on the current stream, behind its queue
    torch.cuda.synchronize()
    assert gdn_stream_status(s) == "GDN_OK"
    for w, g, c in zip(want, got, first):
        assert torch.equal(g, w) and torch.equal(c, w)


@pytest.mark.parametrize("name", ["decode", "gather", "prompt"])
def test_outputs_are_kept_for_the_current_stream(name):
    """The current stream reads an output that is dropped at once; the call's stream must
    not get that memory before the reading is over."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    for _ in range(2):
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
        busy(10)
        copies = [t.clone() for t in got]  # queued behind the work
        shapes = [(t.shape, t.dtype) for t in got]
        del got
        with torch.cuda.stream(s):
            for _ in range(4):
                for shape, dtype in shapes:
                    torch.empty(shape, dtype=dtype, device="cuda").fill_(float("nan"))
        torch.cuda.synchronize()
        for w, c in zip(want, copies):
            assert torch.equal(c, w)


@pytest.mark.parametrize("name", ["decode", "gather", "prompt"])
def test_a_raw_stream_handle(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s.cuda_stream, torch.cuda.current_stream().cuda_stream, torch.cuda.current_stream()):
        got = call(handle)
        s.synchronize()
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(g, w)
    assert gdn_stream_status(s) == "GDN_OK"
