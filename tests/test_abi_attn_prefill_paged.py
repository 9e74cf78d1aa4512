"""Host-checkable errors of attention over the paged cache for packed new tokens, and of its
binding: refused before anything is launched (these calls touch no GPU)."""
import pytest
import torch

import gated_deltanet_linear_recurrence_gb300 as gdn
from gated_deltanet_linear_recurrence_gb300 import _lib
from gated_deltanet_linear_recurrence_gb300.build import build

FAKE = 0x10000  # aligned, never dereferenced: validation fails first
NULL, ARG, SHAPE, DTYPE, ALIGN, SMALL = 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def call(lib, **kw):
    a = dict(q=FAKE, qs=4096, kp=FAKE, vp=FAKE, ke=FAKE, ve=FAKE, table=FAKE, cu=FAKE, lens=FAKE, o=FAKE,
             n=2, t=9, h_q=16, h_kv=2, d=256, page=64, pages=8, max_pages=4, dtype=2, scale=1.0,
             window=0, sinks=0, ws=FAKE, bytes=1 << 30)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_attn_prefill_paged(*a.values(), None)


def test_refusals(lib):
    for p in ("q", "o", "cu", "lens", "ws", "kp", "vp", "table", "ke", "ve"):
        assert call(lib, **{p: None}) == NULL, p
    for p in ("n", "t", "pages", "max_pages", "window", "sinks"):
        assert call(lib, **{p: -1}) == ARG, p
    assert call(lib, h_q=0) == ARG and call(lib, h_kv=0) == ARG and call(lib, d=0) == ARG
    assert call(lib, page=0) == ARG and call(lib, qs=4095) == ARG
    assert call(lib, n=0) == ARG                                # tokens of no sequence
    assert call(lib, h_q=18, h_kv=2, qs=4608) == SHAPE          # nine heads on a KV head
    assert call(lib, h_q=7, h_kv=2, qs=1792) == SHAPE
    assert call(lib, d=64) == SHAPE and call(lib, d=192) == SHAPE
    assert call(lib, page=48) == SHAPE and call(lib, page=4) == SHAPE and call(lib, page=2048) == SHAPE
    assert call(lib, max_pages=1 << 25) == SHAPE and call(lib, pages=1 << 25) == SHAPE
    assert call(lib, t=1 << 31) == SHAPE
    assert call(lib, dtype=0) == DTYPE and call(lib, dtype=3) == DTYPE
    assert call(lib, qs=4100) == ALIGN
    for p in ("q", "o", "ws", "kp", "vp"):
        assert call(lib, **{p: FAKE + 8}) == ALIGN, p
    for p in ("table", "cu", "lens"):
        assert call(lib, **{p: FAKE + 2}) == ALIGN, p
    assert call(lib, ke=FAKE + 4) == ALIGN
    # nothing to do: nothing is launched
    assert call(lib, t=0) == 0 and call(lib, t=0, q=None, o=None, ws=None, bytes=0) == 0
    assert call(lib, n=0, t=0, cu=None, lens=None) == 0


def test_workspace(lib):
    size = gdn.gdn_attn_prefill_paged_workspace_size
    e4m3 = torch.float8_e4m3fn
    for d in (128, 256):
        least = size(16, 2, d)
        assert least > 0 and least % 16 == 0
        assert call(lib, d=d, bytes=least - 1) == SMALL and call(lib, d=d, bytes=0) == SMALL
        # eight heads on a KV head: 32 tokens a tile of queries; room for widened rows from a fourth tile on
        assert size(16, 2, d, e4m3, 96) == least and size(16, 2, d, e4m3, 97) == least + (128 << 20)
        assert size(16, 2, d, torch.bfloat16, 10 ** 9) == least
    assert size(3, 3, 128, e4m3, 768) == size(3, 3, 128) and size(3, 3, 128, e4m3, 769) > size(3, 3, 128)
    for bad in ((16, 2, 64), (18, 2, 256), (0, 1, 128), (16, 2, 256, e4m3, -1)):
        assert size(*bad) == 0
    assert lib.gdn_attn_prefill_paged_workspace_size(16, 2, 256, 7, 0) == 0


def test_binding_refuses_before_the_gpu():
    """Types and devices, on tensors of the CPU."""
    build()
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    pages, table = torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32)
    cu, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prefill_paged(q, pages, pages, table, cu, lens)  # not on the GPU
    with pytest.raises(TypeError):
        gdn.gdn_attn_prefill_paged(q, pages.float(), pages.float(), table, cu, lens)
    with pytest.raises(TypeError):
        gdn.gdn_attn_prefill_paged(q, None, pages, table, cu, lens)
