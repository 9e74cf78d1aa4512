"""Host-checkable errors of the paged cache's and prompt attention's entry points:
refused before anything is launched (these calls touch no GPU)."""
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


def rows(lib, name, **kw):
    a = dict(k=FAKE, v=FAKE, ks=512, vs=512, kp=FAKE, vp=FAKE, ke=FAKE, ve=FAKE, table=FAKE, cu=FAKE,
             start=FAKE, n=1, t=4, h_kv=2, d=256, page=64, pages=8, max_pages=4, dtype=2)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(lib, name)(*a.values(), None)


@pytest.mark.parametrize("name", ["gdn_kv_append", "gdn_kv_gather"])
def test_rows_calls_refuse(lib, name):
    r = lambda **kw: rows(lib, name, **kw)  # noqa: E731
    for p in ("k", "v", "kp", "vp", "table", "cu", "start", "ke", "ve"):
        assert r(**{p: None}) == NULL, p
    for p in ("n", "t", "pages", "max_pages"):
        assert r(**{p: -1}) == ARG, p
    assert r(h_kv=0) == ARG and r(d=0) == ARG and r(page=0) == ARG
    assert r(ks=511) == ARG and r(vs=0) == ARG          # less than a token
    assert r(n=0) == ARG                                # tokens of no sequence
    assert r(ks=516) == ALIGN and r(vs=520 + 4) == ALIGN  # not whole 16-byte steps
    assert r(d=64, ks=128, vs=128) == SHAPE and r(d=192) == SHAPE
    assert r(page=48) == SHAPE and r(page=4) == SHAPE and r(page=2048) == SHAPE
    assert r(max_pages=1 << 25) == SHAPE                # 2^31 positions
    assert r(pages=1 << 25) == SHAPE                    # 2^32 rows
    assert r(t=1 << 31) == SHAPE
    assert r(dtype=0) == DTYPE and r(dtype=3) == DTYPE
    for p in ("k", "v", "kp", "vp"):
        assert r(**{p: FAKE + 8}) == ALIGN, p
    for p in ("table", "cu", "start"):
        assert r(**{p: FAKE + 2}) == ALIGN, p
    assert r(ke=FAKE + 4) == ALIGN
    # nothing to do: nothing is launched and no row pointer is wanted
    assert r(t=0) == 0 and r(t=0, k=None, v=None) == 0 and r(n=0, t=0, cu=None, start=None) == 0


def paged(lib, **kw):
    a = dict(q=FAKE, qs=4096, kp=FAKE, vp=FAKE, ke=FAKE, ve=FAKE, table=FAKE, lens=FAKE, o=FAKE, b=2,
             h_q=16, h_kv=2, d=256, page=64, pages=8, max_pages=4, dtype=2, scale=1.0, ws=FAKE,
             bytes=1 << 30)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_attn_decode_paged(*a.values(), None)


def test_paged_decode_refuses(lib):
    for p in ("q", "o", "lens", "ws", "kp", "vp", "table", "ke", "ve"):
        assert paged(lib, **{p: None}) == NULL, p
    assert paged(lib, b=-1) == ARG and paged(lib, h_q=0) == ARG and paged(lib, qs=4095) == ARG
    assert paged(lib, h_q=18, h_kv=2) == SHAPE            # nine heads on a KV head
    assert paged(lib, h_q=7, h_kv=2, qs=1792) == SHAPE
    assert paged(lib, d=64) == SHAPE and paged(lib, page=40) == SHAPE
    assert paged(lib, qs=4100) == ALIGN and paged(lib, o=FAKE + 8) == ALIGN
    assert paged(lib, lens=FAKE + 1) == ALIGN and paged(lib, ws=FAKE + 8) == ALIGN
    assert paged(lib, dtype=1, ke=None, ve=None, bytes=16) == SMALL  # bf16 needs no exponents
    need = lib.gdn_attn_decode_paged_workspace_size(16, 2, 256)
    assert need > 0 and paged(lib, bytes=need - 1) == SMALL
    assert lib.gdn_attn_decode_paged_workspace_size(16, 2, 64) == 0
    assert lib.gdn_attn_decode_paged_workspace_size(0, 2, 256) == 0
    assert paged(lib, b=0) == 0


def prompt(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, cq=FAKE, ck=FAKE, n=2, tq=10, tk=12, h_q=16, h_kv=2, d=256,
             qs=4096, ks=512, vs=512, dtype=1, scale=1.0)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_attn_prefill(*a.values(), None)


def test_prompt_attention_refuses(lib):
    for p in ("q", "k", "v", "o", "cq", "ck"):
        assert prompt(lib, **{p: None}) == NULL, p
        assert prompt(lib, **{p: FAKE + 2}) == ALIGN, p
    for p in ("n", "tq", "tk"):
        assert prompt(lib, **{p: -1}) == ARG, p
    assert prompt(lib, n=0) == ARG and prompt(lib, qs=4088) == ARG and prompt(lib, ks=0) == ARG
    assert prompt(lib, qs=4100) == ALIGN and prompt(lib, vs=516) == ALIGN
    assert prompt(lib, d=64) == SHAPE and prompt(lib, h_q=17) == SHAPE and prompt(lib, h_q=18) == SHAPE
    assert prompt(lib, tq=1 << 31) == SHAPE and prompt(lib, tk=1 << 31) == SHAPE
    assert prompt(lib, dtype=0) == DTYPE and prompt(lib, dtype=2) == DTYPE
    assert prompt(lib, tq=0) == 0 and prompt(lib, n=0, tq=0, tk=0, cq=None, ck=None) == 0


def test_binding_refuses_before_the_library(lib):
    """Shapes, types and places that the binding checks (tensors on the CPU are refused)."""
    bf, i32 = torch.bfloat16, torch.int32
    pages = torch.zeros((4, 2, 16, 128), dtype=bf)
    table, cu, start = (torch.zeros(s, dtype=i32) for s in ((1, 2), (2,), (1,)))
    k = torch.zeros((3, 2, 128), dtype=bf)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(k, k, pages, pages, table, cu, start)             # not on the GPU
    with pytest.raises(TypeError):
        gdn.gdn_kv_append(k, k, pages.float(), pages.float(), table, cu, start)
    with pytest.raises(ValueError):
        gdn.gdn_kv_gather(pages[0], pages[0], table, cu, start, 3)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode_paged(k[:1], pages, pages, table, start)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prefill(k, k, k, cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prefill(k.float(), k.float(), k.float(), cu)


def test_token_stride(lib):
    stride = _lib.binding().token_stride
    fused = torch.zeros((5, 12, 128))
    assert stride(fused) == 12 * 128
    assert stride(fused[:, 2:6]) == 12 * 128
    assert stride(fused[:1, 2:6]) == 4 * 128  # one token: no step is taken
    assert stride(fused[::2, 3:4]) == 24 * 128
    for bad in (fused[..., ::2], fused[:, ::2], fused.transpose(0, 1)):
        with pytest.raises(ValueError):
            stride(bad)
    with pytest.raises(ValueError):
        stride(fused[0])
    with pytest.raises(TypeError):
        stride(5)
