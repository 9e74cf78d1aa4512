"""Host-checkable errors of the norms' and rotations' entry points, and of their binding:
refused before anything is launched (these calls touch no GPU)."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_recurrence_gb300 as gdn
from gated_deltanet_linear_recurrence_gb300 import _lib
from gated_deltanet_linear_recurrence_gb300.build import build

FAKE = 0x10000  # aligned, never dereferenced: validation fails first
NULL, ARG, SHAPE, DTYPE, ALIGN = 1, 2, 3, 4, 5
NORM, PAIRS = 1, 2
THIRDS = (ctypes.c_uint8 * 32)(*[i % 3 for i in range(32)])


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def dense(lib, **kw):
    a = dict(q=FAKE, k=FAKE, qs=4096, ks=512, qo=FAKE, ko=FAKE, qos=4096, kos=512, pos=FAKE, axes=1,
             axis_of=None, freq=FAKE, rot=64, qw=FAKE, kw=FAKE, eps=1e-6, t=4, h_q=16, h_kv=2,
             d=256, dtype=1, options=NORM)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_qk_norm_rope(*a.values(), None)


def paged(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=4096, ks=512, vs=512, qo=FAKE, qos=4096, kp=FAKE, vp=FAKE,
             ke=FAKE, ve=FAKE, table=FAKE, cu=FAKE, start=FAKE, pos=FAKE, axes=1, axis_of=None,
             freq=FAKE, rot=64, qw=FAKE, kw=FAKE, eps=1e-6, n=1, t=4, h_q=16, h_kv=2, d=256,
             page=64, pages=8, max_pages=4, dtype=2, options=NORM)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.gdn_kv_append_rope(*a.values(), None)


@pytest.mark.parametrize("call", [dense, paged])
def test_both_refuse(lib, call):
    r = lambda **kw: call(lib, **kw)  # noqa: E731
    for p in ("q", "k", "qo", "freq"):
        assert r(**{p: None}) == NULL, p
    assert r(t=-1) == ARG and r(d=0) == ARG and r(h_q=-1) == ARG and r(h_kv=0) == ARG
    assert r(rot=0) == ARG and r(rot=-8) == ARG and r(axes=0) == ARG
    assert r(rot=264) == SHAPE and r(rot=60) == SHAPE and r(rot=4) == SHAPE
    assert r(d=128, rot=136) == SHAPE and r(d=192) == SHAPE and r(d=64) == SHAPE
    assert r(h_q=65536, qs=1 << 24, qos=1 << 24) == SHAPE and r(t=1 << 31) == SHAPE
    assert r(options=4) == ARG and r(options=0) == ARG  # weights without the norm
    assert r(options=0, qw=None) == ARG and r(options=0, kw=None) == ARG
    for eps in (-1e-9, float("nan"), float("-inf")):
        assert r(eps=eps) == ARG
    assert r(qs=4095) == ARG and r(ks=0) == ARG and r(qos=8) == ARG
    assert r(qs=4100) == ALIGN and r(ks=516) == ALIGN and r(qos=4108) == ALIGN
    for p in ("q", "k", "qo", "qw", "kw"):
        assert r(**{p: FAKE + 8}) == ALIGN, p
    assert r(pos=FAKE + 2) == ALIGN and r(freq=FAKE + 1) == ALIGN
    # axes
    assert r(axes=3) == NULL and r(axes=3, axis_of=THIRDS, pos=None) == NULL
    assert r(axes=2, axis_of=THIRDS) == ARG  # an axis that is not there
    assert r(axes=5, axis_of=THIRDS) == SHAPE
    # nothing to do
    assert r(t=0) == 0 and r(t=0, q=None, k=None, qo=None) == 0
    assert r(t=0, axes=3, axis_of=THIRDS) == 0 and r(t=0, options=NORM | PAIRS) == 0
    assert r(t=0, options=0, qw=None, kw=None) == 0


def test_dense_refuses(lib):
    assert dense(lib, pos=None) == NULL and dense(lib, ko=None) == NULL
    assert dense(lib, h_q=0) == ARG and dense(lib, kos=511) == ARG and dense(lib, kos=516) == ALIGN
    assert dense(lib, ko=FAKE + 8) == ALIGN and dense(lib, dtype=0) == DTYPE


def test_paged_refuses(lib):
    r = lambda **kw: paged(lib, **kw)  # noqa: E731
    for p in ("v", "kp", "vp", "table", "cu", "start", "ke", "ve"):
        assert r(**{p: None}) == NULL, p
    for p in ("n", "pages", "max_pages"):
        assert r(**{p: -1}) == ARG, p
    assert r(page=0) == ARG and r(vs=511) == ARG and r(n=0) == ARG
    assert r(page=48) == SHAPE and r(page=4) == SHAPE and r(pages=1 << 25) == SHAPE
    assert r(dtype=0) == DTYPE and r(vs=516) == ALIGN
    for p in ("v", "kp", "vp"):
        assert r(**{p: FAKE + 8}) == ALIGN, p
    for p in ("table", "cu", "start"):
        assert r(**{p: FAKE + 2}) == ALIGN, p
    assert r(ke=FAKE + 4) == ALIGN
    assert r(n=0, t=0, cu=None, start=None) == 0


def test_binding_refuses_before_the_gpu():
    """Types and devices, on tensors of the CPU."""
    build()
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    f, p = torch.ones(32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(x, x, p, f)  # not on the GPU
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm_rope(x.numpy, x, p, f)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(x[0], x, p, f)
    pages, table = torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append_rope(x, x, x, pages, pages, table, p[:2], p[:1], f)
    with pytest.raises(TypeError):
        gdn.gdn_kv_append_rope(x, x, x, pages.float(), pages.float(), table, p[:2], p[:1], f)
