"""The cache and both attention forms together, as examples/attention_layer.py runs them:
a prompt in pieces gives what the whole prompt gives, and a decoding step what prompt
attention gives for the same token."""
import importlib.util
import os

import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import (gdn_attn_prefill, gdn_kv_append, gdn_kv_gather,
                                                    gdn_stream_status)
from tests.attention_util import BF16, gen, normal, offsets

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("sequences,prompt,new", [(1, 1, 1), (3, 500, 5), (5, 2100, 3)])
def test_example(example, sequences, prompt, new, bits):
    """Both forms round o to bf16 (2^-8 each), prompt attention its weights too (2^-8);
    random values: the outputs' size is near the largest weighted sum of |v| only up to
    a factor of about 4 at these lengths."""
    assert example.serve(sequences, prompt, new, bits, piece=256) <= 4 * 3 * BF16


@pytest.mark.parametrize("D", [128, 256])
def test_pieces_over_the_cache_give_the_whole_prompt(D):
    """A bf16 cache holds the rows unchanged, so each piece's output is within the two
    calls' own rounding of the whole prompt's: the key tiles begin at the same keys, and
    the weights are rounded relative to references that may differ."""
    T, cut, page = 500, 333, 16
    x = normal(gen(1), T, 8 + 2 * 2, D).cuda()
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    whole = gdn_attn_prefill(q, k, v, offsets([T]))
    pages = torch.empty((40, 2, page, D), dtype=torch.bfloat16, device="cuda")
    kp, vp = pages.clone(), pages
    table = torch.randperm(40, generator=gen(2))[:32].int().cuda()[None].contiguous()
    out = []
    for a, b in ((0, cut), (cut, T)):
        start = torch.tensor([a], dtype=torch.int32, device="cuda")
        gdn_kv_append(k[a:b], v[a:b], kp, vp, table, offsets([b - a]), start)
        gk, gv = gdn_kv_gather(kp, vp, table, offsets([b]), torch.zeros_like(start), b)
        assert torch.equal(gk, k[:b]) and torch.equal(gv, v[:b])
        out.append(gdn_attn_prefill(q[a:b], gk, gv, offsets([b - a]), offsets([b])))
    assert gdn_stream_status() == "GDN_OK"
    got = torch.cat(out).double()
    wabs = gdn_attn_prefill(q, k, v.abs(), offsets([T])).double() * (1 + BF16)
    bound = 2 * ((BF16 + 2.0 ** -10) * wabs + BF16 * whole.double().abs() + 1e-6)
    assert ((got - whole.double()).abs() <= bound).all()
