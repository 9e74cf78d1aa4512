"""Attention over the paged cache in a window, by a server that gives back the pages behind it:
a page of which no query sees a key may be missing, named wrongly or another sequence's by
now, without an error and without an effect; one that some query sees may not."""
import numpy as np
import pytest
import torch

from gated_deltanet_linear_recurrence_gb300 import gdn_stream_status
from oracle.window_attention import seen
from tests.test_gpu_attn_prefill_paged import Batch

pytestmark = pytest.mark.gpu


def seen_entries(b, n, window, sinks):
    """Truth values: which entries of sequence n's table hold a key that some query sees."""
    if b.new[n] == 0:
        return np.zeros(b.table.shape[1], dtype=bool)
    see = seen(b.new[n], b.lengths[n], window, sinks).any(axis=0)
    return np.array([see[i * b.page:(i + 1) * b.page].any() for i in range(b.table.shape[1])])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [8, 16, 64, 256])
def test_pages_behind_the_window_may_be_gone(page, D, fp8):
    """Single tokens, drafted ones and pieces of prompts (whose e4m3 rows are widened once), at
    lengths that put the window's first key everywhere in a tile of 128 keys."""
    new = [1, 1, 3, 150, 40, 1, 0]
    for shift in (0, 1, 7, 8, 60, 119, 127):
        lengths = [700 + shift, 1001 + shift, 640 + shift, 900 + shift, 1200 + shift, 33, 400]
        b = Batch(new, lengths, 8, 1, D, page, fp8, page + shift)
        keep = b.table.clone()
        for window, sinks in ((200, 0), (129, 4), (333, 130), (1, 0), (1, 9)):
            b.table.copy_(keep)
            want = b.run(window=window, sinks=sinks)
            assert gdn_stream_status() == "GDN_OK"
            for value in (-1, 10 ** 6, 0):
                for n in range(len(new)):
                    for i in np.nonzero(~seen_entries(b, n, window, sinks))[0]:
                        b.table[n, i] = value
                got = b.run(window=window, sinks=sinks)
                assert gdn_stream_status() == "GDN_OK", (shift, window, sinks, value)
                assert torch.equal(got, want), (shift, window, sinks, value)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_that_are_seen_may_not(fp8):
    """The first and the last page that some query sees, at each end of the window and among the
    first keys."""
    window, sinks, page = 200, 20, 16
    new, lengths = [2, 150], [711, 1030]
    b = Batch(new, lengths, 8, 1, 128, page, fp8, 4)
    keep = b.table.clone()
    for n in range(2):
        entries = np.nonzero(seen_entries(b, n, window, sinks))[0]
        first = entries[entries > sinks // page][0]
        for entry in (0, sinks // page, first, entries[-1]):
            b.table.copy_(keep)
            b.table[n, entry] = -1
            gone = [np.arange(x) // page == (entry if i == n else -1) for i, x in enumerate(lengths)]
            b.check(window=window, sinks=sinks, gone=gone)
