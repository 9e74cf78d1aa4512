"""One full-attention layer's serving path on the paged cache: prompts in pieces, then
decoding, for a ragged batch of sequences.

    python examples/attention_layer.py [--bits 8] [--sequences 4] [--prompt 3000] [--new 16]

A layer's projections leave q, k and v side by side; here they are random.  Per piece
of the prompts the layer writes the new rows (gdn_kv_append), reads back every row of
the sequences so far (gdn_kv_gather) and attends over them (gdn_attn_prefill); per new
token it writes one row a sequence and attends over the cache where it lies
(gdn_attn_decode_paged).  At the end the last token's output is compared with prompt
attention over the whole sequences, whose keys and values come from the same cache.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_recurrence_gb300 as gdn  # noqa: E402

H_Q, H_KV, D, PAGE = 16, 2, 256, 64


class PagedCache:
    """The pool of one layer, and the pages of its sequences (given out as they grow)."""

    def __init__(self, sequences, tokens, bits):
        per_seq = -(-tokens // PAGE)
        shape = (sequences * per_seq, H_KV, PAGE, D)
        dtype = torch.float8_e4m3fn if bits == 8 else torch.bfloat16
        self.k = torch.empty(shape, dtype=dtype, device="cuda")
        self.v = torch.empty_like(self.k)
        exp = lambda: torch.empty(shape[:3], dtype=torch.uint8, device="cuda")  # noqa: E731
        self.exps = dict(k_exp=exp(), v_exp=exp()) if bits == 8 else {}
        self.free = torch.randperm(shape[0]).tolist()
        self.pages = [[] for _ in range(sequences)]
        self.lengths = [0] * sequences
        self.table = torch.full((sequences, per_seq), -1, dtype=torch.int32, device="cuda")

    def grow(self, new):
        """Room for new[n] more rows of each sequence; returns (offsets, start positions)."""
        start = list(self.lengths)
        for n, extra in enumerate(new):
            self.lengths[n] += extra
            while len(self.pages[n]) * PAGE < self.lengths[n]:
                self.pages[n].append(self.free.pop())
                self.table[n, len(self.pages[n]) - 1] = self.pages[n][-1]
        return ints(offsets(new)), ints(start)

    def append(self, k, v, cu, start):
        gdn.gdn_kv_append(k, v, self.k, self.v, self.table, cu, start, **self.exps)

    def all_rows(self):
        cu = ints(offsets(self.lengths))
        k, v = gdn.gdn_kv_gather(self.k, self.v, self.table, cu, ints([0] * len(self.lengths)),
                                 sum(self.lengths), **self.exps)
        return k, v, cu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def projections(tokens):
    x = torch.randn((tokens, H_Q + 2 * H_KV, D), device="cuda").to(torch.bfloat16)
    return x[:, :H_Q], x[:, H_Q:H_Q + H_KV], x[:, H_Q + H_KV:]


def serve(sequences=4, prompt=3000, new_tokens=16, bits=8, piece=1024, seed=0):
    """Returns the largest difference between decoding and prompt attention at the last
    token, relative to the largest output."""
    torch.manual_seed(seed)
    prompts = [max(1, prompt * (n + 1) // sequences) for n in range(sequences)]
    cache = PagedCache(sequences, max(prompts) + new_tokens, bits)
    left = list(prompts)
    while any(left):
        new = [min(piece, n) for n in left]
        left = [n - a for n, a in zip(left, new)]
        q, k, v = projections(sum(new))
        cu, start = cache.grow(new)
        cache.append(k, v, cu, start)
        rows_k, rows_v, cu_k = cache.all_rows()
        gdn.gdn_attn_prefill(q, rows_k, rows_v, cu, cu_k)
    workspace = torch.empty(gdn.gdn_attn_decode_paged_workspace_size(H_Q, H_KV, D),
                            dtype=torch.uint8, device="cuda")
    for _ in range(new_tokens):
        q, k, v = projections(sequences)
        cu, start = cache.grow([1] * sequences)
        cache.append(k, v, cu, start)
        o = gdn.gdn_attn_decode_paged(q, cache.k, cache.v, cache.table, ints(cache.lengths),
                                      workspace=workspace, **cache.exps)
    rows_k, rows_v, cu_k = cache.all_rows()
    ref = gdn.gdn_attn_prefill(q, rows_k, rows_v, ints(list(range(sequences + 1))), cu_k)
    status = gdn.gdn_stream_status()
    if status != "GDN_OK":
        raise RuntimeError(status)
    return float((o.float() - ref.float()).abs().max() / ref.float().abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--bits", type=int, choices=(8, 16), default=8)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=3000)
    ap.add_argument("--new", type=int, default=16)
    a = ap.parse_args()
    diff = serve(a.sequences, a.prompt, a.new, a.bits)
    print(f"{a.sequences} sequences, prompts up to {a.prompt} tokens, {a.new} new tokens, {a.bits}-bit "
          f"cache: decoding and prompt attention differ by {diff:.2e} of the largest output")


if __name__ == "__main__":
    main()
