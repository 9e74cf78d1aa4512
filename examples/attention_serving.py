"""One attention layer of a server that mixes prompts, decoding and drafted tokens in every
step, over the paged cache, with norms and rotary positions of queries and keys.

    python examples/attention_serving.py [--bits 8] [--window 512] [--steps 12]

A step's new tokens of all sequences lie side by side, as the layer's projection leaves them
(here they are random): pieces of prompts that are still being read, one token of a sequence
that decodes, a few drafted tokens of one that checks them.  gdn_kv_append_rope normalises
and rotates their q and k and writes k and v into the cache; gdn_attn_prefill_paged attends
to it, with a window and the first tokens where the layer has one.  Drafted tokens that are
not accepted are taken back by the sequence's length alone: the next step writes over them.
At the end the last step is compared with the rows read back and attended to densely:
gdn_kv_gather, then gdn_attn_prefill, or with a window a plain softmax over what it shows.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_recurrence_gb300 as gdn  # noqa: E402

H_Q, H_KV, D, ROTARY, PAGE, PIECE, DRAFTED, SINKS = 16, 2, 256, 64, 64, 256, 4, 4


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


class Layer:
    """The layer's weights and its pool of pages; sequence n has the pages n * per_seq ..."""

    def __init__(self, sequences, tokens, bits, window):
        per_seq = -(-tokens // PAGE)
        shape = (sequences * per_seq, H_KV, PAGE, D)
        dtype = torch.float8_e4m3fn if bits == 8 else torch.bfloat16
        self.k, self.v = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
        exp = lambda: torch.empty(shape[:3], dtype=torch.uint8, device="cuda")  # noqa: E731
        self.exps = dict(k_exp=exp(), v_exp=exp()) if bits == 8 else {}
        self.table = ints(torch.randperm(shape[0]).view(sequences, per_seq).tolist())
        self.window = window
        n = ROTARY // 2
        self.inv_freq = (1e7 ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda()
        self.norms = dict(q_weight=1 + 0.1 * torch.randn(D, device="cuda"),
                          k_weight=1 + 0.1 * torch.randn(D, device="cuda"), norm_eps=1e-6)

    def step(self, qkv, new, start):
        """o of the new tokens (new[n] of sequence n, at its positions start[n] ..)."""
        cu, length = ints(offsets(new)), ints([s + n for s, n in zip(start, new)])
        q, k, v = qkv[:, :H_Q], qkv[:, H_Q:H_Q + H_KV], qkv[:, H_Q + H_KV:]
        # (in place: the projection's q is not needed any more)
        gdn.gdn_kv_append_rope(q, k, v, self.k, self.v, self.table, cu, ints(start), self.inv_freq, q_out=q,
                               **self.norms, **self.exps)
        return gdn.gdn_attn_prefill_paged(q, self.k, self.v, self.table, cu, length, window=self.window,
                                          sinks=SINKS if self.window else 0, **self.exps)


def in_window(q, k, v, new, full, window, sinks):
    """The same attention in plain fp32: row p sees the window keys up to itself and the first few."""
    o = torch.zeros(q.shape, device=q.device)
    t = u = 0
    for a, n in zip(new, full):
        p, j = torch.arange(n - a, n, device=q.device)[:, None], torch.arange(n, device=q.device)
        see = (j <= p) & ((j > p - window) | (j < sinks))
        kk, vv = (x[u:u + n].float().repeat_interleave(H_Q // H_KV, 1) for x in (k, v))
        s = torch.einsum("ahd,nhd->han", q[t:t + a].float(), kk) * D ** -0.5
        o[t:t + a] = torch.einsum("han,nhd->ahd", s.masked_fill(~see, float("-inf")).softmax(-1), vv)
        t, u = t + a, u + n
    return o


def serve(sequences=5, prompt=1500, steps=12, bits=8, window=None, seed=0):
    """Returns the largest difference of the last step from dense attention over the rows read
    back, relative to the largest output."""
    torch.manual_seed(seed)
    prompts = [max(1, prompt * (n + 1) // sequences) for n in range(sequences)]
    layer = Layer(sequences, max(prompts) + steps * (DRAFTED + 1), bits, window)
    length = [0] * sequences
    for _ in range(steps):
        # a piece of the prompt, one token, or drafted tokens with the one before them
        new = [min(PIECE, p - x) if x < p else (1 if n % 2 else 1 + DRAFTED)
               for n, (x, p) in enumerate(zip(length, prompts))]
        start = list(length)
        qkv = torch.randn((sum(new), H_Q + 2 * H_KV, D), device="cuda").to(torch.bfloat16)
        o = layer.step(qkv, new, start)
        accepted = [a if x < p else 1 + (a - 1) // 2 for a, x, p in zip(new, start, prompts)]
        length = [x + a for x, a in zip(start, accepted)]
    full = [s + a for s, a in zip(start, new)]
    k, v = gdn.gdn_kv_gather(layer.k, layer.v, layer.table, ints(offsets(full)), ints([0] * sequences), sum(full),
                             **layer.exps)
    if window:
        ref = in_window(qkv[:, :H_Q], k, v, new, full, window, SINKS)
    else:
        ref = gdn.gdn_attn_prefill(qkv[:, :H_Q], k, v, ints(offsets(new)), ints(offsets(full)))
    status = gdn.gdn_stream_status()
    if status != "GDN_OK":
        raise RuntimeError(status)
    return float((o.float() - ref.float()).abs().max() / ref.float().abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--bits", type=int, choices=(8, 16), default=8)
    ap.add_argument("--sequences", type=int, default=5)
    ap.add_argument("--prompt", type=int, default=1500)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--window", type=int, default=None)
    a = ap.parse_args()
    diff = serve(a.sequences, a.prompt, a.steps, a.bits, a.window)
    print(f"{a.sequences} sequences, prompts up to {a.prompt} tokens, {a.steps} steps, {a.bits}-bit cache"
          + (f", window {a.window}" if a.window else "")
          + f": attention over the pages and over the rows read back differ by {diff:.2e} of the largest output")


if __name__ == "__main__":
    main()
