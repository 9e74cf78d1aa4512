"""Inputs and bounds shared by the GPU tests of prompt attention and the paged cache.

Bounds, from the arithmetic.  With A = sum_j w_j |v_j| (the oracle's attention over
|v|; A >= |o|) and a rounding to type t off by at most eps(t) / 2 of the value (bf16
2^-8, fp16 2^-11):

* o is stored in bf16: 2^-8 |o|;
* prompt attention rounds each weight to bf16 before the product with V, the sums stay
  unrounded: 2^-8 A.  Decode rounds the weights to bf16 pairs (2^-16 A) or, over an
  e4m3 cache, to fp16 (2^-11 A; below fp16's normal range, 2^-14 of the largest
  weighted unit, 2^-25 of that unit at most: inside the term below);
* scores are exact products of the inputs summed in fp32 and scaled: for scores up to 64
  in size an error of at most D 2^-24 64 absolutely, each weight off by that share; the
  base-2 exponential of the hardware adds 2^-22, the sum of L weights L 2^-24.  Taken
  together 2^-10 A covers D = 256, L = 2^13 (the tests' scores and lengths); plus 1e-6
  where everything cancels.
"""
import numpy as np
import torch

BF16, F16 = 2.0 ** -8, 2.0 ** -11


def check(got, ref, wabs, weights, name=""):
    got = got.detach().double().cpu().numpy()
    err = np.abs(got - ref)
    bound = (weights + 2.0 ** -10) * wabs + BF16 * np.abs(ref) + 1e-6
    assert np.isfinite(got).all(), f"{name}: not finite"
    worst = np.unravel_index((err - bound).argmax(), err.shape)
    assert (err <= bound).all(), f"{name}: err {err[worst]:.3e} > bound {bound[worst]:.3e} at {worst}"


def normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, dtype=torch.float64).to(dtype)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def offsets(lens, device="cuda"):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=device)
