"""Pins for the fp64 oracle of prompt attention and of the 8-bit cache rows: brute
force over single entries, the format's own definition, invariances.  The pins of
prompt attention also run against copies of it with one planted mistake each, every
one of which must fail at least one."""
import numpy as np
import pytest
import torch

from oracle import paged_attention as oracle
from oracle.attention import gqa_decode


def case(seed=0, lens=((3, 3), (1, 4), (0, 0), (5, 2), (4, 6)), h_q=4, h_kv=2, D=8):
    r = np.random.default_rng(seed)
    cq = np.cumsum([0] + [a for a, _ in lens])
    ck = np.cumsum([0] + [b for _, b in lens])
    q = r.standard_normal((cq[-1], h_q, D))
    k, v = r.standard_normal((2, ck[-1], h_kv, D))
    return q, k, v, cq, ck


def brute(q, k, v, cq, ck, scale, h_kv=2):
    o = np.zeros(q.shape)
    G = q.shape[1] // h_kv
    for n in range(len(cq) - 1):
        a, b = cq[n + 1] - cq[n], ck[n + 1] - ck[n]
        for i in range(a):
            for h in range(q.shape[1]):
                num, den = np.zeros(q.shape[2]), 0.0
                for j in range(b):
                    if j <= i + b - a:
                        w = np.exp(scale * np.dot(q[cq[n] + i, h], k[ck[n] + j, h // G]))
                        num, den = num + w * v[ck[n] + j, h // G], den + w
                if den > 0:
                    o[cq[n] + i, h] = num / den
    return o


def pin_brute_force(f):
    q, k, v, cq, ck = case()
    assert np.allclose(f(q, k, v, cq, ck, 0.6), brute(q, k, v, cq, ck, 0.6), atol=1e-13)


def pin_last_query_is_decode(f):
    q, k, v, cq, ck = case(1, lens=((6, 9),))
    ref = gqa_decode(q[-1:], k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None], [9], 0.6)
    assert np.allclose(f(q, k, v, cq, ck, 0.6)[-1:], ref, atol=1e-13)


def pin_pieces_are_the_whole(f):
    q, k, v, cq, ck = case(2, lens=((7, 7),))
    whole = f(q, k, v, cq, ck, 0.6)
    for s in (1, 3, 6):
        part = f(q[s:], k, v, [0, 7 - s], [0, 7], 0.6)
        assert np.allclose(part, whole[s:], atol=1e-13)


def pin_unseen_entries_do_nothing(f):
    q, k, v, cq, ck = case(3, lens=((4, 4), (3, 3)))
    ref = f(q, k, v, cq, ck, 0.6)
    k2, v2 = k.copy(), v.copy()
    k2[3], v2[3] = np.nan, np.inf  # only query 3 of the first sequence sees key 3
    got = f(q, k2, v2, cq, ck, 0.6)
    keep = [0, 1, 2, 4, 5, 6]
    assert np.allclose(got[keep], ref[keep], atol=1e-13)
    v3 = v.copy()
    v3[2, :, 1] = np.inf
    got = f(q, k, v3, cq, ck, 0.6)
    assert np.isinf(got[2:4, :, 1]).all()
    got[2:4, :, 1] = ref[2:4, :, 1]
    assert np.allclose(got, ref, atol=1e-13)


PINS = [pin_brute_force, pin_last_query_is_decode, pin_pieces_are_the_whole,
        pin_unseen_entries_do_nothing]


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_prompt_oracle(pin):
    pin(oracle.prompt)


def mutants():
    p = oracle.prompt
    roll = lambda x: np.roll(np.asarray(x, float), 1, axis=1)  # noqa: E731
    return {
        "scale dropped": lambda q, k, v, cq, ck, s: p(q, k, v, cq, ck, 1.0),
        "wrong head map": lambda q, k, v, cq, ck, s: p(q, roll(k), v, cq, ck, s),
        "aligned to the first key": lambda q, k, v, cq, ck, s: np.concatenate(
            [p(q[a:b], k[c:c + b - a], v[c:c + b - a], [0, b - a], [0, min(b - a, len(k[c:c + b - a]))], s)
             for a, b, c in zip(cq[:-1], cq[1:], ck[:-1])]),
        "one key short": lambda q, k, v, cq, ck, s: p(q, k, v, cq, [max(0, x - 1) for x in ck], s),
        "values and keys swapped": lambda q, k, v, cq, ck, s: p(q, v, k, cq, ck, s),
        "whole batch as one sequence": lambda q, k, v, cq, ck, s: p(q, k, v, [0, cq[-1]], [0, ck[-1]], s),
    }


@pytest.mark.parametrize("name", sorted(mutants()))
def test_a_planted_mistake_is_caught(name):
    wrong = mutants()[name]
    for pin in PINS:
        try:
            pin(wrong)
        except (AssertionError, ValueError, IndexError):
            return
    pytest.fail(f"no pin catches: {name}")


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, oracle.e4m3_table(), equal_nan=True)


def test_quantise_against_torchs_rounding():
    """The codes of torch's own conversion (nearest, ties to even) in units found from frexp."""
    r = np.random.default_rng(4)
    x = torch.tensor(r.standard_normal((64, 128)) * 10.0 ** r.uniform(-20, 20, (64, 1)),
                     dtype=torch.bfloat16)
    x[0] = 0
    x[1, :3] = torch.tensor([448.0, 1.0, -0.00390625])
    x[1, 3:] = 0
    x[2, 0], x[3, 5], x[4] = float("inf"), float("nan"), float("nan")
    x[5] = 1e-39
    vals, e = oracle.quantise(x)
    xd = x.double()
    amax = torch.where(torch.isfinite(xd), xd.abs(), 0.0).amax(1)
    m, ex = torch.frexp(amax)
    unit = torch.where(m > 0.875, ex - 8, ex - 9).clamp(min=-126)
    unit = torch.where(amax > 0, unit, 0)
    assert np.array_equal(e, unit.numpy())
    y = (xd * torch.exp2(-unit.double())[:, None]).float()
    y[~torch.isfinite(xd)] = float("nan")
    assert np.array_equal(vals, y.to(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    # reading back rounds nothing in bf16, and is near x by half a step of e4m3
    back = oracle.dequantise(vals, e)
    ok = np.isfinite(back)
    assert np.array_equal(torch.tensor(back[ok]).to(torch.bfloat16).double().numpy(), back[ok])
    err = np.abs(back - xd.numpy())[ok]
    bound = np.maximum(2.0 ** -4 * np.abs(xd.numpy()), 2.0 ** -10 * (2.0 ** e)[:, None])[ok]
    assert (err <= bound).all()


def test_ties_go_to_the_even_code():
    vals, e = oracle.quantise(np.array([[448.0, 17.0, 19.0, 21.0, 2.0 ** -10, 3 * 2.0 ** -10]]))
    assert e[0] == 0 and vals[0].tolist() == [448.0, 16.0, 20.0, 20.0, 0.0, 2.0 ** -8]


def test_cached_rows_and_decode():
    r = np.random.default_rng(5)
    pages = r.standard_normal((5, 2, 8, 16))
    rows = oracle.cached_rows(pages, [3, 0, -1], 11, 8)
    assert np.array_equal(rows[:, :8], pages[3]) and np.array_equal(rows[:, 8:], pages[0, :, :3])
    q = r.standard_normal((4, 16))
    ref = gqa_decode(q[None], rows[None], rows[None], [11], 0.4)[0]
    assert np.allclose(oracle.decode(q, rows, rows, 0.4), ref, atol=1e-14)
