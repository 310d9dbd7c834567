"""Attention over long contexts, by the norm of each row's error.

A result over T tokens shrinks like 1 / sqrt(T), so a bound by the largest |v| says little there.  A token's part
p v of a result is off by a factor of its own: three roundings to 16 bits of at most 2^-11 (the weight; its product
with a step, or the value as tiles are expanded, and the factor that follows the maximum) and what the score's
rounding moves, 2^-10.8 at one standard deviation for normal keys, twice that here.  They are independent from token
to token, so the row is off by at most (3 2^-11 + 2^-9.8) sqrt(sum_t p_t^2 |v_t|^2), and by its own rounding, half a
unit of the row type times |out|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import serve_ref as ref
from tests.test_serve import NP_TYPE, attention_case, ld, run_attention  # noqa: F401
from tests.test_serve_numbers import rows_of

gpu = pytest.mark.gpu
FACTOR = 3 * 2.0 ** -11 + 2.0 ** -9.8

# (lens, head_dim, kv heads, query heads of each, type, window)
LONG = [([(20000, 1)], 128, 1, 4, torch.bfloat16, 0), ([(30000, 1)], 64, 1, 1, torch.float16, 0),
        ([(5000, 1), (12, 1), (7000, 1)], 128, 2, 8, torch.bfloat16, 0), ([(9000, 1)], 128, 1, 1, torch.float16, 5000),
        ([(6000, 4), (100, 4)], 128, 1, 4, torch.bfloat16, 0), ([(4000, 2)], 256, 1, 5, torch.float16, 0),
        ([(3000, 300)], 128, 1, 2, torch.bfloat16, 0), ([(4000, 150), (50, 3)], 128, 1, 4, torch.float16, 1000),
        ([(0, 1500)], 128, 1, 1, torch.bfloat16, 0), ([(5000, 40)], 64, 2, 4, torch.float16, 0),
        ([(3000, 90), (700, 1)], 256, 1, 3, torch.bfloat16, 0)]


def results(c, window, values=lambda v: v):
    """Results [n, Q, D] in 64 bits, and the bound of each one's error [n, Q]; the values as ``values`` changes them."""
    q = c["q"].double().cpu().numpy()
    out, bound = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(len(c["seq"])):
        a, e, pos, k, v = rows_of(c, b)
        v = values(v)
        t = np.arange(len(k))
        seen = (t <= pos[:, None]) & ((t > pos[:, None] - window) if window else True)
        for h in range(k.shape[1]):
            g = q.shape[1] // k.shape[1]
            s = np.einsum("ngd,td->ngt", q[a:e, h * g:(h + 1) * g], k[:, h]) * c["D"] ** -0.5
            s = np.where(seen[:, None], s, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[a:e, h * g:(h + 1) * g] = p @ v[:, h]
            bound[a:e, h * g:(h + 1) * g] = FACTOR * np.sqrt(p ** 2 @ (v[:, h] ** 2).sum(-1))
    return out, bound + NP_TYPE[c["dtype"]] / 2 * np.linalg.norm(out, axis=-1)


def long_case(i):
    lens, D, H, group, dtype, _ = LONG[i]
    return attention_case(np.random.default_rng(100 + i), lens, D, H, group, 32, dtype)


@gpu
@pytest.mark.parametrize("i", range(len(LONG)))
def test_rows_of_long_contexts_are_within_their_norm(ld, i):  # noqa: F811
    c, window = long_case(i), LONG[i][-1]
    got, _, err = run_attention(ld, c, window)
    want, bound = results(c, window)
    assert err == 0
    off = np.linalg.norm(got.double().cpu().numpy() - want, axis=-1)
    assert (off <= bound).all(), float((off / bound).max())


def test_the_bound_sees_values_that_are_lost_or_exchanged():
    """In 64 bits, on the CPU: 256 of some 5000 tokens' values zeroed, or put in one another's place."""
    rng = np.random.default_rng(3)
    D, T = 64, 5000
    pages = np.zeros((T // 32 + 1, 1, 2, ref.tile_bytes(D)), np.uint8)
    k, v = (x.astype(np.float16).astype(float) for x in rng.standard_normal((2, T, 1, D)))
    ref.append(pages, k, v, np.arange(T), 32)
    c = {"q": torch.from_numpy(rng.standard_normal((3, 2, D))).half(), "pages": pages, "table": np.arange(T // 32 + 1)[None],
         "start": np.array([0, 3]), "seq": np.array([T]), "P": 32, "D": D, "dtype": torch.float16}
    want, bound = results(c, 0)
    exact = ref.attend(c["q"].double().numpy(), pages, 32, c["table"], c["start"], c["seq"], D ** -0.5, 0)[0]
    assert np.abs(exact - want).max() < 1e-12

    def lost(x):
        return np.concatenate([x[:2000], 0 * x[2000:2256], x[2256:]])

    def exchanged(x):
        return np.concatenate([x[:2000], x[2000:2256][::-1], x[2256:]])

    for values in (lost, exchanged):
        off = np.linalg.norm(results(c, 0, values)[0] - want, axis=-1)
        assert (off > 8 * bound).all()
