"""Infinite and largest values in adapters per row: the second product takes
the first one's sums as terms of a bf16 split, and the result is still the
formula's infinity, NaN or number."""

import numpy as np
import pytest
import torch

import w8a8_int8_linear_amd as cr
from tests.gpu_util import to_dev, to_np
from workloads import to_bf16_values

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}

# rows, adapters: the 16-row tiles and the 64-row ones
SIZES = [(5, 3), (150, 2)]


def _dev(v, dtype):
    return to_dev(np.ascontiguousarray(v), dtype)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,E", SIZES)
@pytest.mark.parametrize("r", [16, 48, 96, 176])
def test_lora_infinite_entries_of_b(cuda, M, E, r, dt):
    """B holds infinities of both signs, where T is positive, negative and
    zero, alone and several in a row: the infinity of the formula (0 x inf and
    inf - inf: NaN), in those features only."""
    g = np.random.default_rng(r + M)
    K, N = 64, 150
    x = to_bf16_values(g.standard_normal((M, K)).astype(np.float32))
    a = to_bf16_values((g.standard_normal((E, r, K)) / 8).astype(np.float32))
    a[:, 3] = 0.0                                       # T[:, 3] is zero
    a[:, 5], a[:, 9, 1:] = 0.0, 0.0
    a[:, 5, 0], a[:, 9, 0] = 0.5, -0.25                 # T[:, 5] and T[:, 9] are products of one value: no second term
    b = to_bf16_values((g.standard_normal((E, N, r)) * 0.3).astype(np.float32))
    inf = np.inf
    b[:, 2, 0], b[:, 17, 1], b[:, 40, r - 1], b[:, 64, 5], b[:, 65, 9] = inf, -inf, inf, inf, -inf
    b[:, 90, 3] = inf                                   # 0 x inf
    b[:, 100, [0, 1, 2]] = inf                          # any signs of T
    b[:, 130, [4, 7]] = [inf, -inf]
    b[0, 149, 6] = -inf                                 # one adapter only
    s = (0.25 + g.random(E)).astype(np.float32)
    s[1] = -s[1]
    y = g.standard_normal((M, N)).astype(np.float32)
    y = to_bf16_values(y) if dt == "bf16" else y
    ids = (np.arange(M) % E).astype(np.int32)
    out = to_np(cr.lora_add_grouped(_dev(x, torch.bfloat16), _dev(a, torch.bfloat16), _dev(b, torch.bfloat16),
                                    _dev(s, torch.float32), _dev(y, TDT[dt]), cr.group_rows(_dev(ids, torch.int32), E)))
    terms = 3 if dt == "f32" else 2
    for m in range(M):
        A, B = a[ids[m]].astype(np.float64), b[ids[m]].astype(np.float64)
        t = A @ x[m].astype(np.float64)
        with np.errstate(invalid="ignore"):
            want = y[m] + float(s[ids[m]]) * (B * t).sum(1)
        bad = ~np.isfinite(B).all(1)
        assert bad.sum() >= 8 and np.isfinite(want[~bad]).all() and not np.isfinite(want[bad]).any()
        assert np.array_equal(out[m, bad], want[bad].astype(np.float32), equal_nan=True), m
        dtm = K * U * (np.abs(A) @ np.abs(x[m]).astype(np.float64)) + 2.0 ** (-8 * terms) * np.abs(t)
        F = np.abs(B[~bad])
        bound = abs(float(s[ids[m]])) * (F @ dtm + (r * terms + 2) * U * (F @ (np.abs(t) + dtm)))
        bound = bound + HALF_STEP[dt] * (np.abs(want[~bad]) + bound)
        assert np.all(np.abs(out[m, ~bad] - want[~bad]) <= bound), m


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,E", SIZES)
def test_lora_sums_next_to_the_largest_number(cuda, M, E, dt):
    """T between bf16's largest number and fp32's, which bf16 rounds to an
    infinity: its first term is bf16's largest number."""
    K, N, r = 32, 70, 32
    x = np.zeros((M, K), dtype=np.float32)
    a = np.zeros((E, r, K), dtype=np.float32)
    x[:, 0], x[:, 1] = 255.0 / 128 * 2.0 ** 64, 2.0 ** 60
    a[:, 7, 0], a[:, 7, 1] = 2.0 ** 63, 0.75 * 2.0 ** 60       # T[:, 7] = (255 + 0.75) 2^120
    x[1::2] *= -1
    b = np.zeros((E, N, r), dtype=np.float32)
    b[:, :, 7] = 2.0 ** -121 * (1 + np.arange(N) % 5)
    y, s = np.zeros((M, N), dtype=np.float32), np.ones(E, dtype=np.float32)
    ids = (np.arange(M) % E).astype(np.int32)
    out = to_np(cr.lora_add_grouped(_dev(x, torch.bfloat16), _dev(a, torch.bfloat16), _dev(b, torch.bfloat16),
                                    _dev(s, torch.float32), _dev(y, TDT[dt]), cr.group_rows(_dev(ids, torch.int32), E)))
    want = np.where(np.arange(M) % 2 == 0, 1.0, -1.0)[:, None] * 127.875 * (1 + np.arange(N) % 5)
    # two terms hold T to 2^-16, three exactly; two additions and the output's rounding
    bound = ((2.0 ** -16 if dt == "bf16" else 0.0) + 4 * U + HALF_STEP[dt]) * np.abs(want) * 1.01
    assert np.all(np.abs(out - want) <= bound)
