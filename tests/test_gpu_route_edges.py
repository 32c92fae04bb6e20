"""The router where fp32 does not carry it: choice values of scores of
different sizes that lie closer than their errors, sums of choice values past
the largest fp32 number, and scores that underflow.  Against the 64-bit
statements of tests/routed_oracle.py and the weights' own below."""

import numpy as np
import pytest
import torch

import tests.routed_oracle as R
import w8a8_int8_linear_amd as cr
from tests.gpu_util import to_dev, to_np

pytestmark = pytest.mark.gpu

LOW = float(np.finfo(np.float32).min)


def _route(x, k, **rule):
    if rule.get("bias") is not None:
        rule["bias"] = to_dev(rule["bias"], torch.float32)
    ids, w = cr.route(to_dev(x, torch.float32), k, **rule)
    return to_np(ids), to_np(w)


@pytest.mark.parametrize("E,k", [(128, 3), (256, 1), (256, 5), (256, 14), (500, 20), (1000, 33), (1024, 64)])
def test_route_near_ties_of_scores_of_different_size(cuda, E, k):
    """Softmax with a bias.  One expert's score is next to 1, and the other
    exponentials of its part of the fp32 sum (runs of four experts, one in 16,
    32 or 64) are about 2^-24: each is lost or counts twice, so the score is
    off by up to 15 units of 2^-24 either way.  More than k experts have no
    score; their choice values are their biases, 2.25 units apart: far enough
    to be told from each other, not from the one.  The choice is that of the
    fp64 values."""
    g = np.random.default_rng(E + k)
    M, n, u, v = 400, k + 10, 2.0 ** -24, 2.0 ** -6
    lanes = 16 if k <= 14 and E <= 256 else 32 if k <= 30 and E <= 512 else 64
    run = np.arange(E) // 4 % lanes == 0
    mates = np.nonzero(run)[0][1:]
    tiny = g.permutation(np.nonzero(~run)[0])[:n]
    x = np.full((M, E), -60.0, dtype=np.float32)
    x[:, 0] = 0.0
    x[:, mates] = np.log(u * g.uniform(0.5, 1.5, (M, 1)))
    bias = np.full(E, -1.0, dtype=np.float32)
    bias[tiny] = v + 2.25 * u * np.arange(n)
    bias[0] = v + 2.25 * u * (n - k) + len(mates) * u - 1   # among the last of the k
    ids, _ = _route(x, k, bias=bias, renormalise=False)
    ids_ref, _ = R.route(x, k, "softmax", bias, renormalise=False)
    assert 0.3 < (ids_ref == 0).any(1).mean() < 0.7
    for m in range(M):
        if not np.array_equal(ids[m], ids_ref[m]):
            # equal up to choices whose fp64 values differ by less than their own rounding
            c = R.choice_values(x[m], "softmax", bias)
            assert np.allclose(c[ids[m]], c[ids_ref[m]], rtol=0, atol=4e-16), m


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_group_values_past_fp32(cuda, score):
    """Biases whose sum over two experts of a group leaves fp32's range (the
    lowest value as a mask, large ones): group values are compared as fp64
    values, so such a group is neither lost nor tied with another."""
    g = np.random.default_rng(5)
    for M, E, groups in ((9, 16, 4), (5, 96, 24), (3, 600, 8)):
        per = E // groups
        x = g.standard_normal((M, E)).astype(np.float32)
        for value in (LOW, -3e38, 3e38):
            for top, k in ((groups, 12), (groups // 2 + 1, 5), (1, 2)):
                bias = (0.1 * g.standard_normal(E)).astype(np.float32)
                far = g.permutation(groups)[:groups // 2 + 1]      # whole groups, in steps of their own
                for i, f in enumerate(far):
                    bias[f * per:(f + 1) * per] = np.float32(value) * np.float32(1 - 0.02 * i)
                bias[far[0] * per] = 0.5                           # one of them has an ordinary expert left
                for renorm in (True, False):
                    ids, w = _route(x, k, score=score, bias=bias, groups=groups, top_groups=top, renormalise=renorm)
                    ids_ref, w_ref = R.route(x, k, score, bias, groups, top, renorm)
                    assert np.array_equal(ids, ids_ref), (E, value, top)
                    assert np.all(np.abs(w - w_ref) <= (64 + E + 16) * R.U * np.abs(w_ref)), (E, value, top)
