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


def _weights(x, ids, score):
    """Renormalised weights of the chosen ids from the logarithms of their
    scores (up to a constant per row): l - log(1 + e^l), or l.  Scores that
    are zero in 64 bits stay zero."""
    l = np.take_along_axis(x.astype(np.float64), np.maximum(ids, 0), 1)
    zero = l < -709.7827 if score == "sigmoid" else l - x.max(1, keepdims=True).astype(np.float64) < -745.14
    if score == "sigmoid":
        l = np.where(l < 0, l - np.log1p(np.exp(np.minimum(l, 0))), -np.log1p(np.exp(-np.maximum(l, 0))))
    e = np.where(zero, 0.0, np.exp(l - l.max(1, keepdims=True)))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def _check_weights(x, ids, w, score, k, scale):
    want = _weights(x, ids, score) * scale
    # exponents of at most 200 that matter (below, the weight is nothing): off
    # by a unit of themselves; exp, sums and quotients a few more.  Weights
    # below the smallest normal number are off by that at most.
    tol = (2 * 200 + 2 * k + 16) * R.U
    assert np.all(np.abs(w - want) <= tol * want + 2.0 ** -126 * scale)
    total = want.sum(1)
    assert np.all(np.abs(w.astype(np.float64).sum(1) - total) <= (2 * k + 4) * R.U * scale)
    assert (total > 0).any()


@pytest.mark.parametrize("E,k", [(8, 3), (128, 8), (256, 20), (1000, 33)])
def test_route_weights_of_scores_that_underflow(cuda, E, k):
    """Renormalised weights depend on the ratios of the chosen scores, which
    stay ordinary numbers where the scores do not: logistic scores of very
    negative logits, and softmax scores far below the row's largest."""
    g = np.random.default_rng(E)
    M = 40
    centre = g.choice([-2.0, -62.0, -87.0, -95.0, -104.0, -160.0, -800.0, -1e4, -1e30], (M, 1))
    x = (centre + 6 * g.standard_normal((M, E))).astype(np.float32)
    x[-1] = LOW
    for bias in (None, (1e-3 * g.standard_normal(E)).astype(np.float32)):
        for groups, top in ((1, 1), (2, 1) if E // 2 >= k else (2, 2)):
            ids, w = _route(x, k, score="sigmoid", bias=bias, groups=groups, top_groups=top, scale=2.5)
            ids_ref, _ = R.route(x, k, "sigmoid", bias, groups, top)
            assert np.array_equal(ids, ids_ref)
            _check_weights(x, ids, w, "sigmoid", k, 2.5)
    # softmax: a bias keeps the experts of large score from being chosen
    x = (centre + 6 * g.standard_normal((M, E))).astype(np.float32)
    x[:, :E // 4] = 0.0
    bias = (1e-3 * g.standard_normal(E)).astype(np.float32)
    bias[:E // 4] = -np.inf
    bias[0] = -3.0
    kk = min(k, E - E // 4)
    ids, w = _route(x, kk, bias=bias, scale=2.5)
    assert np.array_equal(ids, R.route(x, kk, "softmax", bias)[0])
    _check_weights(x, ids, w, "softmax", kk, 2.5)


def test_route_weights_do_not_depend_on_the_path(cuda):
    """Rows of equal scores, of which one in two also holds a near tie and is
    decided in fp64, have equal weights."""
    E, k = 64, 4
    x = np.full((32, E), -140.0, dtype=np.float32)
    x[:, :k] = np.float32([-95.0, -96.5, -97.0, -99.0])
    bias = np.zeros(E, dtype=np.float32)
    bias[:k] = [0.4, 0.3, 0.2, 0.1]
    bias[k:] = -1.0
    bias[40:50] = 0.1  # as the last of the four, and closed in every other row
    x[::2, 40:50], x[1::2, 40:50] = -95.0, -np.inf
    ids, w = _route(x, k, score="sigmoid", bias=bias)
    assert np.array_equal(ids, np.tile(np.arange(k), (32, 1)))
    _check_weights(x, ids, w, "sigmoid", k, 1.0)


@pytest.mark.parametrize("M,E,k,dt", [((1 << 28) + 37, 2, 1, torch.bfloat16), ((1 << 26) + 5, 34, 31, torch.bfloat16)])
def test_route_more_rows_than_one_launch_holds(cuda, M, E, k, dt):
    """A launch holds fewer than 2^32 threads: 2^28 rows of sixteen lanes, or
    2^26 of sixty-four."""
    x = torch.zeros((M, E), dtype=dt, device=cuda)
    x[:, E - 1] = 1.0
    x[0, 0], x[-1, 0], x[M // 2, 0] = 2.0, 2.0, 2.0
    ids, w = cr.route(x, k, ids=torch.full((M, k), -7, dtype=torch.int32, device=cuda))
    first = ids[:, 0]
    assert int((first != E - 1).sum()) == 3
    assert first[0] == 0 and first[-1] == 0 and first[M // 2] == 0
    assert torch.equal(ids[1], ids[-2]) and torch.equal(ids[0], ids[-1])
    assert torch.equal(w[1], w[-2]) and torch.equal(w[0], w[-1])
