"""Rows that choose their weights, on the GPU against the 64-bit statements
of tests/routed_oracle.py (whose error bounds count the roundings of a
correct fp32 evaluation): routing and the plan (equal whole numbers), the
grouped products (also bit for bit against the linears of each group's weight
alone), the weighted sum, adapters per row, and all of them together."""

import numpy as np
import pytest
import torch

import tests.routed_oracle as R
import w8a8_int8_linear_amd as cr
from tests.gpu_util import to_dev, to_np
from workloads import to_bf16_values

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _close(got, want, bound):
    bad = np.abs(got.astype(np.float64) - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float((np.abs(got - want) / bound).max()))


def _vals(a, dt):
    return to_bf16_values(a) if dt == "bf16" else np.asarray(a, dtype=np.float32)


# ------------------------------------------------------------------ routing

def _logits(M, E, seed, dt, closed=0.0):
    g = np.random.default_rng(seed)
    x = _vals((1.5 * g.standard_normal((M, E))).astype(np.float32), dt)
    if closed:
        x[g.random((M, E)) < closed] = -np.inf
    return x


# M, E, k, groups, top_groups
ROUTES = [(1, 1, 1, 1, 1), (1, 128, 8, 1, 1), (3, 7, 7, 1, 1), (5, 64, 6, 1, 1), (130, 65, 4, 5, 2), (33, 256, 8, 8, 4),
          (17, 320, 10, 64, 3), (9, 1024, 64, 1, 1), (12, 1000, 32, 4, 1), (64, 24, 5, 12, 7), (300, 160, 6, 8, 3)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,E,k,groups,top", ROUTES)
def test_route(cuda, M, E, k, groups, top, score, dt):
    for case, (biased, renorm, closed) in enumerate([(False, True, 0.0), (True, True, 0.0), (False, False, 0.0),
                                                     (True, False, 0.5), (False, True, 0.9)]):
        x = _logits(M, E, 10 * M + E + case, dt, closed)
        if closed and M > 2:
            x[M // 2] = -np.inf  # a row with nothing open
        bias = (0.1 * np.random.default_rng(case).standard_normal(E)).astype(np.float32) if biased else None
        ids, w = cr.route(to_dev(x, TDT[dt]), k, score=score, bias=None if bias is None else to_dev(bias, torch.float32),
                          groups=groups, top_groups=top, renormalise=renorm, scale=2.5)
        ids_ref, w_ref = R.route(x, k, score, bias, groups, top, renorm, 2.5)
        assert np.array_equal(to_np(ids), ids_ref), case
        # fp32 scores: the exponent's argument (below 32 here) is off by a unit
        # of itself, exp and the division by a few units, sums by one per term
        tol = (2 * 32 + E + 16) * R.U
        assert np.all(np.abs(to_np(w) - w_ref) <= tol * np.abs(w_ref)), case


def test_route_ties_and_extremes(cuda):
    """Equal logits go to the lowest index; signed zeros are equal; +inf is
    the largest finite value; the lowest finite value can be chosen; NaN and
    a bias of -inf close an expert."""
    inf, low = np.inf, float(np.finfo(np.float32).min)
    x = np.array([[1, 1, 1, 1, 1, 1], [0.0, -0.0, 0.0, -0.0, -1, -1], [inf, 0, inf, 0, 0, 0],
                  [low, low, low, low, low, low], [np.nan, 2, np.nan, 1, -inf, 3], [5, low, low, low, low, low]],
                 dtype=np.float32)
    for score in ("softmax", "sigmoid"):
        for bias in (None, np.zeros(6, np.float32), np.array([0, 0, -inf, 0, 0, 0], np.float32)):
            for groups, top in ((1, 1), (3, 2)):
                ids, w = cr.route(to_dev(x, torch.float32), 3, score=score, groups=groups, top_groups=top,
                                  bias=None if bias is None else to_dev(bias, torch.float32))
                ids_ref, w_ref = R.route(x, 3, score, bias, groups, top)
                assert np.array_equal(to_np(ids), ids_ref), (score, bias, groups)
                assert np.all(np.abs(to_np(w) - w_ref) <= 64 * R.U * np.abs(w_ref)), (score, bias, groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(64, 8, 1, 1), (256, 8, 8, 3), (500, 20, 4, 2), (1024, 40, 16, 5)])
def test_route_near_ties(cuda, score, E, k, groups, top):
    """Values that fp32 does not tell apart: logits a few units apart around
    few levels, and a bias that undoes most of their differences (its own
    rounding leaves some).  The choice is that of the fp64 values."""
    g = np.random.default_rng(E)
    M = 60
    x = (g.integers(0, 4, (M, E)) * 0.5).astype(np.float32)
    x = (x * (1 + g.integers(-3, 4, (M, E)) * 2.0 ** -23)).astype(np.float32)
    for bias in (None, np.zeros(E, np.float32), (g.integers(0, 3, E) * 2.0 ** -24).astype(np.float32)):
        ids, w = cr.route(to_dev(x, torch.float32), k, score=score, groups=groups, top_groups=top,
                          bias=None if bias is None else to_dev(bias, torch.float32), renormalise=False)
        ids_ref, w_ref = R.route(x, k, score, bias, groups, top, False)
        ids = to_np(ids)
        # equal up to choices whose fp64 values differ by less than their own rounding
        for m in range(M):
            if not np.array_equal(ids[m], ids_ref[m]):
                assert bias is not None or groups > 1
                c = R.choice_values(x[m], score, bias)
                assert np.allclose(np.sort(c[ids[m]]), np.sort(c[ids_ref[m]]), rtol=0, atol=4e-16), m
        assert np.all(np.abs(to_np(w) - w_ref) <= (64 + E + 16) * R.U * np.abs(w_ref) + 4e-7 * (groups > 1))


def test_route_strided_logits_and_given_outputs(cuda):
    x = _logits(21, 40, 3, "f32")
    buf = torch.full((21, 53), 9.0, device=cuda)
    buf[:, 5:45] = to_dev(x, torch.float32)
    ids = torch.full((21, 4), 7, dtype=torch.int32, device=cuda)
    w = torch.empty((21, 4), device=cuda)
    got = cr.route(buf[:, 5:45], 4, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w
    assert np.array_equal(to_np(ids), R.route(x, 4, "softmax")[0])


# ---------------------------------------------------------------- the plan

@pytest.mark.parametrize("M,k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 128), (3, 5, 4), (257, 6, 64), (1000, 8, 7), (64, 1, 4096),
                                   (1024, 8, 128), (1025, 8, 33), (4099, 8, 256), (20000, 3, 1000), (70000, 1, 2)])
def test_group_rows(cuda, M, k, E):
    g = np.random.default_rng(M + k + E)
    for kind in ("mixed", "one", "none"):
        if kind == "mixed":
            ids = g.integers(-1, E + 1, size=(M, k)).astype(np.int32)  # some outside on both sides
        else:
            ids = np.full((M, k), E - 1 if kind == "one" else -5, dtype=np.int32)
        p = cr.group_rows(to_dev(ids, torch.int32), E)
        order, offsets = R.plan(ids, E)
        assert np.array_equal(to_np(p.order), order) and np.array_equal(to_np(p.offsets), offsets), kind
        # the row tiles: every group cut evenly (in whole 16 rows) into as few
        # as hold it, in order, the rest last
        t = to_np(p.tiles)
        starts = np.append(offsets, M * k)
        at = 10
        for b in range(5):
            bm = 16 << b
            want = []
            for e in range(E + 1):
                rows = int(starts[e + 1] - starts[e])
                n = -(-rows // bm)
                step = bm if n <= 1 else (-(-rows // n) + 15) // 16 * 16
                want += [(e, int(starts[e]) + i * step) for i in range(n)]
                assert n <= 1 or (n - 1) * step < rows <= n * step <= n * bm
            assert t[b] == sum(e < E for e, _ in want) and t[5 + b] == len(want), (kind, bm)
            assert np.array_equal(t[at:at + 2 * len(want)].reshape(-1, 2), np.array(want, dtype=np.int32).reshape(-1, 2))
            at += 2 * (M * k // bm + min(E + 1, M * k))


def test_group_rows_into_the_same_plan(cuda):
    g = np.random.default_rng(1)
    first = to_dev(g.integers(0, 9, size=(50, 4)).astype(np.int32), torch.int32)
    p = cr.group_rows(first, 9)
    ids = g.integers(0, 9, size=(50, 4)).astype(np.int32)
    assert cr.group_rows(to_dev(ids, torch.int32), 9, out=p) is p
    assert np.array_equal(to_np(p.order), R.plan(ids, 9)[0])


# ------------------------------------------------------- experts' products

def _codes(shape, seed):
    g = np.random.default_rng(seed)
    return np.clip(np.rint(36 * g.standard_normal(shape)), -127, 127).astype(np.int8)


def _scales(n, seed, s):
    return ((0.5 + np.random.default_rng(seed).random(n)) * s / 127).astype(np.float32)


def _packed(q, s, G):
    return cr.Packed(to_dev(q, torch.int8), to_dev(s, torch.float32), G)


def _ids(M, k, E, seed, unused=0.0):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] if k <= E else g.integers(0, E, k) for _ in range(M)]).astype(np.int32)
    ids[g.random((M, k)) < unused] = -1
    return ids.reshape(M, k)


# M, k, E, K, N, G, share of pairs without a group: every kernel the launch
# rules choose (few and many workgroups of the ring's three tile heights, the
# tiled kernel), whole and ragged K and N
PRODUCTS = [(20, 2, 16, 208, 4200, 16, 0.1), (20, 2, 16, 384, 4224, 64, 0), (160, 1, 16, 128, 1350, 64, 0.1),
            (200, 1, 4, 96, 5200, 16, 0.05), (210, 1, 4, 256, 5185, 64, 0.05),
            (900, 1, 2, 1152, 8200, 64, 0.05), (900, 1, 2, 1168, 8195, 16, 0.0), (460, 2, 3, 1040, 8200, 16, 0.02),
            (1, 1, 1, 16, 1, 16, 0), (1, 8, 128, 256, 96, 256, 0), (2, 2, 8, 1152, 100, 64, 0), (16, 2, 8, 1152, 260, 64, 0.2),
            (5, 3, 4, 48, 33, 16, 0.5), (40, 4, 6, 2048, 130, 256, 0.1), (150, 2, 3, 320, 77, 64, 0.1),
            (300, 1, 2, 1040, 200, 16, 0.0), (513, 2, 4, 1152, 300, 64, 0.05), (7, 2, 300, 256, 40, 64, 0.3),
            (700, 2, 3, 256, 513, 64, 0.0), (1300, 1, 2, 208, 272, 16, 0.1)]


@pytest.mark.parametrize("M,k,E,K,N,G,unused", PRODUCTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_linear_grouped(cuda, M, k, E, K, N, G, unused, dt):
    ids = _ids(M, k, E, M + K, unused)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    w, sw = _codes((E * N, K), 1), _scales(E * N, 2, 0.08)
    b = (0.1 * np.random.default_rng(3).standard_normal(E * N)).astype(np.float32)
    pw = _packed(w, sw, G)
    for source, dest, act, bias in [("by_row", "sorted", None, None), ("sorted", "by_pair", None, b),
                                    ("by_pair", "by_pair", "gelu_erf", b), ("by_row", "by_pair", "silu", None),
                                    ("sorted", "sorted", "gelu_tanh", b)]:
        rows = M if source == "by_row" else M * k
        x, sx = _codes((rows, K), 4), _scales(rows, 5, 3.0)
        out = torch.full((M * k, N), -3.0, dtype=TDT[dt], device=cuda)
        got = cr.linear_grouped(_packed(x, sx, G), pw, plan, None if bias is None else to_dev(bias, torch.float32),
                                act=act, source=source, dest=dest, out=out)
        assert got is out
        want, bound, written = R.grouped(x, sx, ids, E, w, sw, bias, act, source, dest, dtype=dt)
        y = to_np(got)
        _close(y[written], want[written], bound[written])
        assert np.all(y[~written] == -3.0)


@pytest.mark.parametrize("M,k,E,K,N,G,unused", PRODUCTS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_linear_gated_grouped(cuda, M, k, E, K, N, G, unused, dt):
    ids = _ids(M, k, E, M + K + 1, unused)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    wg, wu = _codes((E * N, K), 1), _codes((E * N, K), 6)
    sg, su = _scales(E * N, 2, 0.08), _scales(E * N, 7, 0.08)
    g = np.random.default_rng(8)
    bg, bu = (0.1 * g.standard_normal((2, E * N))).astype(np.float32)
    for source, dest, act, biased in [("by_row", "sorted", "silu", False), ("sorted", "by_pair", "gelu_tanh", True),
                                      ("by_pair", "sorted", "gelu_erf", True)]:
        rows = M if source == "by_row" else M * k
        x, sx = _codes((rows, K), 4), _scales(rows, 5, 3.0)
        out = torch.full((M * k, N), -3.0, dtype=TDT[dt], device=cuda)
        got = cr.linear_gated_grouped(_packed(x, sx, G), _packed(wg, sg, G), _packed(wu, su, G), plan,
                                      to_dev(bg, torch.float32) if biased else None,
                                      to_dev(bu, torch.float32) if biased else None, act=act, source=source, dest=dest,
                                      out=out)
        want, bound, written = R.grouped(x, sx, ids, E, wg, sg, bg if biased else None, act, source, dest, wu, su,
                                         bu if biased else None, dt)
        y = to_np(got)
        _close(y[written], want[written], bound[written])
        assert np.all(y[~written] == -3.0)


@pytest.mark.parametrize("M,E,K,N", [(3, 4, 256, 64), (90, 3, 1152, 130), (700, 2, 512, 272), (900, 2, 1152, 8200)])
def test_groups_carry_the_bits_of_the_linear_of_their_weight(cuda, M, E, K, N):
    """The accumulator is exact and the epilogue the same expression, so a
    group's rows equal the linear of its weight alone, bit for bit."""
    G = 64
    ids = _ids(M, 1, E, 9)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    px = _packed(_codes((M, K), 1), _scales(M, 2, 3.0), G)
    ws = [_packed(_codes((E * N, K), 3 + i), _scales(E * N, 5 + i, 0.08), G) for i in range(2)]
    b = to_dev((0.1 * np.random.default_rng(3).standard_normal(E * N)).astype(np.float32), torch.float32)
    y = cr.linear_grouped(px, ws[0], plan, b)
    ya = cr.linear_grouped(px, ws[0], plan, b, act="gelu_erf", out_dtype=torch.float32)
    yg = cr.linear_gated_grouped(px, ws[0], ws[1], plan, b, None, act="gelu_tanh", dest="by_pair")
    for e in range(E):
        rows = torch.from_numpy(np.nonzero(ids[:, 0] == e)[0]).to(cuda)
        if rows.numel() == 0:
            continue
        sub = cr.Packed(px.q[rows].contiguous(), px.scale[rows].contiguous(), G)
        we = [cr.Packed(w.q[e * N:(e + 1) * N], w.scale[e * N:(e + 1) * N].contiguous(), G) for w in ws]
        be = b[e * N:(e + 1) * N].contiguous()
        assert torch.equal(y[rows], cr.linear(sub, we[0], be))
        assert torch.equal(ya[rows], cr.linear_act(sub, we[0], be, "gelu_erf", torch.float32))
        assert torch.equal(yg[rows], cr.linear_gated(sub, we[0], we[1], be, None, "gelu_tanh"))


@pytest.mark.parametrize("M,E,K,N", [(20, 4, 192, 75), (600, 2, 192, 75), (450, 2, 1152, 8203)])
def test_grouped_strided_operands_and_outputs(cuda, M, E, K, N):
    """Row pitches above the width, outputs that start off 16 bytes, padding
    left as it was."""
    G, k = 64, 2
    ids = _ids(M, k, E, 2, 0.1)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    x, sx, w, sw = _codes((M, K), 1), _scales(M, 2, 3.0), _codes((E * N, K), 3), _scales(E * N, 4, 0.08)
    xb = torch.zeros((M, K + 32), dtype=torch.int8, device=cuda)
    wb = torch.zeros((E * N, K + 64), dtype=torch.int8, device=cuda)
    xb[:, :K], wb[:, :K] = to_dev(x, torch.int8), to_dev(w, torch.int8)
    px, pw = cr.Packed(xb[:, :K], to_dev(sx, torch.float32), G), cr.Packed(wb[:, :K], to_dev(sw, torch.float32), G)
    for dt in ("f32", "bf16"):
        buf = torch.full((M * k, N + 9), -3.0, dtype=TDT[dt], device=cuda)
        cr.linear_grouped(px, pw, plan, out=buf[:, 3:3 + N])
        want, bound, written = R.grouped(x, sx, ids, E, w, sw, dtype=dt)
        y = to_np(buf)
        _close(y[written, 3:3 + N], want[written], bound[written])
        assert np.all(y[~written] == -3.0) and np.all(y[:, :3] == -3.0) and np.all(y[:, 3 + N:] == -3.0)


# ----------------------------------------------------------- the weighted sum

@pytest.mark.parametrize("M,k,N", [(0, 2, 8), (1, 1, 1), (1, 8, 2048), (33, 2, 1152), (7, 13, 100), (129, 6, 77), (300, 3, 264)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_combine_rows(cuda, M, k, N, dt):
    g = np.random.default_rng(M + N)
    E = 9
    ids = g.integers(-1, E + 1, size=(M, k)).astype(np.int32)
    if M > 1:
        ids[M // 2] = -1  # a row without any choice becomes zero
    y = _vals(g.standard_normal((M * k, N)).astype(np.float32), dt)
    y[((ids < 0) | (ids >= E)).reshape(-1)] = np.nan  # rows nobody wrote are not read
    w = g.random((M, k)).astype(np.float32)
    yt = torch.from_numpy(y).to(TDT[dt]).to(cuda)
    got = cr.combine_rows(yt, to_dev(w, torch.float32), to_dev(ids, torch.int32), E)
    want, bound = R.combine(y, w, ids, E, dt)
    _close(to_np(got), want, bound)
    if M:
        buf = torch.full((M, N + 5), -3.0, dtype=TDT[dt], device=cuda)
        wide = torch.zeros((M * k, N + 3), dtype=TDT[dt], device=cuda)
        wide[:, :N] = yt
        cr.combine_rows(wide[:, :N], to_dev(w, torch.float32), to_dev(ids, torch.int32), E, out=buf[:, 1:1 + N])
        assert torch.equal(buf[:, 1:1 + N], got)
        assert torch.all(buf[:, 0] == -3.0) and torch.all(buf[:, 1 + N:] == -3.0)


def test_combine_more_outputs_than_one_grid_of_threads(cuda):
    """More outputs than a launch has threads (2^32), a width that takes no
    16-byte pieces."""
    M, N = 1 << 22, 1027
    y = torch.full((M, N), 2.0, dtype=torch.bfloat16, device=cuda)
    y[-1], y[M // 2, 5] = 3.0, -1.0
    w = torch.full((M, 1), 0.5, device=cuda)
    ids = torch.zeros((M, 1), dtype=torch.int32, device=cuda)
    ids[7] = -1
    out = torch.full_like(y, 9.0)
    cr.combine_rows(y, w, ids, 1, out=out)
    y *= 0.5
    y[7] = 0.0
    assert torch.equal(out, y)


# ------------------------------------------------------------- adapters per row

def _adapters(M, E, K, N, r, seed, dt):
    g = np.random.default_rng(seed)
    x = to_bf16_values(g.standard_normal((M, K)).astype(np.float32))
    a = to_bf16_values((g.standard_normal((E, r, K)) / np.sqrt(K)).astype(np.float32))
    b = to_bf16_values((g.standard_normal((E, N, r)) * 0.3).astype(np.float32))
    s = (0.25 + g.random(E)).astype(np.float32)
    y = _vals(g.standard_normal((M, N)).astype(np.float32), dt)
    ids = g.integers(-1, E, size=M).astype(np.int32)
    return x, a, b, s, y, ids


LORAS = [(1, 1, 16, 1, 16), (1, 4, 1152, 130, 16), (48, 64, 1024, 300, 16), (5, 2, 48, 64, 32), (40, 3, 2048, 520, 64),
         (130, 2, 1040, 100, 48), (257, 4, 512, 264, 128), (33, 5, 272, 72, 256), (600, 3, 400, 77, 64),
         (150, 2, 4096, 65, 240), (900, 20, 256, 640, 16)]


@pytest.mark.parametrize("M,E,K,N,r", LORAS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_lora_add_grouped(cuda, M, E, K, N, r, dt):
    x, a, b, s, y, ids = _adapters(M, E, K, N, r, M + K + N, dt)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    ops = [to_dev(t, torch.bfloat16) for t in (x, a, b)]
    sd, yd = to_dev(s, torch.float32), to_dev(y, TDT[dt])
    want, bound = R.lora(x, a, b, s, y, ids, dt)
    out = cr.lora_add_grouped(*ops, sd, yd, plan, out=torch.full_like(yd, 7.0))
    _close(to_np(out), want, bound)
    assert torch.equal(yd, to_dev(y, TDT[dt]))
    # in place: the same bits, rows without an adapter as they were
    assert cr.lora_add_grouped(*ops, sd, yd, plan) is yd
    assert torch.equal(yd, out)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M", [5, 200])
def test_lora_rows_without_an_adapter_keep_their_bits(cuda, M, dt):
    """Copied out of place bit for bit, signed zeros, infinities and NaN
    payloads included; and a bad value in one row, or in an adapter nobody of
    that row uses, stays in its rows."""
    E, K, N, r = 3, 64, 40, 16
    x, a, b, s, y, ids = _adapters(M, E, K, N, r, 8, dt)
    ids[: M // 2] = np.where(np.arange(M // 2) % 2 == 0, -1, E)
    ids[M // 2:] = np.arange(M - M // 2) % 2  # adapter 2 is not used
    y[:, ::7], y[:, 1::7], y[:, 2::7] = -0.0, np.inf, np.nan
    a[2], b[2] = np.nan, np.inf
    x[0] = np.nan                # a row without an adapter
    x[M - 1] = np.inf            # one with
    t = lambda v, d: torch.from_numpy(np.ascontiguousarray(v)).to(d).to(cuda)
    yd = t(y, TDT[dt])
    out = cr.lora_add_grouped(t(x, torch.bfloat16), t(a, torch.bfloat16), t(b, torch.bfloat16), t(s, torch.float32), yd,
                              cr.group_rows(t(ids, torch.int32), E), out=torch.full_like(yd, 7.0))
    bits = torch.int16 if dt == "bf16" else torch.int32
    assert torch.equal(out[: M // 2].view(bits), yd[: M // 2].view(bits))
    rest = to_np(out[M // 2:M - 1])[:, 3::7]
    assert np.isfinite(rest).all()
    keep = slice(M // 2, M - 1)
    want, bound = R.lora(x[keep], a[:2], b[:2], s[:2], y[keep], ids[keep], dt)
    _close(rest, want[:, 3::7], bound[:, 3::7])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,E", [(3, 2), (150, 2)])
def test_lora_infinite_products_stay_infinities(cuda, M, E, dt):
    """An infinite T (its terms would otherwise be inf and inf - inf)."""
    K, N, r = 96, 70, 32
    x, a, b, s, y, ids = _adapters(M, E, K, N, r, 21, dt)
    ids[:] = np.arange(M) % E
    a[:, :, 5], b = (to_bf16_values(np.abs(v) + np.float32(0.125)) for v in (a[:, :, 5], b))
    x[::2, 5] = np.inf
    x[1, 5] = -np.inf
    out = cr.lora_add_grouped(*(to_dev(t, torch.bfloat16) for t in (x, a, b)), to_dev(s, torch.float32),
                              to_dev(y, TDT[dt]), cr.group_rows(to_dev(ids, torch.int32), E))
    got = to_np(out)
    assert np.all(got[::2] == np.inf) and np.all(got[1] == -np.inf)
    rest = np.arange(3, M, 2)
    want, bound = R.lora(x[rest], a, b, s, y[rest], ids[rest], dt)
    _close(got[rest], want, bound)


def test_lora_add_grouped_strided(cuda):
    """Operands inside wider buffers and an output off 16 bytes."""
    M, E, K, N, r = 70, 3, 256, 50, 16
    x, a, b, s, y, ids = _adapters(M, E, K, N, r, 5, "bf16")
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    xb = torch.zeros((M, K + 8), dtype=torch.bfloat16, device=cuda)
    ab = torch.zeros((E, r + 2, K + 16), dtype=torch.bfloat16, device=cuda)
    bb = torch.zeros((E, N + 1, r + 8), dtype=torch.bfloat16, device=cuda)
    yb = torch.full((M, N + 7), -3.0, dtype=torch.bfloat16, device=cuda)
    xb[:, :K], ab[:, :r, :K], bb[:, :N, :r] = (to_dev(t, torch.bfloat16) for t in (x, a, b))
    yb[:, 3:3 + N] = to_dev(y, torch.bfloat16)
    cr.lora_add_grouped(xb[:, :K], ab[:, :r, :K], bb[:, :N, :r], to_dev(s, torch.float32), yb[:, 3:3 + N], plan)
    want, bound = R.lora(x, a, b, s, y, ids, "bf16")
    got = to_np(yb)
    _close(got[:, 3:3 + N], want, bound)
    assert np.all(got[:, :3] == -3.0) and np.all(got[:, 3 + N:] == -3.0)
    # Y and out as column slices of one buffer
    both = torch.zeros((M, 2 * N), dtype=torch.bfloat16, device=cuda)
    both[:, :N] = to_dev(y, torch.bfloat16)
    cr.lora_add_grouped(xb[:, :K], ab[:, :r, :K], bb[:, :N, :r], to_dev(s, torch.float32), both[:, :N], plan,
                        out=both[:, N:])
    assert torch.equal(both[:, N:], yb[:, 3:3 + N]) and torch.equal(both[:, :N], to_dev(y, torch.bfloat16))


def test_layer_with_an_adapter_bank(cuda):
    """A shared int8 projection with the rows' own adapters beside it."""
    M, E, K, N, r, G = 37, 4, 512, 260, 32, 64
    x, a, b, s, _, ids = _adapters(M, E, K, N, r, 6, "bf16")
    g = np.random.default_rng(7)
    layer = cr.ConvRotLinear.from_dense(to_dev(to_bf16_values((0.02 * g.standard_normal((N, K))).astype(np.float32)),
                                               torch.bfloat16), group=G)
    layer.set_lora_bank(to_dev(a, torch.bfloat16), to_dev(b, torch.bfloat16), to_dev(s, torch.float32))
    xd = to_dev(x, torch.bfloat16)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    base = layer(xd, out_dtype=torch.float32)
    got = layer(xd, out_dtype=torch.float32, groups=plan)
    want, bound = R.lora(x, a, b, s, to_np(base), ids, "f32")
    _close(to_np(got), want, bound)


# ------------------------------------------------------------------ together

def _experts(cuda, E, K, I, N, k, **rule):
    g = np.random.default_rng(11)
    def t(*s, sd):
        return to_dev(to_bf16_values((sd * g.standard_normal(s)).astype(np.float32)), torch.bfloat16)
    return cr.ConvRotExperts.from_dense(t(E, K, sd=K ** -0.5), t(E, I, K, sd=0.05), t(E, I, K, sd=0.05),
                                        t(E, N, I, sd=0.05), k, group=64, **rule)


@pytest.mark.parametrize("M", [1, 3, 70, 515])
def test_experts_layer(cuda, M):
    """Router, plan, grouped products, pack and weighted sum against the same
    layer stated in 64 bits from the library's own choices and codes: every
    step's result is the next step's given input, so each bound is its own."""
    E, K, I, N, k, G = 8, 256, 192, 136, 2, 64
    layer = _experts(cuda, E, K, I, N, k, score="sigmoid", bias=0.1 * torch.randn(E, device=cuda), scale=1.5)
    x = to_dev(to_bf16_values(np.random.default_rng(M).standard_normal((M, K)).astype(np.float32)), torch.bfloat16)
    logits = cr.linear_bf16(x, layer.router, out_dtype=torch.float32)
    ids, w = cr.route(logits, **layer.rule)
    plan = cr.group_rows(ids, E)
    px = cr.pack_act(x, G)
    h = cr.linear_gated_grouped(px, layer.gate, layer.up, plan)
    n = lambda t: to_np(t)
    want, bound, written = R.grouped(n(px.q), n(px.scale), n(ids), E, n(layer.gate.q), n(layer.gate.scale), None, "silu",
                                     "by_row", "sorted", n(layer.up.q), n(layer.up.scale), None, "bf16")
    assert written.all()
    _close(n(h), want, bound)
    ph = cr.pack_act(h, G)
    y = cr.linear_grouped(ph, layer.down, plan, source=cr.SORTED)
    want, bound, _ = R.grouped(n(ph.q), n(ph.scale), n(ids), E, n(layer.down.q), n(layer.down.scale), source="sorted",
                               dtype="bf16")
    _close(n(y), want, bound)
    out = layer(x)
    want, bound = R.combine(n(y), n(w), n(ids), E, "bf16")
    _close(n(out), want, bound)
    assert torch.equal(layer(x.reshape(1, M, K)).reshape(M, N), out)


def test_layers_take_no_rows(cuda):
    E, K = 4, 256
    layer = _experts(cuda, E, K, 192, 136, 2)
    assert layer(torch.empty((0, K), dtype=torch.bfloat16, device=cuda)).shape == (0, 136)
    proj = cr.ConvRotLinear.from_dense(torch.ones((8, K), device=cuda), group=64)
    proj.set_lora_bank(torch.ones((E, 16, K), device=cuda), torch.ones((E, 8, 16), device=cuda),
                       torch.ones(E, device=cuda))
    plan = cr.group_rows(torch.empty(0, dtype=torch.int32, device=cuda), E)
    assert proj(torch.empty((0, K), dtype=torch.bfloat16, device=cuda), groups=plan).shape == (0, 8)
    assert torch.equal(plan.offsets, torch.zeros_like(plan.offsets))


def test_experts_and_adapters_replay_in_a_graph(cuda):
    """One captured graph of a whole step (experts, then a projection with
    adapters per row), replayed with new inputs and new ids in place and
    checked against the eager step every time."""
    M, E, K, I, k, r = 24, 8, 256, 192, 2, 16
    layer = _experts(cuda, E, K, I, K, k)
    g = np.random.default_rng(3)
    proj = cr.ConvRotLinear.from_dense(to_dev(to_bf16_values((0.05 * g.standard_normal((136, K))).astype(np.float32)),
                                              torch.bfloat16), group=64)
    _, a, b, s, _, _ = _adapters(1, E, K, 136, r, 4, "bf16")
    proj.set_lora_bank(to_dev(a, torch.bfloat16), to_dev(b, torch.bfloat16), to_dev(s, torch.float32))
    x = torch.randn(M, K, device=cuda, dtype=torch.bfloat16)
    adapter = torch.zeros(M, dtype=torch.int32, device=cuda)

    def step():
        return proj(layer(x), groups=cr.group_rows(adapter, E))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i in range(4):
        x.copy_(torch.randn(M, K, device=cuda, dtype=torch.bfloat16))
        adapter.copy_(torch.from_numpy(np.random.default_rng(i).integers(-1, E, M).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step()), i


def test_two_streams_at_once(cuda):
    """Calls with their own plans and outputs on two streams do not disturb
    each other."""
    E, K, I, N, k = 8, 256, 192, 136, 2
    layer = _experts(cuda, E, K, I, N, k)
    xs = [torch.randn(M, K, device=cuda, dtype=torch.bfloat16) for M in (300, 5)]
    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(layer(x))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
