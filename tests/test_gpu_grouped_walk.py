"""Grouped linears of more tiles than the card has compute units: every
workgroup of the tiled kernel goes on to a second tile (transfers of the next
tile during one's epilogue, staging areas used again), with groups that leave
some of its waves without a position."""

import numpy as np
import pytest
import torch

import tests.routed_oracle as R
import w8a8_int8_linear_amd as cr
from tests.gpu_util import to_dev, to_np

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
# rows of the three groups, and rows without one: six 256-row tiles of the
# first group and one each of the others, times 65 blocks of 256 features (or
# 129 of 128)
ROWS = (1480, 12, 1)
NONE = 7


def _codes(shape, seed):
    g = np.random.default_rng(seed)
    return np.clip(np.rint(36 * g.standard_normal(shape)), -127, 127).astype(np.int8)


def _scales(n, seed, s):
    return ((0.5 + np.random.default_rng(seed).random(n)) * s / 127).astype(np.float32)


def _packed(q, s):
    return cr.Packed(to_dev(q, torch.int8), to_dev(s, torch.float32), 16)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K,N,offset", [(384, 16640, 0), (272, 16640, 0), (384, 16395, 0), (272, 16395, 0),
                                        (384, 16640, 1)])
def test_plain_linear_of_many_tiles(cuda, K, N, offset, dt):
    """offset: the output starts one element into a wider buffer (no 16-byte
    stores)."""
    E, M = len(ROWS), sum(ROWS) + NONE
    g = np.random.default_rng(K + N)
    ids = g.permutation(np.repeat(np.arange(-1, E), (NONE,) + ROWS)).astype(np.int32)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    x, sx, w, sw = _codes((M, K), 1), _scales(M, 2, 3.0), _codes((E * N, K), 3), _scales(E * N, 4, 0.08)
    b = (0.1 * g.standard_normal(E * N)).astype(np.float32)
    px, pw, bd = _packed(x, sx), _packed(w, sw), to_dev(b, torch.float32)
    for source, dest, act in [("by_row", "by_pair", None), ("sorted", "sorted", "silu")]:
        buf = torch.full((M, N + 2 * offset), -3.0, dtype=TDT[dt], device=cuda)
        out = buf[:, offset:offset + N]
        for _ in range(2):  # (the second call meets the first one's leavings in LDS)
            cr.linear_grouped(px, pw, plan, bd, act=act, source=source, dest=dest, out=out)
        want, bound, written = R.grouped(x, sx, ids, E, w, sw, b, act, source, dest, dtype=dt)
        y = to_np(out)
        bad = np.abs(y[written].astype(np.float64) - want[written]) > bound[written]
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
        assert np.all(y[~written] == -3.0)
        assert torch.all(buf[:, :offset] == -3.0) and torch.all(buf[:, offset + N:] == -3.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K,N", [(512, 16640), (400, 16395)])
def test_many_tiles_carry_the_bits_of_each_weight_alone(cuda, K, N, dt):
    """The plain and the gated form over many tiles against the linear of
    each group's weight alone, bit for bit."""
    E, M = len(ROWS), sum(ROWS)
    ids = np.random.default_rng(K).permutation(np.repeat(np.arange(E), ROWS)).astype(np.int32)
    plan = cr.group_rows(to_dev(ids, torch.int32), E)
    px = _packed(_codes((M, K), 1), _scales(M, 2, 3.0))
    ws = [_packed(_codes((E * N, K), 3 + i), _scales(E * N, 5 + i, 0.08)) for i in range(2)]
    y = cr.linear_grouped(px, ws[0], plan, out_dtype=TDT[dt])
    yg = cr.linear_gated_grouped(px, ws[0], ws[1], plan, act="gelu_erf", dest="by_pair", out_dtype=TDT[dt])
    for e in range(E):
        rows = torch.from_numpy(np.nonzero(ids == e)[0]).to(cuda)
        sub = cr.Packed(px.q[rows].contiguous(), px.scale[rows].contiguous(), 16)
        we = [cr.Packed(w.q[e * N:(e + 1) * N], w.scale[e * N:(e + 1) * N].contiguous(), 16) for w in ws]
        assert torch.equal(y[rows], cr.linear(sub, we[0], out_dtype=TDT[dt]))
        assert torch.equal(yg[rows], cr.linear_gated(sub, we[0], we[1], act="gelu_erf", out_dtype=TDT[dt]))


@pytest.mark.parametrize("M,k,E", [(1, 8, 128), (513, 4, 60), (900, 8, 300), (8000, 1, 2000), (8193, 1, 40),
                                   (5000, 4, 1500), (20000, 8, 256)])
def test_a_plan_has_the_same_bits_again(cuda, M, k, E):
    """The same ids give the same plan: in new buffers, and in a plan that
    held another (of the lists what is in use)."""
    g = np.random.default_rng(M + E)
    ids = to_dev(g.integers(-1, E + 1, size=(M, k)).astype(np.int32), torch.int32)
    other = to_dev(np.full((M, k), E - 1, dtype=np.int32), torch.int32)
    first = cr.group_rows(ids, E)
    used, at = torch.zeros_like(first.tiles, dtype=torch.bool), 10
    used[:10] = True
    for b in range(5):
        used[at:at + 2 * int(first.tiles[5 + b])] = True
        at += 2 * (M * k // (16 << b) + min(E + 1, M * k))
    stale = cr.group_rows(other, E)
    for again in (cr.group_rows(ids, E), cr.group_rows(ids, E, out=stale)):
        assert torch.equal(again.order, first.order) and torch.equal(again.offsets, first.offsets)
        assert torch.equal(again.tiles[used], first.tiles[used])
