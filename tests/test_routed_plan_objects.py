"""Plans as Python objects, and calls of the binding for rows that choose
their weights that end before a launch."""

import copy
import pickle

import pytest
import torch

import w8a8_int8_linear_amd as cr
from w8a8_int8_linear_amd import _lib


def _plan(pairs=32, groups=4, per_row=2):
    n = cr.row_groups_tiles(pairs, groups)
    return cr.RowGroups(torch.arange(pairs, dtype=torch.int32), torch.zeros(groups + 1, dtype=torch.int32),
                        torch.zeros(n, dtype=torch.int32), groups, per_row)


def test_a_used_plan_can_be_copied():
    """A plan that has served a call holds the descriptor of its buffers; a
    copy has buffers of its own and takes none of it along."""
    p = _plan()
    object.__setattr__(p, "_checked", _lib.RowGroups(1 << 20, 2 << 20, 3 << 20, 32, 4, 2))  # as after a call
    for q in (copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert torch.equal(q.order, p.order) and q.order.data_ptr() != p.order.data_ptr()
        assert (q.pairs, q.groups, q.per_row) == (32, 4, 2)
        assert "_checked" not in q.__dict__
    assert "_checked" not in copy.copy(p).__dict__
    assert p.descriptor().pairs == 32


@pytest.mark.gpu
def test_a_copied_plan_is_independent(cuda):
    ids = torch.tensor([[0, 2], [1, 2], [2, 0]], dtype=torch.int32, device=cuda)
    p = cr.group_rows(ids, 3)
    q = copy.deepcopy(p)
    want = q.order.clone()
    cr.group_rows(ids.flip(0).contiguous(), 3, out=p)
    assert torch.equal(q.order, want) and not torch.equal(p.order, want)
    cr.group_rows(ids.flip(0).contiguous(), 3, out=q)
    assert torch.equal(q.order, p.order) and torch.equal(q.offsets, p.offsets)


def _packed(rows, K=256):
    return cr.Packed(torch.zeros((rows, K), dtype=torch.int8), torch.ones(rows), 256)


def _packed_w4(rows, K=256):
    return cr.PackedW4(torch.zeros((rows, K // 2), dtype=torch.uint8), torch.ones(rows), K, 256)


@pytest.mark.parametrize("wrong", [_packed_w4(256), torch.zeros(256, 256, dtype=torch.int8)])
def test_grouped_linears_take_int8_rows_only(wrong):
    """A packed int4 weight or bare codes are refused by name, whichever
    operand they are given as."""
    x, w = _packed(16), _packed(256)
    for call in (lambda: cr.linear_grouped(x, wrong, _plan()), lambda: cr.linear_grouped(wrong, w, _plan()),
                 lambda: cr.linear_gated_grouped(x, wrong, w, _plan()),
                 lambda: cr.linear_gated_grouped(x, w, wrong, _plan())):
        with pytest.raises(ValueError, match="must be int8 rows"):
            call()
    with pytest.raises(ValueError, match="must be int8 rows"):
        cr.ConvRotExperts(torch.zeros(4, 256), wrong, w, w, 2)


A, B, C, D = 0x1000000, 0x2000000, 0x3000000, 0x4000000


@pytest.mark.parametrize("ids,order,offsets,tiles", [
    (A, A, B, C), (A + 4 * 19999, A, B, C), (A - 4 * 19999, A, B, C), (B, A, B, C), (B + 4 * 40, A, B, C),
    (C + 4 * 9, A, B, C), (D, A, A + 4 * 7, C), (D, A, B, A), (D, A, C + 8, C)])
def test_group_rows_refuses_buffers_that_overlap(ids, order, offsets, tiles):
    """The ids are read while the plan is written: ids inside one of the
    plan's buffers would change under the workgroups that place them."""
    lib = _lib.load()
    p = _lib.RowGroups(order, offsets, tiles, 20000, 40, 1)
    assert lib.convrot_group_rows(ids, p, None) == _lib.ERR_INVALID_ARG
    assert b"overlap" in lib.convrot_last_error()


def test_group_rows_counts_whole_buffers():
    """The buffers' ends: every byte of the tiles counts, the next does not."""
    lib = _lib.load()
    p = _lib.RowGroups(A, B, C, 20000, 40, 1)
    n = cr.row_groups_tiles(20000, 40)
    assert lib.convrot_group_rows(C + 4 * (n - 1), p, None) == _lib.ERR_INVALID_ARG
    assert b"overlap" in lib.convrot_last_error()
    p = _lib.RowGroups(A, B, A + 4 * 19999, 20000, 40, 1)
    assert lib.convrot_group_rows(D, p, None) == _lib.ERR_INVALID_ARG


@pytest.mark.gpu
def test_group_rows_of_a_plans_own_order(cuda):
    p = cr.group_rows(torch.zeros(50, dtype=torch.int32, device=cuda), 3)
    with pytest.raises(cr.ConvrotError, match="overlap"):
        cr.group_rows(p.order, 3, out=p)
    q = cr.group_rows(p.order, 3)  # into buffers of its own: ids 0, 1, 2 and others
    assert q.offsets.tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("gated,N", [(False, 500000), (True, 250000)])
def test_grouped_launches_of_too_many_threads_are_refused(gated, N):
    """A launch holds fewer than 2^32 threads; the weight-streaming form of
    many narrow groups with very many features would need more."""
    lib = _lib.load()
    E, pairs = 4096, 20480
    p = _lib.RowGroups(A, B, C, pairs, E, 1)
    rot = _lib.Rot(16, _lib.ROT_REGULAR, None)
    act = _lib.Packed(A, B, pairs, 16, 16, rot, _lib.LAYOUT_ROWS)
    w = _lib.Packed(C, D, E * N, 16, 16, rot, _lib.LAYOUT_ROWS)
    if gated:
        st = lib.convrot_linear_gated_grouped(act, w, None, w, None, _lib.ACT_SILU, p, _lib.BY_ROW, _lib.SORTED, D,
                                              _lib.BF16, N, None)
    else:
        st = lib.convrot_linear_grouped(act, w, None, _lib.ACT_NONE, p, _lib.BY_ROW, _lib.SORTED, D, _lib.BF16, N, None)
    assert st == _lib.ERR_INVALID_ARG
    assert b"threads" in lib.convrot_last_error()


@pytest.mark.parametrize("what", ["plain", "gated", "lora"])
def test_widths_next_to_2_31_are_refused(what):
    """Kernels count features in 32 bits, whole blocks past the last one."""
    lib = _lib.load()
    N, wide = (1 << 31) - 1, 1 << 31
    p = _lib.RowGroups(A, B, C, 1, 1, 1)
    rot = _lib.Rot(16, _lib.ROT_REGULAR, None)
    act = _lib.Packed(A, B, 1, 16, 16, rot, _lib.LAYOUT_ROWS)
    w = _lib.Packed(C, D, N, 16, 16, rot, _lib.LAYOUT_ROWS)
    if what == "plain":
        st = lib.convrot_linear_grouped(act, w, None, _lib.ACT_NONE, p, _lib.BY_ROW, _lib.SORTED, D, _lib.BF16, wide, None)
    elif what == "gated":
        st = lib.convrot_linear_gated_grouped(act, w, None, w, None, _lib.ACT_SILU, p, _lib.BY_ROW, _lib.SORTED, D,
                                              _lib.BF16, wide, None)
    else:
        st = lib.convrot_lora_add_grouped(A, 16, 1, 16, B, 16, 256, C, 16, wide * 16, N, 16, D, p, D, wide, _lib.BF16, D,
                                          wide, A, 1 << 20, None)
    assert st == _lib.ERR_INVALID_ARG
    assert b"features" in lib.convrot_last_error()
