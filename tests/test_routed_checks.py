"""What the entry points for rows that choose their weights refuse, on the
host (no call here reaches a launch): the C ABI's statuses with fake device
addresses that validation never reads through, and the Python binding's own
checks."""

import ctypes

import numpy as np
import pytest
import torch

import tests.routed_oracle as R
import w8a8_int8_linear_amd as cr
from w8a8_int8_linear_amd import _lib

A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000
MIS16, MIS4 = 0x10008, 0x10002
INVALID, DTYPE, ALIGN, MISMATCH, OK = (_lib.ERR_INVALID_ARG, _lib.ERR_DTYPE, _lib.ERR_ALIGN, _lib.ERR_MISMATCH, _lib.OK)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def plan(pairs=32, groups=4, per_row=2, order=A, offsets=B, tiles=C):
    return _lib.RowGroups(order, offsets, tiles, pairs, groups, per_row)


def packed(rows, K=256, q=A, scale=B, G=256, layout=_lib.LAYOUT_ROWS):
    return _lib.Packed(q, scale, rows, K, K, _lib.Rot(G, _lib.ROT_REGULAR, None), layout)


def test_struct_layouts():
    assert ctypes.sizeof(_lib.Routing) == 24
    assert ctypes.sizeof(_lib.RowGroups) == 40 and _lib.RowGroups.groups.offset == 32


def route(lib, M=0, E=64, k=4, score=0, groups=1, top=1, dt=_lib.F32, ldl=None, logits=A, bias=None, ids=B, w=C, rule=True):
    r = _lib.Routing(score, k, groups, top, 1, 1.0)
    return lib.convrot_route(logits, dt, E if ldl is None else ldl, M, E, bias, ctypes.byref(r) if rule else None, ids, w,
                             None)


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(groups=64, top=4)), (INVALID, dict(E=0)), (INVALID, dict(E=1025)), (DTYPE, dict(dt=_lib.I32)),
    (INVALID, dict(score=2)), (INVALID, dict(score=-1)), (INVALID, dict(groups=0)), (INVALID, dict(groups=65, E=65)),
    (INVALID, dict(groups=5)), (INVALID, dict(groups=4, top=5)), (INVALID, dict(top=0)), (INVALID, dict(k=0)),
    (INVALID, dict(k=65, E=128)), (INVALID, dict(E=3)), (INVALID, dict(groups=16, top=0)), (INVALID, dict(groups=32, k=3)),
    (INVALID, dict(ldl=63)), (INVALID, dict(M=-1)), (INVALID, dict(M=2, logits=None)), (INVALID, dict(M=2, ids=None)),
    (INVALID, dict(M=2, w=None)), (ALIGN, dict(logits=MIS4)), (ALIGN, dict(bias=MIS4)), (ALIGN, dict(ids=MIS4)),
    (INVALID, dict(rule=False))])
def test_route_checks(lib, want, kw):
    assert route(lib, **kw) == want
    assert (lib.convrot_last_error() == b"") == (want == OK)


def test_row_groups_checks(lib):
    n = ctypes.c_int64(-1)
    for pairs, groups in ((-1, 4), ((1 << 22) + 1, 4), (8, 0), (8, 4097)):
        assert lib.convrot_row_groups_tiles(pairs, groups, ctypes.byref(n)) == INVALID
    assert lib.convrot_row_groups_tiles(8, 4, None) == INVALID
    assert lib.convrot_row_groups_tiles(1 << 22, 4096, ctypes.byref(n)) == OK and n.value > 0
    f = lambda p, ids=D: lib.convrot_group_rows(ids, ctypes.byref(p) if p is not None else None, None)
    assert f(None) == INVALID
    assert f(plan(), None) == INVALID and f(plan(), MIS4) == ALIGN
    for kw in (dict(pairs=-2), dict(pairs=(1 << 22) + 2), dict(groups=0), dict(groups=4097), dict(per_row=0),
               dict(per_row=3), dict(order=None), dict(offsets=None), dict(tiles=None)):
        assert f(plan(**kw)) == INVALID, kw
    for kw in (dict(order=MIS4), dict(offsets=MIS4), dict(tiles=MIS4)):
        assert f(plan(**kw)) == ALIGN, kw


def test_row_tiles_fit_their_lists():
    """The lists' sizes hold every split of pairs into groups."""
    g = np.random.default_rng(0)
    for _ in range(300):
        pairs, E = int(g.integers(1, 400)), int(g.integers(1, 40))
        ids = g.integers(-1, E, pairs) if g.random() < 0.5 else np.full(pairs, int(g.integers(0, E)))
        starts = np.append(R.plan(ids, E)[1], pairs)
        for b in range(5):
            bm = 16 << b
            tiles = sum(-(-int(n) // bm) for n in np.diff(starts))
            assert tiles <= pairs // bm + min(E + 1, pairs)


def grouped(lib, gated=False, act=None, w=None, w2=None, p=None, fn=0, source=0, dest=1, Y=D, ydt=_lib.BF16, ldy=64,
            bias=None):
    act = packed(16) if act is None else act
    w = packed(256) if w is None else w
    p = plan() if p is None else p
    if gated:
        w2 = packed(256) if w2 is None else w2
        return lib.convrot_linear_gated_grouped(ctypes.byref(act), ctypes.byref(w), bias, ctypes.byref(w2), None, fn,
                                                ctypes.byref(p), source, dest, Y, ydt, ldy, None)
    return lib.convrot_linear_grouped(ctypes.byref(act), ctypes.byref(w), bias, fn, ctypes.byref(p), source, dest, Y, ydt,
                                      ldy, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(fn=4)), (INVALID, dict(fn=-1)), (INVALID, dict(source=3)), (INVALID, dict(dest=0)),
    (INVALID, dict(dest=3)), (MISMATCH, dict(act=packed(17))), (MISMATCH, dict(source=1)), (MISMATCH, dict(source=2)),
    (MISMATCH, dict(w=packed(258))), (MISMATCH, dict(w=packed(256, K=512))), (MISMATCH, dict(act=packed(16, G=64))),
    (INVALID, dict(w=packed(256, layout=_lib.LAYOUT_TILE16))), (INVALID, dict(act=packed(16, layout=_lib.LAYOUT_TILE16))),
    (DTYPE, dict(ydt=_lib.I32)), (INVALID, dict(Y=None)), (INVALID, dict(ldy=63)), (ALIGN, dict(Y=0x10001)),
    (ALIGN, dict(bias=MIS4)), (ALIGN, dict(act=packed(16, q=MIS16))), (INVALID, dict(p=plan(per_row=5))),
    (INVALID, dict(act=packed(16, q=None)))])
def test_linear_grouped_checks(lib, want, kw):
    assert grouped(lib, **kw) == want
    if kw.get("fn") is None:
        assert grouped(lib, True, fn=3, **kw) == want


def test_gated_grouped_checks(lib):
    assert grouped(lib, True, fn=0) == INVALID
    assert grouped(lib, True, fn=3, w2=packed(512)) == MISMATCH
    assert grouped(lib, True, fn=3, w2=packed(256, K=512)) == MISMATCH
    assert grouped(lib, True, fn=3, w2=packed(256, G=64)) == MISMATCH


def test_too_many_workgroups_are_refused(lib):
    n = 1 << 22
    p = plan(pairs=n, groups=1, per_row=1)
    w = packed((1 << 31) - 1, K=16, G=16)
    assert grouped(lib, act=packed(n, K=16, G=16), w=w, p=p, ldy=1 << 31) == INVALID
    assert b"workgroups" in lib.convrot_last_error()


def test_empty_products_are_no_ops(lib):
    assert grouped(lib, act=packed(0, q=None, scale=None), p=plan(pairs=0, order=None), Y=None) == OK
    assert grouped(lib, w=packed(0, q=None, scale=None)) == OK


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (OK, dict(N=0)), (DTYPE, dict(dt=2)), (INVALID, dict(M=-1)), (INVALID, dict(k=0)),
    (INVALID, dict(M=1 << 21, k=4)), (INVALID, dict(M=1 << 40, k=1 << 40)), (INVALID, dict(N=-1)), (INVALID, dict(E=0)),
    (INVALID, dict(E=4097)), (INVALID, dict(ldy=7)), (INVALID, dict(ldo=7)), (INVALID, dict(Y=None)),
    (INVALID, dict(out=None)), (INVALID, dict(w=None)), (INVALID, dict(ids=None)), (ALIGN, dict(w=MIS4)),
    (ALIGN, dict(ids=MIS4)), (ALIGN, dict(Y=0x10002, dt=0)), (INVALID, dict(M=1 << 22, k=1, N=(1 << 31) - 1, ldy=1 << 31,
                                                                           ldo=1 << 31)),
    (INVALID, dict(out=A)), (INVALID, dict(out=A, k=1)), (INVALID, dict(out=A + 2 * 46)), (INVALID, dict(out=A - 2 * 18)),
    (INVALID, dict(Y=A, out=A - 64, ldo=1 << 62))])
def test_combine_checks(lib, want, kw):
    a = dict(Y=A, dt=_lib.BF16, ldy=8, w=B, ids=C, M=3, k=2, N=8, E=4, out=D, ldo=8)
    a.update(kw)
    assert lib.convrot_combine_rows(a["Y"], a["dt"], a["ldy"], a["w"], a["ids"], a["M"], a["k"], a["N"], a["E"], a["out"],
                                    a["ldo"], None) == want


@pytest.mark.parametrize("want,kw", [
    (OK, dict(M=0)), (OK, dict(N=0)), (INVALID, dict(K=24)), (INVALID, dict(r=8)), (INVALID, dict(r=272)),
    (INVALID, dict(r=0)), (MISMATCH, dict(p=plan(pairs=32, per_row=2))), (MISMATCH, dict(p=plan(pairs=31, per_row=1))),
    (INVALID, dict(N=-1)), (DTYPE, dict(dt=2)), (INVALID, dict(ldx=64)), (INVALID, dict(lda=64)), (INVALID, dict(ldb=8)),
    (ALIGN, dict(X=MIS16)), (ALIGN, dict(A=MIS16)), (ALIGN, dict(B=MIS16)), (INVALID, dict(sa=16 * 256 - 8)),
    (INVALID, dict(sb=40 * 16 - 8)), (ALIGN, dict(sa=16 * 256 + 4)), (INVALID, dict(scales=None)),
    (ALIGN, dict(scales=MIS4)), (INVALID, dict(ws=None)), (INVALID, dict(wn=64)), (ALIGN, dict(ws=0x90008)),
    (INVALID, dict(out=0x500000 + 80)), (INVALID, dict(ldx=(1 << 62) + 256)), (INVALID, dict(lda=(1 << 62) + 256)),
    (INVALID, dict(out=0x4FFFC0, ldo=1 << 62)), (INVALID, dict(out=0x500000, ldo=48)), (INVALID, dict(Y=None))])
def test_lora_add_grouped_checks(lib, want, kw):
    a = dict(X=A, ldx=256, M=32, K=256, A=B, lda=256, sa=16 * 256, B=C, ldb=16, sb=40 * 16, N=40, r=16, scales=D,
             p=None, Y=0x500000, ldy=40, dt=_lib.BF16, out=0x600000, ldo=40, ws=0x700000, wn=1 << 30)
    a.update(kw)
    p = a["p"] or plan(pairs=a["M"], per_row=1)
    assert lib.convrot_lora_add_grouped(
        a["X"], a["ldx"], a["M"], a["K"], a["A"], a["lda"], a["sa"], a["B"], a["ldb"], a["sb"], a["N"], a["r"],
        a["scales"], ctypes.byref(p), a["Y"], a["ldy"], a["dt"], a["out"], a["ldo"], a["ws"], a["wn"], None) == want


def test_lora_grouped_workspace_query(lib):
    n = ctypes.c_int64(-1)
    f = lambda M, K, r, E: lib.convrot_lora_grouped_workspace_bytes(M, K, r, E, ctypes.byref(n))
    assert f(0, 256, 16, 4) == OK and n.value == 0
    assert f(32, 256, 16, 4) == OK and n.value >= 4 * 32 * 16
    for bad in ((-1, 256, 16, 4), (32, 8, 16, 4), (32, 256, 24, 4), (32, 256, 16, 0), (32, 256, 16, 4097),
                ((1 << 22) + 1, 256, 16, 4)):
        assert f(*bad) == INVALID, bad
    assert lib.convrot_lora_grouped_workspace_bytes(1, 16, 16, 1, None) == INVALID


def test_older_entry_points_keep_their_activations(lib):
    """SiLU belongs to the grouped linears; the others refuse it as before."""
    a, w = packed(4), packed(64)
    assert lib.convrot_linear_act(ctypes.byref(a), ctypes.byref(w), None, _lib.ACT_SILU, D, _lib.BF16, 64, None, 0,
                                  None) == INVALID


# ------------------------------------------------------------ the binding

def _p(rows, K=256):
    return cr.Packed(torch.zeros((rows, K), dtype=torch.int8), torch.ones(rows), 256)


def _plan(pairs=32, groups=4, per_row=2):
    n = cr.row_groups_tiles(pairs, groups)
    return cr.RowGroups(torch.zeros(pairs, dtype=torch.int32), torch.zeros(groups + 1, dtype=torch.int32),
                        torch.zeros(n, dtype=torch.int32), groups, per_row)


def test_binding_refuses_host_tensors_and_wrong_types():
    for call in (lambda: cr.route(torch.zeros(2, 8), 2), lambda: cr.group_rows(torch.zeros(4, dtype=torch.int32), 2),
                 lambda: cr.combine_rows(torch.zeros(4, 8), torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.int32), 4),
                 lambda: _plan().descriptor(),
                 lambda: cr.lora_add_grouped(torch.zeros(4, 16, dtype=torch.bfloat16), None, None, None, None, None)):
        with pytest.raises(ValueError, match="device"):
            call()


@pytest.mark.parametrize("kw", [dict(top_k=0), dict(top_k=9), dict(top_k=(1 << 32) + 2), dict(groups=(1 << 32) + 1),
                                dict(groups=0), dict(top_groups=(1 << 32) + 1)])
def test_binding_route_sizes(kw):
    """Sizes a 32-bit field would wrap are refused before it is filled."""
    with pytest.raises(ValueError, match="experts"):
        cr.route(torch.zeros(2, 8), **(dict(top_k=2) | kw))


@pytest.mark.parametrize("kw,match", [
    (dict(source="rows"), "source"), (dict(dest="by_row"), "dest"), (dict(act="relu"), "activation"),
    (dict(source="sorted"), "32 rows"), (dict(out=torch.zeros(32, 63, dtype=torch.bfloat16)), "shape"),
    (dict(out=torch.zeros(16, 64, dtype=torch.bfloat16)), "shape"), (dict(out_dtype=torch.int32), "float32 or bfloat16"),
    (dict(bias=torch.zeros(64)), "length N")])
def test_binding_linear_grouped_checks(kw, match):
    with pytest.raises(ValueError, match=match):
        cr.linear_grouped(_p(16), _p(256), _plan(), **kw)
    if "bias" in kw:
        kw = dict(b_gate=kw["bias"])
    with pytest.raises(ValueError, match=match):
        cr.linear_gated_grouped(_p(16), _p(256), _p(256), _plan(), **kw)


def test_binding_stacked_weight_must_divide():
    with pytest.raises(ValueError, match="multiple"):
        cr.linear_grouped(_p(16), _p(258), _plan())


def test_layer_checks():
    w = torch.zeros(8, 100)
    layer = cr.ConvRotLinear.from_dense(w, group=64)  # routed to bf16: packs nothing
    with pytest.raises(ValueError, match="bank"):
        layer(torch.zeros(2, 100), groups=_plan(2, 4, 1))
    with pytest.raises(ValueError, match="bank shapes"):
        layer.set_lora_bank(torch.zeros(3, 16, 64), torch.zeros(3, 8, 16), torch.zeros(3))
    with pytest.raises(ValueError, match="do not fit"):
        cr.ConvRotExperts(torch.zeros(4, 256), _p(256), _p(256), _p(256, 256), 2)
