"""Python binding of the operators for rows that choose their weights.

Tokens routed to experts and requests with adapters of their own: ``route``
turns router logits into expert ids and weights, ``group_rows`` turns ids
into a plan (``RowGroups``) of the (row, choice) pairs in the order of their
groups, and the products read that plan: ``linear_grouped``,
``linear_gated_grouped`` (stacked packed weights), ``combine_rows`` (the
weighted sum of every row's outputs) and ``lora_add_grouped`` (adapters per
row).  Group sizes stay on the device: no call waits for the GPU, and all may
be captured into a graph.

As in ``api``, shapes, dtypes, strides and devices are checked here and the
arithmetic is the library's.  Calls run on the current stream of the
operands' device, whichever device is current.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from .api import (GELU_ERF, GELU_TANH, Packed, _check_bias, _check_out, _DT, _ld, _need_cuda, _ptr, _stream, _ws)

# The current stream's handle by device index, without building a Stream
# object (a tenth of the time, for calls that take a few microseconds).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

SILU = "silu"
_FN = {None: _lib.ACT_NONE, GELU_ERF: _lib.ACT_GELU_ERF, GELU_TANH: _lib.ACT_GELU_TANH, SILU: _lib.ACT_SILU}

SOFTMAX = "softmax"
SIGMOID = "sigmoid"
_SCORE = {SOFTMAX: _lib.SCORE_SOFTMAX, SIGMOID: _lib.SCORE_SIGMOID}

BY_ROW = "by_row"
BY_PAIR = "by_pair"
SORTED = "sorted"
_ORDER = {BY_ROW: _lib.BY_ROW, BY_PAIR: _lib.BY_PAIR, SORTED: _lib.SORTED}

_FLOATS = (torch.float32, torch.bfloat16)


def _need_device(t: torch.Tensor, device: torch.device, name: str) -> None:
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the operands on {device}")


def _need_float(t: torch.Tensor, name: str) -> None:
    if t.dtype not in _FLOATS:
        raise ValueError(f"{name} must be float32 or bfloat16")


def _dense(t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> None:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")


def _call(device: torch.device, fn, *args) -> None:
    """fn(*args, stream) on the current stream of ``device``, with that device
    current; raises on an error status."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            _lib.check(fn(*args, _stream(device)))
    else:
        _lib.check(fn(*args, _raw_stream(device.index) if _raw_stream is not None else _stream(device)))


# ---------------------------------------------------------------------------
# The router
# ---------------------------------------------------------------------------

def route(logits: torch.Tensor, top_k: int, score: str = SOFTMAX, bias: torch.Tensor | None = None, groups: int = 1,
          top_groups: int = 1, renormalise: bool = True, scale: float = 1.0, ids: torch.Tensor | None = None,
          weights: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(ids int32 [M, top_k], weights float32 [M, top_k]) of router logits
    [M, E] (float32 or bfloat16): the experts with the largest score plus
    bias, among the ``top_groups`` best of ``groups`` groups of consecutive
    experts, and their scores, renormalised and times ``scale``
    (convrot_route has the rule).  Ties go to the lowest index; a logit of
    -inf closes an expert, and where too few are left the id is -1 and the
    weight 0."""
    experts = logits.shape[-1] if logits.dim() else 0
    for n, name in ((top_k, "top_k"), (groups, "groups"), (top_groups, "top_groups")):
        if not 1 <= n <= experts:
            raise ValueError(f"{name} must be 1 to the {experts} experts")
    _need_cuda(logits, "logits")
    _need_float(logits, "logits")
    if score not in _SCORE:
        raise ValueError(f"score must be one of {sorted(_SCORE)}")
    M, E = logits.shape
    dev = logits.device
    if bias is not None:
        _dense(bias, torch.float32, (E,), "bias")
        _need_device(bias, dev, "bias")
    if ids is None:
        ids = torch.empty((M, top_k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((M, top_k), dtype=torch.float32, device=dev)
    _dense(ids, torch.int32, (M, top_k), "ids")
    _dense(weights, torch.float32, (M, top_k), "weights")
    _need_device(ids, dev, "ids")
    _need_device(weights, dev, "weights")
    rule = _lib.Routing(_SCORE[score], int(top_k), int(groups), int(top_groups), int(bool(renormalise)), float(scale))
    lib = _lib.load()
    _call(dev, lib.convrot_route, logits.data_ptr(), _DT[logits.dtype], _ld(logits), M, E, _ptr(bias),
          ctypes.byref(rule), ids.data_ptr(), weights.data_ptr())
    return ids, weights


# ---------------------------------------------------------------------------
# The plan
# ---------------------------------------------------------------------------

@dataclass(frozen=True, eq=False)
class RowGroups:
    """The (row, choice) pairs of a batch in the order of their groups
    (convrot_row_groups).  Pair p belongs to row p // per_row; group g's
    pairs are ``order[offsets[g]:offsets[g + 1]]``, ascending, and pairs
    without a group come last.  The buffers are fixed (``group_rows`` with
    ``out`` rewrites their contents), so they are checked once."""
    order: torch.Tensor     # [pairs] int32
    offsets: torch.Tensor   # [groups + 1] int32
    tiles: torch.Tensor     # int32, the library's row tiles
    groups: int
    per_row: int

    @property
    def pairs(self) -> int:
        return self.order.shape[0]

    def descriptor(self) -> _lib.RowGroups:
        desc = self.__dict__.get("_checked")
        if desc is None:
            desc = self._check()
            object.__setattr__(self, "_checked", desc)
        return desc

    def __getstate__(self) -> dict:
        # a copy has buffers of its own: it is checked anew
        return {k: v for k, v in self.__dict__.items() if k != "_checked"}

    def _check(self) -> _lib.RowGroups:
        for t, name in ((self.order, "order"), (self.offsets, "offsets"), (self.tiles, "tiles")):
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 vector")
            if not t.is_cuda or t.device != self.order.device:
                raise ValueError("the row groups must be device tensors on one device")
        if self.offsets.numel() != self.groups + 1 or self.tiles.numel() < row_groups_tiles(self.pairs, self.groups):
            raise ValueError("offsets and tiles do not fit the row groups")
        return _lib.RowGroups(self.order.data_ptr(), self.offsets.data_ptr(), self.tiles.data_ptr(), self.pairs,
                              self.groups, self.per_row)


def row_groups_tiles(pairs: int, groups: int) -> int:
    """int32 values of ``RowGroups.tiles`` (convrot_row_groups_tiles)."""
    lib = _lib.load()
    out = ctypes.c_int64(0)
    _lib.check(lib.convrot_row_groups_tiles(pairs, groups, ctypes.byref(out)))
    return out.value


def group_rows(ids: torch.Tensor, groups: int, out: RowGroups | None = None) -> RowGroups:
    """The plan of int32 ids [M] or [M, k] over ``groups`` weights
    (convrot_group_rows); ids outside 0..groups-1 are pairs without a group.
    ``out`` takes a plan of the same sizes to write again (a captured
    graph's, for instance)."""
    if not ids.is_cuda:
        raise ValueError("ids must be a device tensor")
    if ids.dtype != torch.int32 or ids.dim() not in (1, 2) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 tensor of shape [M] or [M, k]")
    per_row = ids.shape[1] if ids.dim() == 2 else 1
    if per_row < 1:
        raise ValueError("ids must hold at least one choice per row")
    pairs, dev = ids.numel(), ids.device
    if out is None:
        sizes = [pairs, groups + 1, row_groups_tiles(pairs, groups)]
        buf = torch.empty((sum(sizes),), dtype=torch.int32, device=dev)
        out = RowGroups(*buf.split(sizes), groups, per_row)
        at = buf.data_ptr()  # (what _check would find)
        object.__setattr__(out, "_checked", _lib.RowGroups(at, at + 4 * sizes[0], at + 4 * (sizes[0] + sizes[1]), pairs,
                                                           groups, per_row))
    elif (out.pairs, out.groups, out.per_row) != (pairs, groups, per_row):
        raise ValueError("out is a plan of other sizes")
    _need_device(out.order, dev, "out")
    desc = out.descriptor()
    lib = _lib.load()
    _call(dev, lib.convrot_group_rows, ids.data_ptr(), ctypes.byref(desc))
    return out


# ---------------------------------------------------------------------------
# The experts' products
# ---------------------------------------------------------------------------

def need_packed(t, name: str) -> None:
    """``t`` must be a packed int8 operand (there are no grouped linears over
    int4 weights)."""
    if not isinstance(t, Packed):
        raise ValueError(f"{name} must be int8 rows (Packed), got {type(t).__name__}")


def _grouped(act: Packed, w: Packed, groups: RowGroups, bias, source: str, dest: str, out, out_dtype, name="bias"):
    need_packed(act, "the activation")
    need_packed(w, "the weight")
    if source not in _ORDER:
        raise ValueError(f"source must be one of {sorted(_ORDER)}")
    if dest not in (BY_PAIR, SORTED):
        raise ValueError(f"dest must be {BY_PAIR!r} or {SORTED!r}")
    if w.rows % groups.groups:
        raise ValueError(f"the stacked weight's {w.rows} rows are no multiple of the {groups.groups} groups")
    rows = groups.pairs // groups.per_row if source == BY_ROW else groups.pairs
    if act.rows != rows:
        raise ValueError(f"the activation must have {rows} rows, got {act.rows}")
    dev = act.q.device
    _need_device(w.q, dev, "the weight")
    _need_device(groups.order, dev, "the row groups")
    N = w.rows // groups.groups
    if out is None:
        if out_dtype not in _FLOATS:
            raise ValueError("output must be float32 or bfloat16")
        out = torch.empty((groups.pairs, N), dtype=out_dtype, device=dev)
    _check_out(out, groups.pairs, N, _FLOATS, dev)
    _check_bias(bias, w.rows, dev, name)
    return out


def linear_grouped(act_in: Packed, w: Packed, groups: RowGroups, bias: torch.Tensor | None = None,
                   act: str | None = None, source: str = BY_ROW, dest: str = BY_PAIR,
                   out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [pairs, N] = act(A s_x s_w + b) of rows that meet the weight of their
    group (convrot_linear_grouped).  ``w`` holds the packed weights stacked
    over the groups, [groups * N, K] (``pack_weight`` of the stacked rows),
    ``bias`` likewise.  ``source`` says which row of ``act_in`` a pair
    reads: BY_ROW (its row's), BY_PAIR, or SORTED (the plan's order);
    ``dest`` where its output goes: BY_PAIR or SORTED.  ``act`` is None,
    "gelu_erf", "gelu_tanh" or "silu".  Rows of pairs without a group are left
    as they were (undefined in a new tensor)."""
    if act not in _FN:
        raise ValueError(f"activation must be None or one of {sorted(k for k in _FN if k)}")
    out = _grouped(act_in, w, groups, bias, source, dest, out, out_dtype)
    a, b, g = act_in.descriptor(), w.descriptor(), groups.descriptor()
    dev = act_in.q.device
    lib = _lib.load()
    _call(dev, lib.convrot_linear_grouped, ctypes.byref(a), ctypes.byref(b), _ptr(bias), _FN[act], ctypes.byref(g),
          _ORDER[source], _ORDER[dest], out.data_ptr(), _DT[out.dtype], _ld(out))
    return out


def linear_gated_grouped(act_in: Packed, w_gate: Packed, w_up: Packed, groups: RowGroups,
                         b_gate: torch.Tensor | None = None, b_up: torch.Tensor | None = None, act: str = SILU,
                         source: str = BY_ROW, dest: str = SORTED, out_dtype: torch.dtype = torch.bfloat16,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [pairs, N] = act(gate) * up over stacked weights in one launch
    (convrot_linear_gated_grouped); arguments as ``linear_grouped``."""
    if act is None or act not in _FN:
        raise ValueError(f"activation must be one of {sorted(k for k in _FN if k)}")
    need_packed(w_up, "the up weight")
    out = _grouped(act_in, w_gate, groups, b_gate, source, dest, out, out_dtype, "b_gate")
    _check_bias(b_up, w_up.rows, act_in.q.device, "b_up")
    _need_device(w_up.q, act_in.q.device, "the up weight")
    a, wg, wu, g = act_in.descriptor(), w_gate.descriptor(), w_up.descriptor(), groups.descriptor()
    dev = act_in.q.device
    lib = _lib.load()
    _call(dev, lib.convrot_linear_gated_grouped, ctypes.byref(a), ctypes.byref(wg), _ptr(b_gate), ctypes.byref(wu),
          _ptr(b_up), _FN[act], ctypes.byref(g), _ORDER[source], _ORDER[dest], out.data_ptr(), _DT[out.dtype], _ld(out))
    return out


def combine_rows(y: torch.Tensor, weights: torch.Tensor, ids: torch.Tensor, groups: int,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """out [M, N] = sum_j weights[m, j] y[m k + j] (convrot_combine_rows), in
    y's dtype, from the outputs y [M * k, N] of a product with
    ``dest=BY_PAIR`` and the router's weights and ids [M, k].  Pairs whose id
    is outside 0..groups-1 are skipped."""
    _need_cuda(y, "y")
    _need_float(y, "y")
    if weights.dim() != 2:
        raise ValueError("weights must be [M, k]")
    M, k = weights.shape
    N, dev = y.shape[1], y.device
    if y.shape[0] != M * k:
        raise ValueError(f"y must have {M * k} rows, got {y.shape[0]}")
    _dense(weights, torch.float32, (M, k), "weights")
    _dense(ids, torch.int32, (M, k), "ids")
    _need_device(weights, dev, "weights")
    _need_device(ids, dev, "ids")
    if out is None:
        out = torch.empty((M, N), dtype=y.dtype, device=dev)
    _check_out(out, M, N, (y.dtype,), dev)
    lib = _lib.load()
    _call(dev, lib.convrot_combine_rows, y.data_ptr(), _DT[y.dtype], _ld(y), weights.data_ptr(), ids.data_ptr(), M, k, N,
          int(groups), out.data_ptr(), _ld(out))
    return out


# ---------------------------------------------------------------------------
# Adapters per row
# ---------------------------------------------------------------------------

def lora_grouped_workspace_bytes(M: int, K: int, r: int, groups: int) -> int:
    """Bytes of device workspace ``lora_add_grouped`` needs on the current
    device (convrot_lora_grouped_workspace_bytes)."""
    lib = _lib.load()
    out = ctypes.c_int64(0)
    _lib.check(lib.convrot_lora_grouped_workspace_bytes(M, K, r, groups, ctypes.byref(out)))
    return out.value


def _lora_workspace(device: torch.device, M: int, K: int, r: int, groups: int) -> int:
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return max(lora_grouped_workspace_bytes(M, K, r, groups), 16)
    return max(lora_grouped_workspace_bytes(M, K, r, groups), 16)


def _need_stack(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda or t.dim() != 3 or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a 3-D bfloat16 device tensor")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")


def _stack_strides(t: torch.Tensor) -> tuple[int, int]:
    """(leading dimension, elements between adapters) of a stack."""
    ld = t.stride(1) if t.shape[1] > 1 else t.shape[2]
    return ld, t.stride(0) if t.shape[0] > 1 else t.shape[1] * ld


def lora_add_grouped(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scales: torch.Tensor, y: torch.Tensor,
                     groups: RowGroups, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[m] + scales[g] (x[m] a[g]^T) b[g]^T with g the group of row m, from
    the unrotated bf16 input x [M, K] and stacked adapters a [groups, r, K],
    b [groups, N, r] (convrot_lora_add_grouped); rows without a group keep
    y.  In place (``out`` None) or into ``out``.  ``groups`` is the plan of
    the rows' adapter ids [M]; one plan serves every layer of a batch.
    ``workspace`` holds ``lora_grouped_workspace_bytes`` bytes (allocated here
    when not given)."""
    _need_cuda(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    _need_stack(a, "a")
    _need_stack(b, "b")
    _need_cuda(y, "y")
    _need_float(y, "y")
    M, K = x.shape
    E, r, N = a.shape[0], a.shape[1], b.shape[1]
    if E != groups.groups or a.shape[2] != K or tuple(b.shape) != (E, N, r) or tuple(y.shape) != (M, N):
        raise ValueError("shapes must be x [M, K], a [groups, r, K], b [groups, N, r], y [M, N]")
    if groups.pairs != M or groups.per_row != 1:
        raise ValueError(f"the row groups must hold one pair for each of the {M} rows")
    dev = x.device
    _dense(scales, torch.float32, (E,), "scales")
    for t, name in ((a, "a"), (b, "b"), (scales, "scales"), (y, "y"), (groups.order, "the row groups")):
        _need_device(t, dev, name)
    _check_out(y, M, N, _FLOATS, dev)
    if out is None:
        out = y
    _check_out(out, M, N, (y.dtype,), dev)
    lda, stride_a = _stack_strides(a)
    ldb, stride_b = _stack_strides(b)
    g = groups.descriptor()
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty((_lora_workspace(dev, M, K, r, E),), dtype=torch.uint8, device=dev)
    wp, wn = _ws(workspace, dev)
    _call(dev, lib.convrot_lora_add_grouped, x.data_ptr(), _ld(x), M, K, a.data_ptr(), lda, stride_a, b.data_ptr(), ldb,
          stride_b, N, r, scales.data_ptr(), ctypes.byref(g), y.data_ptr(), _ld(y), _DT[y.dtype], out.data_ptr(),
          _ld(out), wp, wn)
    return out
