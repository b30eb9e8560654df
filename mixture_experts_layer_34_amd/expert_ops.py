"""The layer's steps as separate operators, for a routing or experts of the
caller's own: pairs sorted by expert, token rows to the experts' rows and back
with their gradients, expert products with 4-bit integer weights, low-rank
adapters beside a projection with their gradients, and the whole layer for a
few tokens, with adapters or without.

Torch plumbing around the C ABI (include/mok.h): tensors are checked, outputs
allocated unless given, and the kernels enqueued on the tensors' device, on
its current stream.  Inputs that are not contiguous (or not 16-byte aligned)
are copied; an output given by the caller has to be both, and apart from every
input (rows, gates, maps and weights).  Nothing is recorded for autograd: the
gradients are the _backward functions', and the forward calls refuse rows, gates,
scales, weights and adapters that require one while gradients are recorded."""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import mok

_DTYPES = {torch.float32: mok.MOK_DTYPE_F32, torch.bfloat16: mok.MOK_DTYPE_BF16, torch.float16: mok.MOK_DTYPE_F16}


def _need(ok: bool, fn: str, what: str):
    if not ok:
        raise ValueError(f"{fn}: {what}")


def _on(fn: str, ref: torch.Tensor, *tensors):
    """Every tensor on the first one's GPU."""
    _need(ref.is_cuda, fn, "tensors on a GPU expected")
    i = ref.get_device()
    for t in tensors:
        if t is not None and t.get_device() != i:
            raise ValueError(f"{fn}: tensors on different devices")


def _unrecorded(fn: str, rows, other=None, out=None, third=None):
    """No gradient is lost without a word."""
    if (rows.requires_grad or (other is not None and other.requires_grad) or (out is not None and out.requires_grad) or
            (third is not None and third.requires_grad)) and torch.is_grad_enabled():
        raise RuntimeError(f"{fn} is not recorded for autograd, but a tensor requires a gradient: call it on detached "
                           "tensors or under torch.no_grad()")


def _ready(t):
    """The tensor itself, or a contiguous, 16-byte aligned copy."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _of_shape(fn: str, name: str, t: torch.Tensor, shape) -> torch.Tensor:
    """An array of a pair map with the type and shape it has to have: checked
    at every use, for a tensor can be resized or given other data in place."""
    if t.dtype != torch.int32 or t.shape != shape:
        raise ValueError(f"{fn}: int32 {name} {list(shape)} of the pair map expected")
    return t


def _output(fn: str, out, shape, dtype, device, *inputs):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.shape != shape or out.dtype != dtype or out.device != device:
        raise ValueError(f"{fn}: out must be {dtype} {shape} on {device}")
    _need(out.is_contiguous() and out.data_ptr() % 16 == 0, fn, "out must be contiguous and 16-byte aligned")
    o, end = out.data_ptr(), out.data_ptr() + out.nbytes
    for t in inputs:
        if t is not None:
            i = t.data_ptr()
            if i < end and o < i + t.nbytes and t.nbytes and out.nbytes:
                raise ValueError(f"{fn}: out must not overlap an input")
    return out


def _call(f, ref, *args):
    """f(*args, stream) on ref's device, on that device's current stream (its
    handle alone: building a torch Stream object takes longer than a small
    call's other checks together)."""
    i = ref.get_device()
    stream = torch._C._cuda_getCurrentRawStream(i)
    if i == torch.cuda.current_device():
        f(*args, stream)
    else:
        with torch.cuda.device(i):
            f(*args, stream)


@dataclass(frozen=True, eq=False)
class PairMap:
    """Where the T * k token-expert pairs sit in the expert-sorted rows
    (mok_sort_pairs): int32 counts [E], offsets [E + 1], row_of_pair [T, k]
    (-1: no row) and pair_of_row [T * k] (-1 past the last row)."""
    T: int
    k: int
    E: int
    expert_begin: int
    expert_end: int
    counts: torch.Tensor
    offsets: torch.Tensor
    row_of_pair: torch.Tensor
    pair_of_row: torch.Tensor

    def __post_init__(self):
        for name, shape in zip(("counts", "offsets", "row_of_pair", "pair_of_row"),
                               ((self.E,), (self.E + 1,), (self.T, self.k), (self.T * self.k,))):
            t = _of_shape("PairMap", name, getattr(self, name), shape)
            _need(t.device == self.counts.device, "PairMap", "arrays on one device expected")

    @classmethod
    def _of(cls, *fields):
        """A map whose arrays are known to fit."""
        m = object.__new__(cls)
        m.__dict__.update(zip(cls.__dataclass_fields__, fields))
        return m


def sort_pairs(topk_idx: torch.Tensor, E: int, expert_begin: int = 0, expert_end: int | None = None) -> PairMap:
    """Sorts the pairs of int32 topk_idx [T, k] by expert, stably.  Indices
    outside [expert_begin, expert_end) (-1: dropped) get no row."""
    fn = "sort_pairs"
    _need(topk_idx.dim() == 2 and topk_idx.dtype == torch.int32, fn, "int32 topk_idx [T, k] expected")
    _on(fn, topk_idx)
    T, k = topk_idx.shape
    ee = E if expert_end is None else expert_end
    dev = topk_idx.device
    nws = mok.mok_sort_pairs_workspace_query(T, k, E)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None
    P = T * k
    if P % 4 or E % 4:
        counts, offsets, row, pair = (torch.empty(s, dtype=torch.int32, device=dev) for s in (E, E + 1, P, P))
    else:  # every part on 16 bytes: one buffer (3.4 us of host time, four 5.3)
        counts, row, pair, offsets = torch.empty(2 * (P + E) + 1, dtype=torch.int32, device=dev).split_with_sizes(
            (E, P, P, E + 1))
    row = row.view(T, k)
    m = PairMap._of(T, k, E, expert_begin, ee, counts, offsets, row, pair)
    _call(mok.mok_sort_pairs, topk_idx, _ready(topk_idx), T, k, E, expert_begin, ee, counts, offsets, row, pair, ws)
    return m


def _rows_args(fn: str, pmap: PairMap, gate, tokens, rows):
    """Checks one [T, d] tensor, one [rows, d] tensor (either may be None) and
    the gates against a pair map; returns (d, dtype code)."""
    ref = tokens if tokens is not None else rows
    dt = _DTYPES.get(ref.dtype)
    _need(dt is not None and ref.dim() == 2, fn, "fp32, bf16 or fp16 matrices expected")
    d = ref.shape[1]
    _need(tokens is None or tokens.shape == (pmap.T, d), fn, "token rows [T, d] expected")
    _need(rows is None or (rows.dim() == 2 and rows.dtype == ref.dtype and rows.shape[1] == d),
          fn, "expert rows [rows, d] of the tokens' type expected")
    pairs = pmap.T, pmap.k
    rop = _of_shape(fn, "row_of_pair", pmap.row_of_pair, pairs)
    _need(gate is None or (gate.dtype == torch.float32 and gate.shape == pairs), fn, "fp32 gate [T, k] expected")
    _on(fn, ref, tokens, rows, gate, rop)
    return d, dt


def permute_rows(x: torch.Tensor, pmap: PairMap, gate: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """xp[row(t, j)] = gate[t, j] * x[t]; xp is [T * k, d] (or `out`, of any
    height).  Rows without a pair are left as they are (uninitialised in a new
    tensor)."""
    fn = "permute_rows"
    d, dt = _rows_args(fn, pmap, gate, x, out)
    _unrecorded(fn, x, gate, out)
    rows = pmap.T * pmap.k if out is None else out.shape[0]
    x, gate, rop = _ready(x), _ready(gate), _ready(pmap.row_of_pair)
    out = _output(fn, out, (rows, d), x.dtype, x.device, x, gate, rop)
    _call(mok.mok_permute_rows, x, x, gate, rop, pmap.T, pmap.k, d, dt, rows, out)
    return out


def permute_rows_backward(dxp: torch.Tensor, pmap: PairMap, gate: torch.Tensor | None = None,
                          x: torch.Tensor | None = None):
    """(dx, dgate) of permute_rows; dgate (None without x) needs the forward's x."""
    fn = "permute_rows_backward"
    d, dt = _rows_args(fn, pmap, gate, x, dxp)
    dx = torch.empty((pmap.T, d), dtype=dxp.dtype, device=dxp.device)
    dgate = None if x is None else torch.empty((pmap.T, pmap.k), dtype=torch.float32, device=dxp.device)
    _call(mok.mok_permute_rows_backward, dxp, _ready(dxp), _ready(x), _ready(gate), _ready(pmap.row_of_pair),
          pmap.T, pmap.k, d, dt, dxp.shape[0], dx, dgate)
    return dx, dgate


def unpermute_rows(y: torch.Tensor, pmap: PairMap, gate: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = sum_j gate[t, j] * y[row(t, j)], in fp32, rounded once."""
    fn = "unpermute_rows"
    d, dt = _rows_args(fn, pmap, gate, None, y)
    _unrecorded(fn, y, gate, out)
    y, gate, rop = _ready(y), _ready(gate), _ready(pmap.row_of_pair)
    out = _output(fn, out, (pmap.T, d), y.dtype, y.device, y, gate, rop)
    _call(mok.mok_unpermute_rows, y, y, gate, rop, pmap.T, pmap.k, d, dt, y.shape[0], out)
    return out


def unpermute_rows_backward(dout: torch.Tensor, pmap: PairMap, gate: torch.Tensor | None = None,
                            y: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """(dy, dgate) of unpermute_rows; dgate (None without y) needs the
    forward's y.  dy is as high as y (or `out`, or T * k rows); rows without a
    pair are left as they are."""
    fn = "unpermute_rows_backward"
    d, dt = _rows_args(fn, pmap, gate, dout, y)
    rows = y.shape[0] if y is not None else pmap.T * pmap.k if out is None else out.shape[0]
    dout, y, gate, rop = _ready(dout), _ready(y), _ready(gate), _ready(pmap.row_of_pair)
    dy = _output(fn, out, (rows, d), dout.dtype, dout.device, dout, y, gate, rop)
    dgate = None if y is None else torch.empty((pmap.T, pmap.k), dtype=torch.float32, device=dout.device)
    _call(mok.mok_unpermute_rows_backward, dout, dout, y, gate, rop, pmap.T, pmap.k, d, dt, rows, dy, dgate)
    return dy, dgate


# ------------------------------------------------------------------ 4-bit integer weights
@dataclass(frozen=True, eq=False)
class Int4Weights:
    """Matrices [E, N, K] in 4-bit integers: uint8 codes [E, N, K / 2] (two per
    byte, the lower element in the low nibble), scales [E, N, K / group] in the
    activations' type, and uint8 zeros (0..15) like the scales (None: 8
    everywhere).  They may be held on the CPU (read, pickled, moved by `to`);
    the products take them on x's GPU."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None = None

    def __post_init__(self):
        for name in ("codes", "scales", "zeros"):
            object.__setattr__(self, name, _ready(getattr(self, name)))
        self.view("Int4Weights")

    def view(self, fn: str):
        """(E, N, K, group, the C view): the arrays checked against each other,
        again only after one of them was given other storage or strides."""
        q, s, z = self.codes, self.scales, self.zeros
        now = (q.data_ptr(), s.data_ptr(), q.shape, s.shape, q.is_contiguous() and s.is_contiguous(),
               None if z is None else (z.data_ptr(), z.shape, z.is_contiguous()))
        seen = self.__dict__.get("_seen")
        if seen is not None and seen[0] == now:
            return seen[1]
        _need(q.dim() == 3 and q.dtype == torch.uint8 and s.dim() == 3 and s.shape[:2] == q.shape[:2], fn,
              "uint8 codes [E, N, K / 2] and scales [E, N, K / group] expected")
        _need(s.dtype in (torch.bfloat16, torch.float16), fn, "bf16 or fp16 scales expected")
        E, N, K = q.shape
        K, G = 2 * K, s.shape[2]
        group = K // G if G else 0
        _need(group in (32, 64, 128) and group * G == K, fn, "groups of 32, 64 or 128 expected")
        _need(z is None or (z.dtype == torch.uint8 and z.shape == s.shape), fn, "uint8 zeros like the scales expected")
        _need(s.device == q.device and (z is None or z.device == q.device), fn, "tensors on different devices")
        _need(all(t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0) for t in (q, s, z)), fn,
              "contiguous, 16-byte aligned arrays expected")
        _need(all(t is None or t.data_ptr() or not t.numel() for t in (q, s, z)), fn, "arrays without memory")
        v = (E, N, K, group, mok.int4_weights(q, s, z))
        self.__dict__["_seen"] = (now, v)
        return v

    def to(self, device) -> Int4Weights:
        return Int4Weights(self.codes.to(device), self.scales.to(device),
                           None if self.zeros is None else self.zeros.to(device))

    def __reduce__(self):
        return Int4Weights, (self.codes, self.scales, self.zeros)


def quantize_int4(w: torch.Tensor, group: int = 128, symmetric: bool = True) -> Int4Weights:
    """4-bit weights of bf16 or fp16 w [N, K] or [E, N, K], in groups along K."""
    _need(w.dim() in (2, 3) and w.dtype in (torch.bfloat16, torch.float16),
          "quantize_int4", "bf16 or fp16 w [N, K] or [E, N, K] expected")
    _on("quantize_int4", w)
    w = _ready(w if w.dim() == 3 else w[None])
    E, N, K = w.shape
    _need(group in (32, 64, 128) and K > 0 and K % group == 0, "quantize_int4",
          "K a multiple of a group of 32, 64 or 128")
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((E, N, K // group), dtype=w.dtype, device=w.device)
    zeros = None if symmetric else torch.empty(scales.shape, dtype=torch.uint8, device=w.device)
    _call(mok.mok_quantize_int4, w, w, E * N, K, group, _DTYPES[w.dtype], codes, scales, zeros)
    return Int4Weights(codes, scales, zeros)


def expert_matvec_int4(x: torch.Tensor, w: Int4Weights, pmap: PairMap | None = None, w_up: Int4Weights | None = None,
                       from_tokens: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """W_e x of each row's expert, or silu(W_e x) * (Wup_e x) with w_up.

    With a pair map x holds the expert-sorted rows [T * k, K], or with
    from_tokens the token rows [T, K], and the result the sorted rows
    [T * k, N] (rows without a pair are left as they are).  Without one, w is
    one matrix and every row of x is its own.  A map over part of its experts is
    expected to have that part of its pairs local; where all of them are, sort
    over those experts alone (E their number)."""
    fn = "expert_matvec_int4"
    E_w, N, K, group, wc = w.view(fn)
    _need(x.dim() == 2 and x.dtype == w.scales.dtype and x.shape[1] == K, fn,
          "x [rows, K] of the scales' type expected")
    uc = us = pair = offsets = None
    if w_up is not None:
        up, us = w_up.view(fn), w_up.scales
        uc = up[4]
        _need(up[:4] == (E_w, N, K, group) and us.dtype == w.scales.dtype and
              (w_up.zeros is None) == (w.zeros is None), fn, "w and w_up of one shape, group and kind expected")
    if pmap is None:
        _need(E_w == 1 and not from_tokens, fn, "one matrix expected without a pair map")
        rows, k, E, eb, ee = x.shape[0], 1, 1, 0, 1
    else:
        rows, k, E, eb, ee = pmap.T * pmap.k, pmap.k, pmap.E, pmap.expert_begin, pmap.expert_end
        _need(E_w == ee - eb, fn, "weights of the map's local experts expected")
        _need(x.shape[0] == (pmap.T if from_tokens else rows), fn, "x of T token rows or T * k sorted rows expected")
        offsets = _of_shape(fn, "offsets", pmap.offsets, (E + 1,))
        if from_tokens:
            pair = _of_shape(fn, "pair_of_row", pmap.pair_of_row, (rows,))
    _on(fn, x, w.codes, us, offsets, pair)
    _unrecorded(fn, x, w.scales, out, us)
    x, pair, offsets = _ready(x), _ready(pair), _ready(offsets)
    if out is None:
        out = torch.empty((rows, N), dtype=x.dtype, device=x.device)
    else:
        read = [t for m in (w, w_up) if m for t in (m.codes, m.scales, m.zeros)]
        out = _output(fn, out, (rows, N), x.dtype, x.device, x, pair, offsets, *read)
    cfg = mok.int4_config(rows, x.shape[0], k, E, eb, ee, N, K, group, _DTYPES[x.dtype])
    _call(mok.mok_expert_matvec_int4, x, x, pair, offsets, wc, uc, cfg, out)
    return out


def int4_experts(x: torch.Tensor, pmap: PairMap, gate: torch.Tensor, w1: Int4Weights, w3: Int4Weights,
                 w2: Int4Weights) -> torch.Tensor:
    """The expert block of a decode step on token rows x [T, d]:
    out[t] = sum_j gate[t, j] W2_e (silu(W1_e x_t) * (W3_e x_t)), e the expert
    of pair (t, j); in three launches after sort_pairs."""
    h = expert_matvec_int4(x, w1, pmap, w_up=w3, from_tokens=True)
    y = expert_matvec_int4(h, w2, pmap)
    return unpermute_rows(y, pmap, gate=gate)


# ------------------------------------------------------------------ low-rank adapters
@dataclass(frozen=True, eq=False)
class LoraWeights:
    """Low-rank adapters scale B A of a projection [N, K]: A [G, r, K] and B
    [G, N, r] of one floating type, 1 <= r <= 128, scale fp32 [G] (None: 1), for
    lora_rows; or A [L, E, r, K], B [L, E, N, r] and scale [L], adapter l of
    expert e, for few_token_layer.  They may be held on the CPU and moved by
    `to`; the operators take them on x's GPU.  A, B and scale are the caller's
    own arrays, read at each call, but for one that is not contiguous (or not
    16-byte aligned): it is copied here, and what is written to the original
    afterwards is not seen."""
    A: torch.Tensor
    B: torch.Tensor
    scale: torch.Tensor | None = None

    def __post_init__(self):
        for name in ("A", "B", "scale"):
            object.__setattr__(self, name, _ready(getattr(self, name)))
        self.view("LoraWeights")

    def view(self, fn: str):
        """(groups, N, K, r, the C view): the arrays checked against each other,
        again only after one of them was given other storage or strides."""
        a, b, s = self.A, self.B, self.scale
        now = (a.data_ptr(), b.data_ptr(), a.shape, b.shape, a.dtype, b.dtype, a.is_contiguous() and b.is_contiguous(),
               None if s is None else (s.data_ptr(), s.shape, s.dtype, s.is_contiguous()))
        seen = self.__dict__.get("_seen")
        if seen is not None and seen[0] == now:
            return seen[1]
        n = a.dim()
        _need(n in (3, 4) and b.dim() == n and a.shape[:-2] == b.shape[:-2] and a.shape[-2] == b.shape[-1], fn,
              "A [G, r, K] and B [G, N, r], or A [L, E, r, K] and B [L, E, N, r] expected")
        r = a.shape[-2]
        _need(a.dtype in _DTYPES and b.dtype == a.dtype, fn, "A and B of one type, fp32, bf16 or fp16, expected")
        _need(1 <= r <= 128, fn, "a rank of 1 to 128 expected")
        _need(s is None or (s.dtype == torch.float32 and s.shape == a.shape[:1]), fn,
              "fp32 scale, one for each adapter, expected")
        _need(b.device == a.device and (s is None or s.device == a.device), fn, "tensors on different devices")
        _need(all(t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0) for t in (a, b, s)), fn,
              "contiguous, 16-byte aligned arrays expected")
        _need(all(t is None or t.data_ptr() or not t.numel() for t in (a, b, s)), fn, "arrays without memory")
        v = (tuple(a.shape[:-2]), b.shape[-2], a.shape[-1], r, mok.lora_weights(a, b, s, r))
        self.__dict__["_seen"] = (now, v)
        return v

    def to(self, device) -> LoraWeights:
        return LoraWeights(self.A.to(device), self.B.to(device), None if self.scale is None else self.scale.to(device))

    def __reduce__(self):
        return LoraWeights, (self.A, self.B, self.scale)


@functools.lru_cache(maxsize=256)
def _lora_plan(rows, E, eb, ee, K, N, dt, r):
    """(the C config, bytes of the forward call's workspace, of the backward call's)."""
    cfg = mok.lora_config(rows, E, eb, ee, K, N, dt)
    return (cfg, *mok.mok_lora_workspace_query(cfg, r))


def _lora_args(fn: str, x, dout, amap: PairMap, w: LoraWeights, sorted_rows: bool):
    """Checks rows [rows, K] and [rows, N] (the latter may be None) against a map
    and its adapters; returns (rows, N, K, r, the weights' C view, the plan, the
    map's arrays)."""
    groups, N, K, r, wc = w.view(fn)
    dt = _DTYPES.get(x.dtype)
    rows = amap.T * amap.k
    _need(len(groups) == 1 and groups[0] == amap.expert_end - amap.expert_begin, fn,
          "adapters A [G, r, K] of the map's local groups expected")
    _need(sorted_rows or amap.k == 1, fn, "a map of one group a row (k = 1) expected, or sorted rows")
    _need(dt is not None and w.A.dtype == x.dtype, fn, "rows of the adapters' type expected")
    _need(x.shape == (rows, K) and (dout is None or (dout.shape == (rows, N) and dout.dtype == x.dtype)), fn,
          "x [rows, K] and y or dout [rows, N] of one type, a row for each of the map's, expected")
    offsets = _of_shape(fn, "offsets", amap.offsets, (amap.E + 1,))
    pair = rop = None
    if not sorted_rows:
        pair = _of_shape(fn, "pair_of_row", amap.pair_of_row, (rows,))
        rop = _of_shape(fn, "row_of_pair", amap.row_of_pair, (amap.T, amap.k))
    _on(fn, x, dout, w.A, offsets, pair, rop)
    plan = _lora_plan(rows, amap.E, amap.expert_begin, amap.expert_end, K, N, dt, r)
    return rows, N, K, r, wc, plan, (_ready(pair), _ready(rop), _ready(offsets))


def _added_to(fn: str, base, out, shape, like, *inputs):
    """The base (contiguous) and the output of a sum, which may be one array."""
    if base is not None:
        _need(base.shape == shape and base.dtype == like.dtype, fn, "rows to add to like the output expected")
        _on(fn, like, base)
    same = out is not None and base is not None and out.data_ptr() == base.data_ptr() and out.is_contiguous() and \
        base.is_contiguous()
    base = _ready(base)
    out = _output(fn, out, shape, like.dtype, like.device, *inputs, None if same else base)
    return base, out


def lora_rows(x: torch.Tensor, amap: PairMap, w: LoraWeights, y: torch.Tensor | None = None,
              sorted_rows: bool = False, out: torch.Tensor | None = None, save: bool = False):
    """out_q = y_q + scale_g B_g (A_g x_q), g the group of row q (y None: 0).

    Many requests' adapters beside one projection: amap =
    sort_pairs(adapter[:, None], G), -1 for a row of the base model, and x
    [T, K], y and out [T, N] in the tokens' order; a row of no adapter gets y.
    One adapter on each expert's projection: the pairs' map with sorted_rows, and
    all of them in the experts' sorted rows; rows of no expert are left as they
    are.  `out` may be y itself.  With save the result is (out, u), u = A_g x_q
    in fp32 [rows, r] and sorted rows (rows of no group uninitialised), for
    lora_rows_backward."""
    fn = "lora_rows"
    rows, N, K, r, wc, (cfg, nws, _), (pair, rop, offsets) = _lora_args(fn, x, y, amap, w, sorted_rows)
    _unrecorded(fn, x, y, out, w.scale)
    _unrecorded(fn, w.A, w.B)
    x = _ready(x)
    y, out = _added_to(fn, y, out, (rows, N), x, x, pair, rop, offsets, w.A, w.B, w.scale)
    u = torch.empty((rows, r), dtype=torch.float32, device=x.device) if save else None
    ws = torch.empty(nws, dtype=torch.uint8, device=x.device)
    _call(mok.mok_lora_rows, x, x, y, pair, rop, offsets, wc, cfg, out, u, ws)
    return (out, u) if save else out


def lora_rows_backward(dout: torch.Tensor, x: torch.Tensor, u: torch.Tensor, amap: PairMap, w: LoraWeights,
                       base: torch.Tensor | None = None, sorted_rows: bool = False, out: torch.Tensor | None = None):
    """(dx, dA, dB) of lora_rows on x, whose u it kept: dx = base + the
    adapters' share (base None: 0; `out` takes dx and may be base itself), dA
    [G, r, K] and dB [G, N, r] in fp32, 0 for a group without rows.  y's
    gradient is dout itself."""
    fn = "lora_rows_backward"
    rows, N, K, r, wc, (cfg, _, nws), (pair, rop, offsets) = _lora_args(fn, x, dout, amap, w, sorted_rows)
    _need(u.dtype == torch.float32 and u.shape == (rows, r), fn, "fp32 u [rows, r] of the forward call expected")
    _on(fn, x, u)
    dout, x, u = _ready(dout), _ready(x), _ready(u)
    base, dx = _added_to(fn, base, out, (rows, K), x, dout, x, u, pair, rop, offsets, w.A, w.B, w.scale)
    dA = torch.empty(w.A.shape, dtype=torch.float32, device=x.device)
    dB = torch.empty(w.B.shape, dtype=torch.float32, device=x.device)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=x.device)
    _call(mok.mok_lora_rows_backward, x, dout, x, u, base, pair, rop, offsets, wc, cfg, dx, dA, dB, ws)
    return dx, dA, dB


# ------------------------------------------------------------------ the layer for a few tokens
_GATING = {"softmax": 0, "sigmoid": mok.MOK_FLAG_SIGMOID_GATES}


@functools.lru_cache(maxsize=256)
def _few_plan(T, d, E, k, F, eb, ee, dt, flags, L, ranks):
    """(the C config, bytes of the workspace); ranks: of the adapters of w1, w3
    and w2 (0: none), or None."""
    cfg = mok.few_token_config(T, d, E, k, F, eb, ee, dt, flags, L)
    lora = None
    if ranks is not None:
        lora = (mok.mok_lora_weights * 3)()
        for m, r in enumerate(ranks):
            if r:
                lora[m] = mok.lora_weights(16, 16, None, r)  # read for their sizes alone
    return cfg, mok.mok_few_token_workspace_query(cfg, lora)


def few_token_layer(x: torch.Tensor, logits: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor,
                    k: int, expert_begin: int = 0, gating: str = "softmax", renorm: bool = False,
                    adapter: torch.Tensor | None = None, lora=None, out: torch.Tensor | None = None):
    """The layer for at most 16 tokens (a decode step), in two launches, four
    with adapters: (out, topk_idx, topk_gate) with out[t] = sum_j gate[t, j]
    W2_e (silu(W1_e x_t) * (W3_e x_t)), e = topk_idx[t, j].

    x [T, d], w1 and w3 [E_loc, F, d], w2 [E_loc, d, F] of one type, fp32, bf16 or
    fp16; logits fp32 [T, E]; the experts [expert_begin, expert_begin + E_loc) are
    local and a token without one of them gets 0.  Routing as in the layer
    (MoeShape.gating, renorm).  lora = (l1, l3, l2), LoraWeights [L, E_loc, ...]
    of w1, w3 and w2 or None each, with int32 adapter [T]: token t's matrices are
    W + scale B A of its adapter; an adapter outside [0, L) is none.  A NaN logit
    ranks last; an infinity or NaN in x or in the weights of an expert reaches the
    tokens of that row or expert and no other."""
    fn = "few_token_layer"
    dt = _DTYPES.get(x.dtype)
    _need(x.dim() == 2 and dt is not None and x.shape[0] <= 16, fn, "fp32, bf16 or fp16 x [T, d], T <= 16, expected")
    T, d = x.shape
    _need(w1.dim() == 3 and w1.dtype == x.dtype and w1.shape[2] == d, fn, "w1 [E_loc, F, d] of x's type expected")
    E_loc, F = w1.shape[:2]
    _need(w3.shape == w1.shape and w3.dtype == x.dtype and w2.shape == (E_loc, d, F) and w2.dtype == x.dtype, fn,
          "w3 [E_loc, F, d] and w2 [E_loc, d, F] of x's type expected")
    _need(logits.dim() == 2 and logits.shape[0] == T and logits.dtype == torch.float32, fn,
          "fp32 logits [T, E] expected")
    E = logits.shape[1]
    _need(gating in _GATING, fn, "gating 'softmax' or 'sigmoid' expected")
    _on(fn, x, logits, w1, w3, w2, adapter)
    _unrecorded(fn, x, logits, out, w1)
    _unrecorded(fn, w3, w2)
    L, lc, read, ranks = 0, None, (), None
    _need((lora is None) == (adapter is None), fn, "lora and adapter expected together")
    if lora is not None:
        _need(adapter.dtype == torch.int32 and adapter.shape == (T,), fn, "int32 adapter [T] expected")
        _need(len(lora) == 3, fn, "lora of w1, w3 and w2 expected")
        lc, read, ranks = (mok.mok_lora_weights * 3)(), [], [0, 0, 0]
        for m, (lw, N, K) in enumerate(zip(lora, (F, F, d), (d, d, F))):
            if lw is None:
                continue
            groups, n, kk, ranks[m], c = lw.view(fn)
            _need(len(groups) == 2 and groups[1] == E_loc and (n, kk) == (N, K) and lw.A.dtype == x.dtype and
                  L in (0, groups[0]) and groups[0], fn, "adapters [L, E_loc, ...] of the weights' type and sizes expected")
            _on(fn, x, lw.A)
            _unrecorded(fn, lw.A, lw.B, lw.scale)
            L = groups[0]
            lc[m] = c
            read += [lw.A, lw.B, lw.scale]
        ranks = tuple(ranks)
    x, logits, w1, w3, w2, adapter = (_ready(t) for t in (x, logits, w1, w3, w2, adapter))
    out = _output(fn, out, (T, d), x.dtype, x.device, x, logits, w1, w3, w2, adapter, *read)
    cfg, nws = _few_plan(T, d, E, k, F, expert_begin, expert_begin + E_loc, dt,
                         _GATING[gating] | (mok.MOK_FLAG_RENORM_GATES if renorm else 0), L, ranks)
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    gate = torch.empty((T, k), dtype=torch.float32, device=x.device)
    ws = torch.empty(nws, dtype=torch.uint8, device=x.device)
    _call(mok.mok_few_token_layer, x, x, logits, w1, w3, w2, adapter, lc, cfg, out, idx, gate, ws)
    return out, idx, gate
