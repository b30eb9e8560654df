"""The layer's steps as separate operators, for a routing or experts of the
caller's own: pairs sorted by expert, token rows to the experts' rows and back
with their gradients, and expert products with 4-bit integer weights.

Torch plumbing around the C ABI (include/mok.h): tensors are checked, outputs
allocated unless given, and the kernels enqueued on the tensors' device, on
its current stream.  Inputs that are not contiguous (or not 16-byte aligned)
are copied; an output given by the caller has to be both, and apart from every
input (rows, gates, maps and weights).  Nothing is recorded for autograd: the
gradients are the _backward functions', and permute_rows, unpermute_rows and the
4-bit products refuse rows, gates and scales that require one while gradients
are recorded."""
from __future__ import annotations

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
