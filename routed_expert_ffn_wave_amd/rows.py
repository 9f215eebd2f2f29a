"""Binding of the row calls (include/ft_moe_rows.h): 8-bit rows and their products, token rows in expert
order, and the gradients of the dispatch and of the weighted combine.

The functions carry the C ABI's names.  Unlike the C calls they see the tensors' types, so they also
refuse (FtError, FT_E_INVAL) a tensor of another type, shape, device or layout than the call reads.
Work is enqueued on the current stream of the tensors' device, or on `stream` (a stream of that device);
outputs that are not given come from that stream's memory, and a tensor that other streams use too is the
caller's to order and to keep (Tensor.record_stream), as with any work of torch's.  The calls are not
recorded by autograd: the gradients are calls of their own.  8-bit codes are
torch.float8_e4m3fn tensors (uint8 is taken too)."""
from __future__ import annotations

import ctypes

import torch

from . import FT_E_INVAL, FT_N_SLOTS, FT_OUT_BF16, FtError, _check, lib

FT_ROWS_F32 = 0x20

_P, _i = ctypes.c_void_p, ctypes.c_int
_SIG = {
    "ft_moe_fp8_scale_cols": [_i],
    "ft_moe_quant_fp8": [_P, _i, _i, _P, _P, _i, _P],
    "ft_moe_swiglu_fp8": [_P, _i, _i, _P, _P, _P],
    "ft_moe_dispatch": [_P, _P, _P, _P, _i, _i, _i, _i, _P, _i, _P],
    "ft_moe_dispatch_fp8": [_P, _P, _P, _P, _i, _i, _i, _i, _P, _P, _i, _P],
    "ft_moe_dispatch_grad": [_P, _P, _P, _P, _i, _i, _i, _i, _P, _i, _P],
    "ft_moe_combine_grad": [_P, _P, _P, _P, _P, _P, _i, _i, _i, _i, _P, _P, _P, _i, _P],
    "ft_moe_fp8_matmul": [_P, _P, _i, _P, _P, _i, _i, _P, _i, _P],
    "ft_moe_fp8_grouped_matmul": [_P, _P, _i, _P, _P, _i, _i, _i, _P, _P, _i, _P, _i, _P],
}
for _name, _args in _SIG.items():
    _f = getattr(lib, _name)
    _f.argtypes, _f.restype = _args, _i

EXPORTED_ROWS = tuple(_SIG)

_E4, _U8, _BF, _F32, _I32 = torch.float8_e4m3fn, torch.uint8, torch.bfloat16, torch.float32, torch.int32
_CODES = (_E4, _U8)
_FLOATS = (_BF, _F32)
_INTS = (_I32,)

# Calls of a few microseconds: the stream handle and the current device are asked for without building objects, where
# this torch has the functions for it (a build without GPU support has not).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(text: str):
    raise FtError(FT_E_INVAL, text)


def _first(t, name: str, dims: int, dtypes, stream=None):
    """Checks a call's first tensor, whose sizes the others follow, and its stream; returns the tensor's GPU and sizes."""
    try:
        shape, dev = t.shape, t.get_device()
        fits = len(shape) == dims and t.dtype in dtypes and t.is_contiguous()
    except AttributeError:
        _refuse(f"{name} must be a tensor")
    if dev < 0:
        _refuse(f"{name} must be on a GPU (it is on {t.device})")
    if not fits:
        _refuse(f"{name} must be a contiguous tensor of {dims} dimensions and type "
                f"{' or '.join(str(d) for d in dtypes)} (got {t.dtype}, {list(t.shape)}, strides {t.stride()})")
    if stream is not None and stream.device_index != dev:
        _refuse(f"the stream is of cuda:{stream.device_index}, {name} is on cuda:{dev}")
    return dev, shape


def _take(t, name: str, dtypes, shape, dev: int):
    """Checks one more tensor; returns its address."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        _refuse(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        _refuse(f"{name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    if t.shape != shape:
        _refuse(f"{name} must have shape {list(shape)} (got {list(t.shape)})")
    if t.get_device() != dev:
        _refuse(f"{name} is on {t.device}, not on cuda:{dev}")
    _refuse(f"{name} must be contiguous")


def _run(fn, dev: int, stream, *args):
    """Enqueues on `stream`, or on the current stream of GPU `dev`, with that GPU as the current one."""
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    if _current_device() == dev:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        _check(rc)


def _new(shape, dtype, dev: int, stream=None):
    """A tensor to write on `stream`: from that stream's memory, which no work of another stream still uses."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")


def _pairs(ids, inv, slot_of_expert, E, T, dev: int, n_slots=None):
    """The pair tables: (their addresses, T, E, k, the flags of n_slots); T None: as many tokens as ids has rows."""
    shape = ids.shape if isinstance(ids, torch.Tensor) else ()
    if len(shape) != 2 or (T is not None and shape[0] != T):
        _refuse(f"ids must be a tensor of shape [{'T' if T is None else T}, k]")
    T, k = shape
    pi = _take(ids, "ids", _INTS, shape, dev)
    pv = _take(inv, "inv", _INTS, (T * k,) if isinstance(inv, torch.Tensor) and inv.dim() == 1 else shape, dev)
    ps = None
    if slot_of_expert is not None:
        n = slot_of_expert.shape[0] if isinstance(slot_of_expert, torch.Tensor) and slot_of_expert.dim() == 1 else -1
        ps = _take(slot_of_expert, "slot_of_expert", (_I32,), (n,), dev)
        if E is not None and E != n:
            _refuse(f"E = {E} does not match slot_of_expert ({n} experts)")
        E = n
    elif E is None:
        _refuse("E is needed when slot_of_expert is not given")
    if E < 1:
        _refuse(f"E must be >= 1 (got {E})")
    if n_slots is None:
        return pi, pv, ps, T, E, k, 0
    if ps is None:
        _refuse("n_slots is given without slot_of_expert")
    return pi, pv, ps, T, E, k, FT_N_SLOTS(n_slots)


def _cols(K: int) -> int:
    return (K + 511) // 512 * 4


def ft_moe_fp8_scale_cols(K: int) -> int:
    """Scale columns of an 8-bit row of K values: one per 128, rounded up to a multiple of 4."""
    return lib.ft_moe_fp8_scale_cols(K)


def _rows_out(codes, scales, rows: int, K: int, dev: int, stream):
    if codes is None:
        codes = _new((rows, K), _E4, dev, stream)
    if scales is None:
        scales = _new((rows, _cols(K)), _F32, dev, stream)
    return codes, scales, _take(codes, "codes", _CODES, (rows, K), dev), _take(scales, "scales", (_F32,), (rows, _cols(K)), dev)


def ft_moe_quant_fp8(x, codes=None, scales=None, stream=None):
    """bf16 or fp32 rows [rows][K] -> (codes [rows][K], scales fp32 [rows][S]): per block of 128 the scale is the
    largest magnitude / 448 and the codes are the nearest e4m3 values of x / scale."""
    dev, (rows, K) = _first(x, "x", 2, _FLOATS, stream)
    codes, scales, pc, ps = _rows_out(codes, scales, rows, K, dev, stream)
    _run(lib.ft_moe_quant_fp8, dev, stream, x.data_ptr(), rows, K, pc, ps, FT_ROWS_F32 if x.dtype is _F32 else 0)
    return codes, scales


def ft_moe_swiglu_fp8(gu, codes=None, scales=None, stream=None):
    """bf16 rows [rows][2 I] = [gate | up] -> the 8-bit rows (codes [rows][I], scales) of SiLU(gate) * up."""
    dev, (rows, I2) = _first(gu, "gu", 2, (_BF,), stream)
    if I2 % 2:
        _refuse(f"gu must have gate and up columns (got {I2})")
    codes, scales, pc, ps = _rows_out(codes, scales, rows, I2 // 2, dev, stream)
    _run(lib.ft_moe_swiglu_fp8, dev, stream, gu.data_ptr(), rows, I2 // 2, pc, ps)
    return codes, scales


def ft_moe_dispatch(x, ids, inv, E=None, slot_of_expert=None, x_sorted=None, stream=None, n_slots=None):
    """Token rows [T][d] (bf16 or fp32) to their places in expert order [T*k][d].  n_slots, here and in the calls
    below: slots outside [0, n_slots) count as not resident too, as in ft_moe_fp8_grouped_matmul."""
    dev, (T, d) = _first(x, "x", 2, _FLOATS, stream)
    pi, pv, pt, T, E, k, fl = _pairs(ids, inv, slot_of_expert, E, T, dev, n_slots)
    if x_sorted is None:
        x_sorted = _new((T * k, d), x.dtype, dev, stream)
    out = _take(x_sorted, "x_sorted", (x.dtype,), (T * k, d), dev)
    _run(lib.ft_moe_dispatch, dev, stream, x.data_ptr(), pi, pv, pt, T, E, k, d, out,
         fl | (FT_ROWS_F32 if x.dtype is _F32 else 0))
    return x_sorted


def ft_moe_dispatch_fp8(x, ids, inv, E=None, slot_of_expert=None, codes=None, scales=None, stream=None, n_slots=None):
    """Token rows [T][d] (bf16 or fp32) to 8-bit rows in expert order: (codes [T*k][d], scales [T*k][S])."""
    dev, (T, d) = _first(x, "x", 2, _FLOATS, stream)
    pi, pv, pt, T, E, k, fl = _pairs(ids, inv, slot_of_expert, E, T, dev, n_slots)
    codes, scales, pc, ps = _rows_out(codes, scales, T * k, d, dev, stream)
    _run(lib.ft_moe_dispatch_fp8, dev, stream, x.data_ptr(), pi, pv, pt, T, E, k, d, pc, ps,
         fl | (FT_ROWS_F32 if x.dtype is _F32 else 0))
    return codes, scales


def ft_moe_dispatch_grad(dx_sorted, ids, inv, E=None, slot_of_expert=None, dx=None, stream=None, n_slots=None):
    """Gradient of ft_moe_dispatch: the sum [T][d] of every token's rows of dx_sorted [T*k][d]."""
    dev, (P, d) = _first(dx_sorted, "dx_sorted", 2, _FLOATS, stream)
    pi, pv, pt, T, E, k, fl = _pairs(ids, inv, slot_of_expert, E, None, dev, n_slots)
    if P != T * k:
        _refuse(f"dx_sorted must have {T * k} rows (got {P})")
    if dx is None:
        dx = _new((T, d), dx_sorted.dtype, dev, stream)
    out = _take(dx, "dx", (dx_sorted.dtype,), (T, d), dev)
    _run(lib.ft_moe_dispatch_grad, dev, stream, dx_sorted.data_ptr(), pi, pv, pt, T, E, k, d, out,
         fl | (FT_ROWS_F32 if dx_sorted.dtype is _F32 else 0))
    return dx


def ft_moe_combine_grad(dout, y_sorted, ids, w, inv, E=None, slot_of_expert=None, dy_sorted=None, dw=None, dlogits=None,
                        want_dlogits: bool = True, stream=None, n_slots=None):
    """Gradient of ft_moe_combine for dout [T][d] (fp32 or bf16): (dy_sorted bf16 [T*k][d], dw fp32 [T][k],
    dlogits fp32 [T][E] through the renormalised softmax of the chosen logits, or None)."""
    dev, (T, d) = _first(dout, "dout", 2, _FLOATS, stream)
    pi, pv, pt, T, E, k, fl = _pairs(ids, inv, slot_of_expert, E, T, dev, n_slots)
    py = _take(y_sorted, "y_sorted", (_BF,), (T * k, d), dev)
    pw = _take(w, "w", (_F32,), (T, k), dev)
    if dy_sorted is None:
        dy_sorted = _new((T * k, d), _BF, dev, stream)
    if dw is None:
        dw = _new((T, k), _F32, dev, stream)
    if dlogits is None and want_dlogits:
        dlogits = _new((T, E), _F32, dev, stream)
    pl = None if dlogits is None else _take(dlogits, "dlogits", (_F32,), (T, E), dev)
    _run(lib.ft_moe_combine_grad, dev, stream, dout.data_ptr(), py, pi, pw, pv, pt, T, E, k, d,
         _take(dy_sorted, "dy_sorted", (_BF,), (T * k, d), dev), _take(dw, "dw", (_F32,), (T, k), dev), pl,
         fl | (FT_OUT_BF16 if dout.dtype is _BF else 0))
    return dy_sorted, dw, dlogits


def _product_out(out, out_dtype, shape, dev: int, stream):
    if out is None:
        if out_dtype not in _FLOATS:
            _refuse(f"out_dtype must be torch.bfloat16 or torch.float32 (got {out_dtype})")
        out = _new(shape, out_dtype, dev, stream)
    return out, _take(out, "out", _FLOATS, shape, dev), FT_OUT_BF16 if out.dtype is _BF else 0


def ft_moe_fp8_matmul(a, a_scales, w, w_scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """8-bit rows a [M][K] (scales [M][S]) times w [N][K] transposed (fp32 scales [ceil(N/128)][ceil(K/128)]):
    [M][N] in bf16, or in fp32 with out_dtype=torch.float32 (or an fp32 `out`).  fp32 results add exact products in
    fp32; bf16 results of more than a few rows cut each product at 2^-13 of the largest of its group of 8 before adding,
    which shows where products cancel."""
    dev, (M, K) = _first(a, "a", 2, _CODES, stream)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        _refuse("w must be a tensor of shape [N, K]")
    N = w.shape[0]
    psa = _take(a_scales, "a_scales", (_F32,), (M, _cols(K)), dev)
    pw = _take(w, "w", _CODES, (N, K), dev)
    psw = _take(w_scales, "w_scales", (_F32,), ((N + 127) // 128, (K + 127) // 128), dev)
    out, po, flags = _product_out(out, out_dtype, (M, N), dev, stream)
    _run(lib.ft_moe_fp8_matmul, dev, stream, a.data_ptr(), psa, M, pw, psw, N, K, po, flags)
    return out


def ft_moe_fp8_grouped_matmul(a, a_scales, w, w_scales, offsets, slot_of_expert, out=None, out_dtype=torch.bfloat16,
                              stream=None):
    """8-bit rows a [P][K] in expert order, each expert's rows times its matrix of w [n_slots][N][K] transposed
    (fp32 scales [n_slots][ceil(N/128)][ceil(K/128)]): [P][N] in bf16 or fp32, as in ft_moe_fp8_matmul.  Rows of
    experts without a slot are left as they were (with out=None: unset)."""
    dev, (P, K) = _first(a, "a", 2, _CODES, stream)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        _refuse("w must be a tensor of shape [n_slots, N, K]")
    n_slots, N, _ = w.shape
    psa = _take(a_scales, "a_scales", (_F32,), (P, _cols(K)), dev)
    pw = _take(w, "w", _CODES, (n_slots, N, K), dev)
    psw = _take(w_scales, "w_scales", (_F32,), (n_slots, (N + 127) // 128, (K + 127) // 128), dev)
    E = slot_of_expert.shape[0] if isinstance(slot_of_expert, torch.Tensor) and slot_of_expert.dim() == 1 else 0
    pt = _take(slot_of_expert, "slot_of_expert", (_I32,), (E,), dev)
    pf = _take(offsets, "offsets", (_I32,), (E + 1,), dev)
    out, po, flags = _product_out(out, out_dtype, (P, N), dev, stream)
    _run(lib.ft_moe_fp8_grouped_matmul, dev, stream, a.data_ptr(), psa, P, pw, psw, n_slots, N, K, pf, pt, E, po, flags)
    return out


# ------------------------------------------------------------------------------------- one layer on 8-bit rows

class Fp8MoELayer:
    """One MoE layer whose expert products run on 8-bit rows and the experts' 8-bit matrices as they are stored:
    route, permute, token rows to 8-bit rows in expert order, gate/up product, SwiGLU to 8-bit rows, down product,
    weighted combine.  w13 [n_slots][2I][d] ([gate ; up] rows) and w2 [n_slots][d][I] are e4m3 codes with
    fp32 scales per 128 x 128 block (s13, s2); slot_of_expert int32 [E], -1 for experts that are not resident
    (left to the residual mask; entries outside [0, n_slots) count as -1).  Every buffer is allocated here for a
    fixed (T, k): forward() allocates nothing and can be captured into a graph.  The accuracy is that of one e4m3 term per activation,
    where MoELayer carries two.  One forward() at a time: its results and buffers are the next one's.  forward() runs on
    any stream: the buffers are free of earlier work when the layer is made (that waits for the current stream), and
    their memory is kept for the streams they were used on (Tensor.record_stream) when the layer goes; a graph that
    holds a forward() needs the layer as long as it is replayed."""

    def __init__(self, w13, s13, w2, s2, slot_of_expert, k: int, T: int, out_bf16: bool = False):
        dev, (self.n_slots, I2, self.d) = _first(w13, "w13", 3, _CODES)
        self.I = I2 // 2
        nb = lambda v: (v + 127) // 128  # noqa: E731
        _take(w2, "w2", _CODES, (self.n_slots, self.d, self.I), dev)
        _take(s13, "s13", (_F32,), (self.n_slots, nb(I2), nb(self.d)), dev)
        _take(s2, "s2", (_F32,), (self.n_slots, nb(self.d), nb(self.I)), dev)
        _first(slot_of_expert, "slot_of_expert", 1, (_I32,))
        _take(slot_of_expert, "slot_of_expert", (_I32,), slot_of_expert.shape, dev)
        E = slot_of_expert.shape[0]
        if T < 0 or T * k > 1 << 30 or I2 % 32 or self.d % 16 or self.d * self.I == 0 or not 1 <= self.n_slots < 1 << 23 or E > 1024 or not 1 <= k <= min(E, 32):
            _refuse(f"invalid layer shape T={T}, k={k}, E={E}, d={self.d}, w13 rows={I2}, slots={self.n_slots}")
        self.dev = dev
        self.w13, self.s13, self.w2, self.s2, self.slot_of = w13, s13, w2, s2, slot_of_expert
        self.E, self.k, self.T, self.slots = E, k, T, FT_N_SLOTS(self.n_slots)
        self.flags = self.slots | (FT_OUT_BF16 if out_bf16 else 0)
        new = lambda *shape, dtype: _new(shape, dtype, dev)  # noqa: E731
        P, e4, f32, bf, i32 = T * k, _E4, _F32, _BF, _I32
        self.ids, self.w, self.inv = new(T, k, dtype=i32), new(T, k, dtype=f32), new(max(P, 1), dtype=i32)
        self.counts, self.offsets, self.gather = new(self.E, dtype=i32), new(self.E + 1, dtype=i32), new(max(P, 1), dtype=i32)
        self.perm_ws = new(max(lib.ft_moe_permute_workspace(T, self.E, k), 16), dtype=torch.uint8)
        S = _cols
        self.x8, self.xs = new(P, self.d, dtype=e4), new(P, S(self.d), dtype=f32)
        self.gu = new(P, I2, dtype=bf)
        self.h8, self.hs = new(P, self.I, dtype=e4), new(P, S(self.I), dtype=f32)
        self.y_sorted = new(P, self.d, dtype=bf)
        self.out, self.mask = new(T, self.d, dtype=bf if out_bf16 else f32), new(max(T, 1), dtype=i32)
        self._buffers = (self.ids, self.w, self.inv, self.counts, self.offsets, self.gather, self.perm_ws, self.x8, self.xs, self.gu,
                         self.h8, self.hs, self.y_sorted, self.out, self.mask)
        # The buffers are memory of the stream that is current here, whose work on tensors freed before may still run.
        self._streams = {_raw_stream(dev)}
        with torch.cuda.device(dev):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _use_on(self, stream):
        """Keeps the buffers' memory, once they are freed, until the work on `stream` is done."""
        for b in self._buffers:
            b.record_stream(stream)
        self._streams.add(stream.cuda_stream)

    def forward(self, logits, x, stream=None):
        """logits fp32 [T][E], x bf16 [T][d] -> (out [T][d], residual mask [T])."""
        dev, T, E, k = self.dev, self.T, self.E, self.k
        if stream is not None and stream.device_index != dev:
            _refuse(f"the stream is of cuda:{stream.device_index}, the layer is on cuda:{dev}")
        px = _take(x, "x", (_BF,), (T, self.d), dev)
        pl = _take(logits, "logits", (_F32,), (T, E), dev)
        if T == 0:
            return self.out, self.mask[:0]
        if (_raw_stream(dev) if stream is None else stream.cuda_stream) not in self._streams:
            self._use_on(torch.cuda.current_stream(dev) if stream is None else stream)
        inv, slot = self.inv.view(T, k), self.slot_of
        pi, pw, pv, pt = self.ids.data_ptr(), self.w.data_ptr(), inv.data_ptr(), slot.data_ptr()
        _run(lib.ft_moe_route, dev, stream, pl, T, E, k, pi, pw)
        _run(lib.ft_moe_permute, dev, stream, pi, T, E, k, self.counts.data_ptr(), self.offsets.data_ptr(),
             self.gather.data_ptr(), pv, self.perm_ws.data_ptr(), self.perm_ws.numel())
        _run(lib.ft_moe_dispatch_fp8, dev, stream, px, pi, pv, pt, T, E, k, self.d, self.x8.data_ptr(), self.xs.data_ptr(),
             self.slots)
        ft_moe_fp8_grouped_matmul(self.x8, self.xs, self.w13, self.s13, self.offsets, slot, out=self.gu, stream=stream)
        ft_moe_swiglu_fp8(self.gu, codes=self.h8, scales=self.hs, stream=stream)
        ft_moe_fp8_grouped_matmul(self.h8, self.hs, self.w2, self.s2, self.offsets, slot, out=self.y_sorted, stream=stream)
        _run(lib.ft_moe_combine, dev, stream, self.y_sorted.data_ptr(), None, pi, pw, pv, pt, T, E, k, self.d,
             self.out.data_ptr(), self.mask.data_ptr(), self.flags)
        return self.out, self.mask[:T]
