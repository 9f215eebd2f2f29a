"""Binding of the row calls (include/ft_moe_rows.h): 8-bit rows and their products, token rows in expert
order, and the gradients of the dispatch and of the weighted combine.

The functions carry the C ABI's names.  Unlike the C calls they see the tensors' types, so they also
refuse (FtError, FT_E_INVAL) a tensor of another type, shape, device or layout than the call reads.
Work is enqueued on the current stream of the tensors' device, or on `stream`.  8-bit codes are
torch.float8_e4m3fn tensors (uint8 is taken too)."""
from __future__ import annotations

import ctypes

import torch

from . import FT_E_INVAL, FT_OUT_BF16, FtError, _check, _ptr, lib

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

_CODES = (torch.float8_e4m3fn, torch.uint8)
_FLOATS = (torch.bfloat16, torch.float32)


def _refuse(text: str):
    raise FtError(FT_E_INVAL, text)


class _Call:
    """The tensors of one call: each checked for type, shape and layout, all on one GPU."""

    def __init__(self, first: torch.Tensor, name: str):
        if not isinstance(first, torch.Tensor):
            _refuse(f"{name} must be a tensor")
        self.device = first.device
        if self.device.type != "cuda":
            _refuse(f"{name} must be on a GPU (it is on {self.device})")

    def take(self, t, name, dtypes, shape, optional=False):
        """Checks one tensor; `shape` holds sizes, None where any will do."""
        if t is None and optional:
            return None
        if not isinstance(t, torch.Tensor):
            _refuse(f"{name} must be a tensor")
        dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
        if t.dtype not in dtypes:
            _refuse(f"{name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
        if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
            want = ", ".join("any" if s is None else str(s) for s in shape)
            _refuse(f"{name} must have shape [{want}] (got {list(t.shape)})")
        if t.device != self.device:
            _refuse(f"{name} is on {t.device}, not on {self.device}")
        if not t.is_contiguous():
            _refuse(f"{name} must be contiguous")
        return t

    def out(self, t, name, dtypes, shape):
        """An output: the caller's tensor, or a new one of the first type."""
        first = dtypes[0] if isinstance(dtypes, tuple) else dtypes
        return torch.empty(shape, dtype=first, device=self.device) if t is None else self.take(t, name, dtypes, shape)

    def run(self, fn, *args, stream=None):
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        with torch.cuda.device(self.device):
            _check(fn(*args, ctypes.c_void_p(s.cuda_stream)))

    def pairs(self, ids, inv, slot_of_expert, E, T=None):
        """The pair tables; returns (T, E, k)."""
        self.take(ids, "ids", torch.int32, (T, None))
        T, k = ids.shape
        if not isinstance(inv, torch.Tensor) or inv.numel() != T * k:
            _refuse(f"inv must hold T*k = {T * k} entries")
        self.take(inv, "inv", torch.int32, (T, k) if inv.dim() == 2 else (T * k,))
        if slot_of_expert is not None:
            self.take(slot_of_expert, "slot_of_expert", torch.int32, (None,))
            if E is not None and E != slot_of_expert.shape[0]:
                _refuse(f"E = {E} does not match slot_of_expert ({slot_of_expert.shape[0]} experts)")
            E = slot_of_expert.shape[0]
        if E is None:
            _refuse("E is needed when slot_of_expert is not given")
        return T, E, k


def _f32(t: torch.Tensor) -> int:
    return FT_ROWS_F32 if t.dtype == torch.float32 else 0


def ft_moe_fp8_scale_cols(K: int) -> int:
    """Scale columns of an 8-bit row of K values: one per 128, rounded up to a multiple of 4."""
    return lib.ft_moe_fp8_scale_cols(K)


def ft_moe_quant_fp8(x, codes=None, scales=None, stream=None):
    """bf16 or fp32 rows [rows][K] -> (codes [rows][K], scales fp32 [rows][S]): per block of 128 the scale is the
    largest magnitude / 448 and the codes are the nearest e4m3 values of x / scale."""
    c = _Call(x, "x")
    c.take(x, "x", _FLOATS, (None, None))
    rows, K = x.shape
    codes = c.out(codes, "codes", _CODES, (rows, K))
    scales = c.out(scales, "scales", torch.float32, (rows, ft_moe_fp8_scale_cols(K)))
    c.run(lib.ft_moe_quant_fp8, _ptr(x), rows, K, _ptr(codes), _ptr(scales), _f32(x), stream=stream)
    return codes, scales


def ft_moe_swiglu_fp8(gu, codes=None, scales=None, stream=None):
    """bf16 rows [rows][2 I] = [gate | up] -> the 8-bit rows (codes [rows][I], scales) of SiLU(gate) * up."""
    c = _Call(gu, "gu")
    c.take(gu, "gu", torch.bfloat16, (None, None))
    rows, I2 = gu.shape
    if I2 % 2:
        _refuse(f"gu must have gate and up columns (got {I2})")
    codes = c.out(codes, "codes", _CODES, (rows, I2 // 2))
    scales = c.out(scales, "scales", torch.float32, (rows, ft_moe_fp8_scale_cols(I2 // 2)))
    c.run(lib.ft_moe_swiglu_fp8, _ptr(gu), rows, I2 // 2, _ptr(codes), _ptr(scales), stream=stream)
    return codes, scales


def ft_moe_dispatch(x, ids, inv, E=None, slot_of_expert=None, x_sorted=None, stream=None):
    """Token rows [T][d] (bf16 or fp32) to their places in expert order [T*k][d]."""
    c = _Call(x, "x")
    c.take(x, "x", _FLOATS, (None, None))
    T, E, k = c.pairs(ids, inv, slot_of_expert, E, x.shape[0])
    x_sorted = c.out(x_sorted, "x_sorted", x.dtype, (T * k, x.shape[1]))
    c.run(lib.ft_moe_dispatch, _ptr(x), _ptr(ids), _ptr(inv), _ptr(slot_of_expert), T, E, k, x.shape[1], _ptr(x_sorted),
          _f32(x), stream=stream)
    return x_sorted


def ft_moe_dispatch_fp8(x, ids, inv, E=None, slot_of_expert=None, codes=None, scales=None, stream=None):
    """Token rows [T][d] (bf16 or fp32) to 8-bit rows in expert order: (codes [T*k][d], scales [T*k][S])."""
    c = _Call(x, "x")
    c.take(x, "x", _FLOATS, (None, None))
    T, E, k = c.pairs(ids, inv, slot_of_expert, E, x.shape[0])
    d = x.shape[1]
    codes = c.out(codes, "codes", _CODES, (T * k, d))
    scales = c.out(scales, "scales", torch.float32, (T * k, ft_moe_fp8_scale_cols(d)))
    c.run(lib.ft_moe_dispatch_fp8, _ptr(x), _ptr(ids), _ptr(inv), _ptr(slot_of_expert), T, E, k, d, _ptr(codes),
          _ptr(scales), _f32(x), stream=stream)
    return codes, scales


def ft_moe_dispatch_grad(dx_sorted, ids, inv, E=None, slot_of_expert=None, dx=None, stream=None):
    """Gradient of ft_moe_dispatch: the sum [T][d] of every token's rows of dx_sorted [T*k][d]."""
    c = _Call(dx_sorted, "dx_sorted")
    T, E, k = c.pairs(ids, inv, slot_of_expert, E)
    c.take(dx_sorted, "dx_sorted", _FLOATS, (T * k, None))
    d = dx_sorted.shape[1]
    dx = c.out(dx, "dx", dx_sorted.dtype, (T, d))
    c.run(lib.ft_moe_dispatch_grad, _ptr(dx_sorted), _ptr(ids), _ptr(inv), _ptr(slot_of_expert), T, E, k, d, _ptr(dx),
          _f32(dx_sorted), stream=stream)
    return dx


def ft_moe_combine_grad(dout, y_sorted, ids, w, inv, E=None, slot_of_expert=None, dy_sorted=None, dw=None, dlogits=None,
                        want_dlogits: bool = True, stream=None):
    """Gradient of ft_moe_combine for dout [T][d] (fp32 or bf16): (dy_sorted bf16 [T*k][d], dw fp32 [T][k],
    dlogits fp32 [T][E] through the renormalised softmax of the chosen logits, or None)."""
    c = _Call(dout, "dout")
    c.take(dout, "dout", _FLOATS, (None, None))
    T, E, k = c.pairs(ids, inv, slot_of_expert, E, dout.shape[0])
    d = dout.shape[1]
    c.take(y_sorted, "y_sorted", torch.bfloat16, (T * k, d))
    c.take(w, "w", torch.float32, (T, k))
    dy_sorted = c.out(dy_sorted, "dy_sorted", torch.bfloat16, (T * k, d))
    dw = c.out(dw, "dw", torch.float32, (T, k))
    dlogits = c.out(dlogits, "dlogits", torch.float32, (T, E)) if want_dlogits or dlogits is not None else None
    c.run(lib.ft_moe_combine_grad, _ptr(dout), _ptr(y_sorted), _ptr(ids), _ptr(w), _ptr(inv), _ptr(slot_of_expert), T, E,
          k, d, _ptr(dy_sorted), _ptr(dw), _ptr(dlogits), FT_OUT_BF16 if dout.dtype == torch.bfloat16 else 0,
          stream=stream)
    return dy_sorted, dw, dlogits


def _matmul_out(c, out, out_dtype, shape):
    if out is None:
        if out_dtype not in _FLOATS:
            _refuse(f"out_dtype must be torch.bfloat16 or torch.float32 (got {out_dtype})")
        return torch.empty(shape, dtype=out_dtype, device=c.device)
    return c.take(out, "out", _FLOATS, shape)


def ft_moe_fp8_matmul(a, a_scales, w, w_scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """8-bit rows a [M][K] (scales [M][S]) times w [N][K] transposed (fp32 scales [ceil(N/128)][ceil(K/128)]):
    [M][N] in bf16, or in fp32 with out_dtype=torch.float32 (or an fp32 `out`)."""
    c = _Call(a, "a")
    c.take(a, "a", _CODES, (None, None))
    M, K = a.shape
    c.take(a_scales, "a_scales", torch.float32, (M, ft_moe_fp8_scale_cols(K)))
    c.take(w, "w", _CODES, (None, K))
    N = w.shape[0]
    c.take(w_scales, "w_scales", torch.float32, ((N + 127) // 128, (K + 127) // 128))
    out = _matmul_out(c, out, out_dtype, (M, N))
    c.run(lib.ft_moe_fp8_matmul, _ptr(a), _ptr(a_scales), M, _ptr(w), _ptr(w_scales), N, K, _ptr(out),
          FT_OUT_BF16 if out.dtype == torch.bfloat16 else 0, stream=stream)
    return out


def ft_moe_fp8_grouped_matmul(a, a_scales, w, w_scales, offsets, slot_of_expert, out=None, out_dtype=torch.bfloat16,
                              stream=None):
    """8-bit rows a [P][K] in expert order, each expert's rows times its matrix of w [n_slots][N][K] transposed
    (fp32 scales [n_slots][ceil(N/128)][ceil(K/128)]): [P][N] in bf16 or fp32.  Rows of experts without a slot
    are left as they were (with out=None: unset)."""
    c = _Call(a, "a")
    c.take(a, "a", _CODES, (None, None))
    P, K = a.shape
    c.take(a_scales, "a_scales", torch.float32, (P, ft_moe_fp8_scale_cols(K)))
    c.take(w, "w", _CODES, (None, None, K))
    n_slots, N = w.shape[:2]
    c.take(w_scales, "w_scales", torch.float32, (n_slots, (N + 127) // 128, (K + 127) // 128))
    c.take(slot_of_expert, "slot_of_expert", torch.int32, (None,))
    E = slot_of_expert.shape[0]
    c.take(offsets, "offsets", torch.int32, (E + 1,))
    out = _matmul_out(c, out, out_dtype, (P, N))
    c.run(lib.ft_moe_fp8_grouped_matmul, _ptr(a), _ptr(a_scales), P, _ptr(w), _ptr(w_scales), n_slots, N, K,
          _ptr(offsets), _ptr(slot_of_expert), E, _ptr(out), FT_OUT_BF16 if out.dtype == torch.bfloat16 else 0,
          stream=stream)
    return out


# ------------------------------------------------------------------------------------- one layer on 8-bit rows

class Fp8MoELayer:
    """One MoE layer whose expert products run on 8-bit rows and the experts' 8-bit matrices as they are stored:
    route, permute, token rows to 8-bit rows in expert order, gate/up product, SwiGLU to 8-bit rows, down product,
    weighted combine.  w13 [n_slots][2I][d] ([gate ; up] rows) and w2 [n_slots][d][I] are e4m3 codes with
    fp32 scales per 128 x 128 block (s13, s2); slot_of_expert int32 [E], -1 for experts that are not resident
    (left to the residual mask).  Every buffer is allocated here for a fixed (T, k): forward() allocates
    nothing and can be captured into a graph.  The accuracy is that of one e4m3 term per activation,
    where MoELayer carries two."""

    def __init__(self, w13, s13, w2, s2, slot_of_expert, k: int, T: int, out_bf16: bool = False):
        c = _Call(w13, "w13")
        c.take(w13, "w13", _CODES, (None, None, None))
        self.n_slots, I2, self.d = w13.shape
        self.I = I2 // 2
        nb = lambda v: (v + 127) // 128  # noqa: E731
        c.take(w2, "w2", _CODES, (self.n_slots, self.d, self.I))
        c.take(s13, "s13", torch.float32, (self.n_slots, nb(I2), nb(self.d)))
        c.take(s2, "s2", torch.float32, (self.n_slots, nb(self.d), nb(self.I)))
        c.take(slot_of_expert, "slot_of_expert", torch.int32, (None,))
        if T < 0 or I2 % 2:
            _refuse(f"invalid layer shape T={T}, w13 rows={I2}")
        self.w13, self.s13, self.w2, self.s2, self.slot_of = w13, s13, w2, s2, slot_of_expert
        self.E, self.k, self.T, self.flags = slot_of_expert.shape[0], k, T, FT_OUT_BF16 if out_bf16 else 0
        new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=c.device)  # noqa: E731
        P, e4, f32, bf, i32 = T * k, torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32
        self.ids, self.w, self.inv = new(T, k, dtype=i32), new(T, k, dtype=f32), new(max(P, 1), dtype=i32)
        self.counts, self.offsets, self.gather = new(self.E, dtype=i32), new(self.E + 1, dtype=i32), new(max(P, 1), dtype=i32)
        self.perm_ws = new(max(lib.ft_moe_permute_workspace(T, self.E, k), 16), dtype=torch.uint8)
        S = ft_moe_fp8_scale_cols
        self.x8, self.xs = new(P, self.d, dtype=e4), new(P, S(self.d), dtype=f32)
        self.gu = new(P, I2, dtype=bf)
        self.h8, self.hs = new(P, self.I, dtype=e4), new(P, S(self.I), dtype=f32)
        self.y_sorted = new(P, self.d, dtype=bf)
        self.out, self.mask = new(T, self.d, dtype=bf if out_bf16 else f32), new(max(T, 1), dtype=i32)

    def forward(self, logits, x, stream=None):
        """logits fp32 [T][E], x bf16 [T][d] -> (out [T][d], residual mask [T])."""
        c = _Call(x, "x")
        c.take(x, "x", torch.bfloat16, (self.T, self.d))
        c.take(logits, "logits", torch.float32, (self.T, self.E))
        if self.T == 0:
            return self.out, self.mask[:0]
        inv = self.inv.view(self.T, self.k)
        c.run(lib.ft_moe_route, _ptr(logits), self.T, self.E, self.k, _ptr(self.ids), _ptr(self.w), stream=stream)
        c.run(lib.ft_moe_permute, _ptr(self.ids), self.T, self.E, self.k, _ptr(self.counts), _ptr(self.offsets),
              _ptr(self.gather), _ptr(inv), _ptr(self.perm_ws), self.perm_ws.numel(), stream=stream)
        ft_moe_dispatch_fp8(x, self.ids, inv, slot_of_expert=self.slot_of, codes=self.x8, scales=self.xs, stream=stream)
        ft_moe_fp8_grouped_matmul(self.x8, self.xs, self.w13, self.s13, self.offsets, self.slot_of, out=self.gu, stream=stream)
        ft_moe_swiglu_fp8(self.gu, codes=self.h8, scales=self.hs, stream=stream)
        ft_moe_fp8_grouped_matmul(self.h8, self.hs, self.w2, self.s2, self.offsets, self.slot_of, out=self.y_sorted,
                                  stream=stream)
        c.run(lib.ft_moe_combine, _ptr(self.y_sorted), None, _ptr(self.ids), _ptr(self.w), _ptr(inv), _ptr(self.slot_of),
              self.T, self.E, self.k, self.d, _ptr(self.out), _ptr(self.mask), self.flags, stream=stream)
        return self.out, self.mask[: self.T]
