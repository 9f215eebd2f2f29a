"""Binding of the product calls (include/ft_moe_products.h): bf16 products of token rows with one matrix per expert and
their gradients, SwiGLU rows with their gradient, and low-rank adapters of many requests beside a shared projection.

As in rows.py the functions carry the C ABI's names, refuse (FtError, FT_E_INVAL) a tensor of another type, shape,
device or layout than the call reads, enqueue on the current stream of the tensors' device or on `stream`, and take
outputs that are not given from that stream's memory.  The calls are not recorded by autograd: the gradients are calls
of their own."""
from __future__ import annotations

import ctypes

import torch

from . import FT_N_SLOTS, FT_OUT_BF16, lib
from .rows import (_BF, _F32, _FLOATS, _I32, _first, _new, _product_out, _raw_stream, _refuse, _run, _take, ft_moe_combine_grad,
                   ft_moe_dispatch, ft_moe_dispatch_grad)

FT_ADD_TO_OUT = 0x40

_P, _i, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIG = {
    "ft_moe_grouped_matmul_wgrad_workspace": [_i, _i, _i],
    "ft_moe_grouped_matmul": [_P, _i, _P, _i, _i, _i, _P, _P, _i, _P, _i, _P],
    "ft_moe_grouped_matmul_grad": [_P, _i, _P, _i, _i, _i, _P, _P, _i, _P, _i, _P],
    "ft_moe_grouped_matmul_wgrad": [_P, _P, _i, _i, _i, _P, _P, _i, _P, _P, _z, _i, _P],
    "ft_moe_swiglu": [_P, _i, _i, _P, _P],
    "ft_moe_swiglu_grad": [_P, _P, _i, _i, _P, _P],
    "ft_moe_lora_workspace": [_i, _i, _i, _i, _i],
    "ft_moe_lora": [_P, _P, _i, _P, _P, _P, _i, _i, _i, _i, _P, _P, _P, _i, _P, _P, _z, _i, _P],
}
for _name, _args in _SIG.items():
    _f = getattr(lib, _name)
    _f.argtypes, _f.restype = _args, _i
lib.ft_moe_lora_workspace.restype = lib.ft_moe_grouped_matmul_wgrad_workspace.restype = _z

EXPORTED_PRODUCTS = tuple(_SIG)


def _groups(offsets, slots, name: str, dev: int):
    """The tables: (their addresses, the number of experts)."""
    n = offsets.shape[0] if isinstance(offsets, torch.Tensor) and offsets.dim() == 1 else 0
    if n < 2:
        _refuse("offsets must be a tensor of shape [E + 1]")
    pf = _take(offsets, "offsets", (_I32,), (n,), dev)
    return pf, None if slots is None else _take(slots, name, (_I32,), (n - 1,), dev), n - 1


def _matrices(w, name: str):
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        _refuse(f"{name} must be a tensor of 3 dimensions")
    return w.shape


def _workspace(ws, need, dev: int, stream, *args):
    """(the workspace tensor, its address, its bytes): `ws`, or where the call needs one, a new one of need(*args) bytes."""
    if ws is None:
        n = need(*args)
        if n == 0:
            return None, None, 0
        ws = _new((n,), torch.uint8, dev, stream)
    elif not isinstance(ws, torch.Tensor) or ws.get_device() != dev or not ws.is_contiguous():
        _refuse(f"ws must be a contiguous tensor on cuda:{dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def ft_moe_grouped_matmul_wgrad_workspace(N: int, K: int, E: int) -> int:
    return lib.ft_moe_grouped_matmul_wgrad_workspace(N, K, E)


def ft_moe_grouped_matmul(a, w, offsets, slot_of_expert=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """bf16 rows a [P][K] in expert order, each expert's rows times its matrix of w [n_slots][N][K] transposed: [P][N]
    in bf16, or in fp32 with out_dtype=torch.float32 (or an fp32 `out`).  Rows of experts without a slot are left as they
    were (with out=None: unset).  slot_of_expert None: expert e has matrix e."""
    dev, (P, K) = _first(a, "a", 2, (_BF,), stream)
    n_slots, N, _ = _matrices(w, "w")
    pw = _take(w, "w", (_BF,), (n_slots, N, K), dev)
    pf, pt, E = _groups(offsets, slot_of_expert, "slot_of_expert", dev)
    out, po, flags = _product_out(out, out_dtype, (P, N), dev, stream)
    _run(lib.ft_moe_grouped_matmul, dev, stream, a.data_ptr(), P, pw, n_slots, N, K, pf, pt, E, po, flags)
    return out


def ft_moe_grouped_matmul_grad(dout, w, offsets, slot_of_expert=None, da=None, out_dtype=torch.bfloat16, stream=None):
    """Gradient of ft_moe_grouped_matmul's rows: dout [P][N] in expert order times the experts' matrices of
    w [n_slots][N][K]: [P][K] in bf16 or fp32."""
    dev, (P, N) = _first(dout, "dout", 2, (_BF,), stream)
    n_slots, _, K = _matrices(w, "w")
    pw = _take(w, "w", (_BF,), (n_slots, N, K), dev)
    pf, pt, E = _groups(offsets, slot_of_expert, "slot_of_expert", dev)
    da, po, flags = _product_out(da, out_dtype, (P, K), dev, stream)
    _run(lib.ft_moe_grouped_matmul_grad, dev, stream, dout.data_ptr(), P, pw, n_slots, N, K, pf, pt, E, po, flags)
    return da


def ft_moe_grouped_matmul_wgrad(dout, a, offsets, slot_of_expert=None, dw=None, out_dtype=torch.float32, add=False, stream=None,
                                n_slots=None, ws=None):
    """Gradient of ft_moe_grouped_matmul's matrices, by expert: dw[e] = dout_e^T a_e [E][N][K] of the rows dout [P][N] and
    a [P][K] of every expert, in fp32 (add: dw += it) or bf16; zeros for an expert without rows.  Experts that
    slot_of_expert gives no slot (in [0, n_slots), where n_slots is given) are left as they were.  `ws`:
    ft_moe_grouped_matmul_wgrad_workspace(N, K, E) bytes (made for the call when not given)."""
    dev, (P, N) = _first(dout, "dout", 2, (_BF,), stream)
    K = a.shape[1] if isinstance(a, torch.Tensor) and a.dim() == 2 else 0
    pa = _take(a, "a", (_BF,), (P, K), dev)
    pf, pt, E = _groups(offsets, slot_of_expert, "slot_of_expert", dev)
    if add and (dw is None or not isinstance(dw, torch.Tensor) or dw.dtype is not _F32):
        _refuse("add needs an fp32 dw")
    if n_slots is not None and pt is None:
        _refuse("n_slots is given without slot_of_expert")
    fl = (0 if n_slots is None else FT_N_SLOTS(n_slots)) | (FT_ADD_TO_OUT if add else 0)
    dw, po, flags = _product_out(dw, out_dtype, (E, N, K), dev, stream)
    ws, pws, nw = _workspace(ws, lib.ft_moe_grouped_matmul_wgrad_workspace, dev, stream, N, K, E)
    _run(lib.ft_moe_grouped_matmul_wgrad, dev, stream, dout.data_ptr(), pa, P, N, K, pf, pt, E, po, pws, nw, flags | fl)
    return dw


def ft_moe_swiglu(gu, h=None, stream=None):
    """bf16 rows [rows][2 I] = [gate | up] -> SiLU(gate) * up, bf16 [rows][I]."""
    dev, (rows, I2) = _first(gu, "gu", 2, (_BF,), stream)
    if I2 % 2:
        _refuse(f"gu must have gate and up columns (got {I2})")
    if h is None:
        h = _new((rows, I2 // 2), _BF, dev, stream)
    _run(lib.ft_moe_swiglu, dev, stream, gu.data_ptr(), rows, I2 // 2, _take(h, "h", (_BF,), (rows, I2 // 2), dev))
    return h


def ft_moe_swiglu_grad(gu, dh, dgu=None, stream=None):
    """Gradient of ft_moe_swiglu for dh [rows][I]: bf16 [rows][2 I] (dgu may be gu itself)."""
    dev, (rows, I2) = _first(gu, "gu", 2, (_BF,), stream)
    if I2 % 2:
        _refuse(f"gu must have gate and up columns (got {I2})")
    pd = _take(dh, "dh", (_BF,), (rows, I2 // 2), dev)
    if dgu is None:
        dgu = _new((rows, I2), _BF, dev, stream)
    _run(lib.ft_moe_swiglu_grad, dev, stream, gu.data_ptr(), pd, rows, I2 // 2, _take(dgu, "dgu", (_BF,), (rows, I2), dev))
    return dgu


def ft_moe_lora_workspace(T: int, E: int, r: int, N: int, K: int) -> int:
    return lib.ft_moe_lora_workspace(T, E, r, N, K)


def ft_moe_lora(base, x, a, b, offsets, gather, slot_of_adapter=None, scale=None, out=None, ws=None, stream=None):
    """base [T][N] (bf16 or fp32) plus every row's adapter: scale (x a^T) b^T with x bf16 [T][K], a bf16 [n_slots][r][K],
    b bf16 [n_slots][N][r] and scale fp32 [n_slots] (None: 1).  offsets [E + 1] and gather [T] list the rows of the E
    adapters (ft_moe_permute of the rows' adapters, k = 1); rows without an adapter stand before or behind them or with
    one that has no slot, and get base.  out may be base itself.  `ws`: ft_moe_lora_workspace(T, E, r, N, K) bytes."""
    dev, (T, N) = _first(base, "base", 2, _FLOATS, stream)
    K = x.shape[1] if isinstance(x, torch.Tensor) and x.dim() == 2 else 0
    px = _take(x, "x", (_BF,), (T, K), dev)
    n_slots, r, _ = _matrices(a, "a")
    pa = _take(a, "a", (_BF,), (n_slots, r, K), dev)
    pb = _take(b, "b", (_BF,), (n_slots, N, r), dev)
    ps = None if scale is None else _take(scale, "scale", (_F32,), (n_slots,), dev)
    pf, pt, E = _groups(offsets, slot_of_adapter, "slot_of_adapter", dev)
    pg = _take(gather, "gather", (_I32,), (T,), dev)
    if out is None:
        out = _new((T, N), base.dtype, dev, stream)
    po = _take(out, "out", (base.dtype,), (T, N), dev)
    ws, pw, nw = _workspace(ws, lib.ft_moe_lora_workspace, dev, stream, T, E, r, N, K)
    _run(lib.ft_moe_lora, dev, stream, base.data_ptr(), px, T, pa, pb, ps, n_slots, r, N, K, pf, pg, pt, E, po, pw, nw,
         FT_OUT_BF16 if base.dtype is _BF else 0)
    return out


# ------------------------------------------------------------------------------------- one layer with its gradient

class Bf16MoELayer:
    """One MoE layer in bf16 with its gradient, for training steps: route, permute, token rows in expert order, gate/up
    product, SwiGLU, down product, weighted combine; and back.  w13 bf16 [n_slots][2I][d] ([gate ; up] rows) and
    w2 bf16 [n_slots][d][I] as they are stored; slot_of_expert int32 [E], -1 for experts that are not resident (left to
    the residual mask; entries outside [0, n_slots) count as -1); None: expert e has matrix e.  Every buffer is allocated
    here for a fixed (T, k): forward() and backward() allocate nothing and can be captured into a graph.  backward()
    returns the gradients of x, of the logits and, by expert, of w13 and w2 (fp32; zeros for an expert without rows;
    what the buffers hold for one without a slot); add=True adds the latter two to what the buffers hold: zeros when the
    layer is made.  It takes what the last forward() left in the buffers and refuses to run before one, or after one that
    raised on its way.  One step at a time; streams as in Fp8MoELayer."""

    def __init__(self, w13, w2, slot_of_expert=None, k: int = 1, T: int = 1, out_bf16: bool = False):
        dev, (self.n_slots, I2, self.d) = _first(w13, "w13", 3, (_BF,))
        self.I = I2 // 2
        _take(w2, "w2", (_BF,), (self.n_slots, self.d, self.I), dev)
        if slot_of_expert is None:
            E = self.n_slots
        else:
            _first(slot_of_expert, "slot_of_expert", 1, (_I32,))
            _take(slot_of_expert, "slot_of_expert", (_I32,), slot_of_expert.shape, dev)
            E = slot_of_expert.shape[0]
        if T < 0 or T * k > 1 << 30 or I2 % 16 or self.d % 8 or self.d * self.I == 0 or not 1 <= self.n_slots < 1 << 23 or E > 1024 or not 1 <= k <= min(E, 32):
            _refuse(f"invalid layer shape T={T}, k={k}, E={E}, d={self.d}, w13 rows={I2}, slots={self.n_slots}")
        new = lambda *shape, dtype: _new(shape, dtype, dev)  # noqa: E731
        own = () if slot_of_expert is not None else (torch.arange(E, dtype=torch.int32, out=new(E, dtype=torch.int32)),)
        self.dev, self.w13, self.w2, self.slot_of = dev, w13, w2, own[0] if own else slot_of_expert
        self.E, self.k, self.T, self.out_bf16 = E, k, T, out_bf16
        P, f32, bf, i32 = T * k, _F32, _BF, _I32
        out = bf if out_bf16 else f32
        self.ids, self.w, self.inv = new(T, k, dtype=i32), new(T, k, dtype=f32), new(max(P, 1), dtype=i32)
        self.counts, self.offsets, self.gather = new(E, dtype=i32), new(E + 1, dtype=i32), new(max(P, 1), dtype=i32)
        self.perm_ws = new(max(lib.ft_moe_permute_workspace(T, E, k), 16), dtype=torch.uint8)
        self.xs, self.gu, self.h, self.y_sorted = new(P, self.d, dtype=bf), new(P, I2, dtype=bf), new(P, self.I, dtype=bf), new(P, self.d, dtype=bf)
        self.out, self.mask = new(T, self.d, dtype=out), new(max(T, 1), dtype=i32)
        self.dy, self.dh, self.dgu, self.dxs = new(P, self.d, dtype=bf), new(P, self.I, dtype=bf), new(P, I2, dtype=bf), new(P, self.d, dtype=bf)
        self.dx = new(T, self.d, dtype=bf)
        self.dw, self.dlogits = new(T, k, dtype=f32), new(T, E, dtype=f32)
        self.dw13, self.dw2 = new(E, I2, self.d, dtype=f32).zero_(), new(E, self.d, self.I, dtype=f32).zero_()
        need = max(ft_moe_grouped_matmul_wgrad_workspace(I2, self.d, E), ft_moe_grouped_matmul_wgrad_workspace(self.d, self.I, E))
        self.grad_ws = new(max(need, 16), dtype=torch.uint8)
        self._buffers = (self.ids, self.w, self.inv, self.counts, self.offsets, self.gather, self.perm_ws, self.xs, self.gu, self.h,
                         self.y_sorted, self.out, self.mask, self.dy, self.dh, self.dgu, self.dxs, self.dx, self.dw, self.dlogits, self.dw13,
                         self.dw2, self.grad_ws, *own)
        if P == 0:
            self.offsets.zero_()  # no forward() does
        self._ran = P == 0
        # The buffers are memory of the stream that is current here, whose work on tensors freed before may still run.
        self._streams = {_raw_stream(dev)}
        with torch.cuda.device(dev):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _on(self, stream):
        """Keeps the buffers' memory, once they are freed, until the work on `stream` is done."""
        if stream is not None and stream.device_index != self.dev:
            _refuse(f"the stream is of cuda:{stream.device_index}, the layer is on cuda:{self.dev}")
        if (_raw_stream(self.dev) if stream is None else stream.cuda_stream) not in self._streams:
            s = torch.cuda.current_stream(self.dev) if stream is None else stream
            for b in self._buffers:
                b.record_stream(s)
            self._streams.add(s.cuda_stream)

    def forward(self, logits, x, stream=None):
        """logits fp32 [T][E], x bf16 [T][d] -> (out [T][d], residual mask [T])."""
        dev, T, E, k, slot, off = self.dev, self.T, self.E, self.k, self.slot_of, self.offsets
        self._on(stream)
        _take(x, "x", (_BF,), (T, self.d), dev)
        pl = _take(logits, "logits", (_F32,), (T, E), dev)
        if T == 0:
            return self.out, self.mask[:0]
        self._ran = False  # until every step of this one is enqueued
        inv = self.inv[: T * k].view(T, k)
        pi, pw, pv, pt = self.ids.data_ptr(), self.w.data_ptr(), inv.data_ptr(), slot.data_ptr()
        _run(lib.ft_moe_route, dev, stream, pl, T, E, k, pi, pw)
        _run(lib.ft_moe_permute, dev, stream, pi, T, E, k, self.counts.data_ptr(), off.data_ptr(), self.gather.data_ptr(), pv,
             self.perm_ws.data_ptr(), self.perm_ws.numel())
        ft_moe_dispatch(x, self.ids, inv, slot_of_expert=slot, x_sorted=self.xs, stream=stream, n_slots=self.n_slots)
        ft_moe_grouped_matmul(self.xs, self.w13, off, slot_of_expert=slot, out=self.gu, stream=stream)
        ft_moe_swiglu(self.gu, h=self.h, stream=stream)
        ft_moe_grouped_matmul(self.h, self.w2, off, slot_of_expert=slot, out=self.y_sorted, stream=stream)
        _run(lib.ft_moe_combine, dev, stream, self.y_sorted.data_ptr(), None, pi, pw, pv, pt, T, E, k, self.d,
             self.out.data_ptr(), self.mask.data_ptr(), FT_N_SLOTS(self.n_slots) | (FT_OUT_BF16 if self.out_bf16 else 0))
        self._ran = True
        return self.out, self.mask[:T]

    def backward(self, dout, add: bool = False, stream=None):
        """dout [T][d] (bf16 or fp32) of the last forward() -> (dx bf16 [T][d], dlogits fp32 [T][E], dw13 fp32 [E][2I][d],
        dw2 fp32 [E][d][I])."""
        T, slot, off, n = self.T, self.slot_of, self.offsets, self.n_slots
        self._on(stream)
        _take(dout, "dout", _FLOATS, (T, self.d), self.dev)
        if not self._ran:
            _refuse("backward() needs a forward() before it")
        if T == 0:
            inv = None
        else:
            inv = self.inv[: T * self.k].view(T, self.k)
            ft_moe_combine_grad(dout, self.y_sorted, self.ids, self.w, inv, slot_of_expert=slot, dy_sorted=self.dy, dw=self.dw,
                                dlogits=self.dlogits, stream=stream, n_slots=n)
            ft_moe_grouped_matmul_grad(self.dy, self.w2, off, slot_of_expert=slot, da=self.dh, stream=stream)
        grads = dict(slot_of_expert=slot, add=add, stream=stream, n_slots=n, ws=self.grad_ws)
        ft_moe_grouped_matmul_wgrad(self.dy, self.h, off, dw=self.dw2, **grads)
        if T > 0:
            ft_moe_swiglu_grad(self.gu, self.dh, dgu=self.dgu, stream=stream)
        ft_moe_grouped_matmul_wgrad(self.dgu, self.xs, off, dw=self.dw13, **grads)
        if T > 0:
            ft_moe_grouped_matmul_grad(self.dgu, self.w13, off, slot_of_expert=slot, da=self.dxs, stream=stream)
            ft_moe_dispatch_grad(self.dxs, self.ids, inv, slot_of_expert=slot, dx=self.dx, stream=stream, n_slots=n)
        return self.dx, self.dlogits, self.dw13, self.dw2
