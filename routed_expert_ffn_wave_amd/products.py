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
from .rows import _BF, _F32, _FLOATS, _I32, _first, _new, _product_out, _refuse, _run, _take

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
    adapters (ft_moe_permute of the rows' adapters, k = 1); rows without an adapter stand behind them or with one that
    has no slot, and get base.  out may be base itself.  `ws`: ft_moe_lora_workspace(T, E, r, N, K) bytes."""
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
