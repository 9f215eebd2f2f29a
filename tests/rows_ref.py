"""The row calls' definitions in 64 bits on the CPU, and the bounds that their tests hold the kernels to.

A rounding is off by at most half a step: 2^-24 of the value in fp32, 2^-8 in bf16 (torch.finfo(t).eps / 2)."""
from __future__ import annotations

import numpy as np
import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8
FLOOR = 2.0 ** -100


def cols(K: int) -> int:
    return (K + 511) // 512 * 4


def e4m3_step(q: torch.Tensor) -> torch.Tensor:
    """The spacing of e4m3 values at fp64 magnitudes q: 8 a binade, 2^-9 below 2^-6."""
    exp = torch.frexp(q.abs())[1] - 1
    return torch.ldexp(torch.ones_like(q), exp.clamp(min=-6) - 3)


def e4m3_nearest(q: torch.Tensor) -> torch.Tensor:
    step = e4m3_step(q)
    return (torch.round(q / step) * step).clamp(-448, 448)  # torch.round: ties to even


def quotients(x: torch.Tensor):
    """fp64 rows -> (448 x / top, top / 448) with top per 128 values, [rows][K] and [rows][ceil(K/128)]."""
    rows, K = x.shape
    nb = (K + 127) // 128
    q, s = torch.empty_like(x), torch.empty(rows, nb, dtype=torch.float64)
    for b in range(nb):
        part = x[:, 128 * b: 128 * b + 128]
        top = part.abs().amax(1).clamp(min=FLOOR)
        q[:, 128 * b: 128 * b + 128] = 448 * part / top[:, None]
        s[:, b] = top / 448
    return q, s


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """What 8-bit rows stand for, fp64."""
    K = codes.shape[1]
    return codes.double() * scales.double().repeat_interleave(128, 1)[:, :K]


def weight_values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    N, K = codes.shape
    return codes.double() * scales.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def random_weights(gen, *shape):
    """e4m3 codes [..., N, K] and scales per 128 x 128."""
    codes = (torch.randn(*shape, generator=gen) * 112).clamp(-448, 448).to(torch.float8_e4m3fn)
    N, K = shape[-2:]
    scales = torch.rand(*shape[:-2], (N + 127) // 128, (K + 127) // 128, generator=gen) * 0.01 + 1e-3
    return codes, scales


def random_rows(gen, rows, K):
    """8-bit rows as a caller may have them: any codes but NaN, scales with zero columns behind the last block."""
    codes = (torch.randn(rows, K, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.zeros(rows, cols(K))
    scales[:, : (K + 127) // 128] = torch.rand(rows, (K + 127) // 128, generator=gen) * 0.02 + 1e-3
    return codes, scales


def product(a, sa, w, sw):
    """(product, sum of the magnitudes of its terms), fp64."""
    x, y = values(a, sa), weight_values(w, sw)
    return x @ y.t(), x.abs() @ y.abs().t()


def product_bound(ref, mag, K, bf16):
    """fp32 results: exact products; a block's 128 terms are added in 127 steps of at most 2^-23 each (the matrix
    instruction may cut instead of round), the two scales' product, the multiply-add and the sums over
    ceil(K/128) blocks and 8 waves one rounding each.  bf16 results on the 8-bit instructions: each product
    of a group of 8 is cut at 2^-13 of the group's largest, so 7 of them lose up to 7 * 2^-13 of
    the group's largest, and the result is rounded once."""
    bound = (2 * 127 + (K + 127) // 128 + 10) * U32 * mag
    return bound + 7 * 2.0 ** -13 * mag + UBF * ref.abs() if bf16 else bound


def routing(gen, T, E, k, held=None):
    """ids, w, counts' offsets, inv and a slot table that holds `held` experts (None: all), CPU tensors."""
    logits = torch.randn(T, E, generator=gen)
    top, ids = logits.topk(k, dim=1) if T else (torch.zeros(0, k), torch.zeros(0, k, dtype=torch.long))
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * k)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    slot = torch.full((E,), -1, dtype=torch.int32)
    n = E if held is None else held
    slot[torch.randperm(E, generator=gen)[:n]] = torch.arange(n, dtype=torch.int32)
    return dict(logits=logits, ids=ids.int(), w=top.softmax(1), inv=inv.int().view(T, k), offsets=offsets, slot=slot)


def pair_rows(ids, inv, E, slot=None):
    """Row of every pair, -1 where it has none."""
    ok = (ids >= 0) & (ids < E) & (inv >= 0) & (inv < ids.numel())
    if slot is not None:
        ok &= slot[ids.clamp(0, E - 1).long()] >= 0
    return torch.where(ok, inv, torch.full_like(inv, -1)).long()


def combine_grad(dout, y, w, rows, ids, E):
    """fp64 (dw, dlogits) of out[t] = sum_j w_j y[rows_j], w the softmax of the chosen logits, and the sums of
    magnitudes that bound their errors."""
    T, k = ids.shape
    has = (rows >= 0).double()
    yj = y.double()[rows.clamp(min=0)]
    terms = dout.double()[:, None, :] * yj * has[:, :, None]
    dw, mag = terms.sum(2), terms.abs().sum(2)
    wd = w.double()
    dl = wd * (dw - (wd * dw).sum(1, keepdim=True))
    out = torch.zeros(T, E, dtype=torch.float64)
    valid = (ids >= 0) & (ids < E)
    for j in range(k):
        t = torch.nonzero(valid[:, j])[:, 0]
        out[t, ids[t, j].long()] += dl[t, j]
    return dw, mag, out


def softmax_weights(logits, ids):
    z = np.take_along_axis(logits, ids, 1)
    z = np.exp(z - z.max(1, keepdims=True))
    return z / z.sum(1, keepdims=True)
