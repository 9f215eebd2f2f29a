"""The product calls' definitions in 64 bits on the CPU, and the bounds that their tests hold the kernels to.

A rounding is off by at most half a step: 2^-24 of the value in fp32, 2^-8 in bf16 (torch.finfo(t).eps / 2)."""
from __future__ import annotations

import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -126  # fp32 and bf16 values below it may count as 0, before and after a sum


def groups(offsets, slot, E, P, n_slots):
    """(expert, first row, past the last, slot) of every expert with a slot; offsets clipped, slot None: its number."""
    o = [min(max(int(v), 0), P) for v in offsets.tolist()]
    for e in range(E):
        s = e if slot is None else int(slot[e])
        if 0 <= s < n_slots:
            yield e, o[e], max(o[e], o[e + 1]), s


def sum_bound(ref, mag, terms, dtype):
    """`terms` exact products added in fp32 in any order: each addition is off by at most a whole step (the matrix
    instruction may cut instead of round) of a partial sum that is at most mag; then one rounding to the output."""
    return 2 * terms * U32 * mag + (UBF * ref.abs() if dtype == torch.bfloat16 else 0) + TINY


def forward(a, w, offsets, slot, out):
    """(rows that have a result, fp64 results, sums of magnitudes), [P][N]."""
    P, E = a.shape[0], offsets.numel() - 1
    has = torch.zeros(P, dtype=torch.bool)
    ref, mag = torch.zeros(P, w.shape[1], dtype=torch.float64), torch.zeros(P, w.shape[1], dtype=torch.float64)
    for _, r0, r1, s in groups(offsets, slot, E, P, w.shape[0]):
        x, y = a[r0:r1].double(), w[s].double()
        ref[r0:r1], mag[r0:r1] = x @ y.t(), x.abs() @ y.abs().t()
        has[r0:r1] = True
    return has, ref, mag


def matrix_gradient(dout, a, offsets, slot, n_slots):
    """(experts that have one, fp64 gradients, sums of magnitudes, rows of the largest expert), [E][N][K]."""
    P, E = a.shape[0], offsets.numel() - 1
    has = torch.zeros(E, dtype=torch.bool)
    ref = torch.zeros(E, dout.shape[1], a.shape[1], dtype=torch.float64)
    mag, most = torch.zeros_like(ref), 0
    for e, r0, r1, _ in groups(offsets, slot, E, P, n_slots):
        x, y = dout[r0:r1].double(), a[r0:r1].double()
        ref[e], mag[e] = x.t() @ y, x.abs().t() @ y.abs()
        has[e], most = True, max(most, r1 - r0)
    return has, ref, mag, most


def swiglu(gu):
    """(h, what its fp32 steps may be off by), fp64.  The exponent's argument is off by |g| log2(e) roundings, its power
    and the reciprocal by two units, the sum and the two products by a rounding each; 1 / (1 + e^-g) below 2^-126
    may count as 0."""
    g, u = gu.double().chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    return h, (g.abs() + 10) * U32 * h.abs() + g.abs() * u.abs() * TINY


def swiglu_gradient(gu, dh):
    """([dg | du], what their fp32 steps may be off by), fp64: the sigmoid s carries (|g| + 5) roundings, 1 - s one more of
    1, and they meet in s + g s (1 - s), whose two terms may cancel."""
    g, u = gu.double().chunk(2, 1)
    d, s = dh.double(), torch.sigmoid(g)
    e = (g.abs() + 12) * U32
    slope, size = s + g * s * torch.sigmoid(-g), s + (g * s).abs() * (torch.sigmoid(-g) + 1)
    dg, du = d * u * slope, d * g * s
    off_g = (d * u).abs() * (e * size + (1 + g.abs()) * TINY)
    off_u = (d * g).abs() * (e * s + TINY)
    return torch.cat([dg, du], 1), torch.cat([off_g, off_u], 1)


def adapters(base, x, a, b, offsets, gather, slot, scale, left=2.0 ** -16):
    """(fp64 out, bound): rows without an adapter are base; a hidden value is a sum of K products in fp32 (in splits) times the
    scale (a rounding), in two bf16 terms that leave 2^-16 of it (2^-8 of 2^-8), or in three that leave 2^-24 (left); the outer sum has 2 r terms; base is
    added and the sum rounded."""
    T, E, n_slots, r, K = base.shape[0], offsets.numel() - 1, a.shape[0], a.shape[1], a.shape[2]
    ref, bound = base.double().clone(), torch.zeros(base.shape, dtype=torch.float64)
    for _, r0, r1, s in groups(offsets, slot, E, T, n_slots):
        rows = gather[r0:r1].long()
        rows = rows[(rows >= 0) & (rows < T)]
        sc = 1.0 if scale is None else float(scale[s])
        A, B, xr = a[s].double(), b[s].double(), x[rows].double()
        hid, hmag = xr @ A.t(), xr.abs() @ A.abs().t()
        hoff = 2 * (K + 20) * U32 * hmag + left * hid.abs()
        delta = sc * (hid @ B.t())
        ref[rows] += delta
        bound[rows] = abs(sc) * ((hoff + 2 * (2 * r + 2) * U32 * hid.abs()) @ B.abs().t()) + 2 * U32 * (delta.abs() + base[rows].double().abs())
        if base.dtype == torch.bfloat16:
            bound[rows] += UBF * ref[rows].abs()
        bound[rows] += TINY
    return ref, bound
