"""Row calls without a GPU: exports, argument checks of the C ABI and of the binding, and the reference formulas
against differences."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import routed_expert_ffn_wave_amd as ft
import rows_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ft_moe_rows.h")
A, B = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)  # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10008)
L = ft.lib


def err(rc, status, text):
    assert rc == status, (rc, ft.ft_moe_last_error())
    assert text in ft.ft_moe_last_error(), ft.ft_moe_last_error()


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*int\s+(ft_moe_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(ft.EXPORTED_ROWS)
    out = subprocess.run(["nm", "-D", "--defined-only", ft.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(ft_moe_\w+)", out))
    assert int(re.search(r"#define FT_ROWS_F32 (0x\w+)", open(HEADER).read()).group(1), 16) == ft.FT_ROWS_F32


@pytest.mark.parametrize("K, S", [(-5, 0), (0, 0), (1, 4), (16, 4), (512, 4), (513, 8), (768, 8), (7168, 56)])
def test_scale_cols(K, S):
    assert ft.ft_moe_fp8_scale_cols(K) == S


def test_quant_refusals():
    q = lambda x=A, rows=4, K=64, c=B, s=B, f=0: L.ft_moe_quant_fp8(x, rows, K, c, s, f, None)  # noqa: E731
    err(q(rows=-1), ft.FT_E_INVAL, "rows must be")
    for K in (0, -16, 8, 100, (1 << 20) + 16):
        err(q(K=K), ft.FT_E_INVAL, "K must be")
    err(q(f=0x1), ft.FT_E_INVAL, "unknown flags 0x1")
    err(q(rows=1 << 30, K=1 << 20), ft.FT_E_UNSUPPORTED, "rows too large")
    err(q(x=None), ft.FT_E_INVAL, "x is null")
    err(q(c=MIS), ft.FT_E_INVAL, "codes is not 16-byte")
    err(q(s=None), ft.FT_E_INVAL, "scales is null")
    assert q(x=None, rows=0, c=None, s=None) == ft.FT_OK
    err(L.ft_moe_swiglu_fp8(A, 4, 24, B, B, None), ft.FT_E_INVAL, "I must be")
    err(L.ft_moe_swiglu_fp8(None, 4, 32, B, B, None), ft.FT_E_INVAL, "gu is null")
    assert L.ft_moe_swiglu_fp8(None, 0, 32, None, None, None) == ft.FT_OK


def test_pair_refusals():
    names = ("dispatch", "dispatch_fp8", "dispatch_grad", "combine_grad")
    bad = [(dict(T=-1), "T must be"), (dict(E=0), "E must be"), (dict(E=1025), "E must be"), (dict(k=0), "k must be"),
           (dict(k=9), "k must be"), (dict(k=33, E=64), "k must be"), (dict(d=0), "d must be"), (dict(d=12), "d must be"),
           (dict(d=(1 << 20) + 16), "d must be"), (dict(flags=0x40), "unknown flags"), (dict(ids=None), "ids is null"),
           (dict(inv=MIS), "inv is not 16-byte"), (dict(slot=MIS), "slot_of_expert is not 16-byte"), (dict(x=None), "is null"),
           (dict(out=None), "is null")]
    for kw, text in bad:
        for name in names:
            err(_one(name, **kw), ft.FT_E_INVAL, text)
    for name in names:
        assert _one(name, T=0, x=None, ids=None, inv=None, out=None) == ft.FT_OK
    err(_one("dispatch_fp8", d=24), ft.FT_E_INVAL, "multiple of 16")
    err(_one("dispatch", T=1 << 29, d=1 << 20, k=1), ft.FT_E_UNSUPPORTED, "T too large")
    err(_one("dispatch", flags=ft.FT_OUT_BF16), ft.FT_E_INVAL, "unknown flags 0x4")
    err(_one("combine_grad", flags=ft.FT_ROWS_F32), ft.FT_E_INVAL, "unknown flags 0x20")


def _one(name, T=4, E=8, k=2, d=64, ids=A, inv=A, slot=None, x=A, out=B, flags=0):
    if name == "combine_grad":
        return L.ft_moe_combine_grad(x, A, ids, A, inv, slot, T, E, k, d, out, B, None, flags, None)
    if name == "dispatch_fp8":
        return L.ft_moe_dispatch_fp8(x, ids, inv, slot, T, E, k, d, out, B, flags, None)
    return getattr(L, "ft_moe_" + name)(x, ids, inv, slot, T, E, k, d, out, flags, None)


def test_matmul_refusals():
    m = lambda a=A, sa=A, M=4, w=A, sw=A, N=64, K=64, out=B, f=0: L.ft_moe_fp8_matmul(a, sa, M, w, sw, N, K, out, f, None)  # noqa: E731
    for kw, text in [(dict(M=-1), "M must be"), (dict(M=(1 << 30) + 1), "M must be"), (dict(N=0), "N must be"),
                     (dict(N=(1 << 24) + 1), "N must be"), (dict(K=0), "K must be"), (dict(K=40), "K must be"),
                     (dict(K=(1 << 20) + 16), "K must be"), (dict(f=0x20), "unknown flags 0x20"), (dict(a=None), "a is null"),
                     (dict(sa=MIS), "a_scales is not"), (dict(w=None), "w is null"), (dict(sw=None), "w_scales is null"),
                     (dict(out=MIS), "out is not")]:
        err(m(**kw), ft.FT_E_INVAL, text)
    err(m(M=1 << 30, N=1 << 24), ft.FT_E_UNSUPPORTED, "product too large")
    assert m(M=0, a=None, sa=None, w=None, sw=None, out=None) == ft.FT_OK
    g = lambda P=4, n=3, N=64, K=64, off=A, slot=A, E=8, out=B, f=0: L.ft_moe_fp8_grouped_matmul(  # noqa: E731
        A, A, P, A, A, n, N, K, off, slot, E, out, f, None)
    for kw, text in [(dict(E=0), "E must be"), (dict(E=1025), "E must be"), (dict(n=0), "n_slots must be"), (dict(P=-1), "P must be"),
                     (dict(K=8), "K must be"), (dict(off=None), "offsets is null"), (dict(slot=MIS), "slot_of_expert is not"),
                     (dict(out=None), "out is null"), (dict(f=1), "unknown flags 0x1")]:
        err(g(**kw), ft.FT_E_INVAL, text)
    assert g(P=0, off=None, slot=None, out=None) == ft.FT_OK


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ft.ft_moe_quant_fp8(x), lambda: ft.ft_moe_swiglu_fp8(x), lambda: ft.ft_moe_dispatch(x, i, i, E=4),
                 lambda: ft.ft_moe_dispatch_fp8(x, i, i, E=4), lambda: ft.ft_moe_dispatch_grad(x, i, i, E=4),
                 lambda: ft.ft_moe_combine_grad(x, x, i, x, i, E=4), lambda: ft.ft_moe_fp8_matmul(x, x, x, x),
                 lambda: ft.ft_moe_fp8_grouped_matmul(x, x, x, x, i, i), lambda: ft.ft_moe_quant_fp8(None)):
        with pytest.raises(ft.FtError):
            call()


def test_reference_gradient_against_differences():
    """The reference's dw and dlogits are the differences of sum(dout * out) in fp64."""
    rng = np.random.default_rng(3)
    T, E, k, d = 3, 7, 4, 5
    logits, y, dout = rng.normal(size=(T, E)), rng.normal(size=(T * k, d)), rng.normal(size=(T, d))
    ids = np.argsort(-logits, axis=1)[:, :k]
    rows = rng.permutation(T * k).reshape(T, k)
    rows[1, 2] = -1  # a pair without a row

    def loss(z, w=None):
        w = ref.softmax_weights(z, ids) if w is None else w
        return sum(w[t, j] * dout[t] @ y[rows[t, j]] for t in range(T) for j in range(k) if rows[t, j] >= 0)

    w = ref.softmax_weights(logits, ids)
    dw, _, dl = ref.combine_grad(*(torch.from_numpy(v) for v in (dout, y, w, rows, ids)), E)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            z = [logits.copy(), logits.copy()]
            z[0][t, e] += h
            z[1][t, e] -= h
            assert abs((loss(z[0]) - loss(z[1])) / (2 * h) - dl[t, e].item()) < 1e-8
        for j in range(k):
            v = [w.copy(), w.copy()]
            v[0][t, j] += h
            v[1][t, j] -= h
            assert abs((loss(None, v[0]) - loss(None, v[1])) / (2 * h) - dw[t, j].item()) < 1e-8


def test_sizes_that_a_launch_cannot_count():
    err(L.ft_moe_quant_fp8(A, 1 << 27, 512, B, B, 0, None), ft.FT_E_UNSUPPORTED, "rows too large")
    err(L.ft_moe_swiglu_fp8(A, 1 << 27, 16, B, B, None), ft.FT_E_UNSUPPORTED, "rows too large")
    for name in ("dispatch", "dispatch_fp8", "dispatch_grad", "combine_grad"):
        err(_one(name, T=1 << 26, d=1024, k=1), ft.FT_E_UNSUPPORTED, "T too large")
    err(_one("combine_grad", T=1 << 24, d=8, k=1), ft.FT_E_UNSUPPORTED, "T too large")
    # a table that does not ascend may give all rows to 512 of 1024 experts: more tiles than are counted
    for flags in (0, ft.FT_OUT_BF16):
        err(L.ft_moe_fp8_grouped_matmul(A, A, 1 << 30, A, A, 1, 1, 16, A, A, 1024, B, flags, None), ft.FT_E_UNSUPPORTED, "product too large")
    err(L.ft_moe_fp8_matmul(A, A, 1 << 30, A, A, 1, 16, B, 0, None), ft.FT_E_UNSUPPORTED, "product too large")


def test_scale_cols_of_the_largest_size():
    assert ft.ft_moe_fp8_scale_cols(2 ** 31 - 1) == 4 * 2 ** 22


def test_slot_counts_in_flags():
    assert re.search(r"#define FT_N_SLOTS\(n\) \(\(n\) << 8\)", open(os.path.join(ROOT, "include", "ft_moe.h")).read())
    assert ft.FT_N_SLOTS(5) == 5 << 8 and ft.FT_N_SLOTS((1 << 23) - 1) == 0x7FFFFF00
    for n in (0, -1, 1 << 23):
        with pytest.raises(ft.FtError, match="n_slots must be"):
            ft.FT_N_SLOTS(n)
    for name in ("dispatch", "dispatch_fp8", "dispatch_grad", "combine_grad"):
        err(_one(name, flags=ft.FT_N_SLOTS(5)), ft.FT_E_INVAL, "FT_N_SLOTS without slot_of_expert")
        err(_one(name, flags=ft.FT_N_SLOTS(5), slot=A, out=None), ft.FT_E_INVAL, "is null")
        err(_one(name, flags=-(2 ** 31), slot=A), ft.FT_E_INVAL, "unknown flags 0x80000000")
        assert _one(name, T=0, flags=ft.FT_N_SLOTS(5)) == ft.FT_OK
    # calls that know the bank, or take no table, do not take the flag
    err(L.ft_moe_quant_fp8(A, 4, 64, B, B, ft.FT_N_SLOTS(5), None), ft.FT_E_INVAL, "unknown flags 0x500")
    err(L.ft_moe_fp8_grouped_matmul(A, A, 4, A, A, 3, 64, 64, A, A, 8, B, ft.FT_N_SLOTS(3), None), ft.FT_E_INVAL, "unknown flags 0x300")
    call = lambda flags, out=None: L.ft_moe_combine(A, None, A, A, A, A, 4, 8, 2, 256, out, None, flags, None)  # noqa: E731
    err(call(ft.FT_N_SLOTS(5) | ft.FT_OUT_BF16), ft.FT_E_INVAL, "out is null")
    err(call(-(2 ** 31)), ft.FT_E_INVAL, "unknown flags 0x80000000")


def test_last_sizes_that_a_launch_counts():
    """Whole blocks count: the last sizes below a launch's 2^32 threads pass the check (and fail at the next one, a null
    pointer), the sizes after them are refused."""
    quant = lambda rows, K: L.ft_moe_quant_fp8(None, rows, K, B, B, 0, None)  # noqa: E731
    swiglu = lambda rows, K: L.ft_moe_swiglu_fp8(None, rows, K, B, B, None)  # noqa: E731
    for call in (quant, swiglu):
        err(call((1 << 27) - 8, 512), ft.FT_E_INVAL, "is null")
        for rows in range((1 << 27) - 7, (1 << 27) + 1):
            err(call(rows, 512), ft.FT_E_UNSUPPORTED, "rows too large")
    for name in ("dispatch", "dispatch_grad", "dispatch_fp8"):
        err(_one(name, T=(1 << 26) - 4, d=1024, k=1, x=None) if name != "dispatch_fp8" else _one(name, T=(1 << 26) - 4, d=512, k=1, x=None),
            ft.FT_E_INVAL, "is null")
        for T in range((1 << 26) - 3, (1 << 26) + 1):
            err(_one(name, T=T, d=1024, k=1, x=None), ft.FT_E_UNSUPPORTED, "T too large")
    err(_one("combine_grad", T=(1 << 24) - 1, d=8, k=1, x=None), ft.FT_E_INVAL, "is null")
    # 47 x 178481 tiles of 256 x 256: one less than 2^23, but blocks are launched in multiples of 8
    err(L.ft_moe_fp8_matmul(A, A, 178480 * 256 + 1, A, A, 47 * 256, 16, B, ft.FT_OUT_BF16, None), ft.FT_E_UNSUPPORTED, "product too large")


def test_layer_orders_its_buffers_with_the_streams(monkeypatch):
    """With stand-ins for the GPU: making a layer waits for the current stream, and a forward on a stream that did not make
    it records every buffer for that stream, once."""
    import contextlib
    import types

    from routed_expert_ffn_wave_amd import rows
    made, waits, used = [], [], []

    class Buffer(torch.Tensor):
        def record_stream(self, stream):
            used.append((id(self), stream.cuda_stream))

    def new(shape, dtype, dev, stream=None):
        made.append(torch.zeros(shape).to(dtype).as_subclass(Buffer))
        return made[-1]

    streams = {n: types.SimpleNamespace(cuda_stream=n, device_index=0, synchronize=lambda n=n: waits.append(n)) for n in (1, 2, 3)}
    current = [1]
    monkeypatch.setattr(rows, "_new", new)
    monkeypatch.setattr(rows, "_first", lambda t, name, dims, dtypes, stream=None: (0, t.shape))
    monkeypatch.setattr(rows, "_take", lambda t, name, dtypes, shape, dev: t.data_ptr())
    monkeypatch.setattr(rows, "_run", lambda *a: None)
    monkeypatch.setattr(rows, "_raw_stream", lambda dev: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: streams[current[0]])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    z = lambda *s, dtype=torch.float8_e4m3fn: torch.zeros(s).to(dtype)  # noqa: E731
    layer = rows.Fp8MoELayer(z(2, 64, 64), z(2, 1, 1, dtype=torch.float32), z(2, 64, 32), z(2, 1, 1, dtype=torch.float32),
                             torch.zeros(4, dtype=torch.int32), 2, 4)
    assert waits == [1] and len(made) == 15
    args = (torch.zeros(4, 4), torch.zeros(4, 64, dtype=torch.bfloat16))
    layer.forward(*args)
    assert used == []
    layer.forward(*args, stream=streams[2])
    assert sorted(used) == sorted((id(b), 2) for b in made)
    layer.forward(*args, stream=streams[2])
    current[0] = 3
    layer.forward(*args)
    layer.forward(*args)
    assert sorted(used) == sorted((id(b), n) for b in made for n in (2, 3))
    assert waits == [1]


def test_import_without_torchs_inner_functions():
    """The package imports under a torch build that lacks them, and asks torch's public functions instead."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import types\n"
            "torch.cuda.current_stream = lambda dev: types.SimpleNamespace(cuda_stream=40 + dev)\n"
            "import routed_expert_ffn_wave_amd as ft\n"
            "from routed_expert_ffn_wave_amd import rows\n"
            "assert rows._raw_stream(2) == 42 and rows._current_device is torch.cuda.current_device\n"
            "assert ft.ft_moe_fp8_scale_cols(513) == 8\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
