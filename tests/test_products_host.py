"""Product calls without a GPU: exports, argument checks of the C ABI and of the binding, and the reference formulas
against differences."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import products_ref as ref
import routed_expert_ffn_wave_amd as ft

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ft_moe_products.h")
A, B = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)  # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10008)
L = ft.lib


def err(rc, status, text):
    assert rc == status, (rc, ft.ft_moe_last_error())
    assert text in ft.ft_moe_last_error(), ft.ft_moe_last_error()


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(ft_moe_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(ft.EXPORTED_PRODUCTS)
    out = subprocess.run(["nm", "-D", "--defined-only", ft.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(ft_moe_\w+)", out))
    assert int(re.search(r"#define FT_ADD_TO_OUT (0x\w+)", open(HEADER).read()).group(1), 16) == ft.FT_ADD_TO_OUT


def grouped(name, a=A, P=4, w=A, n=8, N=64, K=64, off=A, slot=None, E=8, out=B, f=0):
    return getattr(L, "ft_moe_grouped_matmul" + name)(a, P, w, n, N, K, off, slot, E, out, f, None)


def wgrad(d=A, a=A, P=4, N=64, K=64, off=A, slot=None, E=8, dw=B, ws=B, nb=1 << 20, f=0):
    return L.ft_moe_grouped_matmul_wgrad(d, a, P, N, K, off, slot, E, dw, ws, nb, f, None)


def lora(base=A, x=A, T=4, a=A, b=A, s=None, n=8, r=16, N=64, K=64, off=A, ga=A, slot=None, E=8, out=B, ws=B, nb=1 << 20, f=0):
    return L.ft_moe_lora(base, x, T, a, b, s, n, r, N, K, off, ga, slot, E, out, ws, nb, f, None)


SIZES = [(dict(E=0), "E must be"), (dict(E=1025), "E must be"), (dict(N=0), "N must be"), (dict(N=12), "N must be"),
         (dict(N=(1 << 20) + 8), "N must be"), (dict(K=-8), "K must be"), (dict(K=4), "K must be"), (dict(K=(1 << 20) + 8), "K must be"),
         (dict(f=1), "unknown flags 0x1")]


@pytest.mark.parametrize("name, a, out", [("", "a", "out"), ("_grad", "dout", "da")])
def test_grouped_refusals(name, a, out):
    for kw, text in SIZES + [(dict(P=-1), "P must be"), (dict(P=(1 << 30) + 1), "P must be"), (dict(n=0), "n_slots must be"),
                             (dict(n=7), "slot_of_expert is needed"), (dict(a=None), a + " is null"), (dict(w=MIS), "w is not 16"),
                             (dict(off=None), "offsets is null"), (dict(slot=MIS), "slot_of_expert is not 16"), (dict(out=None), out + " is null"),
                             (dict(f=ft.FT_ADD_TO_OUT), "unknown flags 0x40"), (dict(f=ft.FT_N_SLOTS(3), slot=A), "unknown flags 0x300")]:
        err(grouped(name, **kw), ft.FT_E_INVAL, text)
    assert grouped(name, P=0, a=None, w=None, off=None, out=None) == ft.FT_OK
    # a table that does not ascend may give all rows to 512 of 1024 experts: more tiles than are counted
    err(grouped(name, P=1 << 30, N=1 << 20, K=1 << 20, E=1024, n=1024), ft.FT_E_UNSUPPORTED, "product too large")


def test_wgrad_refusals():
    for kw, text in SIZES + [(dict(P=-1), "P must be"), (dict(d=None), "dout is null"), (dict(a=MIS), "a is not 16"),
                             (dict(off=None), "offsets is null"), (dict(slot=MIS), "slot_of_expert is not 16"), (dict(dw=None), "dw is null"),
                             (dict(f=ft.FT_ADD_TO_OUT | ft.FT_OUT_BF16), "FT_ADD_TO_OUT needs"),
                             (dict(f=ft.FT_N_SLOTS(3)), "FT_N_SLOTS without")]:
        err(wgrad(**kw), ft.FT_E_INVAL, text)
    assert wgrad(P=0, d=None, a=None, off=None, dw=None, f=ft.FT_ADD_TO_OUT) == ft.FT_OK
    err(wgrad(P=0, d=None, a=None, dw=None), ft.FT_E_INVAL, "dw is null")  # without rows dw is zeroed
    err(wgrad(N=1 << 20, K=1 << 20, E=1024), ft.FT_E_UNSUPPORTED, "gradient too large")


def test_wgrad_workspace():
    need = ft.ft_moe_grouped_matmul_wgrad_workspace
    assert need(1536, 2048, 8) == 0
    big = need(1536, 2048, 128)
    assert 128 * 16 <= big <= 1 << 16
    for bad in ((0, 2048, 128), (1536, 0, 128), (1536, 2048, 1025), (1536, 2048, 0), ((1 << 20) + 8, 2048, 128)):
        assert need(*bad) == 0
    call = lambda **kw: wgrad(P=32768, N=1536, K=2048, E=128, **kw)  # noqa: E731
    err(call(ws=None), ft.FT_E_INVAL, "ws is null")
    err(call(ws=MIS), ft.FT_E_INVAL, "ws is not 16")
    err(call(nb=big - 1), ft.FT_E_WORKSPACE, "workspace of")


def test_swiglu_refusals():
    f = lambda gu=A, rows=4, I=64, h=B: L.ft_moe_swiglu(gu, rows, I, h, None)  # noqa: E731
    g = lambda gu=A, rows=4, I=64, h=B: L.ft_moe_swiglu_grad(gu, A, rows, I, h, None)  # noqa: E731
    for call in (f, g):
        for kw, text in [(dict(rows=-1), "rows must be"), (dict(I=0), "I must be"), (dict(I=12), "I must be"), (dict(I=(1 << 20) + 8), "I must be"),
                         (dict(gu=None), "gu is null"), (dict(h=MIS), "is not 16")]:
            err(call(**kw), ft.FT_E_INVAL, text)
        err(call(rows=1 << 30, I=64), ft.FT_E_UNSUPPORTED, "rows too large")
        assert call(rows=0, gu=None, h=None) == ft.FT_OK
    err(L.ft_moe_swiglu_grad(A, None, 4, 64, B, None), ft.FT_E_INVAL, "dh is null")


def test_lora_refusals():
    for kw, text in SIZES + [(dict(T=-1), "T must be"), (dict(r=0), "r must be"), (dict(r=4), "r must be"), (dict(r=264), "r must be"),
                             (dict(n=0), "n_slots must be"), (dict(n=7), "slot_of_adapter is needed"), (dict(base=None), "base is null"),
                             (dict(x=MIS), "x is not 16"), (dict(a=None), "a is null"), (dict(b=None), "b is null"), (dict(s=MIS), "scale is not"),
                             (dict(off=None), "offsets is null"), (dict(ga=None), "gather is null"), (dict(slot=MIS), "slot_of_adapter is not"),
                             (dict(out=None), "out is null"), (dict(T=300, r=72, ws=None), "ws is null"), (dict(f=0x40), "unknown flags 0x40")]:
        err(lora(**kw), ft.FT_E_INVAL, text)
    need = ft.ft_moe_lora_workspace(300, 8, 72, 64, 64)
    assert need >= 300 * 72 * 4
    err(lora(T=300, r=72, nb=need - 1), ft.FT_E_WORKSPACE, "workspace of")
    err(lora(T=1 << 24), ft.FT_E_UNSUPPORTED, "T too large")
    err(lora(T=(1 << 24) - 1, N=1 << 20, E=1024, n=1024), ft.FT_E_UNSUPPORTED, "T too large")
    assert lora(T=0, base=None, x=None, a=None, b=None, off=None, ga=None, out=None, ws=None, nb=0) == ft.FT_OK
    for bad in ((0, 8, 72, 64, 64), (300, 0, 72, 64, 64), (300, 1025, 72, 64, 64), (300, 8, 0, 64, 64), (300, 8, 264, 64, 64),
                (300, 8, 72, 0, 64), (300, 8, 72, 64, 0), (1 << 24, 8, 72, 64, 64)):
        assert ft.ft_moe_lora_workspace(*bad) == 0


def test_binding_refuses_tensors_off_the_gpu():
    x, w, i = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: ft.ft_moe_grouped_matmul(x, w, i), lambda: ft.ft_moe_grouped_matmul_grad(x, w, i),
                 lambda: ft.ft_moe_grouped_matmul_wgrad(x, x, i), lambda: ft.ft_moe_swiglu(x), lambda: ft.ft_moe_swiglu_grad(x, x),
                 lambda: ft.ft_moe_lora(x, x, w, w, i, i), lambda: ft.ft_moe_grouped_matmul(None, w, i)):
        with pytest.raises(ft.FtError):
            call()


def test_reference_gradients_against_differences():
    """The references' gradients of rows, matrices and SwiGLU are the differences of sum(dout * out) in fp64."""
    g = torch.Generator().manual_seed(3)
    P, E, N, K, h = 7, 3, 8, 8, 1e-5
    off = torch.tensor([0, 4, 4, 7])
    a, w, dout = (torch.randn(s, generator=g).double() for s in ((P, K), (E, N, K), (P, N)))

    def loss(a, w):
        return sum((dout[r0:r1] * (a[r0:r1] @ w[s].t())).sum() for _, r0, r1, s in ref.groups(off, None, E, P, E))

    da = ref.forward(dout, w.transpose(1, 2), off, None, None)[1]
    dw = ref.matrix_gradient(dout, a, off, None, E)[1]
    for t, grad in ((a, da), (w, dw)):
        for i in range(t.numel()):
            flat, at = t.view(-1), t.view(-1)[i].item()
            flat[i] = at + h
            up = loss(a, w)
            flat[i] = at - h
            down = loss(a, w)
            flat[i] = at
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[i]) < 1e-7
    gu, dh = torch.randn(3, 10, generator=g).double() * 3, torch.randn(3, 5, generator=g).double()
    dgu = ref.swiglu_gradient(gu, dh)[0]
    for i in range(gu.numel()):
        v = [gu.clone(), gu.clone()]
        v[0].view(-1)[i] += h
        v[1].view(-1)[i] -= h
        diff = sum(sign * (dh * ref.swiglu(u)[0]).sum() for sign, u in ((1, v[0]), (-1, v[1]))) / (2 * h)
        assert abs(diff - dgu.view(-1)[i]) < 1e-7


def test_layer_orders_its_buffers_with_the_streams(monkeypatch):
    """With stand-ins for the GPU: making a layer waits for the current stream, and a step on a stream that did not make it
    records every buffer for that stream, once."""
    import contextlib
    import types

    from routed_expert_ffn_wave_amd import products
    made, waits, used = [], [], []

    class Buffer(torch.Tensor):
        def record_stream(self, stream):
            used.append((id(self), stream.cuda_stream))

    def new(shape, dtype, dev, stream=None):
        made.append(torch.zeros(shape).to(dtype).as_subclass(Buffer))
        return made[-1]

    streams = {n: types.SimpleNamespace(cuda_stream=n, device_index=0, synchronize=lambda n=n: waits.append(n)) for n in (1, 2, 3)}
    current = [1]
    monkeypatch.setattr(products, "_new", new)
    monkeypatch.setattr(products, "_first", lambda t, name, dims, dtypes, stream=None: (0, t.shape))
    monkeypatch.setattr(products, "_take", lambda t, name, dtypes, shape, dev: t.data_ptr())
    monkeypatch.setattr(products, "_run", lambda *a: None)
    monkeypatch.setattr(products, "_raw_stream", lambda dev: current[0])
    for name in ("ft_moe_dispatch", "ft_moe_dispatch_grad", "ft_moe_combine_grad", "ft_moe_grouped_matmul", "ft_moe_grouped_matmul_grad",
                 "ft_moe_grouped_matmul_wgrad", "ft_moe_swiglu", "ft_moe_swiglu_grad"):
        monkeypatch.setattr(products, name, lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: streams[current[0]])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s).to(dtype)  # noqa: E731
    layer = products.Bf16MoELayer(z(2, 64, 64), z(2, 64, 32), torch.zeros(4, dtype=torch.int32), k=2, T=4)
    assert waits == [1] and sorted(id(b) for b in layer._buffers) == sorted(id(b) for b in made)
    args = (torch.zeros(4, 4), z(4, 64))
    layer.forward(*args)
    layer.backward(z(4, 64))
    assert used == []
    layer.forward(*args, stream=streams[2])
    assert sorted(used) == sorted((id(b), 2) for b in made)
    layer.backward(z(4, 64), stream=streams[2])
    current[0] = 3
    layer.backward(z(4, 64))
    layer.forward(*args)
    assert sorted(used) == sorted((id(b), n) for b in made for n in (2, 3))
    assert waits == [1]
    with pytest.raises(ft.FtError, match="the stream is of cuda:1"):
        layer.forward(*args, stream=types.SimpleNamespace(cuda_stream=9, device_index=1))


class StandInGpu:
    """Stand-ins for the GPU under a Bf16MoELayer: what it allocates (filled with `fill`), which streams it records its buffers for; a
    call named in `fails` raises."""

    def __init__(self, monkeypatch, fill=0.0):
        import contextlib
        import types

        from routed_expert_ffn_wave_amd import products
        self.made, self.used, self.fails = [], [], ()
        gpu = self

        class Buffer(torch.Tensor):
            def record_stream(self, stream):
                gpu.used.append((id(self), stream.cuda_stream))

        def new(shape, dtype, dev, stream=None):
            gpu.made.append(torch.full(shape, fill).to(dtype).as_subclass(Buffer))
            return gpu.made[-1]

        def call(name):
            def stub(*a, **k):
                if name in gpu.fails:
                    raise ft.FtError(ft.FT_E_UNSUPPORTED, name)
            return stub

        self.streams = {n: types.SimpleNamespace(cuda_stream=n, device_index=0, synchronize=lambda: None) for n in (1, 2)}
        monkeypatch.setattr(products, "_new", new)
        monkeypatch.setattr(products, "_first", lambda t, name, dims, dtypes, stream=None: (0, t.shape))
        monkeypatch.setattr(products, "_take", lambda t, name, dtypes, shape, dev: t.data_ptr())
        monkeypatch.setattr(products, "_run", lambda *a: None)
        monkeypatch.setattr(products, "_raw_stream", lambda dev: 1)
        for name in ("ft_moe_dispatch", "ft_moe_dispatch_grad", "ft_moe_combine_grad", "ft_moe_grouped_matmul", "ft_moe_grouped_matmul_grad",
                     "ft_moe_grouped_matmul_wgrad", "ft_moe_swiglu", "ft_moe_swiglu_grad"):
            monkeypatch.setattr(products, name, call(name))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: self.streams[1])
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())

    def layer(self, slot=None):
        bf = torch.bfloat16
        return ft.Bf16MoELayer(torch.zeros(4, 64, 64, dtype=bf), torch.zeros(4, 64, 32, dtype=bf), slot, k=2, T=4)


STEP = (torch.zeros(4, 4), torch.zeros(4, 64, dtype=torch.bfloat16))  # logits, x


def test_layer_keeps_its_own_table_for_the_streams(monkeypatch):
    """A layer that makes the slot table itself records that too for the streams it runs on: its kernels read it there."""
    gpu = StandInGpu(monkeypatch)
    layer = gpu.layer()
    assert torch.equal(layer.slot_of, torch.arange(4).int()) and layer.slot_of.dtype == torch.int32
    layer.forward(*STEP, stream=gpu.streams[2])
    assert (id(layer.slot_of), 2) in gpu.used
    assert sorted(gpu.used) == sorted((id(b), 2) for b in gpu.made)


def test_layer_gradients_start_from_zeros(monkeypatch):
    """A first backward(add=True) adds to zeros, and experts without a slot have zeros as long as nobody writes others."""
    layer = StandInGpu(monkeypatch, fill=7.0).layer(torch.tensor([0, -1, 1, 2]).int())
    assert not layer.dw13.any() and not layer.dw2.any()


def test_layer_refuses_backward_after_a_forward_that_failed(monkeypatch):
    """A forward() that raised on its way leaves buffers of two steps: backward() refuses until another has run."""
    gpu = StandInGpu(monkeypatch)
    layer, dout = gpu.layer(), STEP[1]
    layer.forward(*STEP)
    layer.backward(dout)
    gpu.fails = ("ft_moe_swiglu",)
    with pytest.raises(ft.FtError, match="ft_moe_swiglu"):
        layer.forward(*STEP)
    gpu.fails = ()
    with pytest.raises(ft.FtError, match="needs a forward"):
        layer.backward(dout)
    layer.forward(*STEP)
    layer.backward(dout)
