"""Product calls on the GPU against their definitions in 64 bits (products_ref.py holds the references and derives the
bounds)."""
import pytest
import torch

import products_ref as ref
import routed_expert_ffn_wave_amd as ft
import rows_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FILL = 7.0  # what a call leaves alone holds
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def filled(*shape, dtype):
    return torch.full(shape, FILL, device="cuda").to(dtype)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(BF)


def same_bits(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def dev(t):
    return None if t is None else t.cuda()


def sizes(g, E, P, empty=0.3):
    """Offsets of E experts with P rows in all, some without any and some with most."""
    cuts = torch.randint(0, P + 1, (E - 1,), generator=g)
    cuts[torch.rand(E - 1, generator=g) < empty] = 0
    return torch.cat([torch.zeros(1), torch.sort(cuts)[0], torch.full((1,), P)]).int()


def check_forward(a, w, off, slot, dtype, grad):
    """grad: the rows' gradient, a being dout [P][N]."""
    P = a.shape[0]
    wt = w.transpose(1, 2).contiguous() if grad else w
    has, want, mag = ref.forward(torch.nan_to_num(a), wt, off, slot, None)
    a = a.clone()
    a[~has] = NAN  # rows of experts without a matrix are not read into a result
    out = filled(P, wt.shape[1], dtype=dtype)
    call = ft.ft_moe_grouped_matmul_grad if grad else ft.ft_moe_grouped_matmul
    kw = {"da": out} if grad else {"out": out}
    got = call(a.cuda(), w.cuda(), off.cuda(), slot_of_expert=dev(slot), **kw)
    assert got is out and torch.equal(out[~has.cuda()].cpu(), torch.full((int((~has).sum()), wt.shape[1]), FILL).to(dtype))
    err = (out.cpu().double() - want).abs()[has]
    assert (err <= ref.sum_bound(want, mag, a.shape[1], dtype)[has]).all(), err.max()


# P, E, held (None: no table), N, K
GROUPS = [(1, 1, None, 8, 8), (3, 4, 2, 16, 24), (8, 128, 128, 72, 64), (17, 5, 3, 136, 72), (64, 2, 2, 128, 128), (129, 3, 3, 264, 200),
          (300, 7, None, 520, 136), (333, 64, 40, 256, 520), (700, 9, 6, 1032, 776), (2000, 16, 16, 384, 1160), (5000, 4, 4, 1544, 328),
          (16, 256, 96, 64, 2056), (1500, 1024, 700, 40, 48)]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P, E, held, N, K", GROUPS)
def test_grouped_product(P, E, held, N, K, dtype, grad):
    g = gen(P * E + N)
    slot = None if held is None else rows_ref.routing(g, 0, E, 1, held)["slot"]
    w = normal(g, E if held is None else held, N, K)
    check_forward(normal(g, P, N if grad else K), w, sizes(g, E, P), slot, dtype, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("P", [1, 5, 90, 700])
def test_grouped_product_of_odd_tables(P, grad):
    """Slots past the bank and below -1, a matrix that three experts share, offsets below 0 and past P."""
    g = gen(P)
    E, N, K = 12, 72, 152
    off = sizes(g, E, P, 0.0)
    off[0], off[-1] = -5, P + 1000
    slot = torch.tensor([0, 3, 3, -1, 5, 4, -2 ** 31, 2 ** 31 - 1, 1, 3, 2, 0]).int()  # of 5
    check_forward(normal(g, P, N if grad else K), normal(g, 5, N, K), off, slot, BF, grad)


@pytest.mark.parametrize("grad", [False, True])
def test_grouped_product_of_a_table_that_does_not_ascend(grad):
    """Each value of a row that several experts have is the result of one of them."""
    g = gen(3)
    P, E, N, K = 600, 6, 72, 136
    off = torch.tensor([0, 500, 100, 600, 50, 590, 700]).int()
    a, w = normal(g, P, N if grad else K), normal(g, E, N, K)
    call = ft.ft_moe_grouped_matmul_grad if grad else ft.ft_moe_grouped_matmul
    got = call(a.cuda(), w.cuda(), off.cuda(), out_dtype=F32).cpu().double()
    fits = torch.zeros(got.shape, dtype=torch.bool)
    for e, r0, r1, s in ref.groups(off, None, E, P, E):
        y = w[s].double() if grad else w[s].double().t()
        want, mag = a[r0:r1].double() @ y, a[r0:r1].double().abs() @ y.abs()
        fits[r0:r1] |= (got[r0:r1] - want).abs() <= ref.sum_bound(want, mag, a.shape[1], F32)
    assert fits.all()


@pytest.mark.parametrize("grad", [False, True])
def test_many_tiles_of_a_table_that_does_not_ascend(grad):
    g = gen(9)
    P, E, cols, red = 3000, 40, 4104, 40
    off = torch.randint(-100, P + 200, (E + 1,), generator=g).int()
    off[::2] = off[::2] // 4
    a, w = normal(g, P, red), normal(g, E, *((red, cols) if grad else (cols, red)))
    got = (ft.ft_moe_grouped_matmul_grad if grad else ft.ft_moe_grouped_matmul)(a.cuda(), w.cuda(), off.cuda(), out_dtype=F32).cpu()
    fits, some = torch.zeros(got.shape, dtype=torch.bool), torch.zeros(P, dtype=torch.bool)
    for e, r0, r1, s in ref.groups(off, None, E, P, E):
        y = w[s].double() if grad else w[s].double().t()
        want, mag = a[r0:r1].double() @ y, a[r0:r1].double().abs() @ y.abs()
        fits[r0:r1] |= (got[r0:r1].double() - want).abs() <= ref.sum_bound(want, mag, red, F32)
        some[r0:r1] = True
    assert some.sum() > P // 2 and fits[some].all()


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("P", [6, 200])
def test_special_values_stay_in_their_rows(P, grad):
    """A NaN or an infinity in a row shows in that row only, one in a matrix in its expert's column only; the reduction's
    ragged end (not a multiple of 64) adds nothing to them."""
    g = gen(P)
    E, N, K = 3, 88, 104
    off = torch.tensor([0, P // 3, P // 3, P]).int()
    a, w = normal(g, P, N if grad else K), normal(g, E, N, K)
    a[1, 5], a[P - 1, 70] = NAN, float("inf")
    w[2, N - 1, 3] = -float("inf")
    call = ft.ft_moe_grouped_matmul_grad if grad else ft.ft_moe_grouped_matmul
    got = call(a.cuda(), w.cuda(), off.cuda(), out_dtype=F32).cpu()
    want = torch.zeros_like(got)
    for e, r0, r1, s in ref.groups(off, None, E, P, E):
        y = w[s].double() if grad else w[s].double().t()
        want[r0:r1] = (a[r0:r1].double() @ y).float()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])


@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
@pytest.mark.parametrize("P, E, held, N, K", GROUPS)
def test_matrix_gradient(P, E, held, N, K, kind):
    g = gen(P * E + K)
    slot = None if held is None else rows_ref.routing(g, 0, E, 1, held)["slot"]
    off = sizes(g, E, P)
    dout, a = normal(g, P, N), normal(g, P, K)
    dtype = BF if kind == "bf16" else F32
    has, want, mag, most = ref.matrix_gradient(dout, a, off, slot, E if held is None else held)
    for e in range(E):  # rows of experts that do not count are not read
        if not has[e]:
            dout[off[e]:off[e + 1]], a[off[e]:off[e + 1]] = NAN, NAN
    old = torch.randn(E, N, K, generator=g).to(dtype) if kind == "add" else torch.full((E, N, K), FILL).to(dtype)
    dw = old.cuda()
    got = ft.ft_moe_grouped_matmul_wgrad(dout.cuda(), a.cuda(), off.cuda(), slot_of_expert=dev(slot), dw=dw, add=kind == "add")
    assert got is dw and same_bits(dw[~has.cuda()], old[~has])
    if kind == "add":
        want, mag = want + old.double(), mag + old.double().abs()
    err = (dw.cpu().double() - want).abs()[has]
    assert (err <= ref.sum_bound(want, mag, most + 1, dtype)[has]).all(), err.max()
    if kind == "add":
        none = has & (off[1:] == off[:-1])
        assert same_bits(dw[none.cuda()], old[none])


def test_matrix_gradient_without_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    empty = lambda n: torch.zeros(0, n, dtype=BF, device="cuda")  # noqa: E731
    dw = filled(3, 16, 24, dtype=F32)
    ft.ft_moe_grouped_matmul_wgrad(empty(16), empty(24), off, dw=dw, add=True)
    assert (dw == FILL).all()
    slot = torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda")
    ft.ft_moe_grouped_matmul_wgrad(empty(16), empty(24), off, slot_of_expert=slot, dw=dw, n_slots=4)
    assert (dw[0] == 0).all() and (dw[1:] == FILL).all()


def test_matrix_gradient_keeps_neighbours_apart():
    """The rows before and behind an expert's are other experts': NaN there stays there."""
    g = gen(8)
    off = torch.tensor([0, 3, 70, 71, 200]).int()
    dout, a = normal(g, 200, 40), normal(g, 200, 136)
    dout[:3], a[70], dout[199, 5] = NAN, NAN, NAN
    dw = ft.ft_moe_grouped_matmul_wgrad(dout.cuda(), a.cuda(), off.cuda()).cpu()
    assert torch.isnan(dw[0]).all() and not torch.isnan(dw[1]).any() and torch.isnan(dw[2]).all()
    bad = torch.zeros(40, 136, dtype=torch.bool)
    bad[5] = True
    assert torch.equal(torch.isnan(dw[3]), bad)


def test_offsets_past_32_bits():
    """Rows, matrices, results and gradients whose byte (and value) offsets pass 2^32; checked at the ends."""
    g = torch.Generator(device="cuda").manual_seed(1)
    P, N, K = (1 << 21) + 200, 8, 2056
    a = torch.empty(P, K, dtype=BF, device="cuda").normal_(generator=g)
    w = torch.empty(2, N, K, dtype=BF, device="cuda").normal_(generator=g)
    off = torch.tensor([0, P - 150, P], dtype=torch.int32, device="cuda")
    out = ft.ft_moe_grouped_matmul(a, w, off, out_dtype=F32)
    for s, rows in ((0, slice(0, 3)), (0, slice(P - 153, P - 150)), (1, slice(P - 150, P))):
        x, y = a[rows].cpu().double(), w[s].cpu().double()
        want, mag = x @ y.t(), x.abs() @ y.abs().t()
        assert ((out[rows].cpu().double() - want).abs() <= ref.sum_bound(want, mag, K, F32)).all()
    dout = torch.empty(P, N, dtype=BF, device="cuda").normal_(generator=g)
    da = ft.ft_moe_grouped_matmul_grad(dout, w, off)
    rows = slice(P - 3, P)
    x, y = dout[rows].cpu().double(), w[1].cpu().double()
    assert ((da[rows].cpu().double() - x @ y).abs() <= ref.sum_bound(x @ y, x.abs() @ y.abs(), N, BF)).all()
    dw = ft.ft_moe_grouped_matmul_wgrad(dout, a, off)
    x, y = dout[P - 150:].cpu().double(), a[P - 150:].cpu().double()
    assert ((dw[1].cpu().double() - x.t() @ y).abs() <= ref.sum_bound(x.t() @ y, x.abs().t() @ y.abs(), 150, F32)).all()
    del a, da, out
    n, N, K = 600, 2048, 2056  # 2.5e9 values
    w = torch.empty(n, N, K, dtype=BF, device="cuda")
    w[n - 1].normal_(generator=g)
    a = torch.empty(5, K, dtype=BF, device="cuda").normal_(generator=g)
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    slot = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    out = ft.ft_moe_grouped_matmul(a, w, off, slot_of_expert=slot, out_dtype=F32)
    x, y = a.cpu().double(), w[n - 1].cpu().double()
    assert ((out.cpu().double() - x @ y.t()).abs() <= ref.sum_bound(x @ y.t(), x.abs() @ y.abs().t(), K, F32)).all()
    del w
    off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    off[n] = 5
    dout = torch.empty(5, N, dtype=BF, device="cuda").normal_(generator=g)
    dw = ft.ft_moe_grouped_matmul_wgrad(dout, a, off, out_dtype=BF)
    x, y = dout.cpu().double(), a.cpu().double()
    assert ((dw[n - 1].cpu().double() - x.t() @ y).abs() <= ref.sum_bound(x.t() @ y, x.abs().t() @ y.abs(), 5, BF)).all()
    assert not dw[n - 2].any()


# ---------------------------------------------------------------------------------------------- SwiGLU

ROWS = [(1, 8), (5, 136), (17, 768), (130, 2048), (1000, 264), (3, 7168)]


@pytest.mark.parametrize("rows, I", ROWS)
def test_swiglu_and_gradient(rows, I):
    g = gen(I)
    gu, dh = normal(g, rows, 2 * I, scale=3.0), normal(g, rows, I)
    h = ft.ft_moe_swiglu(gu.cuda())
    want, off = ref.swiglu(gu)
    assert h.dtype == BF and ((h.cpu().double() - want).abs() <= off * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY).all()
    dgu = ft.ft_moe_swiglu_grad(gu.cuda(), dh.cuda())
    want, off = ref.swiglu_gradient(gu, dh)
    assert ((dgu.cpu().double() - want).abs() <= off * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY).all()
    own = gu.cuda()
    assert same_bits(ft.ft_moe_swiglu_grad(own, dh.cuda(), dgu=own), dgu)


def test_swiglu_far_gates_and_special_values():
    g = torch.tensor([-200.0, -95.0, -88.0, -60.0, -1.28125, 0.0, -0.0, 20.0, 90.0, 200.0, 3e38, -3e38]).to(BF)
    u = torch.tensor([3.0, -2.0, 1.5, 0.5]).to(BF)
    gu = torch.cat([g.repeat(4), u.repeat_interleave(12)])[None]
    dh = torch.full((1, 48), 0.75).to(BF)
    for got, (want, off) in ((ft.ft_moe_swiglu(gu.cuda()), ref.swiglu(gu)), (ft.ft_moe_swiglu_grad(gu.cuda(), dh.cuda()), ref.swiglu_gradient(gu, dh))):
        inside = want.abs() < 3e38
        err = (got.cpu().double() - want).abs()
        assert (err <= off * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY)[inside].all()
        assert not torch.isnan(got[:, inside[0].cuda()]).any()
    gu[0, 3], gu[0, 48 + 9] = NAN, NAN
    assert torch.equal(torch.isnan(ft.ft_moe_swiglu(gu.cuda()))[0].nonzero()[:, 0].cpu(), torch.tensor([3, 9]))
    assert torch.isnan(ft.ft_moe_swiglu_grad(gu.cuda(), dh.cuda()))[0].nonzero()[:, 0].tolist() == [3, 9, 51]


# ---------------------------------------------------------------------------------------------- adapters

# T, E, held (None: no table), r, N, K
ADAPTERS = [(1, 1, None, 8, 8, 8), (1, 3, 2, 16, 264, 520), (5, 40, 24, 8, 136, 2056), (16, 16, 16, 16, 4096, 2048), (33, 2, 1, 24, 72, 1032),
            (131, 40, 24, 64, 520, 264), (300, 5, None, 72, 1288, 776), (1000, 3, 2, 128, 256, 136), (70, 1024, 500, 256, 24, 48),
            (2500, 6, 5, 40, 648, 1544)]


def adapter_rows(g, T, E, without=0.2):
    """offsets [E + 1] and gather [T]: rows by adapter, those without one (number E) behind."""
    ids = torch.randint(0, E, (T,), generator=g)
    ids[torch.rand(T, generator=g) < without] = E
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(ids, minlength=E + 1)[:E].cumsum(0)
    return off, torch.sort(ids, stable=True)[1].int()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T, E, held, r, N, K", ADAPTERS)
def test_adapters(T, E, held, r, N, K, dtype):
    g = gen(T + E + r)
    n = E if held is None else held
    slot = None if held is None else rows_ref.routing(g, 0, E, 1, held)["slot"]
    off, gather = adapter_rows(g, T, E)
    base = torch.randn(T, N, generator=g).to(dtype)
    x, a, b = normal(g, T, K), normal(g, n, r, K, scale=K ** -0.5), normal(g, n, N, r)
    scale = torch.rand(n, generator=g) * 2 if E % 2 else None
    want, bound = ref.adapters(base, x, a, b, off, gather, slot, scale)
    args = [dev(t) for t in (base, x, a, b, off, gather)]
    out = ft.ft_moe_lora(*args, slot_of_adapter=dev(slot), scale=dev(scale), out=filled(T, N, dtype=dtype))
    err = (out.cpu().double() - want).abs()
    assert (err <= bound).all(), (err - bound).max()
    bare = (bound == 0).all(1)
    assert same_bits(out[bare.cuda()], base[bare])
    ws = torch.full((max(ft.ft_moe_lora_workspace(T, E, r, N, K), 16),), 255, dtype=torch.uint8, device="cuda")
    again = ft.ft_moe_lora(*args, slot_of_adapter=dev(slot), scale=dev(scale), out=args[0], ws=ws)
    assert again is args[0] and same_bits(again, out)


def test_adapters_with_odd_tables():
    """gather entries outside [0, T), offsets below 0 and past T, slots past the bank: rows that are not named stay."""
    g = gen(2)
    T, E, r, N, K = 60, 4, 16, 40, 72
    off = torch.tensor([-3, 20, 20, 50, 900]).int()
    gather = torch.randperm(T, generator=g).int()
    lost = gather[[4, 25, 55]].long()
    gather[4], gather[25], gather[55] = -1, T, 2 ** 31 - 1
    slot = torch.tensor([1, 0, 7, 0]).int()
    base = torch.randn(T, N, generator=g)
    x, a, b = normal(g, T, K), normal(g, 2, r, K, scale=0.1), normal(g, 2, N, r)
    want, bound = ref.adapters(base, x, a, b, off, gather, slot, None)
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)], slot_of_adapter=slot.cuda(), out=filled(T, N, dtype=F32)).cpu()
    assert (out[lost] == FILL).all()
    rest = torch.ones(T, dtype=torch.bool)
    rest[lost] = False
    assert ((out.double() - want).abs() <= bound)[rest].all()


def test_adapters_special_values_stay_in_their_rows():
    g = gen(4)
    T, E, r, N, K = 40, 3, 8, 72, 136
    off, gather = adapter_rows(g, T, E, 0.0)
    base = torch.randn(T, N, generator=g)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=0.1), normal(g, E, N, r)
    x[7, 3] = NAN
    base[9, 5] = float("inf")
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)]).cpu()
    bad = torch.zeros(T, N, dtype=torch.bool)
    bad[7] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.isinf(out).sum() == 1 and out[9, 5] == float("inf")


@pytest.mark.parametrize("T, E, r, N, K", [(7, 3, 8, 72, 8), (50, 4, 40, 264, 64), (300, 2, 72, 264, 64), (3000, 5, 16, 1288, 136), (200, 3, 256, 64, 32)])
def test_adapters_keep_what_fp32_results_hold(T, E, r, N, K):
    """Short inner sums, whose own error is small beside 2^-16: fp32 results have them whole."""
    g = gen(T + r)
    off, gather = adapter_rows(g, T, E)
    base = torch.zeros(T, N)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=K ** -0.5), normal(g, E, N, r)
    want, bound = ref.adapters(base, x, a, b, off, gather, None, None, left=2.0 ** -24)
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)]).cpu()
    assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("T, E, r, N, K", [(4000, 7, 16, 2056, 1544), (2000, 7, 24, 2056, 1544), (300, 3, 72, 264, 520)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapters_in_two_kernels(T, E, r, N, K, dtype):
    """Hidden rows in memory, for every width of their tiles; an infinite row among them."""
    g = gen(T + r)
    assert ft.ft_moe_lora_workspace(T, E, r, N, K) > 0
    off, gather = adapter_rows(g, T, E)
    base = torch.randn(T, N, generator=g).to(dtype)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=K ** -0.5), normal(g, E, N, r)
    a[:, :, 3], b = a[:, :, 3].abs() + 0.5, b.abs() + 0.5
    want, bound = ref.adapters(base, x, a, b, off, gather, None, None, left=2.0 ** (-24 if dtype is F32 else -16))
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)])
    assert ((out.cpu().double() - want).abs() <= bound).all()
    row = int(gather[T // 3])
    x[row, 3] = float("inf")
    again = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)]).cpu()
    assert (again[row] == float("inf")).all()
    rest = torch.arange(T) != row
    assert same_bits(again[rest], out.cpu()[rest])


@pytest.mark.parametrize("T, r, K", [(40, 8, 136), (40, 56, 136), (900, 40, 520)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapters_of_infinite_rows(T, r, K, dtype):
    """An infinite hidden sum times positive values is infinite, not a NaN; other rows are what they are without it."""
    g = gen(T + r)
    E, N = 3, 72
    off, gather = adapter_rows(g, T, E, 0.0)
    base = torch.randn(T, N, generator=g).to(dtype)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=0.1), normal(g, E, N, r)
    a[:, :, 3], b = a[:, :, 3].abs() + 0.5, b.abs() + 0.5
    plain = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)]).cpu()
    x[7, 3], x[9, 3] = float("inf"), -float("inf")
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)]).cpu()
    assert (out[7] == float("inf")).all() and (out[9] == -float("inf")).all()
    rest = torch.ones(T, dtype=torch.bool)
    rest[[7, 9]] = False
    assert same_bits(out[rest], plain[rest])


# ---------------------------------------------------------------------------------------------- together

def layer_case(seed, T, E, k, d, I, held):
    g = gen(seed)
    n = E if held is None else held
    r = rows_ref.routing(g, T, E, k, held)
    return r, normal(g, T, d), normal(g, n, 2 * I, d, scale=d ** -0.5), normal(g, n, d, I, scale=I ** -0.5), normal(g, T, d)


LAYERS = [(1, 8, 2, 64, 40, None, False), (5, 4, 3, 72, 136, 2, True), (65, 16, 4, 264, 96, 11, False), (400, 8, 8, 128, 264, None, True),
          (900, 40, 5, 520, 328, 33, False)]


@pytest.mark.parametrize("T, E, k, d, I, held, out_bf16", LAYERS)
def test_layer_step_by_step(T, E, k, d, I, held, out_bf16):
    """Every buffer of forward() and backward() against the definition of its step from the buffers before it."""
    r, x, w13, w2, dout = layer_case(T + E, T, E, k, d, I, held)
    slot = None if held is None else r["slot"]
    n = w13.shape[0]
    layer = ft.Bf16MoELayer(w13.cuda(), w2.cuda(), dev(slot), k=k, T=T, out_bf16=out_bf16)
    out, mask = layer.forward(r["logits"].cuda(), x.cuda())
    dx, dl, dw13, dw2 = layer.backward(dout.cuda())
    assert out.dtype == (BF if out_bf16 else F32) and dx.dtype == BF and dw13.dtype == dw2.dtype == F32
    c = {v: getattr(layer, v).cpu() for v in ("ids", "w", "inv", "offsets", "xs", "gu", "h", "y_sorted", "dy", "dh", "dgu", "dxs", "dw")}
    ids, inv, off = c["ids"], c["inv"].view(T, k), c["offsets"]
    rows = rows_ref.pair_rows(ids, inv, E, slot)
    has = rows >= 0
    live = rows[has]
    assert torch.equal(ids, r["ids"])
    assert torch.equal(c["xs"][live], x[:, None, :].expand(T, k, d)[has])

    def close(got, want, bound, at):
        assert ((got.double() - want).abs()[at] <= bound[at]).all()

    def product(name, a, w, grad):
        ok, want, mag = ref.forward(torch.nan_to_num(a), w.transpose(1, 2) if grad else w, off, slot, None)
        assert torch.equal(ok.nonzero()[:, 0], live.sort()[0])
        close(c[name], want, ref.sum_bound(want, mag, a.shape[1], BF), ok)

    product("gu", c["xs"], w13, False)
    want, slack = ref.swiglu(c["gu"])
    close(c["h"], want, slack * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY, live)
    product("y_sorted", c["h"], w2, False)
    y = torch.where(has[:, :, None], c["y_sorted"].double()[rows.clamp(min=0)], torch.zeros((), dtype=torch.float64))
    terms = c["w"].double()[:, :, None] * y
    want = terms.sum(1)
    assert ((out.cpu().double() - want).abs() <= 2 * k * ref.U32 * terms.abs().sum(1) + (ref.UBF * want.abs() if out_bf16 else 0) + ref.TINY).all()
    assert torch.equal(((mask.cpu()[:, None] >> torch.arange(k)) & 1).bool(), ~has)
    # back: the combine's gradient is checked by its own tests
    product("dh", c["dy"], w2, True)
    want, slack = ref.swiglu_gradient(c["gu"], c["dh"])
    close(c["dgu"], want, slack * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY, live)
    product("dxs", c["dgu"], w13, True)
    for got, a, b in ((dw2, "dy", "h"), (dw13, "dgu", "xs")):
        ok, want, mag, most = ref.matrix_gradient(torch.nan_to_num(c[a]), torch.nan_to_num(c[b]), off, slot, n)
        close(got.cpu(), want, ref.sum_bound(want, mag, max(most, 1), F32), ok)
    g = torch.where(has[:, :, None], c["dxs"].double()[rows.clamp(min=0)], torch.zeros((), dtype=torch.float64))
    assert ((dx.cpu().double() - g.sum(1)).abs() <= k * ref.U32 * g.abs().sum(1) + ref.UBF * g.sum(1).abs()).all()


def test_layer_gradients_against_autograd():
    """The whole step against fp64 autograd without roundings.  On the way to a gradient at most six bf16 roundings come
    one after another (gu, h, y or dy, dh, dgu, dx), each within 2^-8 of every value: together they leave less than 6 * 2^-8 of
    a gradient's norm where they do not all point one way; a wrong term leaves a large part of it."""
    T, E, k, d, I = 200, 6, 3, 256, 192
    r, x, w13, w2, dout = layer_case(5, T, E, k, d, I, None)
    layer = ft.Bf16MoELayer(w13.cuda(), w2.cuda(), k=k, T=T)
    out = layer.forward(r["logits"].cuda(), x.cuda())[0].cpu().double()
    got = [t.cpu().double() for t in layer.backward(dout.cuda())]
    leaves = [t.double().requires_grad_() for t in (x, r["logits"], w13, w2)]
    X, L, W13, W2 = leaves
    ids = r["ids"].long()
    w = L.gather(1, ids).softmax(1)
    ffn = []
    for e in range(E):
        gate, up = (X @ W13[e].t()).chunk(2, 1)
        ffn.append((gate * torch.sigmoid(gate) * up) @ W2[e].t())
    want = (w[:, :, None] * torch.stack(ffn, 1).gather(1, ids[:, :, None].expand(T, k, d))).sum(1)
    assert (out - want).norm() <= 3 * ref.UBF * want.norm()
    for mine, theirs in zip(got, torch.autograd.grad((want * dout.double()).sum(), leaves)):
        assert (mine - theirs).norm() <= 6 * ref.UBF * theirs.norm()


def test_layer_without_tokens_and_adding():
    r, x, w13, w2, dout = layer_case(1, 30, 4, 2, 64, 48, 3)
    slot = r["slot"].cuda()
    none = ft.Bf16MoELayer(w13.cuda(), w2.cuda(), slot, k=2, T=0)
    out, mask = none.forward(r["logits"][:0].cuda(), x[:0].cuda())
    assert out.shape == (0, 64) and mask.shape == (0,)
    none.dw13.fill_(FILL)
    dx, dl, dw13, _ = none.backward(dout[:0].cuda(), add=True)
    assert dx.shape == (0, 64) and dl.shape == (0, 4) and (dw13 == FILL).all()
    dw13 = none.backward(dout[:0].cuda())[2]
    assert (dw13[slot >= 0] == 0).all() and (dw13[slot < 0] == FILL).all()
    layer = ft.Bf16MoELayer(w13.cuda(), w2.cuda(), slot, k=2, T=30)
    layer.forward(r["logits"].cuda(), x.cuda())
    once = [t.clone() for t in layer.backward(dout.cuda())]
    again = [t.clone() for t in layer.backward(dout.cuda())]
    held = slot >= 0
    assert all(same_bits(a[held], b[held]) if a.dim() == 3 else same_bits(a, b) for a, b in zip(once, again))
    twice = layer.backward(dout.cuda(), add=True)
    for a, b in zip(once[2:], twice[2:]):
        assert torch.equal(b[held], a[held] * 2)


def capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    return graph, out


def test_layer_refuses_backward_before_forward():
    g = gen(15)
    layer = ft.Bf16MoELayer(normal(g, 4, 32, 64).cuda(), normal(g, 4, 64, 16).cuda(), k=2, T=9)
    dout = normal(g, 9, 64).cuda()
    with pytest.raises(ft.FtError, match="needs a forward"):
        layer.backward(dout)
    layer.forward(torch.randn(9, 4, generator=g).cuda(), normal(g, 9, 64).cuda())
    assert all(torch.isfinite(t).all() for t in layer.backward(dout))


@pytest.mark.parametrize("T", [3, 700])
def test_graph_replays_match_eager_calls(T):
    """A captured training step and a captured adapter call, replayed with other inputs and eager work in between."""
    E, k, d, I, r_, n = 40, 4, 264, 136, 72, 9
    case, x, w13, w2, dout = layer_case(T, T, E, k, d, I, 30)
    slot = case["slot"].cuda()
    layer, eager = (ft.Bf16MoELayer(w13.cuda(), w2.cuda(), slot, k=k, T=T) for _ in range(2))
    g = gen(T)
    off, gather = (t.cuda() for t in adapter_rows(g, T, n))
    a, b = normal(g, n, r_, d, scale=0.1).cuda(), normal(g, n, d, r_).cuda()
    logits, X, D, base = case["logits"].cuda(), x.cuda(), dout.cuda(), torch.zeros(T, d, device="cuda", dtype=BF)
    args = [logits.clone(), X.clone(), D.clone(), base.clone()]

    def step(layer, logits, X, D, base):
        out, mask = layer.forward(logits, X)
        return (out, mask, *layer.backward(D), ft.ft_moe_lora(base, X, a, b, off, gather))

    for m in (layer, eager):
        m.dw13.zero_(), m.dw2.zero_()
    graph, outs = capture(lambda: step(layer, *args))
    for turn in range(4):
        fresh = [torch.randn(t.shape, generator=gen(10 * turn + i)).to(t.dtype).cuda() for i, t in enumerate(args)]
        for t, f in zip(args, fresh):
            t.copy_(f)
        graph.replay()
        got = [t.clone() for t in outs]
        want = step(eager, *fresh)
        torch.cuda.synchronize()
        assert all(same_bits(p, q) for p, q in zip(got, want)), turn


def test_two_streams_at_once():
    """Calls of one kind at the same time on two streams, large ones with workspaces of their own, match calls in turn."""
    g = gen(6)
    E, P, N, K = 128, 3000, 520, 776
    off = sizes(g, E, P).cuda()
    w, a, d = normal(g, E, N, K).cuda(), normal(g, P, K).cuda(), normal(g, P, N).cuda()
    aoff, gather = (t.cuda() for t in adapter_rows(g, P, 7))
    la, lb, base = normal(g, 7, 64, K, scale=0.1).cuda(), normal(g, 7, N, 64).cuda(), torch.randn(P, N, generator=g).cuda()
    assert ft.ft_moe_grouped_matmul_wgrad_workspace(N, K, E) > 0 and ft.ft_moe_lora_workspace(P, 7, 64, N, K) > 0

    def calls():
        return (ft.ft_moe_grouped_matmul(a, w, off), ft.ft_moe_grouped_matmul_grad(d, w, off), ft.ft_moe_grouped_matmul_wgrad(d, a, off),
                ft.ft_moe_lora(base, a, la, lb, aoff, gather))

    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    for outs in got:
        assert all(same_bits(p, q) for p, q in zip(outs, want))


def test_outputs_on_a_given_stream():
    g = gen(7)
    a, w, off = normal(g, 50, 72).cuda(), normal(g, 2, 40, 72).cuda(), torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ft.ft_moe_grouped_matmul(a, w, off, stream=s)
    s.synchronize()
    assert same_bits(got, ft.ft_moe_grouped_matmul(a, w, off))


def test_refused_tensors():
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    off, i32 = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda"), torch.int32
    a, w, d = z(5, 64), z(2, 32, 64), z(5, 32)
    bad = [lambda: ft.ft_moe_grouped_matmul(a.float(), w, off), lambda: ft.ft_moe_grouped_matmul(a.t(), w, off),
           lambda: ft.ft_moe_grouped_matmul(a, w[:, :, :32], off), lambda: ft.ft_moe_grouped_matmul(a, w.float(), off),
           lambda: ft.ft_moe_grouped_matmul(a, w, off.long()), lambda: ft.ft_moe_grouped_matmul(a, w, off[:1]),
           lambda: ft.ft_moe_grouped_matmul(a, w[:1].contiguous(), off), lambda: ft.ft_moe_grouped_matmul(a, w, off, out=z(5, 64)),
           lambda: ft.ft_moe_grouped_matmul(a, w, off, out=z(5, 32, dtype=torch.float16)), lambda: ft.ft_moe_grouped_matmul(a, w, off, out_dtype=torch.float16),
           lambda: ft.ft_moe_grouped_matmul(a, w, off, slot_of_expert=z(3, dtype=i32)), lambda: ft.ft_moe_grouped_matmul(a[:, :60].contiguous(), w[:, :, :60].contiguous(), off),
           lambda: ft.ft_moe_grouped_matmul(a.to_sparse(), w, off), lambda: ft.ft_moe_grouped_matmul(z(6 * 64 + 1)[1:].view(6, 64), w, off),
           lambda: ft.ft_moe_grouped_matmul_grad(a, w, off), lambda: ft.ft_moe_grouped_matmul_wgrad(d, z(4, 64), off),
           lambda: ft.ft_moe_grouped_matmul_wgrad(d, a, off, add=True), lambda: ft.ft_moe_grouped_matmul_wgrad(d, a, off, dw=z(2, 32, 64), add=True),
           lambda: ft.ft_moe_grouped_matmul_wgrad(d, a, off, n_slots=3), lambda: ft.ft_moe_grouped_matmul_wgrad(z(5, 2048), z(5, 2048), torch.zeros(100, dtype=i32, device="cuda"), ws=z(64, dtype=torch.uint8)),
           lambda: ft.ft_moe_swiglu(z(3, 63)), lambda: ft.ft_moe_swiglu(z(3, 24)), lambda: ft.ft_moe_swiglu_grad(z(3, 32), z(3, 32)),
           lambda: ft.ft_moe_swiglu_grad(z(3, 32), z(3, 16, dtype=F32)),
           lambda: ft.ft_moe_lora(d, a, z(2, 8, 64), z(2, 32, 16), off, z(5, dtype=i32)), lambda: ft.ft_moe_lora(d, a, z(2, 4, 64), z(2, 32, 4), off, z(5, dtype=i32)),
           lambda: ft.ft_moe_lora(d, a, z(2, 8, 64), z(2, 32, 8), off, z(4, dtype=i32)), lambda: ft.ft_moe_lora(d, a, z(2, 8, 64), z(2, 32, 8), off, z(5, dtype=i32), scale=z(3, dtype=F32)),
           lambda: ft.ft_moe_lora(d, a, z(2, 8, 64), z(2, 32, 8), off, z(5, dtype=i32), out=z(5, 32, dtype=F32)),
           lambda: ft.ft_moe_lora(d, a, z(2, 8, 64), z(2, 32, 8), off, z(5, dtype=i32), ws=torch.zeros(8)),
           lambda: ft.Bf16MoELayer(z(2, 32, 64), z(2, 64, 8), k=1, T=4), lambda: ft.Bf16MoELayer(z(2, 32, 64), z(2, 64, 16), k=3, T=4)]
    for i, call in enumerate(bad):
        with pytest.raises(ft.FtError):
            call()
            raise AssertionError(i)
    assert ft.ft_moe_grouped_matmul(z(0, 64), w, off).shape == (0, 32) and ft.ft_moe_swiglu(z(0, 32)).shape == (0, 16)
    assert ft.ft_moe_lora(z(0, 32), z(0, 64), z(2, 8, 64), z(2, 32, 8), off, z(0, dtype=i32)).shape == (0, 32)


def test_calls_repeat_bit_for_bit():
    g = gen(12)
    P, E, N, K = 2500, 30, 264, 520
    off = sizes(g, E, P).cuda()
    w, a, d = normal(g, E, N, K).cuda(), normal(g, P, K).cuda(), normal(g, P, N).cuda()
    calls = (lambda: ft.ft_moe_grouped_matmul(a, w, off), lambda: ft.ft_moe_grouped_matmul_grad(d, w, off), lambda: ft.ft_moe_grouped_matmul_wgrad(d, a, off))
    for call in calls:
        first = call()
        for _ in range(3):
            assert same_bits(call(), first)


def test_adapters_beside_an_8_bit_projection():
    """A shared projection on 8-bit rows, the rows' adapters permuted by the library, and the adapters added in place."""
    g = gen(13)
    T, n, r, N, K = 90, 6, 16, 264, 528
    ids = torch.randint(0, n + 1, (T, 1), generator=g).int().cuda()  # n: none
    _, off, gather, _ = ft.ft_moe_permute(ids, n + 1)
    x, w = normal(g, T, K), normal(g, N, K, scale=0.05)
    a, b, scale = normal(g, n, r, K, scale=0.05), normal(g, n, N, r, scale=0.2), torch.rand(n, generator=g)
    codes, scales = ft.ft_moe_quant_fp8(x.cuda())
    wc, ws = rows_ref.random_weights(g, N, K)
    out = ft.ft_moe_fp8_matmul(codes, scales, wc.cuda(), ws.cuda())
    base = out.cpu().clone()
    ft.ft_moe_lora(out, x.cuda(), a.cuda(), b.cuda(), off[: n + 1].contiguous(), gather, scale=scale.cuda(), out=out)
    want, bound = ref.adapters(base, x, a, b, off.cpu()[: n + 1], gather.cpu(), None, scale)
    assert ((out.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("E, P, N, K", [(1024, 90000, 264, 72), (1022, 60000, 520, 136), (128, 40000, 1032, 200), (48, 9000, 520, 448)])
def test_tiles_of_many_experts(E, P, N, K, grad):
    """Tables of experts that leave less LDS to the tiles; groups of every height."""
    g = gen(E)
    check_forward(normal(g, P, N if grad else K), normal(g, E, N, K), sizes(g, E, P), None, BF, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("red", [8, 64, 72, 128, 136, 192, 200, 256, 264, 320, 328])
def test_tiles_of_every_height_and_few_stages(red, grad):
    """Groups of every height of a tile, whole ones and pairs, over reductions of one to six stages, whole and short."""
    counts = torch.tensor([20, 33, 64, 65, 96, 100, 128, 130, 160, 161, 192, 200, 224, 230, 256, 257, 300, 448, 449, 512, 513, 700] * 3)
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int()
    g, cols = gen(red), 1032
    check_forward(normal(g, int(off[-1]), red), normal(g, len(counts), *((red, cols) if grad else (cols, red))), off, None, BF, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("red", [8, 72, 128, 200, 264, 448, 456, 1032])
def test_narrow_tiles(red, grad):
    """Some 60 rows an expert in few tiles, and groups that take several."""
    counts = torch.tensor([17, 64, 65, 0, 100, 128, 129, 200, 257, 1, 30, 64] + [17] * 8)
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int()
    g, cols = gen(red), 1032
    check_forward(normal(g, int(off[-1]), red), normal(g, len(counts), *((red, cols) if grad else (cols, red))), off, None, BF, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("P, low", [(20000, 17), (52000, 1)])
def test_more_tiles_than_a_block_keeps_at_once(P, low, grad):
    """Some 5000 tiles of 1024 experts, of one height in the experts' order, and of all heights by height."""
    g, E, cols, red = gen(P), 1024, 1032, 24
    spare = torch.rand(E, generator=g).pow(2)
    counts = low + ((spare * (P - low * E) / spare.sum()) if low == 1 else torch.ones(E)).long()
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int()
    check_forward(normal(g, int(off[-1]), red), normal(g, E, *((red, cols) if grad else (cols, red))), off, None, BF, grad)


@pytest.mark.parametrize("P, N, K", [(300, 264, 520), (5000, 1032, 2056), (70000, 264, 520)])
def test_planned_matrix_gradient(P, N, K):
    """More tiles than two a compute unit: from queues, with experts of every class of rows, some without a slot."""
    g = gen(P)
    E = 90 if N < 1000 else 20
    cuts = (torch.rand(E - 1, generator=g) ** 4 * P).long().sort()[0]
    off = torch.cat([torch.zeros(1), cuts, torch.full((1,), P)]).int()
    slot = torch.arange(E).int()
    slot[5], slot[11] = -1, E
    dout, a = normal(g, P, N), normal(g, P, K)
    assert ft.ft_moe_grouped_matmul_wgrad_workspace(N, K, E) > 0
    dw = filled(E, N, K, dtype=F32)
    ft.ft_moe_grouped_matmul_wgrad(dout.cuda(), a.cuda(), off.cuda(), slot_of_expert=slot.cuda(), dw=dw, n_slots=E)
    for e in range(E):
        got = dw[e].cpu().double()
        if not 0 <= slot[e] < E:
            assert (got == FILL).all()
            continue
        x, y = dout[off[e]:off[e + 1]].double(), a[off[e]:off[e + 1]].double()
        want, mag = x.t() @ y, x.abs().t() @ y.abs()
        assert ((got - want).abs() <= ref.sum_bound(want, mag, max(x.shape[0], 1), F32)).all(), e


def test_adapters_past_32_bits():
    """Rows of x whose byte offsets pass 2^32, and positions of gather that name them; checked at the ends."""
    g = torch.Generator(device="cuda").manual_seed(2)
    T, r, N, K = (1 << 18) + 77, 8, 16, 8200
    x = torch.empty(T, K, dtype=BF, device="cuda").normal_(generator=g)
    a = torch.empty(2, r, K, dtype=BF, device="cuda").normal_(generator=g) * 0.02
    b = torch.empty(2, N, r, dtype=BF, device="cuda").normal_(generator=g)
    base = torch.empty(T, N, device="cuda").normal_(generator=g)
    gather = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 70, T - 5], dtype=torch.int32, device="cuda")  # the last 70 rows, all but the first 5
    out = ft.ft_moe_lora(base, x, a, b, off, gather)
    assert same_bits(out[:5], base[:5])
    for s, rows in ((0, slice(T - 70, T)), (1, slice(5, 12)), (1, slice(T - 80, T - 70))):
        n = rows.stop - rows.start
        part = torch.tensor([0, n]).int()
        want, bound = ref.adapters(base[rows].cpu(), x[rows].cpu(), a[s:s + 1].cpu(), b[s:s + 1].cpu(), part, torch.arange(n).int(), None, None)
        assert ((out[rows].cpu().double() - want).abs() <= bound).all()


def test_layer_adds_from_the_first_step_on():
    """backward(add=True) of a layer that has run no other: what backward() gives, and zeros for experts without a slot, in
    memory that held other values."""
    r, x, w13, w2, dout = layer_case(4, 60, 6, 2, 136, 72, 4)
    slot = r["slot"].cuda()
    torch.cuda.empty_cache()
    old = [filled(6, n, m, dtype=F32) for n, m in ((144, 136), (136, 72)) for _ in range(3)]
    del old
    adding, plain = (ft.Bf16MoELayer(w13.cuda(), w2.cuda(), slot, k=2, T=60) for _ in range(2))
    outs = []
    for layer, add in ((adding, True), (plain, False)):
        layer.forward(r["logits"].cuda(), x.cuda())
        outs.append(layer.backward(dout.cuda(), add=add)[2:])
    for a, b in zip(*outs):
        assert torch.equal(a, b) and not a[slot < 0].any() and a[slot >= 0].any()


@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
@pytest.mark.parametrize("P, N, K", [(1000, 264, 520), (5000, 1032, 2056), (40000, 264, 520)])
def test_planned_matrix_gradient_of_every_kind(P, N, K, kind):
    """Matrix gradients from queues in both types and added to what is there: experts of one stage to hundreds, whole and
    short last ones, several tiles a block, some experts without rows or without a slot."""
    g = gen(P + N)
    E = 90 if N < 1000 else 20
    cuts = (torch.rand(E - 1, generator=g) ** 4 * P).long().sort()[0]
    cuts[1:4] = cuts[4]  # without rows
    off = torch.cat([torch.zeros(1), cuts, torch.full((1,), P)]).int()
    slot = torch.arange(E).int()
    slot[7], slot[11] = -1, E
    dout, a = normal(g, P, N), normal(g, P, K)
    dtype = BF if kind == "bf16" else F32
    old = torch.randn(E, N, K, generator=g).to(dtype)
    assert ft.ft_moe_grouped_matmul_wgrad_workspace(N, K, E) > 0
    dw = old.cuda()
    ft.ft_moe_grouped_matmul_wgrad(dout.cuda(), a.cuda(), off.cuda(), slot_of_expert=slot.cuda(), dw=dw, n_slots=E, add=kind == "add")
    for e in range(E):
        got = dw[e].cpu().double()
        before = old[e].double()
        if not 0 <= slot[e] < E:
            assert torch.equal(got, before)
            continue
        x, y = dout[off[e]:off[e + 1]].double(), a[off[e]:off[e + 1]].double()
        want, mag = x.t() @ y, x.abs().t() @ y.abs()
        if kind == "add":
            want, mag = want + before, mag + before.abs()
        assert ((got - want).abs() <= ref.sum_bound(want, mag, x.shape[0] + 1, dtype)).all(), e


# T, r, N, K: in one kernel and in two, ranks that end inside 32 and 64 columns
SPECIAL = [(40, 8, 72, 136), (40, 56, 72, 136), (900, 40, 72, 520), (900, 64, 72, 520), (300, 136, 264, 264), (2000, 24, 2056, 1544)]


def special_case(T, r, N, K, dtype):
    """Hidden values of both signs, well away from 0, some of them bf16 values as they are, and a row of zeros."""
    g, E = gen(T + r + K), 3
    off, gather = adapter_rows(g, T, E, 0.1)
    base = torch.randn(T, N, generator=g).to(dtype)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=0.1), normal(g, E, N, r)
    x[::3, 1:], x[::3, 0] = 0, 2.0  # hidden values 2 a[j][0]
    a[:, :, 0] = torch.where(a[:, :, 0] < 0, a[:, :, 0] - 0.5, a[:, :, 0] + 0.5)
    x[6] = 0
    return off, gather, base, x, a, b


def adapter_of_rows(off, gather, T):
    of = torch.full((T,), -1)
    for e in range(off.numel() - 1):
        of[gather[off[e]:off[e + 1]].long()] = e
    return of


@pytest.mark.parametrize("T, r, N, K", SPECIAL)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapters_with_infinite_values_in_b(T, r, N, K, dtype):
    """An infinity in b gives infinities of the hidden value's sign (a NaN where that is 0), a NaN in b NaN, in its column of
    its adapter's rows; every other value is what it is without them."""
    off, gather, base, x, a, b = special_case(T, r, N, K, dtype)
    args = [t.cuda() for t in (base, x, a)]
    tables = (off.cuda(), gather.cuda())
    plain = ft.ft_moe_lora(*args, b.cuda(), *tables).cpu()
    spots = [(0, 3, 1, float("inf")), (0, 71, r - 1, -float("inf")), (1, 0, r // 2, -float("inf")), (2, 40, 2, NAN), (2, 41, r - 2, float("inf"))]
    for e, n, j, v in spots:
        b[e, n, j] = v
    out = ft.ft_moe_lora(*args, b.cuda(), *tables).cpu()
    of, same = adapter_of_rows(off, gather, T), torch.ones(out.shape, dtype=torch.bool)
    for e, n, j, v in spots:
        rows = (of == e).nonzero()[:, 0]
        hid, mag = x[rows].double() @ a[e, j].double(), x[rows].double().abs() @ a[e, j].double().abs()
        sure = (hid.abs() > 2 * K * ref.U32 * mag) | (mag == 0)  # its sign in fp32 is that of fp64
        assert sure.sum() > rows.numel() // 2
        want = (hid * v)[sure].to(dtype)  # the column's other terms and base are finite
        got = out[rows[sure], n]
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])
        same[rows, n] = False
    assert torch.equal(out[same], plain[same])


@pytest.mark.parametrize("T, r, N, K", [(9, 8, 72, 8), (300, 72, 264, 520)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapters_with_hidden_values_past_the_largest_bf16(T, r, N, K, dtype):
    """A hidden value between bf16's largest one and fp32's is finite: so is its product with a small b."""
    top = float(torch.finfo(BF).max)
    x, a = torch.zeros(T, K, dtype=BF), torch.zeros(1, r, K, dtype=BF)
    x[:, 0], x[:, 1] = top, 2.0 ** 119
    a[:, :, 0] = a[:, :, 1] = torch.where(torch.arange(r) % 2 == 0, 1.0, -1.0).to(BF)
    b = torch.zeros(1, N, r, dtype=BF)
    b[:, :, 0], b[:, :, 1] = 2.0 ** -10, 2.0 ** -11
    off, gather, base = torch.tensor([0, T]).int(), torch.arange(T).int(), torch.zeros(T, N).to(dtype)
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)]).cpu().double()
    want, bound = ref.adapters(base, x, a, b, off, gather, None, None)
    assert want.min() > 1e35 and ((out - want).abs() <= bound).all()


@pytest.mark.parametrize("T, r, N, K", SPECIAL)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapters_of_infinite_scales(T, r, N, K, dtype):
    """An infinite scale gives infinities of the outer sum's sign (a NaN where that is 0)."""
    off, gather, base, x, a, b = special_case(T, r, N, K, dtype)
    scale = torch.tensor([float("inf"), 0.75, -float("inf")])
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)], scale=scale.cuda()).cpu()
    of = adapter_of_rows(off, gather, T)
    total, slack = ref.adapters(torch.zeros(base.shape), x, a, b, off, gather, None, None)
    sure = (total.abs() > slack) | (torch.arange(T) == 6)[:, None]  # its sign in fp32 is that of fp64
    for e in (0, 2):
        mine = sure & (of == e)[:, None]
        assert mine.sum() > (of == e).sum() * N // 2
        want, got = (total * scale[e].double())[mine].to(dtype), out[mine]
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])
    rows = of == 1
    want, bound = ref.adapters(base, x, a, b, off, gather, None, scale)
    assert ((out.double() - want).abs() <= bound)[rows].all()


@pytest.mark.parametrize("T, r, N, K", [(60, 16, 40, 72), (1, 8, 8, 8), (900, 40, 72, 520), (300, 72, 264, 520), (4000, 16, 2056, 1544)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_adapters_of_a_table_that_begins_later(T, r, N, K, dtype):
    """Positions before offsets[0], as a table cut to some of the adapters has them, are rows without an adapter."""
    g = gen(T)
    E = 4
    off, gather = adapter_rows(g, T, E)
    base = torch.randn(T, N, generator=g).to(dtype)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=K ** -0.5), normal(g, E, N, r)
    for first, last in ((2, E), (1, 3), (E - 1, E)):
        part = off[first:last + 1].contiguous()
        slot = torch.arange(first, last).int()
        want, bound = ref.adapters(base, x, a, b, part, gather, slot, None)
        args = [t.cuda() for t in (base, x, a, b, part, gather)]
        out = ft.ft_moe_lora(*args, slot_of_adapter=slot.cuda(), out=filled(T, N, dtype=dtype))
        assert ((out.cpu().double() - want).abs() <= bound).all()
        bare = (bound == 0).all(1)
        assert bare[gather[:part[0]].long()].all() and same_bits(out[bare.cuda()], base[bare])
        assert same_bits(ft.ft_moe_lora(*args, slot_of_adapter=slot.cuda(), out=args[0]), out)


@pytest.mark.parametrize("E", [1, 2, 1023, 1024])
def test_adapters_of_tables_of_every_size_with_rows_around(E):
    """Rows before and behind the table's, beside as many groups as there can be."""
    g = gen(E)
    T, r, N, K = E + 40, 8, 24, 64
    off = (torch.arange(E + 1) + 20).int()
    gather = torch.randperm(T, generator=g).int()
    base = torch.randn(T, N, generator=g)
    x, a, b = normal(g, T, K), normal(g, E, r, K, scale=K ** -0.5), normal(g, E, N, r)
    want, bound = ref.adapters(base, x, a, b, off, gather, None, None)
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)], out=filled(T, N, dtype=F32)).cpu()
    assert ((out.double() - want).abs() <= bound).all()


WIDE = 1 << 20  # the most columns


@pytest.mark.parametrize("N, K", [(WIDE, 8), (8, WIDE)])
def test_products_of_the_most_columns(N, K):
    g = gen(N)
    off = torch.tensor([0, 2, 5]).int()
    a, w, d = normal(g, 5, K), normal(g, 2, N, K), normal(g, 5, N)
    for dtype in (BF, F32):
        check_forward(a, w, off, None, dtype, False)
        check_forward(d, w, off, None, dtype, True)
        has, want, mag, most = ref.matrix_gradient(d, a, off, None, 2)
        got = ft.ft_moe_grouped_matmul_wgrad(d.cuda(), a.cuda(), off.cuda(), out_dtype=dtype)
        assert ((got.cpu().double() - want).abs() <= ref.sum_bound(want, mag, most, dtype)).all()


@pytest.mark.parametrize("T, r", [(3, 16), (3, 256), (40, 8)])
@pytest.mark.parametrize("N, K", [(WIDE, 8), (8, WIDE)])
def test_adapters_of_the_most_columns(T, r, N, K):
    g = gen(N + r)
    off, gather = adapter_rows(g, T, 2)
    base, x = torch.randn(T, N, generator=g), normal(g, T, K)
    a, b = normal(g, 2, r, K, scale=K ** -0.5), normal(g, 2, N, r)
    want, bound = ref.adapters(base, x, a, b, off, gather, None, None)
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)])
    assert ((out.cpu().double() - want).abs() <= bound).all()


def test_swiglu_of_the_most_columns():
    g = gen(1)
    gu, dh = normal(g, 2, 2 * WIDE), normal(g, 2, WIDE)
    for got, (want, off) in ((ft.ft_moe_swiglu(gu.cuda()), ref.swiglu(gu)), (ft.ft_moe_swiglu_grad(gu.cuda(), dh.cuda()), ref.swiglu_gradient(gu, dh))):
        assert ((got.cpu().double() - want).abs() <= off * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY).all()


def test_adapters_that_name_rows_twice():
    """A row that gather names twice, in one group or in two, of one adapter, is formed twice with the same result."""
    g = gen(21)
    T, r, N, K = 80, 16, 72, 136
    gather = torch.arange(T).int()
    gather[10], gather[47], gather[79] = 3, 5, 5  # rows 3 and 5 again; 10, 47 and 79 are not named
    off, slot = torch.tensor([0, 40, T]).int(), torch.zeros(2).int()
    base, x = torch.randn(T, N, generator=g), normal(g, T, K)
    a, b = normal(g, 1, r, K, scale=0.1), normal(g, 1, N, r)
    out = ft.ft_moe_lora(*[t.cuda() for t in (base, x, a, b, off, gather)], slot_of_adapter=slot.cuda(), out=filled(T, N, dtype=F32)).cpu()
    want, bound = ref.adapters(base, x, a, b, torch.tensor([0, T]), torch.arange(T).int(), None, None)
    rest = torch.ones(T, dtype=torch.bool)
    rest[[10, 47, 79]] = False
    assert (out[~rest] == FILL).all() and ((out.double() - want).abs() <= bound)[rest].all()
