"""Row calls on the GPU against their definitions in 64 bits (rows_ref.py holds the references and derives the
bounds)."""
import pytest
import torch

import routed_expert_ffn_wave_amd as ft
import rows_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
FILL = 7.0  # what rows that a call leaves alone hold


def gen(seed):
    return torch.Generator().manual_seed(seed)


def filled(*shape, dtype):
    return torch.full(shape, FILL, device="cuda").to(dtype)


def same_bits(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------------------------------------- 8-bit rows

def check_rows(codes, scales, x, exact, slack=None):
    """codes / scales of rows x (fp64).  exact: bit for bit; else a code may be the other neighbour of a
    quotient that lies within its own error (slack, relative) of a border between two codes."""
    q, s = ref.quotients(x)
    nb = s.shape[1]
    got = codes.cpu().double()
    assert torch.equal(scales[:, nb:].cpu(), torch.zeros(x.shape[0], scales.shape[1] - nb))
    if exact:
        assert torch.equal(scales[:, :nb].cpu(), s.float())
        assert torch.equal(got, ref.e4m3_nearest(q))
        return
    slack = slack if torch.is_tensor(slack) else torch.full_like(q, slack)
    worst = torch.stack([slack[:, 128 * b: 128 * b + 128].amax(1) for b in range(nb)], 1)
    assert ((scales[:, :nb].cpu().double() - s).abs() <= (worst + 2 * ref.U32) * s).all()
    err = q.abs() * (slack + worst.repeat_interleave(128, 1)[:, : q.shape[1]] + 4 * ref.U32)
    assert ((got - q).abs() <= ref.e4m3_step((q.abs() + err).clamp(max=448)) / 2 + err).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, K", [(1, 16), (3, 48), (5, 128), (2, 144), (7, 512), (1, 528), (33, 768), (64, 2000), (9, 7168)])
def test_quant(rows, K, dtype):
    x = (torch.randn(rows, K, generator=gen(rows * K)) * torch.logspace(-6, 6, K)).to(dtype)
    codes, scales = ft.ft_moe_quant_fp8(x.cuda())
    assert codes.dtype == E4 and codes.shape == (rows, K) and scales.shape == (rows, ref.cols(K))
    check_rows(codes, scales, x.double(), dtype == BF, 3 * ref.U32)


def test_quant_every_bf16_magnitude_and_borders():
    """Every finite bf16 pattern beside several block maxima: quotients on borders, subnormals, the largest values."""
    every = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    every = every[torch.isfinite(every.float())]
    for top in (1.0, 1.7578125, 448.0, 3.3895313892515355e38, 2.0 ** -90, 2.0 ** -120, 2.0 ** -133):
        v = every[every.float().abs() <= top]
        v = torch.nn.functional.pad(v, (0, -v.numel() % 127))
        x = torch.cat([v.view(-1, 127), torch.full((v.numel() // 127, 1), top).to(BF)], 1)
        codes, scales = ft.ft_moe_quant_fp8(x.cuda())
        check_rows(codes, scales, x.double(), True)


def test_quant_special_blocks():
    x = torch.randn(6, 256, generator=gen(1)).to(BF)
    x[0, :128] = 0
    x[1, 5], x[2, 130], x[3, 200] = float("nan"), float("inf"), -float("inf")
    x[4, :128] = 2.0 ** -130
    codes, scales = ft.ft_moe_quant_fp8(x.cuda())
    bad = torch.zeros(6, 2, dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = bad[3, 1] = True
    assert torch.equal(torch.isnan(scales[:, :2]).cpu(), bad)
    assert torch.equal(torch.isnan(codes.float()).cpu(), bad.repeat_interleave(128, 1))
    x[1, :128] = 0
    x[2:4, 128:] = 0
    q, s = ref.quotients(x.double())
    keep = ~bad
    assert torch.equal(scales[:, :2].cpu()[keep], s.float()[keep])
    wide = keep.repeat_interleave(128, 1)
    assert torch.equal(codes.cpu().double()[wide], ref.e4m3_nearest(q)[wide])


@pytest.mark.parametrize("rows, I", [(1, 16), (5, 144), (17, 768), (130, 2048)])
def test_swiglu(rows, I):
    gu = (torch.randn(rows, 2 * I, generator=gen(I)) * 3).to(BF)
    gu[0, 0], gu[0, I] = -200.0, 3.0  # e^200 is infinite in fp32: the product is 0
    codes, scales = ft.ft_moe_swiglu_fp8(gu.cuda())
    g, u = gu.double().chunk(2, 1)
    # the exponent's argument is off by |g| log2(e) roundings, its power and the reciprocal by two units, the sum and
    # the two products by a rounding each
    slack = (g.abs() + 10) * ref.U32
    h = g * torch.sigmoid(g) * u
    h[0, 0] = 0
    check_rows(codes, scales, h, False, slack)


# ---------------------------------------------------------------------------------------------- dispatch

PAIRS = [(1, 1, 1, None), (1, 8, 8, None), (3, 4, 2, 2), (16, 256, 8, 96), (65, 40, 9, 17), (200, 1024, 32, 500), (37, 5, 3, 0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [8, 120, 2048, 2056, 7168])
@pytest.mark.parametrize("T, E, k, held", PAIRS)
def test_dispatch_and_gradient(T, E, k, held, d, dtype):
    g = gen(T * E + d)
    r = ref.routing(g, T, E, k, held)
    rows = ref.pair_rows(r["ids"], r["inv"], E, r["slot"])
    x = torch.randn(T, d, generator=g).to(dtype)
    dev = {n: v.cuda() for n, v in r.items()}
    xs = ft.ft_moe_dispatch(x.cuda(), dev["ids"], dev["inv"], slot_of_expert=dev["slot"], x_sorted=filled(T * k, d, dtype=dtype))
    want = torch.full((T * k, d), FILL).to(dtype)
    has = rows >= 0
    want[rows[has]] = x[:, None, :].expand(T, k, d)[has]
    assert same_bits(xs, want)
    dxs = torch.randn(T * k, d, generator=g).to(dtype)
    none = torch.ones(T * k, dtype=torch.bool)
    none[rows[has]] = False
    dxs[none] = float("nan")  # rows that belong to no pair are not read into a sum
    dx = ft.ft_moe_dispatch_grad(dxs.cuda(), dev["ids"], dev["inv"], slot_of_expert=dev["slot"]).cpu()
    assert dx.dtype == dtype
    terms = torch.where(has[:, :, None], dxs.double()[rows.clamp(min=0)], torch.zeros((), dtype=torch.float64))
    total, mag = terms.sum(1), terms.abs().sum(1)
    bound = k * ref.U32 * mag + (ref.UBF * total.abs() if dtype == BF else 0)
    assert ((dx.double() - total).abs() <= bound).all()


def test_dispatch_without_a_slot_table_and_with_bad_tables():
    g = gen(5)
    T, E, k, d = 20, 6, 3, 64
    r = ref.routing(g, T, E, k)
    ids, inv = r["ids"].clone(), r["inv"].clone()
    ids[0, 1], ids[3, 0], ids[4, 2] = -1, E, 2 ** 31 - 1
    inv[5, 0], inv[6, 1], inv[7, 2] = -1, T * k, -(2 ** 31)
    rows = ref.pair_rows(ids, inv, E)
    has = rows >= 0
    assert int((~has).sum()) == 6
    x, dxs = torch.randn(T, d, generator=g).to(BF), torch.randn(T * k, d, generator=g).to(BF)
    xs = ft.ft_moe_dispatch(x.cuda(), ids.cuda(), inv.cuda(), E=E, x_sorted=filled(T * k, d, dtype=BF))
    want = torch.full((T * k, d), FILL).to(BF)
    want[rows[has]] = x[:, None, :].expand(T, k, d)[has]
    assert same_bits(xs, want)
    dx = ft.ft_moe_dispatch_grad(dxs.cuda(), ids.cuda(), inv.cuda().view(-1), E=E).cpu().double()
    terms = torch.where(has[:, :, None], dxs.double()[rows.clamp(min=0)], torch.zeros((), dtype=torch.float64))
    assert ((dx - terms.sum(1)).abs() <= k * ref.U32 * terms.abs().sum(1) + ref.UBF * terms.sum(1).abs()).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T, E, k, held, d", [(1, 8, 8, None, 16), (16, 256, 8, 96, 7168), (65, 40, 9, 17, 768), (50, 64, 32, 40, 528)])
def test_dispatch_fp8_is_quant_of_the_sorted_rows(T, E, k, held, d, dtype):
    g = gen(T + d)
    r = {n: v.cuda() for n, v in ref.routing(g, T, E, k, held).items()}
    x = torch.randn(T, d, generator=g).to(dtype).cuda()
    c0, s0 = filled(T * k, d, dtype=E4), filled(T * k, ref.cols(d), dtype=F32)
    codes, scales = ft.ft_moe_dispatch_fp8(x, r["ids"], r["inv"], slot_of_expert=r["slot"], codes=c0.clone(), scales=s0.clone())
    xc, xscale = ft.ft_moe_quant_fp8(x)
    rows = ref.pair_rows(r["ids"].cpu(), r["inv"].cpu(), E, r["slot"].cpu()).cuda()
    has = rows >= 0
    t = torch.arange(T, device="cuda")[:, None].expand(T, k)[has]
    c0.view(torch.uint8)[rows[has]] = xc.view(torch.uint8)[t]
    s0[rows[has]] = xscale[t]
    assert same_bits(codes, c0) and same_bits(scales, s0)


# ---------------------------------------------------------------------------------------------- combine gradient

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [8, 264, 2048, 7168])
@pytest.mark.parametrize("T, E, k, held", PAIRS)
def test_combine_gradient(T, E, k, held, d, dtype):
    g = gen(T + E + d)
    r = ref.routing(g, T, E, k, held)
    rows = ref.pair_rows(r["ids"], r["inv"], E, r["slot"])
    has = rows >= 0
    dout, y = torch.randn(T, d, generator=g).to(dtype), torch.randn(T * k, d, generator=g).to(BF)
    none = torch.ones(T * k, dtype=torch.bool)
    none[rows[has]] = False
    clean = y.clone()
    y[none] = float("nan")
    dev = {n: v.cuda() for n, v in r.items()}
    dy, dw, dl = ft.ft_moe_combine_grad(dout.cuda(), y.cuda(), dev["ids"], dev["w"], dev["inv"], slot_of_expert=dev["slot"],
                                        dy_sorted=filled(T * k, d, dtype=BF))
    want = torch.full((T * k, d), FILL).to(BF)
    want[rows[has]] = (r["w"][:, :, None] * dout.float()[:, None, :]).to(BF)[has]  # one fp32 product, one rounding
    assert same_bits(dy, want)
    rdw, mag, rdl = ref.combine_grad(dout, clean, r["w"], rows, r["ids"], E)
    # a thread adds d / 2048 pieces of 8 products in turn, then 6 + 2 additions across lanes and waves
    e_dw = (8 * ((d + 2047) // 2048) + 8) * ref.U32 * mag
    assert ((dw.cpu().double() - rdw).abs() <= e_dw).all()
    w = r["w"].double()
    size = (w * rdw.abs()).sum(1, keepdim=True)
    e_dl = w * (e_dw + (w * e_dw).sum(1, keepdim=True) + 10 * ref.U32 * (rdw.abs() + size))
    e_all = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, r["ids"].long(), e_dl)
    assert ((dl.cpu().double() - rdl).abs() <= e_all).all()


def test_combine_gradient_repeated_and_bad_ids_and_no_logits():
    """The same expert twice in one token adds up; ids outside [0, E) have no row and no logit."""
    g = gen(9)
    T, E, k, d = 6, 5, 4, 32
    ids = torch.randint(0, E, (T, k), generator=g).int()
    ids[0] = 2
    ids[1, 0], ids[2, 3] = -1, E
    inv = torch.randperm(T * k, generator=g).int().view(T, k)
    w = torch.rand(T, k, generator=g)
    dout, y = torch.randn(T, d, generator=g), torch.randn(T * k, d, generator=g).to(BF)
    rows = ref.pair_rows(ids, inv, E)
    rdw, mag, rdl = ref.combine_grad(dout, y, w, rows, ids, E)
    args = (dout.cuda(), y.cuda(), ids.cuda(), w.cuda(), inv.cuda())
    dy, dw, dl = ft.ft_moe_combine_grad(*args, E=E)
    assert ((dw.cpu().double() - rdw).abs() <= 16 * ref.U32 * mag).all()
    assert (dl.cpu().double() - rdl).abs().max() <= 64 * ref.U32 * k * mag.max()
    assert torch.equal(dw.cpu()[rows < 0], torch.zeros(2))
    dy2, dw2, none = ft.ft_moe_combine_grad(*args, E=E, want_dlogits=False)
    assert none is None and same_bits(dw, dw2)
    has = rows[rows >= 0].cuda()
    assert same_bits(dy[has], dy2[has])


def test_gradients_against_differences_of_the_library():
    """dlogits and dx against differences of the library's own forward: loss = sum(dout * combine(y)), and
    y = dispatch(x) with identity experts.  The loss is an fp32 result of about 64 terms (error e), the third
    derivative of a softmax weight is below 1, so a central difference of step h is off by at most e / h + h^2 mag."""
    g = gen(11)
    T, E, k, d, h = 4, 8, 3, 64, 2.0 ** -6
    logits = torch.randn(T, E, generator=g)
    x, dout = torch.randn(T, d, generator=g).to(BF).cuda(), torch.randn(T, d, generator=g).cuda()
    scale = torch.linspace(0.5, 2.0, E).cuda()  # expert e multiplies its rows by scale[e]

    def forward(z, grads=False):
        ids, w = ft.ft_moe_route(z.cuda(), k)
        _, off, gather, inv = ft.ft_moe_permute(ids, E)
        xs = ft.ft_moe_dispatch(x, ids, inv, E=E)
        factor = scale[ids.view(-1)[gather.long()].long()][:, None]
        y = (xs.float() * factor).to(BF)
        slot = torch.arange(E, dtype=torch.int32, device="cuda")
        out, _ = ft.ft_moe_combine(y, None, ids, w, inv, slot, d)
        if not grads:
            return (out.double() * dout.double()).sum(1).cpu(), ids.cpu()
        dy, dw, dl = ft.ft_moe_combine_grad(dout, y, ids, w, inv, E=E)
        dx = ft.ft_moe_dispatch_grad((dy.float() * factor).to(BF), ids, inv, E=E)
        return dl.cpu(), dx.cpu(), w, ids.cpu(), factor, inv

    dl, dx, w, ids0, factor, inv = forward(logits, grads=True)
    mag = (x.float().abs() * dout.abs()).sum(1).cpu().double() * 2
    for e in range(E):
        z = [logits.clone(), logits.clone()]
        z[0][:, e] += h
        z[1][:, e] -= h
        (up, iu), (down, idn) = forward(z[0]), forward(z[1])
        for t in range(T):
            if set(iu[t].tolist()) == set(idn[t].tolist()) == set(ids0[t].tolist()):
                tol = (2 * 16 * ref.U32 / h + h * h + ref.UBF * 0) * mag[t]
                # y is the same on both sides (bf16 roundings of x only): only fp32 sums differ
                assert abs((up[t] - down[t]) / (2 * h) - dl[t, e]) <= tol
    # x: out is linear in x with factor sum_j w_j scale_j
    rows = inv.view(T, k).long()
    per = (w * factor[:, 0][rows]).sum(1).cpu().double()
    want = per[:, None] * dout.cpu().double()
    # two bf16 roundings a term and one of the sum
    size = (w * factor[:, 0][rows]).sum(1).cpu().double()[:, None] * dout.cpu().double().abs()
    assert ((dx.double() - want).abs() <= 3.1 * ref.UBF * size).all()


# ---------------------------------------------------------------------------------------------- products

SHAPES = [(1, 1, 16), (1, 16, 128), (1, 130, 2048), (2, 100, 48), (15, 33, 112), (16, 128, 144), (17, 64, 256), (33, 250, 528),
          (64, 256, 768), (65, 129, 2000), (128, 384, 512), (200, 520, 1040), (257, 300, 640), (300, 1536, 2048), (515, 1023, 272),
          (17, 4100, 144), (40, 4096, 1040), (33, 7168, 144), (90, 4096, 400), (700, 4100, 400), (1100, 4096, 144),
          (2050, 4097, 272), (1800, 4104, 528)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_product(M, N, K, dtype):
    g = gen(M + N + K)
    a, sa = ref.random_rows(g, M, K)
    w, sw = ref.random_weights(g, N, K)
    out = ft.ft_moe_fp8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), out_dtype=dtype)
    want, mag = ref.product(a, sa, w, sw)
    assert out.dtype == dtype
    assert ((out.cpu().double() - want).abs() <= ref.product_bound(want, mag, K, dtype == BF)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_of_any_codes(M, dtype):
    """Codes over e4m3's whole range, and NaN codes and scales that reach only their own rows and columns."""
    g = gen(M)
    N, K = 140, 272
    pick = lambda *s: torch.randint(0, 127, s, generator=g).to(torch.uint8) | (torch.randint(0, 2, s, generator=g) << 7).to(torch.uint8)  # noqa: E731
    a, w = pick(M, K).view(E4), pick(N, K).view(E4)
    _, sa = ref.random_rows(g, M, K)
    _, sw = ref.random_weights(g, N, K)
    want, mag = ref.product(a, sa, w, sw)
    a.view(torch.uint8)[1, K - 1] = 0x7F
    w.view(torch.uint8)[N - 1, 3] = 0xFF
    sa[2, 1] = float("nan")
    out = ft.ft_moe_fp8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), out_dtype=dtype).cpu().double()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[1] = bad[2] = True
    bad[:, N - 1] = True
    assert torch.equal(torch.isnan(out), bad)
    assert ((out - want).abs() <= ref.product_bound(want, mag, K, dtype == BF))[~bad].all()


GROUPS = [(1, 1, 1, None, 16, 16), (1, 8, 8, 3, 130, 144), (16, 256, 8, 96, 256, 512), (40, 12, 4, 7, 100, 272),
          (300, 16, 4, 11, 264, 256), (700, 6, 2, 5, 384, 768), (37, 5, 3, 0, 64, 64), (6, 24, 2, 20, 520, 4112),
          (64, 32, 8, 32, 1536, 768), (400, 16, 4, 16, 1032, 144), (1500, 16, 4, 12, 1040, 144), (900, 6, 3, 6, 2056, 272), (3000, 4, 4, 4, 2056, 144)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T, E, k, held, N, K", GROUPS)
def test_grouped_product(T, E, k, held, N, K, dtype):
    g = gen(T * E + N)
    r = ref.routing(g, T, E, k, held)
    P, n = T * k, max(1, E if held is None else held)
    a, sa = ref.random_rows(g, P, K)
    w, sw = ref.random_weights(g, n, N, K)
    out = ft.ft_moe_fp8_grouped_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), r["offsets"].cuda(), r["slot"].cuda(),
                                       out=filled(P, N, dtype=dtype)).cpu().double()
    for e in range(E):
        r0, r1, s = int(r["offsets"][e]), int(r["offsets"][e + 1]), int(r["slot"][e])
        if s < 0:
            assert (out[r0:r1] == FILL).all()
        elif r1 > r0:
            want, mag = ref.product(a[r0:r1], sa[r0:r1], w[s], sw[s])
            assert ((out[r0:r1] - want).abs() <= ref.product_bound(want, mag, K, dtype == BF)).all()


@pytest.mark.parametrize("P", [5, 90, 700])
def test_grouped_product_of_odd_tables(P):
    """Slots outside the bank, rows of no expert, and offsets past the rows are left alone or clipped."""
    g = gen(P)
    E, n, N, K = 6, 3, 72, 160
    a, sa = ref.random_rows(g, P, K)
    w, sw = ref.random_weights(g, n, N, K)
    cut = P // 5
    offsets = torch.tensor([-3, cut, cut, 2 * cut, 3 * cut, 4 * cut, P + 50], dtype=torch.int32)
    slot = torch.tensor([2, 1, 0, n, -7, 1], dtype=torch.int32)
    out = ft.ft_moe_fp8_grouped_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), offsets.cuda(), slot.cuda(),
                                       out=filled(P, N, dtype=F32)).cpu().double()
    for lo, hi, s in ((0, cut, 2), (cut, 2 * cut, 0), (2 * cut, 4 * cut, None), (4 * cut, P, 1)):
        if s is None:
            assert (out[lo:hi] == FILL).all()
        else:
            want, mag = ref.product(a[lo:hi], sa[lo:hi], w[s], sw[s])
            assert ((out[lo:hi] - want).abs() <= ref.product_bound(want, mag, K, False)).all()
    short = torch.tensor([2] * 4 + [4, 4, 4], dtype=torch.int32)  # rows 0, 1 and from 4 on belong to nobody
    out = ft.ft_moe_fp8_grouped_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), short.cuda(),
                                       torch.tensor([0, 0, 0, 2, 0, 0], dtype=torch.int32).cuda(), out=filled(P, N, dtype=F32)).cpu().double()
    want, mag = ref.product(a[2:4], sa[2:4], w[2], sw[2])
    assert ((out[2:4] - want).abs() <= ref.product_bound(want, mag, K, False)).all()
    assert (out[:2] == FILL).all() and (out[4:] == FILL).all()


@pytest.mark.parametrize("M", [1, 70, 400])
def test_products_repeat_bit_for_bit(M):
    g = gen(M)
    a, sa = (v.cuda() for v in ref.random_rows(g, M, 1040))
    w, sw = (v.cuda() for v in ref.random_weights(g, 520, 1040))
    first = ft.ft_moe_fp8_matmul(a, sa, w, sw)
    for _ in range(5):
        assert same_bits(ft.ft_moe_fp8_matmul(a, sa, w, sw), first)


def test_offsets_past_32_bits():
    """A bank and a row array of more than 4 GiB: the last slot and the last rows are reached."""
    g = gen(2)
    N, K, n = 4096, 7168, 150
    w = torch.zeros(n, N, K, dtype=torch.uint8, device="cuda").view(E4)
    last, slast = ref.random_weights(g, 256, K)
    w.view(torch.uint8)[n - 1, :256] = last.view(torch.uint8).cuda()
    sw = torch.ones(n, N // 128, K // 128, device="cuda")
    sw[n - 1, :2] = slast.cuda()
    a, sa = ref.random_rows(g, 20, K)
    off = torch.tensor([0, 0, 20], dtype=torch.int32).cuda()
    out = ft.ft_moe_fp8_grouped_matmul(a.cuda(), sa.cuda(), w, sw, off, torch.tensor([0, n - 1], dtype=torch.int32).cuda(), out_dtype=F32)
    want, mag = ref.product(a, sa, last, slast)
    assert ((out[:, :256].cpu().double() - want).abs() <= ref.product_bound(want, mag, K, False)).all()
    del w
    T, k, d = 90000, 4, 7168  # 5.2 GB of sorted rows
    x = torch.randn(T, d, device="cuda").to(BF)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).view(T, k)
    xs = ft.ft_moe_dispatch(x, ids, inv, E=32)
    at = inv.long()
    for t in (0, 1, 44999, T - 1):
        assert all(same_bits(xs[at[t, j]], x[t]) for j in range(k))
    dx = ft.ft_moe_dispatch_grad(xs, ids, inv, E=32)
    assert same_bits(dx[:3], (4 * x[:3].float()).to(BF)) and same_bits(dx[-3:], (4 * x[-3:].float()).to(BF))
    codes, scales = ft.ft_moe_dispatch_fp8(x, ids, inv, E=32)
    c, s = ft.ft_moe_quant_fp8(x)
    for t in (0, T - 1):
        assert all(same_bits(codes[at[t, j]], c[t]) and same_bits(scales[at[t, j]], s[t]) for j in range(k))
    # M K past 2^32 codes: the last rows of a dense product
    w, sw = (v.cuda() for v in ref.random_weights(g, 16, d))
    M = T * k * 2
    big = torch.zeros(M, d, dtype=torch.uint8, device="cuda").view(E4)
    sbig = torch.zeros(M, ref.cols(d), device="cuda")
    big.view(torch.uint8)[M - 20:] = a.view(torch.uint8).cuda()
    sbig[M - 20:] = sa.cuda()
    out = ft.ft_moe_fp8_matmul(big, sbig, w, sw, out_dtype=F32)
    want, mag = ref.product(a, sa, w.cpu(), sw.cpu())
    assert ((out[M - 20:].cpu().double() - want).abs() <= ref.product_bound(want, mag, d, False)).all()
    assert (out[: M - 20] == 0).all()


# ---------------------------------------------------------------------------------------------- the run of them

def layer_inputs(seed, T, E, k, d, I, held):
    g = gen(seed)
    w13, s13 = ref.random_weights(g, held, 2 * I, d)
    w2, s2 = ref.random_weights(g, held, d, I)
    r = ref.routing(g, T, E, k, held)
    return [v.cuda() for v in (w13, s13 / d ** 0.5, w2, s2 / I ** 0.5, r["slot"], r["logits"], torch.randn(T, d, generator=g).to(BF))]


@pytest.mark.parametrize("T, E, k, d, I, held, out_bf16", [(1, 8, 2, 256, 128, 8, False), (16, 32, 8, 512, 384, 20, True),
                                                          (300, 16, 4, 384, 256, 16, False), (33, 64, 6, 144, 80, 50, False)])
def test_layer_on_8_bit_rows(T, E, k, d, I, held, out_bf16):
    """Every step of the layer against its definition, each on the previous step's own results."""
    w13, s13, w2, s2, slot, logits, x = layer_inputs(T, T, E, k, d, I, held)
    layer = ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T, out_bf16=out_bf16)
    out, mask = layer.forward(logits, x)
    torch.cuda.synchronize()
    ids, w, inv, off = layer.ids.cpu(), layer.w.cpu(), layer.inv.cpu().view(T, k), layer.offsets.cpu()
    rows = ref.pair_rows(ids, inv, E, slot.cpu())
    has = rows >= 0
    assert torch.equal(mask.cpu().long(), sum(((~has[:, j]).long() << j) for j in range(k)))
    c, s = ft.ft_moe_quant_fp8(x)
    t = torch.arange(T)[:, None].expand(T, k)[has]
    assert same_bits(layer.x8.view(torch.uint8)[rows[has].cuda()], c.view(torch.uint8)[t.cuda()])
    for e in range(E):
        r0, r1, sl = int(off[e]), int(off[e + 1]), int(slot[e])
        if sl < 0 or r1 == r0:
            continue
        want, mag = ref.product(layer.x8[r0:r1].cpu(), layer.xs[r0:r1].cpu(), w13[sl].cpu(), s13[sl].cpu())
        assert ((layer.gu[r0:r1].cpu().double() - want).abs() <= ref.product_bound(want, mag, d, True)).all()
        g, u = layer.gu[r0:r1].cpu().double().chunk(2, 1)
        check_rows(layer.h8[r0:r1], layer.hs[r0:r1], g * torch.sigmoid(g) * u, False, (g.abs() + 10) * ref.U32)
        want, mag = ref.product(layer.h8[r0:r1].cpu(), layer.hs[r0:r1].cpu(), w2[sl].cpu(), s2[sl].cpu())
        assert ((layer.y_sorted[r0:r1].cpu().double() - want).abs() <= ref.product_bound(want, mag, I, True)).all()
    terms = torch.where(has[:, :, None], w.double()[:, :, None] * layer.y_sorted.cpu().double()[rows.clamp(min=0)],
                        torch.zeros((), dtype=torch.float64))
    bound = (k + 1) * ref.U32 * terms.abs().sum(1) + (ref.UBF * terms.sum(1).abs() if out_bf16 else 0)
    assert ((out.cpu().double() - terms.sum(1)).abs() <= bound).all()


def test_layer_close_to_the_unquantised_layer():
    """Against the 64-bit layer on the same weights without quantised activations: an e4m3 code is off by at most 2^-4 of its
    value (uniformly: 2^-4 / sqrt(3)), independently per value, in x and in h; the norm of the error stays
    under twice one such rounding."""
    T, E, k, d, I = 40, 8, 2, 512, 256
    w13, s13, w2, s2, slot, logits, x = layer_inputs(7, T, E, k, d, I, E)
    layer = ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T)
    out = layer.forward(logits, x)[0].cpu().double()
    want = torch.zeros(T, d, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            sl = int(slot[layer.ids[t, j]])
            a = ref.weight_values(w13[sl].cpu(), s13[sl].cpu()) @ x[t].cpu().double()
            h = a[:I] * torch.sigmoid(a[:I]) * a[I:]
            want[t] += layer.w[t, j].cpu().double() * (ref.weight_values(w2[sl].cpu(), s2[sl].cpu()) @ h)
    assert (out - want).norm() <= 2 * 2.0 ** -4 * want.norm()


def capture(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    return graph


@pytest.mark.parametrize("T", [4, 260])
def test_graph_replays_match_eager_calls(T):
    """A serving step and a training step's gradients, captured once and replayed between eager work on new inputs."""
    E, k, d, I = 16, 4, 256, 128
    w13, s13, w2, s2, slot, logits, x = layer_inputs(T, T, E, k, d, I, 12)
    layer, eager = (ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T) for _ in range(2))
    dout = torch.randn(T, d, device="cuda")
    bufs = [dict(dy_sorted=torch.zeros(T * k, d, dtype=BF, device="cuda"), dw=torch.zeros(T, k, device="cuda"),
                 dlogits=torch.zeros(T, E, device="cuda")) for _ in range(2)]
    dx = [torch.zeros(T, d, dtype=BF, device="cuda") for _ in range(2)]

    def step(i, ly):
        ly.forward(logits, x)
        inv = ly.inv.view(T, k)
        ft.ft_moe_combine_grad(dout, ly.y_sorted, ly.ids, ly.w, inv, slot_of_expert=slot, **bufs[i])
        ft.ft_moe_dispatch_grad(bufs[i]["dy_sorted"], ly.ids, inv, slot_of_expert=slot, dx=dx[i])

    graph = capture(lambda: step(0, layer))
    for n in range(4):
        x.copy_(torch.randn(T, d, device="cuda"))
        logits.copy_(torch.randn(T, E, device="cuda"))
        dout.copy_(torch.randn(T, d, device="cuda"))
        for b in bufs:
            b["dy_sorted"].zero_()
        torch.cuda.synchronize()
        graph.replay()
        step(1, eager)
        torch.cuda.synchronize()
        assert same_bits(layer.out, eager.out) and same_bits(dx[0], dx[1])
        assert all(same_bits(bufs[0][m], bufs[1][m]) for m in bufs[0])


def test_two_streams_at_once():
    """Calls on two streams, from tensors made on a third, do not disturb each other."""
    g = gen(4)
    jobs = []
    for M in (5, 300):
        a, sa = (v.cuda() for v in ref.random_rows(g, M, 2048))
        w, sw = (v.cuda() for v in ref.random_weights(g, 1024, 2048))
        x = torch.randn(M, 2048, generator=g).to(BF).cuda()
        jobs.append((a, sa, w, sw, x, ft.ft_moe_fp8_matmul(a, sa, w, sw), ft.ft_moe_quant_fp8(x)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[] for _ in jobs]
    for _ in range(20):
        for i, (a, sa, w, sw, x, _, _) in enumerate(jobs):
            out = torch.zeros(a.shape[0], 1024, dtype=BF, device="cuda")
            streams[i].wait_stream(torch.cuda.current_stream())
            ft.ft_moe_fp8_matmul(a, sa, w, sw, out=out, stream=streams[i])
            with torch.cuda.stream(streams[i]):
                q = ft.ft_moe_quant_fp8(x)
            outs[i].append((out, q))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for out, (c, s) in outs[i]:
            assert same_bits(out, job[5]) and same_bits(c, job[6][0]) and same_bits(s, job[6][1])


def test_empty_calls_and_refused_tensors():
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    assert ft.ft_moe_quant_fp8(z(0, 64))[0].shape == (0, 64)
    assert ft.ft_moe_dispatch(z(0, 64), z(0, 2, dtype=i32), z(0, 2, dtype=i32), E=4).shape == (0, 64)
    assert ft.ft_moe_combine_grad(z(0, 64), z(0, 64), z(0, 2, dtype=i32), z(0, 2, dtype=F32), z(0, 2, dtype=i32), E=4)[2].shape == (0, 4)
    assert ft.ft_moe_fp8_matmul(z(0, 64, dtype=E4), z(0, 4, dtype=F32), z(8, 64, dtype=E4), z(1, 1, dtype=F32)).shape == (0, 8)
    x, ids = z(4, 64), z(4, 2, dtype=i32)
    a, sa, w, sw = z(4, 64, dtype=E4), z(4, 4, dtype=F32), z(8, 64, dtype=E4), z(1, 1, dtype=F32)
    for call in (lambda: ft.ft_moe_quant_fp8(x.half()), lambda: ft.ft_moe_quant_fp8(x.t()), lambda: ft.ft_moe_quant_fp8(z(4, 60)),
                 lambda: ft.ft_moe_quant_fp8(x, codes=z(4, 32, dtype=E4)), lambda: ft.ft_moe_quant_fp8(x, scales=z(4, 1, dtype=F32)),
                 lambda: ft.ft_moe_quant_fp8(z(4, 128)[:, :64]), lambda: ft.ft_moe_swiglu_fp8(z(4, 33)),
                 lambda: ft.ft_moe_dispatch(x, ids.long(), ids, E=4), lambda: ft.ft_moe_dispatch(x, ids, ids),
                 lambda: ft.ft_moe_dispatch(x, ids, ids[:2], E=4), lambda: ft.ft_moe_dispatch(x, ids, ids.cpu(), E=4),
                 lambda: ft.ft_moe_dispatch(x, ids, ids, E=4, slot_of_expert=z(5, dtype=i32)),
                 lambda: ft.ft_moe_dispatch_grad(x, ids, ids, E=4), lambda: ft.ft_moe_combine_grad(x, x, ids, x, ids, E=4),
                 lambda: ft.ft_moe_fp8_matmul(a, sa[:, :1].contiguous(), w, sw), lambda: ft.ft_moe_fp8_matmul(a, sa, w[:, :32].contiguous(), sw),
                 lambda: ft.ft_moe_fp8_matmul(a, sa, w, sw, out_dtype=torch.float16),
                 lambda: ft.ft_moe_fp8_grouped_matmul(a, sa, w[None], sw[None], ids.view(-1), z(4, dtype=i32))):
        with pytest.raises(ft.FtError):
            call()


# tables of 1024 experts take 16 KiB of the LDS that the largest tiles would need
MANY = [(40, 1024, 8, 700, 96, 4112), (1500, 1024, 8, 1024, 264, 144), (16000, 1024, 4, 1024, 200, 144), (16000, 1024, 8, 1000, 200, 144)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T, E, k, held, N, K", MANY)
def test_grouped_product_of_many_experts(T, E, k, held, N, K, dtype):
    g = gen(T + E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(256)]).repeat((T + 255) // 256, 1)[:T]
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(ids.reshape(-1), minlength=E).cumsum(0)
    slot = torch.full((E,), -1, dtype=torch.int32)
    slot[torch.randperm(E, generator=g)[:held]] = torch.randperm(held, generator=g).to(torch.int32)
    P = T * k
    a, sa = ref.random_rows(g, P, K)
    w, sw = ref.random_weights(g, held, N, K)
    out = ft.ft_moe_fp8_grouped_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), offsets.cuda(), slot.cuda(),
                                       out=filled(P, N, dtype=dtype)).cpu().double()
    for e in range(0, E, 1 if P < 20000 else 29):
        r0, r1, s = int(offsets[e]), int(offsets[e + 1]), int(slot[e])
        if s < 0:
            assert (out[r0:r1] == FILL).all()
        elif r1 > r0:
            want, mag = ref.product(a[r0:r1], sa[r0:r1], w[s], sw[s])
            assert ((out[r0:r1] - want).abs() <= ref.product_bound(want, mag, K, dtype == BF)).all()


@pytest.mark.parametrize("P, N, K", [(50, 64, 4112), (600, 200, 144), (3000, 600, 144)])
def test_grouped_product_of_a_table_that_does_not_ascend(P, N, K):
    """Every second expert has all rows: a row holds the result of one of them."""
    g = gen(P)
    E, n = 6, 3
    a, sa = ref.random_rows(g, P, K)
    w, sw = ref.random_weights(g, n, N, K)
    offsets = torch.tensor([0, P, 0, P, 0, P, 0], dtype=torch.int32)
    slot = torch.tensor([0, 0, 1, 0, 2, 0], dtype=torch.int32)
    out = ft.ft_moe_fp8_grouped_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), offsets.cuda(), slot.cuda(), out_dtype=F32).cpu().double()
    near = torch.zeros(P, N, dtype=torch.bool)
    for s in range(n):
        want, mag = ref.product(a, sa, w[s], sw[s])
        near |= (out - want).abs() <= ref.product_bound(want, mag, K, False)
    assert near.all()


def test_streams_of_another_gpu_are_refused():
    import types
    other = types.SimpleNamespace(device_index=1, cuda_stream=0)
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    x, ids, i1 = z(4, 64), z(4, 2, dtype=torch.int32), z(1, dtype=torch.int32)
    a, sa, w, sw = z(4, 64, dtype=E4), z(4, 4, dtype=F32), z(64, 64, dtype=E4), z(1, 1, dtype=F32)
    layer = ft.Fp8MoELayer(z(1, 64, 64, dtype=E4), z(1, 1, 1, dtype=F32), z(1, 64, 32, dtype=E4), z(1, 1, 1, dtype=F32), i1, 1, 4)
    for call in (lambda: ft.ft_moe_quant_fp8(x, stream=other), lambda: ft.ft_moe_swiglu_fp8(x, stream=other),
                 lambda: ft.ft_moe_dispatch(x, ids, ids, E=4, stream=other), lambda: ft.ft_moe_dispatch_fp8(x, ids, ids, E=4, stream=other),
                 lambda: ft.ft_moe_dispatch_grad(z(8, 64), ids, ids, E=4, stream=other),
                 lambda: ft.ft_moe_combine_grad(x, z(8, 64), ids, z(4, 2, dtype=F32), ids, E=4, stream=other),
                 lambda: ft.ft_moe_fp8_matmul(a, sa, w, sw, stream=other),
                 lambda: ft.ft_moe_fp8_grouped_matmul(a, sa, w[None], sw[None], z(2, dtype=torch.int32), i1, stream=other),
                 lambda: layer.forward(z(4, 1, dtype=F32), x, stream=other)):
        with pytest.raises(ft.FtError, match="stream"):
            call()


def test_outputs_made_for_another_stream_wait_for_nobody():
    """Outputs of a call on a side stream come from that stream's memory: work of the current stream that still
    writes a freed tensor of the same size cannot reach them."""
    g = gen(6)
    M, K = 2048, 2048
    x = torch.randn(M, K, generator=g).to(BF).cuda()
    want = ft.ft_moe_quant_fp8(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        busy = torch.randn(4096, 4096, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            busy = busy @ busy * 1e-3
        late = [torch.full((M, K), 1, dtype=torch.uint8, device="cuda"), torch.full((M, ref.cols(K)), 2.0, device="cuda")]
        del late
        got = ft.ft_moe_quant_fp8(x, stream=side)
        torch.cuda.synchronize()
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])


# sizes where blocks share K between groups of waves: shares of no, one and several blocks, with and without a short one
SHARED = [(400, 4100, 16), (400, 4100, 128), (400, 4100, 144), (390, 4100, 256), (400, 4100, 400), (400, 4090, 1040), (1000, 4096, 16),
          (1000, 4096, 272), (970, 4090, 384), (1000, 4096, 656)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, N, K", SHARED)
def test_product_with_shares_of_k(M, N, K, dtype):
    test_product(M, N, K, dtype)


@pytest.mark.parametrize("P, N, K", [(3, 128, 256), (90, 272, 400), (700, 1040, 528)])
def test_gradient_of_the_rows_is_the_product_with_the_transposed_matrix(P, N, K):
    """For out = rows . w^T and a gradient in 8-bit rows g: d rows = g . w, dense and by expert, against the formula's own
    gradient and against differences (out is linear: exact up to the products' roundings)."""
    g = gen(P + N)
    E = 3
    w, sw = ref.random_weights(g, E, N, K)
    wt, swt = w.view(torch.uint8).transpose(1, 2).contiguous().view(E4), sw.transpose(1, 2).contiguous()
    dout, sd = ref.random_rows(g, P, N)
    cut = P // 3
    offsets = torch.tensor([0, cut, cut, P], dtype=torch.int32)
    slot = torch.tensor([2, 1, 0], dtype=torch.int32)
    dense = ft.ft_moe_fp8_matmul(dout.cuda(), sd.cuda(), wt[1].cuda(), swt[1].cuda(), out_dtype=F32).cpu().double()
    by = ft.ft_moe_fp8_grouped_matmul(dout.cuda(), sd.cuda(), wt.cuda(), swt.cuda(), offsets.cuda(), slot.cuda(), out_dtype=F32).cpu().double()
    a, sa = ref.random_rows(g, P, K)
    dy = ref.values(dout, sd)
    for got, parts in ((dense, [(0, P, 1)]), (by, [(0, cut, 2), (cut, P, 0)])):
        for lo, hi, s in parts:
            if lo == hi:
                continue
            x = ref.values(a[lo:hi], sa[lo:hi]).requires_grad_()
            y = ref.weight_values(w[s], sw[s])
            ((x @ y.t()) * dy[lo:hi]).sum().backward()
            want, mag = ref.product(dout[lo:hi], sd[lo:hi], wt[s], swt[s])
            bound = ref.product_bound(want, mag, N, False)
            assert ((got[lo:hi] - x.grad).abs() <= bound).all()
            # differences between these rows and others
            b, sb = ref.random_rows(g, hi - lo, K)
            up, mu = ref.product(b, sb, w[s], sw[s])
            dn, md = ref.product(a[lo:hi], sa[lo:hi], w[s], sw[s])
            o = [ft.ft_moe_fp8_matmul(c.cuda(), sc.cuda(), w[s].cuda(), sw[s].cuda(), out_dtype=F32).cpu().double()
                 for c, sc in ((b, sb), (a[lo:hi].contiguous(), sa[lo:hi].contiguous()))]
            step = ref.values(b, sb) - x.detach()
            slack = ((ref.product_bound(up, mu, K, False) + ref.product_bound(dn, md, K, False)) * dy[lo:hi].abs()).sum(1)
            lhs, rhs = ((o[0] - o[1]) * dy[lo:hi]).sum(1), (got[lo:hi] * step).sum(1)
            assert ((lhs - rhs).abs() <= slack + (bound * step.abs()).sum(1)).all()


def test_refusals_before_anything_is_allocated():
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    x, ids = z(4, 64), z(4, 2, dtype=torch.int32)
    for E in (0, -1):
        with pytest.raises(ft.FtError, match="E must be"):
            ft.ft_moe_combine_grad(x, z(8, 64), ids, z(4, 2, dtype=F32), ids, E=E)

    def layer(d=64, I=32, E=4, k=2, T=4, n=2):
        nb = lambda v: (v + 127) // 128  # noqa: E731
        return ft.Fp8MoELayer(z(n, 2 * I, d, dtype=E4), z(n, nb(2 * I), nb(d), dtype=F32), z(n, d, I, dtype=E4), z(n, nb(d), nb(I), dtype=F32),
                              z(E, dtype=torch.int32), k, T)

    layer()
    for kw in (dict(d=24), dict(I=8), dict(E=1025), dict(k=5), dict(k=0), dict(T=-1), dict(n=0), dict(d=0), dict(E=64, k=33)):
        with pytest.raises(ft.FtError, match="invalid layer shape"):
            layer(**kw)


def test_sparse_tensors_are_refused():
    x = torch.ones(4, 64, device="cuda").to(BF)
    with pytest.raises(ft.FtError, match="must be"):
        ft.ft_moe_quant_fp8(x.to_sparse())
    with pytest.raises(ft.FtError, match="must be"):
        ft.ft_moe_quant_fp8(x, scales=torch.ones(4, 4, device="cuda").to_sparse())


# ---------------------------------------------------------------------------------------------- slots past the bank

def past_the_bank(slot, n):
    """The same table with entries at and past the bank's n slots in place of some, and with -1 there."""
    past, none = slot.clone(), slot.clone()
    held = torch.nonzero(slot >= 0)[:, 0]
    for e, v in zip(held[:3].tolist(), (n, n + 5, 2 ** 31 - 1)):
        past[e], none[e] = v, -1
    return past, none


@pytest.mark.parametrize("T, out_bf16", [(1, False), (40, True), (300, False)])
def test_layer_with_slots_past_the_bank(T, out_bf16):
    """They count as not resident in every step: the rows that the products leave alone reach no output, and the pair
    is left to the residual mask."""
    E, k, d, I, held = 8, 4, 256, 128, 6
    w13, s13, w2, s2, slot, logits, x = layer_inputs(T, T, E, k, d, I, held)
    got = []
    for table in past_the_bank(slot.cpu(), held):
        layer = ft.Fp8MoELayer(w13, s13, w2, s2, table.cuda(), k, T, out_bf16=out_bf16)
        for b in (layer.gu, layer.y_sorted):
            b.fill_(float("nan"))
        got.append([v.clone() for v in layer.forward(logits, x)])
    assert torch.isfinite(got[0][0].float()).all()
    assert same_bits(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pair_calls_with_slots_past_the_bank(dtype):
    g = gen(21)
    T, E, k, d, held = 30, 9, 4, 272, 6
    r = ref.routing(g, T, E, k, held)
    past, none = past_the_bank(r["slot"], held)
    rows = ref.pair_rows(r["ids"], r["inv"], E, none)
    away = torch.ones(T * k, dtype=torch.bool)
    away[rows[rows >= 0]] = False
    x, dout = torch.randn(T, d, generator=g).to(dtype).cuda(), torch.randn(T, d, generator=g).to(dtype).cuda()
    y, dxs = torch.randn(T * k, d, generator=g).to(BF), torch.randn(T * k, d, generator=g).to(dtype)
    y[away], dxs[away] = float("nan"), float("nan")
    y, dxs, ids, inv, w = y.cuda(), dxs.cuda(), r["ids"].cuda(), r["inv"].cuda(), r["w"].cuda()
    got = []
    for table, kw in ((past.cuda(), dict(n_slots=held)), (none.cuda(), {})):
        kw["slot_of_expert"] = table
        out = [ft.ft_moe_dispatch(x, ids, inv, x_sorted=filled(T * k, d, dtype=dtype), **kw)]
        out += ft.ft_moe_dispatch_fp8(x, ids, inv, codes=filled(T * k, d, dtype=E4), scales=filled(T * k, ref.cols(d), dtype=F32), **kw)
        out += [ft.ft_moe_dispatch_grad(dxs, ids, inv, **kw)]
        out += ft.ft_moe_combine_grad(dout, y, ids, w, inv, dy_sorted=filled(T * k, d, dtype=BF), **kw)
        out += ft.ft_moe_combine(y, None, ids, w, inv, table, d, flags=ft.FT_N_SLOTS(held) if "n_slots" in kw else 0)
        got.append(out)
    assert torch.isfinite(got[0][3].float()).all() and torch.isfinite(got[0][5]).all() and torch.isfinite(got[0][6]).all()
    assert all(same_bits(a, b) for a, b in zip(*got))


def test_four_calls_with_slots_past_the_bank():
    """MoELayer's two modes agree on such a table."""
    import synth
    from gpu_util import device_bank
    w = synth.Workload("slots_past_the_bank", 93, T=16, d=256, E=8, k=4, I=128, fmt=synth.FMT_BF16)
    li = synth.layer_inputs(w, layer=0, T=16)
    bank = device_bank(li.bank)
    past, none = past_the_bank(li.slot_of_expert.cpu(), li.bank.n_slots)
    got = []
    for table in (past, none):
        layer = ft.MoELayer(bank, table.cuda(), w.k, 16, mode="calls")
        layer.y_sorted.fill_(float("nan"))
        got.append([v.clone() for v in layer.forward(li.logits.cuda(), li.x.cuda())])
    assert torch.isfinite(got[0][0]).all()
    assert same_bits(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---------------------------------------------------------------------------------------------- the layer's buffers and streams

def zeroed_copies(layer):
    """Tensors of the buffers' sizes, zeroed on the current stream (zeros are harmless tables)."""
    return [torch.zeros_like(b.view(torch.uint8)) for b in layer._buffers]


def long_work():
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(8):
        busy = busy @ busy * 1e-3


def test_layer_made_while_its_stream_is_busy():
    """Work that still writes freed tensors of the buffers' sizes does not reach a forward() on another stream."""
    T, E, k, d, I = 64, 8, 4, 256, 128
    w13, s13, w2, s2, slot, logits, x = layer_inputs(5, T, E, k, d, I, E)
    first = ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T)
    want = first.forward(logits, x)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for use in (lambda ly: ly.forward(logits, x, stream=side), None):
        long_work()
        late = zeroed_copies(first)
        del late
        layer = ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T)
        if use:
            out, _ = use(layer)
        else:
            with torch.cuda.stream(side):
                out, _ = layer.forward(logits, x)
        torch.cuda.synchronize()
        assert same_bits(out, want)


def test_layer_freed_while_another_stream_uses_it():
    """Tensors made on the constructing stream after the layer is gone do not overwrite what a forward() on another
    stream still works on."""
    T, E, k, d, I = 64, 8, 4, 256, 128
    w13, s13, w2, s2, slot, logits, x = layer_inputs(6, T, E, k, d, I, E)
    first = ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T)
    want = first.forward(logits, x)[0].clone()
    side = torch.cuda.Stream()
    for given in (True, False):
        layer = ft.Fp8MoELayer(w13, s13, w2, s2, slot, k, T)
        with torch.cuda.stream(side):
            long_work()
            out = (layer.forward(logits, x, stream=side) if given else layer.forward(logits, x))[0]
        del layer
        over = zeroed_copies(first)
        torch.cuda.synchronize()
        assert same_bits(out, want)
        del over
