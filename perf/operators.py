"""Cases of four operators around the expert FFN: rows quantised to 8-bit floating point with a scale
per 128, the matrix product of such rows with 128 x 128 block-scaled weights (dense and grouped by
expert), token rows sorted by expert with their gradient, and the gradient of the weighted combine.

`run` computes a case in plain torch operations, or with `own` through the library's calls."""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # the largest magnitude of a block counts as at least this


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode batch's activations on their way into an 8-bit projection: launch latency
        dict(name="quantise-16", op="quant", form="rows", T=16, d=7168, k=1, E=1, x="bf16", zipf=False),
        # a prompt chunk's rows quantised straight into expert order, popular experts as in the Zipf prefill
        dict(name="sorted-codes-4096", op="quant", form="sorted", T=4096, d=2048, k=8, E=128, x="bf16", zipf=True),
        # gate and up products of a large chunk turned into the down product's rows
        dict(name="swiglu-codes-43541", op="quant", form="swiglu", T=43541, d=2048, k=1, E=1, x="bf16", zipf=False),
        # one token through one matrix: bound by the weights' bytes
        dict(name="product-1", op="product", M=1, N=4096, K=7168, out="bf16"),
        # a short prompt, odd length, 32-bit results
        dict(name="product-77-f32", op="product", M=77, N=7168, K=2048, out="f32"),
        # a long prompt chunk: bound by the matrix cores
        dict(name="product-8192", op="product", M=8192, N=4096, K=7168, out="bf16"),
        # one decode step over the resident experts: a few rows an expert
        dict(name="experts-decode-16", op="experts", T=16, k=8, E=256, slots=96, N=4096, K=7168, zipf=False, out="bf16"),
        # Zipf-routed prefill: groups from none to thousands of rows
        dict(name="experts-prefill-4096", op="experts", T=4096, k=8, E=128, slots=128, N=1536, K=2048, zipf=True, out="bf16"),
        # a training step's rows to their experts
        dict(name="dispatch-4096", op="dispatch", grad=False, T=4096, d=7168, k=8, E=256, x="bf16", zipf=False),
        # and the gradient back, in 32 bits
        dict(name="dispatch-grad-1023", op="dispatch", grad=True, T=1023, d=2048, k=8, E=128, x="f32", zipf=True),
        # the combine's gradient of a training step: rows, weights and router logits
        dict(name="combine-grad-4096", op="combine_grad", T=4096, d=2048, k=8, E=128, dout="bf16", zipf=True),
        # the same for a few tokens: launch latency
        dict(name="combine-grad-8", op="combine_grad", T=8, d=2048, k=8, E=128, dout="f32", zipf=False),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["quant", "product", "experts", "dispatch", "combine_grad"])
    if op == "quant":
        form = rng.choice(["rows", "sorted", "swiglu"])
        E = log(4, 256)
        return dict(op=op, form=form, T=log(1, 4096 if form == "sorted" else 40000), d=16 * log(8, 256),
                    k=min(E, rng.randint(1, 8)) if form == "sorted" else 1, E=E if form == "sorted" else 1,
                    x="bf16" if form == "swiglu" else rng.choice(["bf16", "f32"]), zipf=rng.random() < 0.5)
    if op == "product":
        return dict(op=op, M=log(1, 8192), N=log(100, 4096), K=16 * log(16, 448), out=rng.choice(["bf16", "f32"]))
    if op == "experts":
        E = log(4, 128)
        return dict(op=op, T=log(1, 4096), k=min(E, rng.randint(1, 8)), E=E, slots=rng.randint((E + 1) // 2, E),
                    N=8 * log(32, 256), K=16 * log(16, 128), zipf=rng.random() < 0.5, out="bf16")
    E = log(4, 256)
    case = dict(op=op, T=log(1, 4096), d=8 * log(16, 512), k=min(E, rng.randint(1, 8)), E=E, zipf=rng.random() < 0.5)
    if op == "dispatch":
        return dict(case, grad=rng.random() < 0.5, x=rng.choice(["bf16", "f32"]))
    return dict(case, dout=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------------------------------ inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def _cols(K):
    """Columns of a row's scale array: one per 128 values, rounded up to a multiple of 4."""
    return (K + 4 * BLOCK - 1) // (4 * BLOCK) * 4


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=gen.device).to(dtype)


def _chosen(gen, T, E, k, zipf):
    """Top-k experts of random logits, popular ones first under Zipf."""
    logits = _normal(gen, T, E)
    if zipf:
        rank = torch.randperm(E, generator=gen, device=gen.device) + 1
        logits -= 1.1 * torch.log(rank.float())
    return logits.topk(k, dim=1)


def _routing(gen, T, E, k, zipf):
    """The chosen experts, their weights, and the stable permutation of the pairs by expert."""
    top, ids = _chosen(gen, T, E, k, zipf)
    gather = torch.sort(ids.reshape(-1), stable=True)[1]
    inv = torch.empty_like(gather)
    inv[gather] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return dict(ids=ids.int(), w=top.softmax(1), inv=inv.int().view(T, k), offsets=offsets)


def _row_codes(gen, rows, K):
    x = _normal(gen, rows, K)
    return _quantise(x)


def _weight_codes(gen, slots, N, K):
    codes = torch.empty(slots, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    for s in range(slots):  # one at a time: the 32-bit values of all would not fit next to them
        codes[s] = (_normal(gen, N, K) * 112).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    grid = (slots, -(-N // BLOCK), -(-K // BLOCK))
    return codes, (0.8 + 0.4 * torch.rand(grid, generator=gen, device="cuda")) * (0.02 / 112)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "quant":
        T, d = c["T"], c["d"]
        s["x"] = _normal(gen, T, 2 * d if c["form"] == "swiglu" else d, dtype=_type(c["x"]))
        rows = T
        if c["form"] == "sorted":
            s.update(_routing(gen, T, c["E"], c["k"], c["zipf"]))
            rows = T * c["k"]
        s["codes"] = torch.zeros(rows, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["scales"] = torch.zeros(rows, _cols(d), device="cuda")
    elif c["op"] in ("product", "experts"):
        rows, slots = (c["M"], 1) if c["op"] == "product" else (c["T"] * c["k"], c["slots"])
        s["a"], s["sa"] = _row_codes(gen, rows, c["K"])
        s["b"], s["sb"] = _weight_codes(gen, slots, c["N"], c["K"])
        s["out"] = torch.zeros(rows, c["N"], dtype=_type(c["out"]), device="cuda")
        if c["op"] == "experts":
            s.update(_routing(gen, c["T"], c["E"], c["k"], c["zipf"]))
            slot = torch.full((c["E"],), -1, dtype=torch.int32, device="cuda")
            held = torch.randperm(c["E"], generator=gen, device="cuda")[: c["slots"]]
            slot[held] = torch.arange(c["slots"], dtype=torch.int32, device="cuda")
            s["slot"] = slot
            # what a program without a grouped product has at hand on the host: the groups
            o, h = s["offsets"].tolist(), slot.tolist()
            s["groups"] = [(o[e], o[e + 1], h[e]) for e in range(c["E"]) if o[e + 1] > o[e] and h[e] >= 0]
    else:
        T, d, k, E = c["T"], c["d"], c["k"], c["E"]
        s.update(_routing(gen, T, E, k, c["zipf"]))
        if c["op"] == "dispatch":
            s["x"] = _normal(gen, T * k if c["grad"] else T, d, dtype=_type(c["x"]))
            s["out"] = torch.zeros(T if c["grad"] else T * k, d, dtype=_type(c["x"]), device="cuda")
        else:
            s["dout"] = _normal(gen, T, d, dtype=_type(c["dout"]))
            s["y"] = _normal(gen, T * k, d, dtype=torch.bfloat16)
            s["dy"] = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
            s["dw"] = torch.zeros(T, k, device="cuda")
            s["dlogits"] = torch.zeros(T, E, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _blocks(x):
    """[rows][K] -> [rows][scale columns][128], zeros behind the last column."""
    rows, K = x.shape
    S = _cols(K)
    return torch.nn.functional.pad(x, (0, S * BLOCK - K)).view(rows, S, BLOCK)


def _quantise(x):
    """fp32 rows -> e4m3 codes of 448 x / top and a scale of top / 448 for each 128, top the largest magnitude."""
    b = _blocks(x)
    top = b.abs().amax(2).clamp(min=AMAX_FLOOR)
    codes = (b * E4M3_MAX / top[:, :, None]).to(torch.float8_e4m3fn).view(x.shape[0], -1)[:, : x.shape[1]]
    scale = top / E4M3_MAX
    scale[:, -(-x.shape[1] // BLOCK):] = 0
    return codes.contiguous(), scale


def _swiglu(gu):
    g, u = gu.float().chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _rows(a, sa):
    return (_blocks(a.float()) * sa[:, :, None]).view(a.shape[0], -1)[:, : a.shape[1]]


def _weights(b, sb):
    N, K = b.shape
    return b.float() * sb.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quant":
        if c["form"] == "swiglu":
            codes, scale = _quantise(_swiglu(s["x"]))
        else:
            codes, scale = _quantise(s["x"].float())
        if c["form"] == "sorted":
            at = s["inv"].long().view(-1)
            s["codes"].view(torch.uint8)[at] = codes.view(torch.uint8).repeat_interleave(c["k"], 0)
            s["scales"][at] = scale.repeat_interleave(c["k"], 0)
        else:
            s["codes"].copy_(codes)
            s["scales"].copy_(scale)
        return dict(codes=s["codes"], scales=s["scales"])
    if c["op"] == "product":
        s["out"].copy_(_rows(s["a"], s["sa"]) @ _weights(s["b"][0], s["sb"][0]).t())
        return s["out"]
    if c["op"] == "experts":
        a = _rows(s["a"], s["sa"])
        for r0, r1, slot in s["groups"]:
            s["out"][r0:r1] = (a[r0:r1] @ _weights(s["b"][slot], s["sb"][slot]).t()).to(s["out"].dtype)
        return s["out"]
    at = s["inv"].long()
    if c["op"] == "dispatch":
        if c["grad"]:
            s["out"].copy_(s["x"].float()[at].sum(1))
        else:
            s["out"][at.view(-1)] = s["x"].repeat_interleave(c["k"], 0)
        return s["out"]
    g, y = s["dout"].float(), s["y"].float()[at]
    s["dy"][at.view(-1)] = (s["w"][:, :, None] * g[:, None, :]).to(torch.bfloat16).view(-1, c["d"])
    s["dw"].copy_((y * g[:, None, :]).sum(2))
    dl = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True))
    s["dlogits"].zero_().scatter_(1, s["ids"].long(), dl)
    return dict(dy=s["dy"], dw=s["dw"], dlogits=s["dlogits"])


# ------------------------------------------------------------------------------------------ the library's calls

def _run_own(s):
    import routed_expert_ffn_wave_amd as ft
    c = s["case"]
    if c["op"] == "quant":
        if c["form"] == "swiglu":
            codes, scales = ft.ft_moe_swiglu_fp8(s["x"], codes=s["codes"], scales=s["scales"])
        elif c["form"] == "rows":
            codes, scales = ft.ft_moe_quant_fp8(s["x"], codes=s["codes"], scales=s["scales"])
        else:
            codes, scales = ft.ft_moe_dispatch_fp8(s["x"], s["ids"], s["inv"], E=c["E"], codes=s["codes"],
                                                   scales=s["scales"])
        return dict(codes=codes, scales=scales)
    if c["op"] == "product":
        return ft.ft_moe_fp8_matmul(s["a"], s["sa"], s["b"][0], s["sb"][0], out=s["out"])
    if c["op"] == "experts":
        return ft.ft_moe_fp8_grouped_matmul(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["slot"], out=s["out"])
    if c["op"] == "dispatch":
        if c["grad"]:
            return ft.ft_moe_dispatch_grad(s["x"], s["ids"], s["inv"], E=c["E"], dx=s["out"])
        return ft.ft_moe_dispatch(s["x"], s["ids"], s["inv"], E=c["E"], x_sorted=s["out"])
    dy, dw, dlogits = ft.ft_moe_combine_grad(s["dout"], s["y"], s["ids"], s["w"], s["inv"], E=c["E"],
                                             dy_sorted=s["dy"], dw=s["dw"], dlogits=s["dlogits"])
    return dict(dy=dy, dw=dw, dlogits=dlogits)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "quant":
        T, d = c["T"], c["d"]
        rows = T * c["k"]
        read = T * d * _size(c["x"]) * (2 if c["form"] == "swiglu" else 1) + (8 * rows if c["form"] == "sorted" else 0)
        return dict(bytes=read + rows * (d + 4 * _cols(d)), flops=T * d * (8 if c["form"] == "swiglu" else 3))
    if c["op"] in ("product", "experts"):
        N, K = c["N"], c["K"]
        if c["op"] == "product":
            rows, slots = c["M"], 1
        else:  # the pairs whose expert has a slot, and the experts that have any: of one routing like the case's
            ids = _chosen(torch.Generator().manual_seed(1), c["T"], c["E"], c["k"], c["zipf"])[1]
            hit = torch.bincount(ids.reshape(-1), minlength=c["E"])
            rows = max(1, int(hit.sum()) * c["slots"] // c["E"])
            slots = max(1, int((hit > 0).sum()) * c["slots"] // c["E"])
        weights = slots * (N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK))
        return dict(bytes=weights + rows * (K + 4 * _cols(K) + N * _size(c["out"])), flops=2 * rows * N * K)
    T, d, k = c["T"], c["d"], c["k"]
    if c["op"] == "dispatch":
        return dict(bytes=(T + T * k) * d * _size(c["x"]) + 8 * T * k, flops=T * k * d if c["grad"] else 0)
    return dict(bytes=T * d * _size(c["dout"]) + 2 * T * k * d * 2 + 16 * T * k + 4 * T * c["E"], flops=3 * T * k * d)


# ------------------------------------------------------------------------------------------ exact values

def _e4m3_nearest(q):
    """The e4m3 value nearest to each fp64 value, ties to the even code (|q| <= 448)."""
    exp = torch.frexp(q.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(q), exp.clamp(min=-6) - 3)
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_codes(x, d):
    """x fp64 [rows][d] -> code values and scales."""
    rows, S = x.shape[0], _cols(d)
    codes, scales = torch.zeros_like(x), torch.zeros(rows, S, dtype=torch.float64, device=x.device)
    for b in range(-(-d // BLOCK)):
        part = x[:, b * BLOCK: (b + 1) * BLOCK]
        top = torch.clamp(part.abs().max(dim=1)[0], min=AMAX_FLOOR)
        scales[:, b] = top / 448
        codes[:, b * BLOCK: (b + 1) * BLOCK] = _e4m3_nearest(448 * part / top[:, None])
    return codes, scales


def _exact_product(a, sa, b, sb):
    """sum over blocks of 128 of the codes' products, each times its two scales."""
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    per_row = torch.arange(b.shape[0], device=a.device) // BLOCK
    for i in range(sb.shape[1]):
        ks = slice(i * BLOCK, min(a.shape[1], (i + 1) * BLOCK))
        out += (a[:, ks].double() * sa[:, i, None].double()) @ (b[:, ks].double() * sb[per_row, i, None].double()).t()
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        x = s["x"].double()
        if c["form"] == "swiglu":
            x = x[:, : c["d"]] * torch.sigmoid(x[:, : c["d"]]) * x[:, c["d"]:]
        codes, scales = _exact_codes(x, c["d"])
        if c["form"] == "sorted":
            token = torch.empty(c["T"] * c["k"], dtype=torch.long, device="cuda")
            token[s["inv"].long()] = torch.arange(c["T"], device="cuda")[:, None].expand(-1, c["k"])
            codes, scales = codes[token], scales[token]
        return dict(codes=codes, scales=scales)
    if c["op"] == "product":
        return _exact_product(s["a"], s["sa"], s["b"][0], s["sb"][0])
    if c["op"] == "experts":
        out = torch.zeros(c["T"] * c["k"], c["N"], dtype=torch.float64, device="cuda")
        for r0, r1, slot in s["groups"]:
            out[r0:r1] = _exact_product(s["a"][r0:r1], s["sa"][r0:r1], s["b"][slot], s["sb"][slot])
        return out
    T, k, d = c["T"], c["k"], c["d"]
    at = s["inv"].long()
    if c["op"] == "dispatch":
        x = s["x"].double()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            if c["grad"]:
                out += x[at[:, j]]
            else:
                out[at[:, j]] = x
        return out
    # the gradient of sum(dout * out), out = sum_j w_j y_j and w the softmax of the chosen logits
    g, y, w = s["dout"].double(), s["y"].double(), s["w"].double()
    dy = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        dy[at[:, j]] = w[:, j, None] * g
        dw[:, j] = (g * y[at[:, j]]).sum(1)
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    dlogits = torch.zeros(T, c["E"], dtype=torch.float64, device="cuda")
    dlogits[torch.arange(T, device="cuda")[:, None], s["ids"].long()] = (jac @ dw[:, :, None])[:, :, 0]
    return dict(dy=dy, dw=dw, dlogits=dlogits)
