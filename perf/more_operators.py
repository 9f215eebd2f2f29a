"""Cases of five operators around a trained or adapted expert FFN: the bf16 product of token rows with one matrix
per expert, the gradients of its rows and of its matrices, SwiGLU with its gradient, and low-rank adapters of many
requests beside a shared projection.

`run` computes a case in plain torch operations, or with `own` through the library's calls."""
import math

import torch

own = False


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token's eight experts, gate and up rows: bound by the matrices' bytes
        dict(name="product-1", op="product", T=1, k=8, E=128, slots=128, N=1536, K=2048, zipf=False, out="bf16"),
        # a prompt chunk or training batch with popular and unpopular experts, groups from none to thousands of rows
        dict(name="product-4096", op="product", T=4096, k=8, E=128, slots=128, N=1536, K=2048, zipf=True, out="bf16"),
        # a short odd batch of wide experts, some of them not resident, 32-bit results
        dict(name="product-333-f32", op="product", T=333, k=8, E=64, slots=40, N=2048, K=1032, zipf=False, out="f32"),
        # the same batch on its way back: gradient of the rows
        dict(name="rows-grad-4096", op="rows_grad", T=4096, k=8, E=128, slots=128, N=1536, K=2048, zipf=True, out="bf16"),
        # a small odd batch, 32-bit gradient
        dict(name="rows-grad-77-f32", op="rows_grad", T=77, k=4, E=32, slots=32, N=2048, K=768, zipf=False, out="f32"),
        # the gradient of every expert's matrix in 32 bits: bound by writing it
        dict(name="matrix-grad-4096", op="matrix_grad", T=4096, k=8, E=128, slots=128, N=1536, K=2048, zipf=True, out="f32"),
        # few large experts and a long batch: bound by the matrix cores
        dict(name="matrix-grad-8192", op="matrix_grad", T=8192, k=2, E=8, slots=8, N=4096, K=7168, zipf=False, out="bf16"),
        # gate and up products of the training batch, forward and back
        dict(name="swiglu-32768", op="swiglu", grad=False, rows=32768, I=768),
        dict(name="swiglu-grad-32768", op="swiglu", grad=True, rows=32768, I=768),
        # one decode step of sixteen requests with adapters of their own: launch latency
        dict(name="adapters-16", op="adapters", T=16, n=16, slots=16, r=16, N=4096, K=2048, packed=False, out="bf16"),
        # requests that share adapters, in no order, 32-bit sums
        dict(name="adapters-131-f32", op="adapters", T=131, n=40, slots=24, r=8, N=2048, K=7168, packed=False, out="f32"),
        # five prompts of a chunk one after another
        dict(name="adapters-4096", op="adapters", T=4096, n=5, slots=5, r=64, N=4096, K=7168, packed=True, out="bf16"),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["product", "rows_grad", "matrix_grad", "swiglu", "adapters"])
    if op == "swiglu":
        return dict(op=op, grad=rng.random() < 0.5, rows=log(1, 32768), I=8 * log(4, 96))
    if op == "adapters":
        n = log(1, 64)
        return dict(op=op, T=log(1, 4096), n=n, slots=rng.randint((n + 1) // 2, n), r=8 * log(1, 8), N=8 * log(32, 512),
                    K=8 * log(32, 896), packed=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    E = log(4, 128)
    return dict(op=op, T=log(1, 4096), k=min(E, rng.randint(1, 8)), E=E,
                slots=rng.randint((E + 1) // 2, E), N=8 * log(32, 192), K=8 * log(32, 256),
                zipf=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------------------------------ inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def _normal(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device=gen.device)
    for part in out.view(-1, shape[-1]).split(1 << 16):  # the 32-bit values of all would not fit next to them
        part.copy_(torch.randn(part.shape, generator=gen, device=gen.device) * scale)
    return out


def _chosen(gen, T, E, k, zipf):
    """Top-k experts of random logits, popular ones first under Zipf."""
    logits = torch.randn(T, E, generator=gen, device=gen.device)
    if zipf:
        rank = torch.randperm(E, generator=gen, device=gen.device) + 1
        logits -= 1.1 * torch.log(rank.float())
    return logits.topk(k, dim=1)[1]


def _offsets(ids, E):
    out = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    out[1:] = torch.bincount(ids.reshape(-1), minlength=E)[:E].cumsum(0)
    return out


def _slots(gen, E, slots):
    table = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    table[torch.randperm(E, generator=gen, device="cuda")[:slots]] = torch.arange(slots, dtype=torch.int32, device="cuda")
    return table


def _adapter_of_row(gen, c):
    """The adapter of every row, n for rows without one (about one in ten)."""
    if c["packed"]:  # prompts one after another
        cuts = torch.sort(torch.randint(0, c["T"] + 1, (c["n"] - 1,), generator=gen, device=gen.device))[0]
        return torch.bucketize(torch.arange(c["T"], device=gen.device), cuts, right=True)
    ids = torch.randint(0, c["n"], (c["T"],), generator=gen, device=gen.device)
    ids[torch.rand(c["T"], generator=gen, device=gen.device) < 0.1] = c["n"]
    return ids


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "swiglu":
        s["gu"] = _normal(gen, c["rows"], 2 * c["I"])
        s["dh"] = _normal(gen, c["rows"], c["I"], scale=0.1)
        s["out"] = torch.zeros(c["rows"], c["I"] * (2 if c["grad"] else 1), dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] == "adapters":
        T, r, N, K = c["T"], c["r"], c["N"], c["K"]
        ids = _adapter_of_row(gen, c)
        s["offsets"] = _offsets(ids, c["n"])
        s["gather"] = torch.sort(ids, stable=True)[1].int()
        s["slot"] = _slots(gen, c["n"], c["slots"])
        s["scale"] = 0.5 + 1.5 * torch.rand(c["slots"], generator=gen, device="cuda")
        s["x"] = _normal(gen, T, K)
        s["a"] = _normal(gen, c["slots"], r, K, scale=K ** -0.5)
        s["b"] = _normal(gen, c["slots"], N, r, scale=0.1)
        s["base"] = _normal(gen, T, N, dtype=_type(c["out"]))
        s["out"] = torch.zeros_like(s["base"])
    else:
        P, N, K, E = c["T"] * c["k"], c["N"], c["K"], c["E"]
        s["offsets"] = _offsets(_chosen(gen, c["T"], E, c["k"], c["zipf"]), E)
        s["slot"] = _slots(gen, E, c["slots"])
        if c["op"] != "matrix_grad":
            s["w"] = _normal(gen, c["slots"], N, K, scale=K ** -0.5)
        if c["op"] != "rows_grad":
            s["a"] = _normal(gen, P, K)
        if c["op"] != "product":
            s["dout"] = _normal(gen, P, N, scale=0.1)
        shape = {"product": (P, N), "rows_grad": (P, K), "matrix_grad": (E, N, K)}[c["op"]]
        s["out"] = torch.zeros(shape, dtype=_type(c["out"]), device="cuda")
    # what a program without a grouped product has at hand on the host: the groups
    o, h = s["offsets"].tolist(), s["slot"].tolist()
    s["groups"] = [(e, o[e], o[e + 1], h[e]) for e in range(len(h)) if o[e + 1] > o[e] and h[e] >= 0]
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _run_plain(s):
    c, out = s["case"], s["out"]
    if c["op"] == "swiglu":
        g, u = s["gu"].float().chunk(2, dim=1)
        sig = 1 / (1 + torch.exp(-g))
        if not c["grad"]:
            out.copy_(g * sig * u)
            return out
        dh = s["dh"].float()
        out[:, : c["I"]] = dh * u * sig * (1 + g * (1 - sig))
        out[:, c["I"]:] = dh * g * sig
        return out
    if c["op"] == "adapters":
        out.copy_(s["base"])
        x = s["x"].float()
        for _, r0, r1, slot in s["groups"]:
            rows = s["gather"][r0:r1].long()
            delta = x[rows] @ s["a"][slot].float().t() @ s["b"][slot].float().t()
            out[rows] = (s["base"][rows].float() + s["scale"][slot] * delta).to(out.dtype)
        return out
    if c["op"] == "product":
        for _, r0, r1, slot in s["groups"]:
            out[r0:r1] = (s["a"][r0:r1].float() @ s["w"][slot].float().t()).to(out.dtype)
    elif c["op"] == "rows_grad":
        for _, r0, r1, slot in s["groups"]:
            out[r0:r1] = (s["dout"][r0:r1].float() @ s["w"][slot].float()).to(out.dtype)
    else:
        out.zero_()
        for e, r0, r1, _ in s["groups"]:
            out[e] = (s["dout"][r0:r1].float().t() @ s["a"][r0:r1].float()).to(out.dtype)
    return out


# ------------------------------------------------------------------------------------------ the library's calls

def _run_own(s):
    import routed_expert_ffn_wave_amd as ft
    c = s["case"]
    if c["op"] == "swiglu":
        if c["grad"]:
            return ft.ft_moe_swiglu_grad(s["gu"], s["dh"], dgu=s["out"])
        return ft.ft_moe_swiglu(s["gu"], h=s["out"])
    if c["op"] == "adapters":
        return ft.ft_moe_lora(s["base"], s["x"], s["a"], s["b"], s["offsets"], s["gather"], slot_of_adapter=s["slot"],
                              scale=s["scale"], out=s["out"])
    if c["op"] == "product":
        return ft.ft_moe_grouped_matmul(s["a"], s["w"], s["offsets"], slot_of_expert=s["slot"], out=s["out"])
    if c["op"] == "rows_grad":
        return ft.ft_moe_grouped_matmul_grad(s["dout"], s["w"], s["offsets"], slot_of_expert=s["slot"], da=s["out"])
    return ft.ft_moe_grouped_matmul_wgrad(s["dout"], s["a"], s["offsets"], slot_of_expert=s["slot"], dw=s["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "swiglu":
        n = c["rows"] * c["I"] * 2
        return dict(bytes=n * (5 if c["grad"] else 3), flops=c["rows"] * c["I"] * (12 if c["grad"] else 5))
    if c["op"] == "adapters":
        gen = torch.Generator().manual_seed(1)  # one batch like the case's
        ids = _adapter_of_row(gen, c)
        held = c["slots"] / c["n"]
        used = max(1, round(ids[ids < c["n"]].unique().numel() * held))
        rows = max(1, round((ids < c["n"]).sum().item() * held))
        weights = used * c["r"] * (c["K"] + c["N"]) * 2
        return dict(bytes=weights + rows * c["K"] * 2 + 2 * c["T"] * c["N"] * _size(c["out"]) + 4 * c["T"],
                    flops=2 * rows * c["r"] * (c["K"] + c["N"]))
    # the pairs whose expert has a slot, and the experts that have any: of one routing like the case's
    N, K, E = c["N"], c["K"], c["E"]
    ids = _chosen(torch.Generator().manual_seed(1), c["T"], E, c["k"], c["zipf"])
    hit = torch.bincount(ids.reshape(-1), minlength=E)
    rows = max(1, int(hit.sum()) * c["slots"] // E)
    if c["op"] == "matrix_grad":
        return dict(bytes=rows * (N + K) * 2 + c["slots"] * N * K * _size(c["out"]), flops=2 * rows * N * K)
    used = max(1, int((hit > 0).sum()) * c["slots"] // E)
    read, written = (K, N) if c["op"] == "product" else (N, K)
    return dict(bytes=used * N * K * 2 + rows * (read * 2 + written * _size(c["out"])), flops=2 * rows * N * K)


# ------------------------------------------------------------------------------------------ exact values

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "swiglu":
        g, u = s["gu"][:, : c["I"]].double(), s["gu"][:, c["I"]:].double()
        silu = g * torch.sigmoid(g)
        if not c["grad"]:
            return silu * u
        slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
        return torch.cat([s["dh"].double() * u * slope, s["dh"].double() * silu], 1)
    if c["op"] == "adapters":
        out = s["base"].double()
        slot_of_row = torch.full((c["T"],), -1, dtype=torch.long, device="cuda")
        for i in range(c["n"]):
            rows = s["gather"][s["offsets"][i]: s["offsets"][i + 1]].long()
            slot_of_row[rows] = s["slot"][i].long()
        for j in range(c["slots"]):
            rows = torch.nonzero(slot_of_row == j)[:, 0]
            hidden = s["x"][rows].double() @ s["a"][j].double().t()
            out[rows] += s["scale"][j].double() * (hidden @ s["b"][j].double().t())
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        r0, r1, slot = int(s["offsets"][e]), int(s["offsets"][e + 1]), int(s["slot"][e])
        if slot < 0 or r0 == r1:
            continue
        if c["op"] == "product":
            out[r0:r1] = torch.matmul(s["a"][r0:r1].double(), s["w"][slot].double().t())
        elif c["op"] == "rows_grad":
            out[r0:r1] = torch.matmul(s["dout"][r0:r1].double(), s["w"][slot].double())
        else:
            out[e] = torch.matmul(s["dout"][r0:r1].double().t(), s["a"][r0:r1].double())
    return out
