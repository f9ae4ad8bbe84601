"""The 16-bit products of a routed model, as measured cases: the products grouped by expert (plain and with
SwiGLU), the product with bias, activation and residual in its epilogue, and the softmax cross entropy over a
large vocabulary; each with its gradients.

``run`` computes a case in plain form, elementary torch operations in 32 bits rounded once at the end, or, where
``own`` is true, by the package's calls (``quantized_moe_routed_amd.dense``).
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------------------------- cases
def listed():
    e = dict(H=4096, I=2048, E=256, k=8, zipf=0.0, own_of=1)
    return [
        # one token decoded: 8 experts of 256 read once, the smallest call of the experts
        dict(e, name="swiglu_decode", op="swiglu", T=1, dtype="bf16"),
        # a prompt of 2048 tokens with the experts' popularity Zipf(1.1): from one row to hundreds for an expert
        dict(e, name="swiglu_prefill", op="swiglu", T=2048, dtype="bf16", zipf=1.1),
        # fine-tuning the first half of the experts: every gradient, an odd number of tokens, 64 experts
        dict(e, name="swiglu_grad", op="swiglu_grad", T=2051, E=64, dtype="bf16"),
        # 32 sequences decoded together: the down product into the slots' fp32 rows that the combine reads
        dict(e, name="matmul_batch", op="matmul", T=32, dtype="bf16"),
        # one device's share of 128 tokens, 128 of 256 experts owned
        dict(e, name="matmul_share", op="matmul", T=128, dtype="fp16", own_of=2),
        # fine-tuning the down product, few experts with long ragged row runs
        dict(e, name="matmul_grad", op="matmul_grad", T=4099, E=32, dtype="fp16", zipf=0.6),
        # a dense projection of one token, with bias, activation and the residual stream
        dict(name="linear_decode", op="linear", T=1, N=4096, K=4096, act="silu", dtype="bf16"),
        # the same for a prompt, odd rows
        dict(name="linear_prefill", op="linear", T=4093, N=8192, K=4096, act="gelu", dtype="bf16"),
        # and its gradients
        dict(name="linear_grad", op="linear_grad", T=4093, N=8192, K=4096, act="silu", dtype="fp16"),
        # the likelihood of one token over a large vocabulary
        dict(name="loss_decode", op="loss", T=1, V=100003, H=4096, dtype="bf16", ignored=0.0),
        # the likelihoods of a held-out text
        dict(name="loss_eval", op="loss", T=2048, V=131072, H=4096, dtype="bf16", ignored=0.0),
        # a training step of the vocabulary product: loss and both gradients, odd sizes, a part of the targets ignored
        dict(name="loss_train", op="loss_grad", T=4093, V=50257, H=4096, dtype="bf16", ignored=0.1),
    ]


def _log(rng, lo, hi, step=1):
    """A whole number of [lo, hi], even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["swiglu", "swiglu_grad", "matmul", "matmul_grad", "linear", "linear_grad", "loss", "loss_grad"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]))
    if op in ("swiglu", "swiglu_grad", "matmul", "matmul_grad"):
        grad = op.endswith("grad")
        E = rng.choice([8, 16, 32, 64, 128, 256])
        c.update(T=_log(rng, 1, 4099 if E <= 64 or not grad else 1024), H=_log(rng, 256, 4096, 8), I=_log(rng, 128, 2048, 8), E=E,
                 k=rng.choice([1, 2, 4, 6, 8]), zipf=rng.choice([0.0, 0.6, 1.1]), own_of=rng.choice([1, 1, 2]))
        if op == "swiglu_grad":
            c["T"] = min(c["T"], 2051)
    elif op in ("linear", "linear_grad"):
        c.update(T=_log(rng, 1, 4099), N=_log(rng, 64, 8192, 8), K=_log(rng, 64, 4096, 8), act=rng.choice(["none", "relu", "silu", "gelu"]))
    else:
        c.update(T=_log(rng, 1, 2051), V=_log(rng, 1000, 131072 if op == "loss" else 65537), H=_log(rng, 256, 4096, 8),
                 ignored=rng.choice([0.0, 0.1, 0.5]))
    return c


# --------------------------------------------------------------------------------------------- inputs
def _randn(gen, shape, std, dt):
    return torch.empty(shape, dtype=dt, device=DEV).normal_(0.0, std, generator=gen)


def _route(case, gen, device):
    """The grouping of T*k slots: k distinct experts for each token, popularity uniform or Zipf."""
    T, E, k = case["T"], case["E"], case["k"]
    z = torch.randn((T, E), generator=gen, device=device)
    z = z - case["zipf"] * torch.log(torch.randperm(E, generator=gen, device=device).float() + 1.0)
    ids = torch.topk(z, min(k, E), dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    slots = torch.sort(ids, stable=True).indices.to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=device)
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, slots


def _g2l(case):
    """Every second expert owned where own_of is 2, else every one."""
    E = case["E"]
    if case["own_of"] == 1:
        return None, E
    t = np.full(E, -1, np.int32)
    t[::2] = np.arange((E + 1) // 2)
    return t, (E + 1) // 2


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    dt, op, T = DT[case["dtype"]], case["op"], case["T"]
    s = {}
    if op in ("swiglu", "swiglu_grad", "matmul", "matmul_grad"):
        H, I = case["H"], case["I"]
        offsets, slots = _route(case, gen, DEV)
        table, E_local = _g2l(case)
        R = slots.numel()
        s.update(offsets=offsets, slots=slots, table=None if table is None else torch.from_numpy(table).to(DEV), E_local=E_local)
        # what a program that plans on the host keeps: (local expert, first position, rows)
        off = offsets.tolist()
        s["spans"] = [(e if table is None else int(table[e]), off[e], off[e + 1]) for e in range(case["E"])
                      if off[e + 1] > off[e] and (table is None or table[e] >= 0)]
        if op in ("swiglu", "swiglu_grad"):
            s.update(x=_randn(gen, (T, H), 1.0, dt), gate=_randn(gen, (E_local, I, H), 0.02, dt), up=_randn(gen, (E_local, I, H), 0.02, dt))
            if op == "swiglu":
                s["out"] = torch.zeros((R, I), dtype=dt, device=DEV)
            else:      # g and u are what the forward pass kept
                s.update(dh=_randn(gen, (R, I), 0.01, dt), g=_randn(gen, (R, I), 1.2, dt), u=_randn(gen, (R, I), 1.2, dt))
                s["dx"] = torch.zeros((R, H), dtype=dt, device=DEV)
        else:
            s.update(h=_randn(gen, (R, I), 0.7, dt), w=_randn(gen, (E_local, H, I), 0.02, dt))
            if op == "matmul":
                s["out"] = torch.zeros((R, H), dtype=torch.float32, device=DEV)
            else:
                s["dy"] = _randn(gen, (R, H), 0.01, dt)
                s["dx"] = torch.zeros((R, I), dtype=dt, device=DEV)
    elif op in ("linear", "linear_grad"):
        N, K = case["N"], case["K"]
        s.update(x=_randn(gen, (T, K), 1.0, dt), w=_randn(gen, (N, K), 0.02, dt))
        if op == "linear":
            s.update(bias=_randn(gen, (N,), 0.1, torch.float32), res=_randn(gen, (T, N), 1.0, dt))
        else:
            s.update(pre=_randn(gen, (T, N), 1.3, dt), dy=_randn(gen, (T, N), 0.01, dt))
    else:
        V, H = case["V"], case["H"]
        s.update(x=_randn(gen, (T, H), 1.0, dt), w=_randn(gen, (V, H), 0.03, dt))
        tgt = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
        drop = torch.rand((T,), generator=gen, device=DEV) < case["ignored"]
        s["target"] = torch.where(drop, torch.full_like(tgt, -100), tgt)
        if op == "loss_grad":
            kept = (~drop).sum().clamp(min=1)
            s["dnll"] = torch.where(drop, 0.0, 1.0 / kept.float()).to(torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    return s


# ------------------------------------------------------------------------------------------ plain form
def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain(s):
    c = s["case"]
    op, dt = c["op"], DT[c["dtype"]]
    f = lambda a: a.float()  # noqa: E731
    # the groups are ragged, so each expert's rows are a product of their own
    if op == "swiglu":
        tok = (s["slots"] // min(c["k"], c["E"])).long()
        for e, a, b in s["spans"]:
            xe = f(s["x"][tok[a:b]])
            g, u = xe @ f(s["gate"][e]).t(), xe @ f(s["up"][e]).t()
            s["out"][a:b] = (g * torch.sigmoid(g) * u).to(dt)
        return s["out"]
    if op == "swiglu_grad":
        tok = (s["slots"] // min(c["k"], c["E"])).long()
        dgate, dup = torch.zeros_like(s["gate"]), torch.zeros_like(s["up"])
        for e, a, b in s["spans"]:
            xe, dh, g, u = f(s["x"][tok[a:b]]), f(s["dh"][a:b]), f(s["g"][a:b]), f(s["u"][a:b])
            p = torch.sigmoid(g)
            dg, du = dh * u * p * (1 + g * (1 - p)), dh * g * p
            s["dx"][a:b] = (dg @ f(s["gate"][e]) + du @ f(s["up"][e])).to(dt)
            dgate[e], dup[e] = (dg.t() @ xe).to(dt), (du.t() @ xe).to(dt)
        return {"dx": s["dx"], "dgate": dgate, "dup": dup}
    if op == "matmul":
        to = s["slots"].long()
        for e, a, b in s["spans"]:
            s["out"][to[a:b]] = f(s["h"][a:b]) @ f(s["w"][e]).t()
        return s["out"]
    if op == "matmul_grad":
        at = s["slots"].long()
        dw = torch.zeros_like(s["w"])
        for e, a, b in s["spans"]:
            dy = f(s["dy"][at[a:b]])
            s["dx"][a:b] = (dy @ f(s["w"][e])).to(dt)
            dw[e] = (dy.t() @ f(s["h"][a:b])).to(dt)
        return {"dx": s["dx"], "dw": dw}
    if op == "linear":
        return (f(s["res"]) + _act(f(s["x"]) @ f(s["w"]).t() + s["bias"], c["act"])).to(dt)
    if op == "linear_grad":
        dz = f(s["dy"]) * _act_slope(f(s["pre"]), c["act"])
        return {"dx": (dz @ f(s["w"])).to(dt), "dw": (dz.t() @ f(s["x"])).to(dt), "dbias": dz.sum(0)}
    x, w, t = f(s["x"]), f(s["w"]), s["target"]
    keep = t >= 0
    at = t.clamp(min=0).long()[:, None]
    z = x @ w.t()
    top = z.max(1, keepdim=True).values
    p = torch.exp(z - top)
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    nll = torch.where(keep, lse - z.gather(1, at)[:, 0], 0.0)
    if op == "loss":
        return {"nll": nll, "lse": lse}
    p.div_(total)
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    p.mul_(torch.where(keep, s["dnll"], 0.0)[:, None])
    return {"nll": nll, "lse": lse, "dx": (p @ w).to(dt), "dw": (p.t() @ x).to(dt)}


# --------------------------------------------------------------------------------------- the package's
def _package(s):
    from quantized_moe_routed_amd import dense
    c = s["case"]
    op = c["op"]
    if op in ("swiglu", "swiglu_grad", "matmul", "matmul_grad"):
        groups = dense.Groups(s["offsets"], s["slots"], c["T"], min(c["k"], c["E"]), g2l=s["table"], E_local=s["E_local"])
        if op == "swiglu":
            return dense.grouped_swiglu(s["x"], s["gate"], s["up"], groups, x_rows=dense.ROWS_TOKEN, out=s["out"])
        if op == "swiglu_grad":
            dx, dgate, dup = dense.grouped_swiglu_grad(s["dh"], s["x"], s["gate"], s["up"], s["g"], s["u"], groups,
                                                       x_rows=dense.ROWS_TOKEN, dx=s["dx"])
            return {"dx": dx, "dgate": dgate, "dup": dup}
        if op == "matmul":
            return dense.grouped_matmul(s["h"], s["w"], groups, out_rows=dense.ROWS_SLOT, out=s["out"])
        dx, dw = dense.grouped_matmul_grad(s["dy"], s["h"], s["w"], groups, dy_rows=dense.ROWS_SLOT, dx=s["dx"])
        return {"dx": dx, "dw": dw}
    if op == "linear":
        return dense.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["res"])
    if op == "linear_grad":
        dx, dw, dbias = dense.linear_grad(s["dy"], s["x"], s["w"], pre=s["pre"], act=c["act"])
        return {"dx": dx, "dw": dw, "dbias": dbias}
    nll, lse = dense.cross_entropy(s["x"], s["w"], s["target"])
    if op == "loss":
        return {"nll": nll, "lse": lse}
    dx, dw = dense.cross_entropy_grad(s["x"], s["w"], s["target"], lse, s["dnll"])
    return {"nll": nll, "lse": lse, "dx": dx, "dw": dw}


def run(state):
    return _package(state) if own else _plain(state)


# -------------------------------------------------------------------------------------------- the floor
def work(case):
    op, b = case["op"], 2
    if op in ("linear", "linear_grad"):
        M, N, K = case["T"], case["N"], case["K"]
        if op == "linear":
            return {"bytes": b * (M * K + N * K + 2 * M * N) + 4 * N, "flops": 2 * M * N * K}
        return {"bytes": b * (2 * M * N + 2 * M * K + 2 * N * K) + 4 * N, "flops": 4 * M * N * K}
    if op in ("loss", "loss_grad"):
        T, V, H = case["T"], case["V"], case["H"]
        if op == "loss":
            return {"bytes": b * (T * H + V * H) + 12 * T, "flops": 2 * T * V * H}
        return {"bytes": b * 2 * (T * H + V * H) + 16 * T, "flops": 6 * T * V * H}
    # the routing is drawn, so its rows and touched experts are those of one draw
    gen = torch.Generator().manual_seed(1)
    offsets, _ = _route(case, gen, "cpu")
    n = np.diff(offsets.numpy())
    table, E_local = _g2l(case)
    n = n if table is None else n[table >= 0]
    R, used, H, I, T = int(n.sum()), int((n > 0).sum()), case["H"], case["I"], case["T"]
    if op == "swiglu":
        return {"bytes": b * (2 * used * I * H + T * H + R * I), "flops": 4 * R * I * H}
    if op == "swiglu_grad":
        return {"bytes": b * (2 * used * I * H + 2 * E_local * I * H + T * H + 3 * R * I + R * H), "flops": 8 * R * I * H}
    if op == "matmul":
        return {"bytes": b * (used * H * I + R * I) + 4 * R * H, "flops": 2 * R * I * H}
    return {"bytes": b * (used * H * I + E_local * H * I + 2 * R * I + R * H), "flops": 4 * R * I * H}


# ------------------------------------------------------------------------------------ 64-bit definition
def _sig64(v):
    return 1.0 / (1.0 + torch.exp(-v))


def exact(case, seed):
    """The definitions in 64 bits; products over blocks of rows or of the vocabulary, so that they fit."""
    s, op = _inputs(case, seed), case["op"]
    d = lambda a: a.to(torch.float64)  # noqa: E731
    if op in ("swiglu", "swiglu_grad", "matmul", "matmul_grad"):
        R = s["slots"].numel()
        slot = s["slots"].long()
        tok = torch.div(slot, min(case["k"], case["E"]), rounding_mode="floor")
        H, I = case["H"], case["I"]
        new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
        if op == "swiglu":
            y = new(R, I)
            for e, a, b in s["spans"]:
                rows = d(s["x"]).index_select(0, tok[a:b])
                g = torch.mm(rows, d(s["gate"][e]).T)
                y[a:b] = g * _sig64(g) * torch.mm(rows, d(s["up"][e]).T)
            return y
        if op == "matmul":
            y = new(R, H)
            for e, a, b in s["spans"]:
                y.index_copy_(0, slot[a:b], torch.mm(d(s["h"][a:b]), d(s["w"][e]).T))
            return y
        if op == "matmul_grad":
            dx, dw = new(R, I), new(s["E_local"], H, I)
            for e, a, b in s["spans"]:
                dy = d(s["dy"]).index_select(0, slot[a:b])
                dx[a:b] = torch.mm(dy, d(s["w"][e]))
                dw[e] = torch.mm(dy.T, d(s["h"][a:b]))
            return {"dx": dx, "dw": dw}
        dx, dgate, dup = new(R, H), new(s["E_local"], I, H), new(s["E_local"], I, H)
        for e, a, b in s["spans"]:
            rows, dh, g, u = d(s["x"]).index_select(0, tok[a:b]), d(s["dh"][a:b]), d(s["g"][a:b]), d(s["u"][a:b])
            sg = _sig64(g)
            du = dh * (g * sg)
            dg = dh * u * (sg + g * sg * (1.0 - sg))
            dx[a:b] = torch.mm(dg, d(s["gate"][e])) + torch.mm(du, d(s["up"][e]))
            dgate[e], dup[e] = torch.mm(dg.T, rows), torch.mm(du.T, rows)
        return {"dx": dx, "dgate": dgate, "dup": dup}
    if op in ("linear", "linear_grad"):
        x, w, act = d(s["x"]), d(s["w"]), case["act"]
        if op == "linear":
            z = torch.addmm(d(s["bias"]), x, w.T)
            a = {"none": lambda v: v, "relu": lambda v: torch.where(v > 0, v, torch.zeros_like(v)), "silu": lambda v: v * _sig64(v),
                 "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2.0))}[act](z)
            return a + d(s["res"])
        z = d(s["pre"])
        if act == "none":
            k = torch.ones_like(z)
        elif act == "relu":
            k = torch.where(z > 0, 1.0, 0.0).double()
        elif act == "silu":
            sg = _sig64(z)
            k = sg + z * sg * (1.0 - sg)
        else:
            k = 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
        dz = d(s["dy"]) * k
        return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.T, x), "dbias": dz.sum(dim=0)}
    # the loss: blocks of the vocabulary, a first pass for the sums and a second for the gradients
    x, t = d(s["x"]), s["target"].long()
    T, V, B = case["T"], case["V"], 8192
    lse = torch.full((T,), -math.inf, dtype=torch.float64, device=DEV)
    hit = torch.zeros(T, dtype=torch.float64, device=DEV)
    for v in range(0, V, B):
        z = torch.mm(x, d(s["w"][v:v + B]).T)
        lse = torch.logaddexp(lse, torch.logsumexp(z, dim=1))
        here = (t >= v) & (t < v + z.shape[1])
        hit = torch.where(here, z[torch.arange(T, device=DEV), torch.where(here, t - v, torch.zeros_like(t))], hit)
    nll = torch.where(t >= 0, lse - hit, torch.zeros_like(lse))
    if op == "loss":
        return {"nll": nll, "lse": lse}
    dx, dw = torch.zeros_like(x), torch.zeros((V, case["H"]), dtype=torch.float64, device=DEV)
    up = torch.where(t >= 0, d(s["dnll"]), torch.zeros_like(lse))
    for v in range(0, V, B):
        wb = d(s["w"][v:v + B])
        ds = torch.exp(torch.mm(x, wb.T) - lse[:, None])
        cols = torch.arange(v, v + wb.shape[0], device=DEV)
        ds = (ds - (t[:, None] == cols[None, :]).double()) * up[:, None]
        dx += torch.mm(ds, wb)
        dw[v:v + B] = torch.mm(ds.T, x)
    return {"nll": nll, "lse": lse, "dx": dx, "dw": dw}
