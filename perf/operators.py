"""Cases for the operators around the routed experts, their plain forms and their exact values.

Operators:
  dispatch   token rows brought into the order of the slots (optionally weighted); with
             `grad`, forward and backward: the gradients of the rows and of the weights
  combine    slot-ordered rows brought back to their tokens, weighted and summed; with
             `grad`, forward and backward
  quantize   rows to 8-bit integers with one scale for each row
  matmul     products of 8-bit integers with scales for each row and channel, over the
             groups of a bucketing (groups > 0) or dense (groups = 0); with `swiglu`,
             the gate and up products and silu(gate) * up

Where `own` is true, `run` makes the framework's calls; otherwise it takes elementary torch
operations.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -126  # the smallest scale of a quantised row


def listed():
    return [
        # the first layer step of 32 sequences: their tokens' rows for experts outside the library
        dict(name="dispatch step", op="dispatch", T=32, H=4096, k=8, G=256, absent=0.0,
             dtype="bf16", weighted=False, grad=False),
        # fine-tuning in 32 bits: a prompt batch, weights applied on the way in
        dict(name="dispatch train fp32", op="dispatch", T=2048, H=4096, k=8, G=166, absent=0.0,
             dtype="fp32", weighted=True, grad=True),
        # a long prefill chunk
        dict(name="dispatch long", op="dispatch", T=8192, H=6144, k=8, G=130, absent=0.0,
             dtype="bf16", weighted=False, grad=False),
        # one decode step of 8 sequences: the experts' rows back to their tokens
        dict(name="combine step", op="combine", T=8, H=4096, k=8, G=230, absent=0.0,
             dtype="bf16", weighted=True, grad=False),
        # an odd batch with few experts resident, so some picks (and whole tokens) have no row
        dict(name="combine odd fp16", op="combine", T=1777, H=1001, k=4, G=16, absent=0.3,
             dtype="fp16", weighted=True, grad=True),
        # a training step over a long chunk
        dict(name="combine train long", op="combine", T=8192, H=6144, k=8, G=130, absent=0.0,
             dtype="bf16", weighted=True, grad=True),
        # activations of one decode step
        dict(name="quantize step", op="quantize", M=8, K=4096, dtype="bf16"),
        # the experts' intermediate rows of a long prefill chunk
        dict(name="quantize long", op="quantize", M=65536, K=2048, dtype="bf16"),
        # a shared expert's gate and up products for a single token
        dict(name="matmul token", op="matmul", T=1, k=1, G=0, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, out="bf16"),
        # the routed experts' gate and up products of one decode step
        dict(name="matmul step", op="matmul", T=8, k=8, G=230, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, out="bf16"),
        # the down products of a prompt batch
        dict(name="matmul prefill", op="matmul", T=2048, k=8, G=166, N=4096, K=2048, swiglu=False,
             by_token=False, absent=0.0, out="bf16"),
        # the gate and up products of a long prefill chunk
        dict(name="matmul long", op="matmul", T=8192, k=8, G=130, N=2048, K=6144, swiglu=True,
             by_token=True, absent=0.0, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "quantize", "matmul", "matmul"])
    if op == "quantize":
        M, K = _log(rng, 1, 65536), _log(rng, 16, 8192)
        return dict(op=op, M=M, K=min(K, max(16, (1 << 27) // M)),
                    dtype=rng.choice(sorted(TYPES)))
    k = rng.randint(1, 8)
    G = rng.randint(8, 256)
    absent = rng.choice([0.0, 0.0, 0.2])
    if op == "matmul":
        T = _log(rng, 1, 8192)
        N, K = _log(rng, 33, 4096), _log(rng, 64, 6144)
        if rng.random() < 0.5:  # a multiple of 128, as most models have
            N, K = -(-N // 128) * 128, -(-K // 128) * 128
        swiglu = rng.random() < 0.5
        if rng.random() < 0.25:
            G, k, absent = 0, 1, 0.0
        return dict(op=op, T=T, k=k, G=G, N=min(N, 2048) if swiglu else N, K=K, swiglu=swiglu,
                    by_token=rng.random() < 0.5, absent=absent, out=rng.choice(sorted(TYPES)))
    T, H = _log(rng, 1, 8192), _log(rng, 32, 6144)
    if rng.random() < 0.5:
        H = -(-H // 32) * 32
    dtype = rng.choice(sorted(TYPES))
    if dtype == "fp32":
        T = min(T, 4096)
    return dict(op=op, T=T, H=H, k=k, G=G, absent=absent, dtype=dtype,
                weighted=op == "combine" or rng.random() < 0.5, grad=rng.random() < 0.6)


def _popularity(G):
    p = [(i + 1.0) ** -0.8 for i in range(G)]
    s = sum(p)
    return [v / s for v in p]


def _routing(case, gen):
    """Picks as a router makes them: k distinct slots of G for each token, popular slots
    more often, some absent; and the bucketing of the assignments by slot."""
    T, k, G = case["T"], case["k"], case["G"]
    dev = "cuda"
    p = torch.tensor(_popularity(G), device=dev).log()
    p = p[torch.randperm(G, device=dev, generator=gen)]
    u = torch.rand(T, G, device=dev, generator=gen).clamp_(1e-12, 1 - 1e-7)
    top = (p - (-u.log()).log()).topk(k, dim=1)
    sel = top.indices.sort(dim=1).values
    if case["absent"]:
        gone = torch.rand(T, k, device=dev, generator=gen) < case["absent"]
        if T > 2:
            gone[T // 2] = True  # a token that has no routable expert at all
        sel = torch.where(gone, torch.full_like(sel, -1), sel)
    weight = torch.rand(T, k, device=dev, generator=gen) + 0.1
    weight = torch.where(sel < 0, torch.zeros_like(weight), weight)
    weight = weight / weight.sum(dim=1, keepdim=True).clamp_min(1e-30)
    key = torch.where(sel < 0, torch.full_like(sel, G), sel).reshape(-1)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=G + 1)
    present = int(counts[:G].sum())
    perm = order.to(torch.int32)
    perm[present:] = -1
    offsets = torch.zeros(G + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts[:G].cumsum(0).to(torch.int32)
    return dict(perm=perm, offsets=offsets, weight=weight.float().contiguous())


def _int8(shape, gen):
    """Whole numbers as quantised weights and activations are: bell-shaped, to +-127."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 28) // shape[-1])
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        part.copy_((torch.randn(part.shape, device="cuda", generator=gen) * 36).round_().clamp_(-127, 127))
    return out


def _padded(q):
    """The rows of q at a distance of a multiple of 16 bytes, as int8.quantize lays them out."""
    K = q.shape[-1]
    if K % 16 == 0:
        return q
    wide = torch.zeros(*q.shape[:-1], -(-K // 16) * 16, dtype=q.dtype, device=q.device)
    wide[..., :K] = q
    return wide[..., :K]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype):
        return torch.randn(*shape, device="cuda", generator=gen).to(dtype)

    s = dict(case)
    op = case["op"]
    if op == "quantize":
        # rows of different sizes, a row of zeros among them
        x = torch.randn(case["M"], case["K"], device="cuda", generator=gen)
        x *= torch.exp(torch.randn(case["M"], 1, device="cuda", generator=gen))
        if case["M"] > 2:
            x[case["M"] // 2] = 0
        s["x"] = x.to(TYPES[case["dtype"]])
        return s
    if op == "matmul":
        T, k, G, N, K = (case[v] for v in ("T", "k", "G", "N", "K"))
        n = T * k
        s.update(_routing(case, gen) if G else dict(perm=None, offsets=None))
        rows_a = T if case["by_token"] else n
        s["a"] = _padded(_int8((rows_a, K), gen))
        s["a_scale"] = torch.rand(rows_a, device="cuda", generator=gen) * 0.02 + 0.01
        wide = 2 * N if case["swiglu"] else N
        lead = (G,) if G else ()
        s["b"] = _padded(_int8((*lead, wide, K), gen))
        s["b_scale"] = torch.rand(*lead, wide, device="cuda", generator=gen) * 4e-4 + 2e-4
        s["y"] = torch.zeros(n, N, dtype=TYPES[case["out"]], device="cuda")
        s["index"] = s["perm"] if G and case["by_token"] else None
        edges = s["offsets"].tolist() if G else [0, n]
        s["spans"] = [(g, lo, hi) for g, (lo, hi) in enumerate(zip(edges, edges[1:])) if hi > lo]
        return s
    s.update(_routing(case, gen))
    T, H, n, dtype = case["T"], case["H"], case["T"] * case["k"], TYPES[case["dtype"]]
    if not case["weighted"]:
        s["weight"] = None
    s["x"] = normal(T if op == "dispatch" else n, H, dtype=dtype)
    if op == "combine":
        # the experts' rows are in hand, with the order that brought them there
        s["pos"] = _positions(s["perm"], T, case["k"])
    if case["grad"]:
        s["gy"] = normal(n if op == "dispatch" else T, H, dtype=dtype)
        s["x"].requires_grad_()
        if s["weight"] is not None:
            s["weight"].requires_grad_()
    return s


# ---------------------------------------------------------------------------- plain forms
def _positions(perm, T, k):
    n = T * k
    pos = torch.full((n + 1,), -1, dtype=torch.int32, device=perm.device)
    to = torch.where(perm < 0, torch.full_like(perm, n), perm).long()
    pos.scatter_(0, to, torch.arange(n, dtype=torch.int32, device=perm.device))
    pos[n] = -1
    return pos[:n].view(T, k)


def _to_rows(x, perm, k, weight):
    """x's rows in the order of perm, weighted, in 32 bits; zero where perm names nothing."""
    a = perm.clamp(min=0).long()
    y = x.float()[a // k]
    if weight is not None:
        y = y * weight.reshape(-1)[a].unsqueeze(1)
    return torch.where((perm < 0).unsqueeze(1), torch.zeros((), device=x.device), y)


def _from_rows(y, pos, weight):
    """Each token's rows [T, k, H] in 32 bits, zero where it has none, and their weighted sum."""
    mine = torch.where((pos < 0).unsqueeze(2), torch.zeros((), device=y.device),
                       y.float()[pos.clamp(min=0).long()])
    total = (mine if weight is None else mine * weight.unsqueeze(2)).sum(dim=1)
    return mine, total


@torch.no_grad()
def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].double()
        scale = (x.abs().amax(dim=1) / 127).clamp(min=TINY).float()
        return {"q": torch.round(x / scale.double().unsqueeze(1)).to(torch.int8), "scale": scale}
    if op == "matmul":
        out, N = s["y"], s["N"]
        a, sa = s["a"], s["a_scale"]
        for g, lo, hi in s["spans"]:  # one product for each group: their matrices differ
            r = s["index"][lo:hi].long() // s["k"] if s["index"] is not None else slice(lo, hi)
            b, sb = (s["b"][g], s["b_scale"][g]) if s["G"] else (s["b"], s["b_scale"])
            y = (a[r].float() @ b.float().t()) * sa[r].unsqueeze(1) * sb
            if s["swiglu"]:
                gate, up = y[:, :N], y[:, N:]
                y = gate / (1 + torch.exp(-gate)) * up
            out[lo:hi] = y.to(out.dtype)
        return {"y": out}
    x, perm, w, k, dtype = s["x"], s["perm"], s["weight"], s["k"], s["x"].dtype
    if op == "dispatch":
        pos = _positions(perm, s["T"], k)
        out = {"y": _to_rows(x, perm, k, w).to(dtype), "pos": pos}
        if s["grad"]:
            mine, total = _from_rows(s["gy"], pos, w)
            out["gx"] = total.to(dtype)
            if w is not None:
                out["gw"] = (mine * x.float().unsqueeze(1)).sum(dim=2)
        return out
    pos = s["pos"]
    mine, total = _from_rows(x, pos, w)
    out = {"y": total.to(dtype)}
    if s["grad"]:
        out["gx"] = _to_rows(s["gy"], perm, k, w).to(dtype)
        if w is not None:
            out["gw"] = (mine * s["gy"].float().unsqueeze(1)).sum(dim=2)
    return out


# ---------------------------------------------------------------------------- own calls
def _own(s):
    from resident_expert_routing_amd import int8, rows

    op = s["op"]
    if op == "quantize":
        q, scale = int8.quantize(s["x"])
        return {"q": q, "scale": scale}
    if op == "matmul":
        y = int8.matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], offsets=s["offsets"],
                        index=s["index"], index_div=s["k"], swiglu=s["swiglu"], out=s["y"])
        return {"y": y}
    x, w = s["x"], s["weight"]
    if op == "dispatch":
        order = rows.RowOrder(s["perm"], s["T"], s["k"])
        y = rows.dispatch(x, order, w)
        out = {"y": y, "pos": order.pos}
    else:
        y = rows.combine(x, rows.RowOrder(s["perm"], s["T"], s["k"], pos=s["pos"]), w)
        out = {"y": y}
    if s["grad"]:
        grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["gy"])
        out["gx"] = grads[0]
        if w is not None:
            out["gw"] = grads[1]
    return out


def run(state):
    return _own(state) if own else _plain(state)


def _active(case):
    """The groups that a routing of this case is expected to use."""
    if not case["G"]:
        return 1.0
    q = [min(1.0, v * case["k"] * (1 - case["absent"])) for v in _popularity(case["G"])]
    return sum(1 - (1 - v) ** case["T"] for v in q)


def work(case):
    if case["op"] == "quantize":
        e = torch.empty(0, dtype=TYPES[case["dtype"]]).element_size()
        return {"bytes": case["M"] * (case["K"] * (e + 1) + 4), "flops": 2 * case["M"] * case["K"]}
    T, k, n = case["T"], case["k"], case["T"] * case["k"]
    live = n * (1 - case["absent"])
    if case["op"] == "matmul":
        N, K = case["N"], case["K"]
        wide = 2 * N if case["swiglu"] else N
        e = torch.empty(0, dtype=TYPES[case["out"]]).element_size()
        return {"bytes": (T if case["by_token"] else live) * (K + 4) + _active(case) * wide * (K + 4)
                + live * N * e + (4 * n if case["by_token"] and case["G"] else 0),
                "flops": 2 * live * wide * K}
    H = case["H"]
    e = torch.empty(0, dtype=TYPES[case["dtype"]]).element_size()
    one, many, w = T * H * e, live * H * e, 4 * n if case["weighted"] else 0
    full = n * H * e  # rows in the slots' order are all written
    if case["op"] == "dispatch":
        total = one + full + 8 * n + w
        if case["grad"]:
            total += many + one + 4 * n + (2 * w + one if case["weighted"] else 0)
    else:
        total = many + one + 4 * n + w
        if case["grad"]:
            total += one + full + 4 * n + (2 * w + many if case["weighted"] else 0)
    return {"bytes": total, "flops": (4 if case["grad"] else 2) * live * H}


def exact(case, seed):
    """The same from the definitions in 64 bits, token by token and group by group."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].detach().to(torch.float64)
        top = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
        scale = torch.maximum(top / 127.0, torch.full_like(top, TINY)).to(torch.float32).to(torch.float64)
        low = torch.floor(x / scale[:, None])
        rest = x / scale[:, None] - low
        up = (rest > 0.5) | ((rest == 0.5) & (low % 2 != 0))
        return {"q": (low + up).to(torch.int8), "scale": scale}
    T, k, n = case["T"], case["k"], case["T"] * case["k"]
    if op == "matmul":
        N, K = case["N"], case["K"]
        wide = 2 * N if case["swiglu"] else N
        if 2.0 * n * wide * K > 4e14 or (case["G"] or 1) * wide * K > 4e9:
            return None
        y = torch.zeros(n, N, dtype=torch.float64, device="cuda")
        for g, lo, hi in s["spans"]:
            r = torch.arange(lo, hi, device="cuda")
            if s["index"] is not None:
                r = torch.div(s["index"][lo:hi].to(torch.int64), k, rounding_mode="floor")
            left = s["a"][r].to(torch.float64) * s["a_scale"][r].to(torch.float64)[:, None]
            b, sb = (s["b"][g], s["b_scale"][g]) if case["G"] else (s["b"], s["b_scale"])
            right = b.to(torch.float64) * sb.to(torch.float64)[:, None]
            z = left @ right.t().contiguous()
            y[lo:hi] = torch.nn.functional.silu(z[:, :N]) * z[:, N:] if case["swiglu"] else z
        return {"y": y}
    if n * case["H"] > 2 ** 29:
        return None
    src = s["x"].detach().to(torch.float64)
    w = torch.ones(T, k, dtype=torch.float64, device="cuda") if s["weight"] is None \
        else s["weight"].detach().to(torch.float64)
    there = torch.nonzero(s["perm"] >= 0).reshape(-1)  # the rows that hold an assignment
    a = s["perm"][there].to(torch.int64)
    t, j = a // k, a % k

    def spread(v):
        out = torch.zeros(n, case["H"], dtype=torch.float64, device="cuda")
        out[there] = v[t] * w[t, j][:, None]
        return out

    def gather(v):
        out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, t, v[there] * w[t, j][:, None])

    def dots(many, one):
        out = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        out[t, j] = (many[there] * one[t]).sum(dim=1)
        return out

    if op == "dispatch":
        pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        pos[a] = there.to(torch.int32)
        out = {"y": spread(src), "pos": pos.view(T, k)}
    else:
        out = {"y": gather(src)}
    if case["grad"]:
        gy = s["gy"].to(torch.float64)
        out["gx"] = gather(gy) if op == "dispatch" else spread(gy)
        if s["weight"] is not None:
            out["gw"] = dots(gy, src) if op == "dispatch" else dots(src, gy)
    return out
