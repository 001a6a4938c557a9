"""Cases for the products of the routed experts in floating point and in 4-bit weights, their
plain forms and their exact values.

Operators:
  grouped  products of ragged groups of rows, one matrix for each group, with `swiglu` the gate
           and up products and silu(gate) * up; with `grad`, forward and backward: the
           gradients of the rows (of the tokens, where rows are named by token) and of the
           matrices.  layout "nk": a group's matrix has a row for each output, "kn": a row
           for each input
  int4     products with weights of 4 bits, a scale (and, with `zeros`, a zero point) for
           each `group` weights of a row, over the groups of a bucketing (G > 0) or dense
           (G = 0); with `swiglu` as above

Where `own` is true, `run` makes the framework's calls; otherwise it takes elementary torch
operations.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token through a small layer, where the call's latency counts
        dict(name="grouped token", op="grouped", T=1, k=4, G=10, N=128, K=256, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", layout="nk", grad=False),
        # the gate and up products of one decode step of 8 sequences
        dict(name="grouped step", op="grouped", T=8, k=8, G=230, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", layout="nk", grad=False),
        # the down products of a prompt batch
        dict(name="grouped prefill", op="grouped", T=2048, k=8, G=166, N=4096, K=2048,
             swiglu=False, by_token=False, absent=0.0, dtype="bf16", layout="nk", grad=False),
        # the gate and up products of a long prefill chunk
        dict(name="grouped long", op="grouped", T=8192, k=8, G=130, N=2048, K=6144, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", layout="nk", grad=False),
        # a training step's gate and up products: one rank's tokens over one rank's experts
        dict(name="grouped train", op="grouped", T=4096, k=8, G=64, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", layout="nk", grad=True),
        # the down products of the same, matrices kept with a row for each input, some picks
        # not routable
        dict(name="grouped train kn fp16", op="grouped", T=2048, k=8, G=32, N=4096, K=2048,
             swiglu=False, by_token=False, absent=0.1, dtype="fp16", layout="kn", grad=True),
        # a small odd model trained in 32 bits, as one does to check gradients
        dict(name="grouped train odd fp32", op="grouped", T=333, k=3, G=7, N=515, K=259,
             swiglu=True, by_token=True, absent=0.2, dtype="fp32", layout="nk", grad=True),
        # a shared expert's gate and up products for a single token
        dict(name="int4 token", op="int4", T=1, k=1, G=0, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", group=128, zeros=False),
        # the routed experts' gate and up products of one decode step of 8 sequences
        dict(name="int4 step", op="int4", T=8, k=8, G=230, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", group=128, zeros=False),
        # their down products, from weights with zero points
        dict(name="int4 step down zeros", op="int4", T=8, k=8, G=230, N=4096, K=2048,
             swiglu=False, by_token=False, absent=0.0, dtype="fp16", group=64, zeros=True),
        # a step of many sequences, fine groups
        dict(name="int4 batch", op="int4", T=256, k=8, G=166, N=2048, K=4096, swiglu=True,
             by_token=True, absent=0.0, dtype="bf16", group=32, zeros=True),
        # a small odd model, activations in 32 bits, some picks not routable
        dict(name="int4 odd fp32", op="int4", T=37, k=3, G=9, N=515, K=1000, swiglu=False,
             by_token=True, absent=0.2, dtype="fp32", group=64, zeros=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "int4"])
    N, K = _log(rng, 33, 4096), _log(rng, 64, 6144)
    if rng.random() < 0.5:  # a multiple of 128, as most models have
        N, K = -(-N // 128) * 128, -(-K // 128) * 128
    swiglu = rng.random() < 0.5
    if swiglu:
        N = min(N, 2048)
    k, G = rng.randint(1, 8), rng.randint(2, 230)
    absent = rng.choice([0.0, 0.0, 0.2])
    by_token = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"])
    if op == "int4":
        T = _log(rng, 1, 256)
        if rng.random() < 0.25:
            G, k, absent = 0, 1, 0.0
        return dict(op=op, T=T, k=k, G=G, N=N, K=K, swiglu=swiglu, by_token=by_token,
                    absent=absent, dtype=dtype, group=rng.choice([32, 64, 128]),
                    zeros=rng.random() < 0.5)
    grad = rng.random() < 0.5
    wide = 2 * N if swiglu else N
    T = _log(rng, 1, 8192)
    most = 3e12 if dtype != "fp32" else 4e11  # flops
    T = max(1, min(T, int(most / (2 * k * wide * K * (3 if grad else 1)))))
    if grad:
        G = max(2, min(G, int(1e9 / (wide * K))))
    return dict(op=op, T=T, k=min(k, G), G=G, N=N, K=K, swiglu=swiglu, by_token=by_token,
                absent=absent, dtype=dtype, layout=rng.choice(["nk", "kn"]), grad=grad)


def _popularity(G):
    p = [(i + 1.0) ** -0.8 for i in range(G)]
    s = sum(p)
    return [v / s for v in p]


def _routing(case, gen):
    """Picks as a router makes them: k distinct slots of G for each token, popular slots
    more often, some absent; and the bucketing of the assignments by slot."""
    T, k, G = case["T"], min(case["k"], case["G"]), case["G"]
    dev = "cuda"
    p = torch.tensor(_popularity(G), device=dev).log()
    p = p[torch.randperm(G, device=dev, generator=gen)]
    u = torch.rand(T, G, device=dev, generator=gen).clamp_(1e-12, 1 - 1e-7)
    sel = (p - (-u.log()).log()).topk(k, dim=1).indices.sort(dim=1).values
    if k < case["k"]:  # fewer slots than picks: the rest have no row
        sel = torch.nn.functional.pad(sel, (0, case["k"] - k), value=-1)
    if case["absent"]:
        gone = torch.rand(T, case["k"], device=dev, generator=gen) < case["absent"]
        if T > 2:
            gone[T // 2] = True  # a token that has no routable expert at all
        sel = torch.where(gone, torch.full_like(sel, -1), sel)
    key = torch.where(sel < 0, torch.full_like(sel, G), sel).reshape(-1)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=G + 1)
    present = int(counts[:G].sum())
    perm = order.to(torch.int32)
    perm[present:] = -1
    offsets = torch.zeros(G + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts[:G].cumsum(0).to(torch.int32)
    return perm, offsets


def _packed(codes, scale, zero):
    """Codes [.., N, K] (K a multiple of 128 here, N of 16) and a scale and zero point for
    each group [.., N, groups], as a program that serves them keeps them: codes in tiles of
    16 rows by 128 weights, 64 bytes a row, in words of eight weights whose weight 2j is at
    bit 4j and whose weight 2j+1 is at bit 16+4j; scales and zero points by 16 rows."""
    *lead, N, K = codes.shape
    c = codes.view(-1, N // 16, 16, K // 128, 16, 4, 2)
    out = torch.empty(c.shape[0], N // 16, K // 128, 16, 16, 2, 2, dtype=torch.uint8,
                      device=codes.device)
    for i in range(c.shape[0]):
        t = c[i].permute(0, 2, 1, 3, 5, 4)  # [N/16, K/128, row, word, parity, pair]
        out[i] = t[..., 0::2] | (t[..., 1::2] << 4)
    rows16 = lambda t: t.view(*lead, N // 16, 16, -1).transpose(-1, -2).contiguous()
    return (out.view(*lead, N // 16, K // 128, 16, 64), rows16(scale),
            None if zero is None else rows16(zero))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    T, k, G, N, K = (case[v] for v in ("T", "k", "G", "N", "K"))
    n, wide = T * k, 2 * N if case["swiglu"] else N
    s = dict(case)
    s["perm"], s["offsets"] = _routing(case, gen) if G else (None, None)
    edges = s["offsets"].tolist() if G else [0, n]
    s["spans"] = [(g, lo, hi) for g, (lo, hi) in enumerate(zip(edges, edges[1:])) if hi > lo]
    s["last"] = edges[-1]
    s["index"] = s["perm"] if G and case["by_token"] else None
    s["x"] = torch.randn(T if case["by_token"] else n, K, device="cuda", generator=gen).to(dtype)
    lead = (G,) if G else ()
    if case["op"] == "grouped":
        # weights of about unit gain; in "kn" the view that the product takes is transposed
        shape = (wide, K) if case["layout"] == "nk" else (K, wide)
        b = torch.empty(G, *shape, dtype=dtype, device="cuda")
        for g in range(G):
            b[g] = (torch.randn(*shape, device="cuda", generator=gen) * K ** -0.5).to(dtype)
        if case["grad"]:
            b.requires_grad_()
            s["x"].requires_grad_()
            s["gy"] = torch.randn(n, N, device="cuda", generator=gen).to(dtype)
        s["b"] = b
        return s
    # codes as a quantiser leaves them: bell-shaped around the zero point, cut at both ends
    Np, Kp, gs = -(-wide // 16) * 16, -(-K // 128) * 128, case["group"]
    codes = torch.zeros(*lead, Np, Kp, dtype=torch.uint8, device="cuda")
    for part in (codes.view(-1, Np, Kp)):
        w = torch.randn(wide, K, device="cuda", generator=gen) * 2.7 + 8
        part[:wide, :K] = w.round_().clamp_(0, 15).to(torch.uint8)
    sdt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
    scale = torch.zeros(*lead, Np, Kp // gs, dtype=sdt, device="cuda")
    live = (wide, -(-K // gs))
    scale[..., :wide, :live[1]] = (torch.rand(*lead, *live, device="cuda", generator=gen) + 0.5) \
        .mul_(0.37 * K ** -0.5).to(sdt)
    zero = None
    if case["zeros"]:
        zero = torch.zeros(*lead, Np, Kp // gs, dtype=torch.uint8, device="cuda")
        zero[..., :wide, :live[1]] = torch.randint(5, 12, (*lead, *live), device="cuda",
                                                   generator=gen).to(torch.uint8)
    s["packed"] = _packed(codes, scale, zero)
    s["codes"] = codes[..., :wide, :K]
    s["scale"] = scale[..., :wide, :live[1]]
    s["zero"] = None if zero is None else zero[..., :wide, :live[1]]
    s["y"] = torch.zeros(n, N, dtype=dtype, device="cuda")  # the layer's own buffer
    return s


# ---------------------------------------------------------------------------- plain forms
def _rows_of(s, lo, hi):
    return s["index"][lo:hi].long() // s["k"] if s["index"] is not None else slice(lo, hi)


def _silu(gate):
    """sigmoid, and silu, of gates in 32 bits."""
    p = 1 / (1 + torch.exp(-gate))
    return p, gate * p


def _plain_int4(s):
    out, N, K, gs = s["y"], s["N"], s["K"], s["group"]
    for g, lo, hi in s["spans"]:  # one product for each group: their matrices differ
        at = (g,) if s["G"] else ()
        zero = 8.0 if s["zero"] is None else \
            s["zero"][at].float().repeat_interleave(gs, dim=1)[:, :K]
        b = (s["codes"][at].float() - zero) * s["scale"][at].float().repeat_interleave(
            gs, dim=1)[:, :K]
        y = s["x"][_rows_of(s, lo, hi)].float() @ b.t()
        if s["swiglu"]:
            y = _silu(y[:, :N])[1] * y[:, N:]
        out[lo:hi] = y.to(out.dtype)
    return {"y": out}


def _plain_grouped(s):
    x, b, N, dtype = s["x"], s["b"], s["N"], s["x"].dtype
    n = s["T"] * s["k"]
    y = torch.zeros(n, N, dtype=dtype, device=x.device)
    nk = s["layout"] == "nk"
    if s["grad"]:
        gx = torch.zeros(x.shape, device=x.device)
        gb = torch.zeros_like(b)
    for g, lo, hi in s["spans"]:  # one product for each group: their matrices differ
        r = _rows_of(s, lo, hi)
        a, w = x[r].float(), b[g].float()
        z = a @ (w.t() if nk else w)
        if s["swiglu"]:
            p, v = _silu(z[:, :N])
            y[lo:hi] = (v * z[:, N:]).to(dtype)
        else:
            y[lo:hi] = z.to(dtype)
        if not s["grad"]:
            continue
        gz = s["gy"][lo:hi].float()
        if s["swiglu"]:
            gz = torch.cat([gz * z[:, N:] * (p + v * (1 - p)), gz * v], dim=1)
        ga = gz @ (w if nk else w.t())
        if s["index"] is None:
            gx[lo:hi] = ga
        else:  # a token has at most one row in a group
            gx[r] += ga
        gb[g] = (gz.t() @ a if nk else a.t() @ gz).to(dtype)
    if not s["grad"]:
        return {"y": y}
    return {"y": y, "gx": gx.to(dtype), "gb": gb}


# ---------------------------------------------------------------------------- own calls
def _own(s):
    from resident_expert_routing_amd import grouped, int4, rows

    if s["op"] == "int4":
        w = int4.Int4Weight(*s["packed"], N=s["codes"].shape[-2], K=s["K"])
        y = int4.matmul(s["x"], w, offsets=s["offsets"], index=s["index"], index_div=s["k"],
                        swiglu=s["swiglu"], out=s["y"])
        return {"y": y}
    b = s["b"] if s["layout"] == "nk" else s["b"].transpose(1, 2)
    if not s["grad"]:
        y = grouped.matmul(s["x"], b, s["offsets"], index=s["index"], index_div=s["k"],
                           swiglu=s["swiglu"])
        return {"y": y}
    order = rows.RowOrder(s["perm"], s["T"], s["k"]) if s["index"] is not None else None
    y = grouped.matmul(s["x"], b, s["offsets"], order=order, swiglu=s["swiglu"])
    gx, gb = torch.autograd.grad(y, [s["x"], s["b"]], s["gy"])
    return {"y": y, "gx": gx, "gb": gb}


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain_int4(state) if state["op"] == "int4" else _plain_grouped(state)


def _active(case):
    """The groups that a routing of this case is expected to use."""
    if not case["G"]:
        return 1.0
    q = [min(1.0, v * min(case["k"], case["G"]) * (1 - case["absent"]))
         for v in _popularity(case["G"])]
    return sum(1 - (1 - v) ** case["T"] for v in q)


def work(case):
    T, k, N, K = (case[v] for v in ("T", "k", "N", "K"))
    n = T * k
    live = T * (min(k, case["G"]) if case["G"] else k) * (1 - case["absent"])
    wide = 2 * N if case["swiglu"] else N
    e = torch.empty(0, dtype=TYPES[case["dtype"]]).element_size()
    rows = T if case["by_token"] else live
    order = 4 * n if case["by_token"] and case["G"] else 0
    if case["op"] == "int4":
        groups = -(-K // case["group"])
        matrix = wide * (K / 2 + groups * (3 if case["zeros"] else 2))
        return {"bytes": rows * K * e + order + _active(case) * matrix + live * N * e,
                "flops": 2 * live * wide * K}
    total = rows * K * e + order + _active(case) * wide * K * e + n * N * e
    if case["grad"]:
        total += live * N * e + (T if case["by_token"] else n) * K * e + case["G"] * wide * K * e
    return {"bytes": total, "flops": (6 if case["grad"] else 2) * live * wide * K}


def exact(case, seed):
    """The same from the definitions in 64 bits, group by group."""
    s = prepare(case, seed)
    T, k, N, K = (case[v] for v in ("T", "k", "N", "K"))
    n, f64 = T * k, torch.float64
    x = s["x"].detach().to(f64)
    y = torch.zeros(n, N, dtype=f64, device="cuda")
    grad = case["op"] == "grouped" and case["grad"]
    if grad:
        gx = torch.zeros(x.shape, dtype=f64, device="cuda")
        gb = torch.zeros(s["b"].shape, dtype=f64, device="cuda")
    for g, lo, hi in s["spans"]:
        r = torch.arange(lo, hi, device="cuda")
        if s["index"] is not None:
            r = torch.div(s["index"][lo:hi].to(torch.int64), k, rounding_mode="floor")
        if case["op"] == "int4":
            of = torch.arange(K, device="cuda") // case["group"]  # the group of each weight
            c, sc, z = (t if t is None or not case["G"] else t[g]
                        for t in (s["codes"], s["scale"], s["zero"]))
            z = torch.full_like(sc, 8, dtype=f64) if z is None else z.to(f64)
            w = (c.to(f64) - z[:, of]) * sc.to(f64)[:, of]
        else:
            w = s["b"].detach()[g].to(f64)
            if case["layout"] == "kn":
                w = w.t().contiguous()
        a = x[r]
        z = torch.matmul(a, w.t().contiguous())
        if case["swiglu"]:
            gate, up = z[:, :N], z[:, N:]
            sig = torch.sigmoid(gate)
            y[lo:hi] = gate * sig * up
        else:
            y[lo:hi] = z
        if grad:
            d = s["gy"][lo:hi].to(f64)
            if case["swiglu"]:
                d = torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * gate * sig], dim=1)
            gx.index_add_(0, r, torch.matmul(d, w))
            gw = torch.matmul(d.t().contiguous(), a)
            gb[g] = gw if case["layout"] == "nk" else gw.t()
    return {"y": y, "gx": gx, "gb": gb} if grad else {"y": y}
