"""Float64 reference of the grouped products, with a bound on what float32 sums and the
roundings of the element type may add to each value.

A sum of K products in float32 is off by at most K * 2^-23 of the sum of their magnitudes
(2^-24 for each addition rounded to nearest, twice that where the matrix instruction cuts
instead); a rounding to the element type by half a step, eps / 2 of the value, plus half
the smallest step near zero."""
import torch

STEP = 2.0 ** -23


def rounding(v, dtype):
    f = torch.finfo(dtype)
    return v.abs() * (f.eps / 2) * 1.0001 + f.smallest_normal * f.eps


def bucketing(counts, gen=None, k=1, T=None, tail=0):
    """(perm, offsets) of groups with these rows: assignments in a shuffled order, `tail`
    rows more in no group (perm -1)."""
    n = sum(counts)
    offsets = torch.zeros(len(counts) + 1, dtype=torch.int32)
    offsets[1:] = torch.tensor(counts).cumsum(0).int()
    total = n + tail
    perm = torch.randperm(total, generator=gen)[:n].int()
    return torch.cat([perm, torch.full((tail,), -1, dtype=torch.int32)]), offsets


def silu(g):
    return g * torch.sigmoid(g)


def dsilu(g):
    s = torch.sigmoid(g)
    return s * (1 + g * (1 - s))


class Reference:
    """out, and with `grad` (the gradient of out) da and db, each with its bound; a [rows, K]
    and b [G, wide, K], index the row of a for each row of out (None: itself)."""

    def __init__(self, a, b, offsets, index, M, swiglu, dtype, grad=None, token_sum=False):
        a, b = a.double(), b.double()
        G, wide, K = b.shape
        N = wide // 2 if swiglu else wide
        dev = a.device
        new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
        self.out, self.out_tol = new(M, N), new(M, N)
        if grad is not None:
            d_all = grad.double()
            self.da, self.da_tol = new(*a.shape), new(*a.shape)
            self.db, self.db_tol = new(G, wide, K), new(G, wide, K)
            rows_of = new(a.shape[0])
        edges = offsets.clamp(0, M).tolist()
        for g in range(G):
            lo, hi = edges[g], edges[g + 1]
            if hi <= lo:
                continue
            p = torch.arange(lo, hi, device=dev)
            r = p if index is None else index[lo:hi].long()
            ok = (r >= 0) & (r < a.shape[0])
            p, r = p[ok], r[ok]
            x, w = a[r], b[g]
            z = x @ w.t().contiguous()
            dz_sum = K * STEP * (x.abs() @ w.abs().t().contiguous())
            if swiglu:
                gt, up = z[:, :N], z[:, N:]
                eg, eu = dz_sum[:, :N], dz_sum[:, N:]
                y = silu(gt) * up
                tol = 1.1 * eg * (up.abs() + eu) + silu(gt).abs() * eu + \
                    (1.25 * gt.abs() + 12) * 2.0 ** -24 * y.abs()
            else:
                y, tol = z, dz_sum
            self.out[p] = y
            self.out_tol[p] = tol + rounding(y.abs() + tol, dtype)
            if grad is None:
                continue
            d = d_all[p]
            if swiglu:
                # kept before SwiGLU in float32; the gradient through it is rounded to the type
                dz = torch.cat([d * up * dsilu(gt), d * silu(gt)], 1)
                f32 = 2.0 ** -24 * (24 + 2.5 * gt.abs())
                e = torch.cat([
                    d.abs() * (1.1 * eu + 0.5 * eg * (up.abs() + eu)
                               + up.abs() * (1.1 + gt.abs()) * f32),
                    d.abs() * (1.1 * eg + silu(gt).abs() * f32)], 1)
                e = e + rounding(dz.abs() + e, dtype)
            else:
                dz, e = d, torch.zeros_like(d)
            full = dz.abs() + e
            da = dz @ w
            da_tol = e @ w.abs() + wide * STEP * (full @ w.abs())
            da_tol = da_tol + rounding(da.abs() + da_tol, dtype)
            self.da.index_add_(0, r, da)
            self.da_tol.index_add_(0, r, da_tol)
            rows_of.index_add_(0, r, torch.ones_like(r, dtype=torch.float64))
            t = lambda v: v.t().contiguous()
            self.db[g] = t(dz) @ x
            db_tol = t(e) @ x.abs() + (hi - lo) * STEP * (t(full) @ x.abs())
            self.db_tol[g] = db_tol + rounding(self.db[g].abs() + db_tol, dtype)
        if grad is not None and token_sum:
            # the sum of a token's rows: float32 additions and one rounding
            self.da_tol += (self.da.abs() + self.da_tol) * rows_of[:, None] * 2.0 ** -22
            self.da_tol += rounding(self.da.abs() + self.da_tol, dtype)


def worst(got, want, tol):
    """The largest of |got - want| / tol; infinite for a NaN or an infinity."""
    if got.numel() == 0:
        return 0.0
    d = (got.double() - want).abs()
    ratio = torch.where(d <= 0, torch.zeros_like(d), d / tol.clamp_min(1e-300))
    return float(torch.where(torch.isfinite(got.double()), ratio,
                             torch.full_like(ratio, float("inf"))).max())


def within(got, want, tol) -> bool:
    """worst() at most 1 (a name of its own, so that a failure prints one number)."""
    ratio = worst(got, want, tol)
    if not ratio <= 1:
        print(f"off by {ratio:.3f} of the bound", flush=True)
    return ratio <= 1
