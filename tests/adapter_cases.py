"""Inputs of the tests of low-rank adapters and of the layer for a few tokens,
their plain forms in 64 bits, and how far an fp32 computation of them may be off.

U = 2^-24 bounds one fp32 rounding.  A sum of n products in fp32, in any order, is
off by at most gam(n) = 2 (n + 8) U times the sum of the products' magnitudes (a
matrix instruction need not round to nearest: 2 U a step; 8 for the sums of lanes
and waves and for a factor applied in between)."""
import torch

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # a subnormal step
# u and du enter a 16-bit product as a rounded part and its rounded rest
SPLIT = {"f32": 0.0, "bf16": 2.0 ** -16, "f16": 2.0 ** -22}


def gam(n):
    return 2 * (n + 8) * U


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, shape, dt="f32", std=1.0):
    return (torch.randn(shape, generator=g) * std).to(DT[dt]).cuda()


def close(got, ref, tol, what):
    got, ref, tol = got.double().cpu(), ref.double().cpu(), tol.double().cpu()
    assert got.shape == ref.shape, what
    assert not torch.isnan(got).any(), what
    bad = (got - ref).abs() - tol
    assert bad.numel() == 0 or float(bad.max()) <= 0, \
        f"{what}: {float((got - ref).abs().max())} off, {float(bad.max())} past the bound"


# ------------------------------------------------------------------ adapters beside a projection
def lora64(x, ids, A, B, scale, y=None):
    """(out, its bound before rounding, u, its bound) of rows in the order of ids."""
    xd = x.double().cpu()
    out = torch.zeros((len(ids), B.shape[1]), dtype=torch.float64) if y is None else y.double().cpu().clone()
    err = 2 * U * out.abs()
    u = torch.zeros((len(ids), A.shape[1]), dtype=torch.float64)
    uerr = torch.zeros_like(u)
    K, r = A.shape[2], A.shape[1]
    dt = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[x.dtype]
    for g in range(A.shape[0]):
        rows = (ids == g).nonzero()[:, 0]
        if not len(rows):
            continue
        a, b = A[g].double().cpu(), B[g].double().cpu()
        s = 1.0 if scale is None else float(scale[g])
        u[rows] = xd[rows] @ a.t()
        uerr[rows] = gam(K) * (xd[rows].abs() @ a.abs().t())
        out[rows] += s * (u[rows] @ b.t())
        mag = (u[rows].abs() + uerr[rows]) @ b.abs().t()
        err[rows] += abs(s) * (uerr[rows] @ b.abs().t() + (gam(2 * r) + SPLIT[dt]) * mag) + 2 * U * out[rows].abs()
    return out, err, u, uerr


def rounded(ref, err, dt):
    """The bound of a value off by err and then rounded to dt."""
    return err * (1 + HALF[dt]) + HALF[dt] * ref.abs() + TINY[dt]


def lora_grad64(dout, x, u, ids, A, B, scale, base=None):
    """{name: (value, bound)} of dx, dA, dB, in the order of ids."""
    rev = lora64(dout, ids, B.transpose(1, 2), A.transpose(1, 2), scale, base)
    dx, dxerr, du, duerr = rev
    G, r, K = A.shape
    N = B.shape[1]
    xd, yd, ud = x.double().cpu(), dout.double().cpu(), u.double().cpu()
    dA, eA = torch.zeros((G, r, K), dtype=torch.float64), torch.zeros((G, r, K), dtype=torch.float64)
    dB, eB = torch.zeros((G, N, r), dtype=torch.float64), torch.zeros((G, N, r), dtype=torch.float64)
    for g in range(G):
        rows = (ids == g).nonzero()[:, 0]
        s = 1.0 if scale is None else float(scale[g])
        n = len(rows)
        dA[g] = s * du[rows].t() @ xd[rows]
        eA[g] = abs(s) * (duerr[rows].t() @ xd[rows].abs() + gam(n) * (du[rows].abs() + duerr[rows]).t() @ xd[rows].abs())
        dB[g] = s * yd[rows].t() @ ud[rows]
        eB[g] = abs(s) * gam(n) * yd[rows].abs().t() @ ud[rows].abs()
    return {"dx": (dx, dxerr), "dA": (dA, eA), "dB": (dB, eB)}


# ------------------------------------------------------------------ the layer for a few tokens
def route64(logits, k, gating, renorm):
    """Experts by (logit descending, index ascending) and their gates."""
    ld = logits.double().cpu()
    ld = torch.where(torch.isnan(ld), torch.full_like(ld, -float("inf")), ld)
    idx = torch.sort(ld, dim=1, descending=True, stable=True).indices[:, :k]
    p = torch.sigmoid(ld) if gating == "sigmoid" else torch.softmax(ld, 1)
    gate = torch.gather(p, 1, idx)
    return idx, gate / gate.sum(1, keepdim=True) if renorm else gate


def layer64(x, logits, w1, w3, w2, k, eb=0, gating="softmax", renorm=False, adapter=None, lora=None):
    """(out, its bound before rounding, idx, gate): every pair by itself."""
    dt = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[x.dtype]
    idx, gate = route64(logits, k, gating, renorm)
    T, d = x.shape
    F = w1.shape[1]
    # a gate: exp of a rounded difference, a sum of E exps, a division, k of them added
    gerr = 2.0 ** -18
    out, err = torch.zeros((T, d), dtype=torch.float64), torch.zeros((T, d), dtype=torch.float64)
    xd = x.double().cpu()

    def product(w, v, verr, m, e, l):
        """W v and its bound, the adapter's share in it; v off by verr."""
        w = w[e].double().cpu()
        z, zerr = w @ v, gam(w.shape[1]) * (w.abs() @ v.abs()) + w.abs() @ verr
        if l >= 0 and lora[m] is not None:
            a, b = lora[m].A[l, e].double().cpu(), lora[m].B[l, e].double().cpu()
            s = 1.0 if lora[m].scale is None else float(lora[m].scale[l])
            u, uerr = a @ v, gam(a.shape[1]) * (a.abs() @ v.abs()) + a.abs() @ verr
            z = z + s * (b @ u)
            zerr = zerr + abs(s) * (b.abs() @ (uerr + gam(b.shape[1]) * u.abs()))
        return z, zerr + 4 * U * z.abs()

    for t in range(T):
        l = -1 if adapter is None else int(adapter[t])
        if lora is not None and not 0 <= l < max(w.A.shape[0] for w in lora if w is not None):
            l = -1
        for j in range(k):
            e = int(idx[t, j]) - eb
            if not 0 <= e < w1.shape[0]:
                continue
            none = torch.zeros(d, dtype=torch.float64)
            a, aerr = product(w1, xd[t], none, 0, e, l)
            b, berr = product(w3, xd[t], none, 1, e, l)
            silu = a * torch.sigmoid(a)
            gt = float(gate[t, j])
            h = gt * silu * b
            # |silu'| <= 1.1; the fast exp and the division: 2^-18 of silu
            herr = gt * (1.1 * aerr * (b.abs() + berr) + (silu.abs() + 1.1 * aerr) * berr) + \
                (gerr + 2.0 ** -18 + 4 * U) * h.abs()
            herr = herr + HALF[dt] * (h.abs() + herr) + TINY[dt]
            y, yerr = product(w2, h, herr, 2, e, l)
            out[t] += y
            # every sum goes on over the token's experts: its length, not F alone
            err[t] += yerr + gam(k * F) * (w2[e].double().cpu().abs() @ (h.abs() + herr))
    return out, err + 4 * U * out.abs(), idx, gate
