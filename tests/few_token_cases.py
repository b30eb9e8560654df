"""The layer for a few tokens in 64 bits with the bound of one rounding, out's own:
h is handed on from the first products to the second with 16 bits of mantissa or
more and fp32's range, whatever the type of the weights.

U and gam are those of tests/adapter_cases.py.  Beside 16-bit weights h is handed on
as a bf16 part and its bf16 rest, half a step each: 2^-8 of the rest, which is at
most 2^-8 of h, so it is off by 2^-16 of itself at most.  (fp16 weights are two bf16
parts exactly: 8 bits cut off of 11, and 3.)"""
import torch

from tests.adapter_cases import U, gam, route64

SPLIT_H = {"f32": 0.0, "bf16": 2.0 ** -16, "f16": 2.0 ** -16}
TINY_H = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -133}  # a subnormal step


def layer_once64(x, logits, w1, w3, w2, k, eb=0, gating="softmax", renorm=False, adapter=None, lora=None):
    """(out, its bound before its one rounding)."""
    dt = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[x.dtype]
    idx, gate = route64(logits, k, gating, renorm)
    T, d = x.shape
    F = w1.shape[1]
    out, err = torch.zeros((T, d), dtype=torch.float64), torch.zeros((T, d), dtype=torch.float64)
    xd = x.double().cpu()

    def product(w, v, verr, terms, m, e, l):
        w = w[e].double().cpu()
        z, zerr = w @ v, gam(terms) * (w.abs() @ (v.abs() + verr)) + w.abs() @ verr
        if l >= 0 and lora[m] is not None:
            a, b = lora[m].A[l, e].double().cpu(), lora[m].B[l, e].double().cpu()
            s = 1.0 if lora[m].scale is None else float(lora[m].scale[l])
            u, uerr = a @ v, gam(a.shape[1]) * (a.abs() @ (v.abs() + verr)) + a.abs() @ verr
            z = z + s * (b @ u)
            zerr = zerr + abs(s) * (b.abs() @ (uerr + gam(b.shape[1] + 2) * (u.abs() + uerr)))
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
            a, aerr = product(w1, xd[t], none, d, 0, e, l)
            b, berr = product(w3, xd[t], none, d, 1, e, l)
            silu = a * torch.sigmoid(a)
            gt = float(gate[t, j])
            h = gt * silu * b
            # |silu'| <= 1.1; the fast exp and the division, and the gate's: 2^-18 each
            herr = gt * (1.1 * aerr * (b.abs() + berr) + (silu.abs() + 1.1 * aerr) * berr) + \
                (2.0 ** -17 + 4 * U) * h.abs()
            herr = herr + SPLIT_H[dt] * (h.abs() + herr) + TINY_H[dt]
            # the sum goes on over the token's experts, up to four products an element
            y, yerr = product(w2, h, herr, 4 * k * F, 2, e, l)
            out[t] += y
            err[t] += yerr
    return out, err + 4 * U * out.abs()
