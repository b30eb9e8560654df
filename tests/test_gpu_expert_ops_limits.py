"""The separate expert operators on the GPU at the ends of their ranges,
against plain implementations in 64 bits.  Tolerances: U = 2^-24 bounds one
fp32 rounding, HALF[t] half a step of the output type; a 4-bit product takes at
most 33 steps of 2 U each per matrix instruction, four of them in a chain, then
the group's correction and the sum over groups and waves."""
import pytest
import torch

from mixture_experts_layer_34_amd import expert_ops as X
from tests.test_gpu_expert_ops import _close, _gen, _product_ref, _randn, _weights

pytestmark = pytest.mark.gpu

MIN, MAX = -2 ** 31, 2 ** 31 - 1


def test_offsets_far_outside_the_rows():
    """Neighbouring offsets whose difference passes 32 bits: empty ranges stay
    empty, and the one expert whose range covers the buffer has every row."""
    T, k, E, N, K = 10, 3, 6, 40, 128
    g = _gen(16)
    w = _weights(g, E, N, K, 64, True, "bf16")
    x = _randn(g, (T, K), "bf16")
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([5, MIN, MAX, MIN, -1, -5, 0], dtype=torch.int32, device="cuda")
    pairs = torch.arange(T * k, dtype=torch.int32, device="cuda")
    m = X.PairMap(T, k, E, 0, E, z(E), offsets, z(T, k), pairs)
    out = X.expert_matvec_int4(x, w, m, from_tokens=True)
    ref, tol = _product_ref(x.double()[pairs.long() // k], torch.ones(T * k, dtype=torch.long, device="cuda"), w, None,
                            "bf16")
    _close(out, ref, tol, "expert 1's rows")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
def test_quantize_the_widest_finite_group(group, symmetric):
    """Groups whose ends lie further apart than fp32 reaches, to the largest
    bf16 values: finite scales, and the codes and zero points of the same
    groups 2^-8 times as large, whose scales are 2^-8 times these, bit for bit
    (a power of two moves no rounding)."""
    big = torch.finfo(torch.bfloat16).max
    v = (torch.rand((6, 2 * group), generator=_gen(group)) * 2 - 1) * big
    v[0, 0], v[0, 1] = big, -big
    v[1, 3], v[1, 9] = big, -1.0
    v[2] = -v[2].abs()
    v = v.clamp(-big, big).bfloat16()
    assert float((v.double().amax(1) - v.double().amin(1)).max()) > torch.finfo(torch.float32).max
    w, small = (X.quantize_int4(u.cuda(), group, symmetric) for u in (v, v * 2.0 ** -8))
    assert torch.isfinite(w.scales).all()
    assert torch.equal(w.codes, small.codes) and torch.equal(w.scales, small.scales * 2.0 ** 8)
    assert symmetric or torch.equal(w.zeros, small.zeros)
