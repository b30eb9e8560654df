"""The layer for a few tokens rounds to its type once, at the end: h keeps fp32's
range and 16 bits of mantissa or more between the two products, against 64 bits
(tests/few_token_cases.py derives the bounds)."""
import pytest
import torch

from mixture_experts_layer_34_amd import expert_ops as X
from tests.adapter_cases import DT, close, gen, randn, rounded
from tests.few_token_cases import layer_once64
from tests.gpu_case import note

pytestmark = pytest.mark.gpu


def _case(T, d, F, E, dt, seed, up=1.0, down=1.0):
    """up, down: factors on W1 and W3 each, and on W2."""
    g = gen(seed)
    return [randn(g, (T, d), dt), randn(g, (T, E)), randn(g, (E, F, d), dt, up * d ** -0.5),
            randn(g, (E, F, d), dt, up * d ** -0.5), randn(g, (E, d, F), dt, down * F ** -0.5)]


def _lora(T, d, F, E, L, r, dt, seed, up=1.0, down=1.0):
    g = gen(seed)
    ws = [X.LoraWeights(randn(g, (L, E, r, K), dt, s * K ** -0.5), randn(g, (L, E, N, r), dt, 0.5 * r ** -0.5),
                        torch.rand(L, generator=g).cuda() + 0.5)
          for N, K, s in ((F, d, up), (F, d, up), (d, F, down))]
    return torch.randint(-1, L, (T,), generator=g, dtype=torch.int32).cuda(), ws


def _check(args, k, dt, **kw):
    got, _, _ = X.few_token_layer(*args, k, **kw)
    ref, err = layer_once64(*args, k, **kw)
    close(got, ref, rounded(ref, err, dt), "out")
    return got, ref


# at most eight tokens (both parts of h in one matrix instruction) and more; less than
# a chunk of 128 columns of h, whole ones, a part at the end, rows of less than 16
# bytes, odd rows, and widths of out past 4096 (two column tiles a workgroup)
SHAPES = [(1, 64, 128, 4, 2, "bf16"), (16, 96, 256, 8, 4, "bf16"), (5, 130, 67, 9, 4, "bf16"),
          (3, 40, 5, 4, 2, "bf16"), (7, 4200, 129, 4, 2, "bf16"), (4, 4100, 130, 3, 2, "bf16"),
          (1, 64, 128, 4, 2, "f16"), (16, 96, 256, 8, 4, "f16"), (5, 130, 67, 9, 4, "f16"), (3, 40, 5, 4, 2, "f16"),
          (7, 4200, 129, 4, 2, "f16"), (4, 4100, 130, 3, 2, "f16"), (2, 4160, 64, 3, 1, "f16"),
          (16, 200, 1411, 6, 3, "f16"), (8, 72, 1411, 6, 3, "bf16"), (9, 72, 1411, 6, 3, "bf16"),
          (8, 4104, 67, 3, 2, "f16"), (9, 4104, 67, 3, 2, "f16"), (10, 40, 5, 4, 2, "bf16"), (12, 40, 1, 4, 2, "f16"),
          (11, 4100, 129, 3, 1, "bf16"), (6, 64, 97, 5, 2, "f32")]
# more than eight tokens an expert: one expert, all of them, some of many (in both
# halves of a thread's slots), beside ones with eight or fewer
SHAPES += [(16, 72, 136, 1, 1, "bf16"), (9, 64, 64, 1, 1, "f16"), (16, 72, 264, 3, 3, "bf16"),
           (13, 4104, 72, 2, 2, "f16"), (16, 48, 40, 700, 64, "bf16"), (16, 64, 48, 4, 2, "f16"),
           (16, 40, 24, 90, 50, "bf16"), (10, 200, 520, 5, 4, "f16"), (12, 56, 130, 5, 3, "bf16"),
           (11, 4104, 66, 3, 2, "f16"), (14, 4104, 258, 2, 2, "bf16")]


@pytest.mark.parametrize("T,d,F,E,k,dt", SHAPES)
@pytest.mark.parametrize("with_lora", [False, True])
def test_out_is_rounded_once(T, d, F, E, k, dt, with_lora):
    note(f"few tokens, one rounding T={T} d={d} F={F} E={E} k={k} {dt} lora={with_lora}")
    args = _case(T, d, F, E, dt, T + d + F)
    kw = {}
    if with_lora:
        kw["adapter"], kw["lora"] = _lora(T, d, F, E, 2, 5, dt, T + F)
    _check(args, k, dt, **kw)


@pytest.mark.parametrize("F", [48, 128, 321])
@pytest.mark.parametrize("with_lora", [False, True])
def test_h_past_the_types_largest_number(F, with_lora):
    """silu(W1 x) * (W3 x) of 1e6 to 1e9 and a W2 that brings it back: nothing
    overflows in fp16 on the way."""
    T, d, E, k = 5, 64, 4, 2
    up, down = 2.0 ** 13, 2.0 ** -18
    args = _case(T, d, F, E, "f16", F, up, down * F ** 0.5)
    kw = {}
    if with_lora:
        kw["adapter"], kw["lora"] = _lora(T, d, F, E, 3, 8, "f16", F + 1, 1.0, 2.0 ** -16)
    got, ref = _check(args, k, "f16", **kw)
    z = args[0].double() @ args[2][0].double().t(), args[0].double() @ args[3][0].double().t()
    assert float((z[0] * z[1]).abs().max()) > 1e6 and 0.1 < float(ref.abs().max()) < 65504
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("F", [48, 128, 321])
@pytest.mark.parametrize("with_lora", [False, True])
def test_gates_near_zero(F, with_lora):
    """Sigmoid gates of 1e-4 to 1e-9, not renormalised, and a W2 that scales the
    sum back up: gate * h below fp16's smallest number is not lost."""
    T, d, E, k = 6, 64, 8, 3
    args = _case(T, d, F, E, "f16", F + 2, 1.0, 2.0 ** 14)
    args[1] = args[1] - torch.arange(9, 21, 2, device="cuda")[:, None]
    kw = dict(gating="sigmoid")
    if with_lora:
        kw["adapter"], kw["lora"] = _lora(T, d, F, E, 3, 8, "f16", F + 3, 1.0, 2.0 ** 12)
    got, ref = _check(args, k, "f16", **kw)
    assert float(ref[0].abs().max()) > 2.0 ** -3


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_spread_of_h_within_a_row(dt):
    """Columns of h 2^20 apart, and the rows of W2 that read the small ones alone."""
    T, d, F, E, k = 4, 48, 300, 3, 2
    args = _case(T, d, F, E, dt, 77, 1.0, 2.0 ** 12)
    step = torch.pow(2.0, -20.0 * (torch.arange(F, device="cuda") % 4 != 0))
    args[3] = (args[3].float() * step[:, None].clamp(min=2.0 ** -12)).to(DT[dt])
    args[2] = (args[2].float() * step[:, None].clamp(min=2.0 ** -8)).to(DT[dt])
    args[4][:, ::2, ::4] = 0
    _check(args, k, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_a_token_of_zeros_gets_zero(dt):
    args = _case(4, 64, 160, 4, dt, 5)
    args[0][2] = 0
    got = X.few_token_layer(*args, 2)[0]
    assert not got[2].any() and got[[0, 1, 3]].any(1).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [8, 9, 15, 16])
def test_experts_of_most_tokens_beside_experts_of_one(T, dt):
    """Slots past 512 with more than eight tokens each beside slots with one."""
    d, F, E, k = 40, 24, 1024, 40
    args = _case(T, d, F, E, dt, T)
    hot = torch.arange(E - 25, E, device="cuda")
    args[1][:, hot] = 20.0 - 0.25 * (hot - hot[0]).float()       # every token's first 25
    args[1][1::2, hot[::3]] = -20.0                              # (half of them lack a third)
    _, idx, _ = X.few_token_layer(*args, k)
    n = torch.bincount(idx.flatten().long(), minlength=E)
    assert (n == 1).any() and ((n > 8).sum() >= 16 or T == 8) and (n > 0).sum() > 128
    _check(args, k, dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_sixteen_tokens_are_eight_and_eight(dt):
    """A token's output does not depend on the tokens beside it: the bits of a
    call of sixteen against two calls' of eight, but for the order of their sums."""
    args = _case(16, 96, 264, 12, dt, 21)
    whole = X.few_token_layer(*args, 3)[0]
    for half in (slice(0, 8), slice(8, 16)):
        part = X.few_token_layer(args[0][half], args[1][half], *args[2:], 3)[0]
        ref, err = layer_once64(args[0][half], args[1][half], *args[2:], 3)
        close(whole[half], part, 2 * rounded(ref, err, dt), "out")
