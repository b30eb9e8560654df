"""Low-rank adapters' gradients on maps that name rows and tokens outside the
arrays, or whose offsets fall: nothing outside is read or written, and the rows
that are named rightly are right."""
import pytest
import torch

from mixture_experts_layer_34_amd import expert_ops as X
from tests.adapter_cases import DT, U, close, gen, lora_grad64, randn, rounded
from tests.gpu_case import note

pytestmark = pytest.mark.gpu


def _case(T, K, N, G, r, dt):
    g = gen(T + K)
    w = X.LoraWeights(randn(g, (G, r, K), dt, K ** -0.5), randn(g, (G, N, r), dt, r ** -0.5))
    x, dout = randn(g, (T, K), dt), randn(g, (T, N), dt)
    m = X.sort_pairs(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), G)  # row q is token q
    _, u = X.lora_rows(x, m, w, save=True)
    return x, dout, u, w, m


def _check(x, dout, u, w, m, ids, dt, left):
    """left: tokens that no row names; their dx is left as it was."""
    T, K = x.shape
    guard = torch.full((T + 2, K), 9.0, dtype=DT[dt], device="cuda")
    dx, dA, dB = X.lora_rows_backward(dout, x, u, m, w, out=guard[1:T + 1])
    ref = lora_grad64(dout, x, u, ids, w.A, w.B, w.scale)
    keep = torch.ones(T, dtype=torch.bool)
    keep[left] = False
    close(dx[keep.cuda()], ref["dx"][0][keep], rounded(*ref["dx"], dt)[keep], "dx")
    assert (guard[0] == 9).all() and (guard[-1] == 9).all() and (dx[(~keep).cuda()] == 9).all()
    close(dA, ref["dA"][0], ref["dA"][1] + 2 * U * ref["dA"][0].abs(), "dA")
    close(dB, ref["dB"][0], ref["dB"][1] + 2 * U * ref["dB"][0].abs(), "dB")


# widths past 49152 in all share the rows of the gradients' sums out in one range, lesser ones in several
WIDTHS = [(25088, 24576, "bf16"), (64, 72, "bf16"), (12500, 12100, "f32"), (96, 40, "f32")]


@pytest.mark.parametrize("K,N,dt", WIDTHS)
@pytest.mark.parametrize("offsets,rows", [([0, 50, 30], (0, 30, 0)), ([10, 0, 20], (10, 20, 1)),
                                          ([0, 2 ** 31 - 1, 17], (0, 17, 0)),
                                          ([-(2 ** 31), 64, 2 ** 31 - 1], (0, 64, 0)),
                                          ([40, -5, 2 ** 31 - 1], (40, 64, 1)), ([30, 10, 5], (0, 0, 0))])
def test_gradients_of_falling_offsets(K, N, dt, offsets, rows):
    note(f"lora grad, falling offsets {offsets} K={K} N={N} {dt}")
    T, G, r = 64, 2, 8
    x, dout, u, w, m = _case(T, K, N, G, r, dt)
    m.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    lo, hi, g = rows
    if g:  # u is of the group's own A
        u[lo:hi] = X.lora_rows(x, X.sort_pairs(torch.full((T, 1), g, dtype=torch.int32, device="cuda"), G), w,
                               save=True)[1][lo:hi]
    ids = torch.full((T,), -1)
    ids[lo:hi] = g
    _check(x, dout, u, w, m, ids, dt, [t for t in range(T) if not lo <= t < hi])


@pytest.mark.parametrize("K,N,dt", WIDTHS)
def test_gradients_of_tokens_outside(K, N, dt):
    note(f"lora grad, tokens outside K={K} N={N} {dt}")
    T, G, r = 64, 2, 8
    x, dout, u, w, m = _case(T, K, N, G, r, dt)
    for row, token in ((10, T), (11, -7), (12, 2 ** 31 - 1), (63, -(2 ** 31))):
        m.pair_of_row[row] = token
    ids = torch.zeros(T, dtype=torch.long)
    ids[[10, 11, 12, 63]] = -1
    _check(x, dout, u, w, m, ids, dt, [10, 11, 12, 63])
