"""Gradients of adapters over rows past 4 GiB: dA and dB, whose gathers have
offsets of their own.  dout is zero but for rows at both ends, at the groups'
border and about the 4 GiB line, so the others add exact zeros and a row taken
from a wrong place is seen whole."""
import pytest
import torch

from mixture_experts_layer_34_amd import expert_ops as X
from tests.adapter_cases import U, close, gen, lora_grad64, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("turned", [False, True])
def test_weight_gradients_past_four_gib(turned):
    """turned: the sorted rows run against the tokens, so the gathers do too."""
    rows, K, r = (1 << 19) + 3, 4096, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    border = rows // 2
    at = torch.cat([torch.arange(n, n + 40) for n in (0, border - 20, (1 << 19) - 20 - 40, rows - 40)]).unique().cuda()
    dout = torch.zeros_like(x)
    dout[at] = torch.empty((len(at), K), dtype=x.dtype, device="cuda").normal_(generator=g)
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ids[border:] = 1
    amap = X.sort_pairs((1 - ids if turned else ids)[:, None].contiguous(), 2)
    w = X.LoraWeights(randn(gen(1), (2, r, K), "bf16", K ** -0.5), randn(gen(2), (2, K, r), "bf16", r ** -0.5))
    _, u = X.lora_rows(x, amap, w, save=True)
    _, dA, dB = X.lora_rows_backward(dout, x, u, amap, w)
    own = (1 - ids if turned else ids)[at].cpu().long()
    ref = lora_grad64(dout[at], x[at], u[amap.row_of_pair[at, 0].long()], own, w.A, w.B, None)
    for got, (want, err), what in ((dA, ref["dA"], "dA"), (dB, ref["dB"], "dB")):
        assert want.abs().max() > 1
        close(got, want, err + 2 * U * want.abs(), what)
