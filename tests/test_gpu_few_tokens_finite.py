"""The layer for a few tokens on weights that hold an infinity or a NaN: the
tokens of that expert or adapter are not finite, the others are bit for bit what
they are without it."""
import pytest
import torch

from mixture_experts_layer_34_amd import expert_ops as X
from tests.adapter_cases import gen, randn
from tests.gpu_case import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,F,dt", [(6, 64, 128, "bf16"), (6, 64, 128, "f16"), (6, 64, 128, "f32"),
                                      (7, 67, 131, "bf16"), (16, 72, 321, "f16"), (13, 40, 5, "bf16"), (12, 4104, 136, "bf16"),
                                      (5, 4104, 67, "f16"), (16, 96, 40, "f32")])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", range(3))
def test_an_experts_weights_reach_its_own_tokens_alone(T, d, F, dt, bad, at):
    note(f"few tokens, weights not finite T={T} d={d} F={F} {dt} {bad} {at}")
    E, k = 6, 2
    g = gen(T + F)
    x, logits = randn(g, (T, d), dt), randn(g, (T, E))
    w = [randn(g, (E, F, d), dt, d ** -0.5), randn(g, (E, F, d), dt, d ** -0.5), randn(g, (E, d, F), dt, F ** -0.5)]
    logits[:, 3] = 9.0            # an expert of the even tokens
    logits[1::2, 3] = -9.0
    logits[T - 1] = logits[0]     # (and of the last)
    clean, idx, _ = X.few_token_layer(x, logits, *w, k)
    has = (idx == 3).any(1)
    assert has.any() and not has.all()
    w[at][3, 1, ::3] = bad
    w[at][3, -1, -1] = bad
    got, again, _ = X.few_token_layer(x, logits, *w, k)
    assert torch.equal(idx, again) and torch.equal(got[~has], clean[~has])
    assert not torch.isfinite(got[has]).all(1).any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("at", range(3))
def test_an_adapters_weights_reach_its_own_tokens_alone(dt, bad, at):
    T, d, F, E, k, L, r = 11, 64, 72, 4, 4, 3, 6
    g = gen(8)
    x, logits = randn(g, (T, d), dt), randn(g, (T, E))
    w = [randn(g, (E, F, d), dt, d ** -0.5), randn(g, (E, F, d), dt, d ** -0.5), randn(g, (E, d, F), dt, F ** -0.5)]
    lora = [X.LoraWeights(randn(g, (L, E, r, K), dt, K ** -0.5), randn(g, (L, E, N, r), dt, 0.5 * r ** -0.5))
            for N, K in ((F, d), (F, d), (d, F))]
    adapter = (torch.arange(T, dtype=torch.int32) % 4 - 1).cuda()
    clean = X.few_token_layer(x, logits, *w, k, adapter=adapter, lora=lora)[0]
    for t in (lora[at].A, lora[at].B):
        kept = t.clone()
        t[1, 2, 1] = bad
        got = X.few_token_layer(x, logits, *w, k, adapter=adapter, lora=lora)[0]
        t.copy_(kept)
        own = adapter == 1
        assert torch.equal(got[~own], clean[~own]) and not torch.isfinite(got[own]).all(1).any()
