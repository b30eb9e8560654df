"""Every configuration of the 4-bit product's kernel on the GPU against plain
products in 64 bits: tiles of 4, 16 and 32 rows, one matrix and pairs, groups of
32, 64 and 128, K over 1, 2, 4 and 8 waves, one and two column groups a wave,
whole and part chunks of K, both types, with zero points in one and without in
the other.  Tolerances as in test_gpu_expert_ops
(33 steps of 2^-23 a matrix instruction, four in a chain, the group's
correction, the sum over groups and waves, one rounding to the type)."""
import pytest
import torch

from mixture_experts_layer_34_amd import expert_ops as X
from tests.gpu_case import note
from tests.int4_cases import DENSE, ROUTED, config
from tests.test_gpu_expert_ops import DT, _close, _gen, _product_ref, _randn, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,N,K,group,zeros,pair", ROUTED)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_routed(T, k, E, N, K, group, zeros, pair, dt):
    note(f"{config(T * k, E, E, True, N, K, group, pair)} {dt}")
    g = _gen(T + N + K + group)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if T * k > 4:
        idx[torch.rand((T, k), generator=g) < 0.1] = -1
    idx = idx.cuda()
    m = X.sort_pairs(idx, E)
    P = int(m.offsets[E])
    w = [_weights(g, E, N, K, group, zeros != (dt == "f16"), dt) for _ in range(2 if pair else 1)]
    up = w[1] if pair else None
    pr = m.pair_of_row[:P].long()
    expert = idx.reshape(-1)[pr].long()
    x = _randn(g, (T, K), dt)
    out = torch.full((T * k, N), float("nan"), dtype=DT[dt], device="cuda")
    got = X.expert_matvec_int4(x, w[0], m, w_up=up, from_tokens=True, out=out)
    assert torch.isnan(got[P:]).all()
    ref, tol = _product_ref(x.double()[pr // k], expert, w[0], up, dt)
    _close(got[:P], ref, tol, "from tokens")
    rows = torch.full((T * k, K), float("nan"), dtype=DT[dt], device="cuda")
    rows[:P] = x[pr // k]
    assert torch.equal(X.expert_matvec_int4(rows, w[0], m, w_up=up)[:P], got[:P])


@pytest.mark.parametrize("rows,N,K,group,zeros,pair", DENSE)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_dense(rows, N, K, group, zeros, pair, dt):
    note(f"{config(rows, 1, 1, False, N, K, group, pair)} {dt}")
    g = _gen(rows + N + K + group)
    w = [_weights(g, 1, N, K, group, zeros != (dt == "f16"), dt) for _ in range(2 if pair else 1)]
    up = w[1] if pair else None
    x = _randn(g, (rows, K), dt)
    got = X.expert_matvec_int4(x, w[0], w_up=up)
    ref, tol = _product_ref(x.double(), torch.zeros(rows, dtype=torch.long, device="cuda"), w[0], up, dt)
    _close(got, ref, tol, "one matrix")
    assert torch.equal(X.expert_matvec_int4(x, w[0], w_up=up), got)


@pytest.mark.parametrize("T,k,E,eb,ee,N,K,group,pair", [
    (128, 8, 256, 32, 64, 528, 640, 128, True),     # four rows an expert: in sixteens
    (128, 8, 256, 224, 256, 1040, 384, 32, False),
    (16, 8, 128, 0, 16, 272, 1152, 64, True),       # one row: in fours
    (256, 4, 64, 60, 64, 2000, 640, 64, False),     # sixteen rows
    (300, 8, 16, 3, 4, 4100, 384, 128, False),      # 150 rows: thirty-twos; local, workgroups loop
    (1, 8, 128, 0, 16, 144, 640, 32, True),         # one row for all of them
])
@pytest.mark.parametrize("pairs", ["anywhere", "local", "one expert"])
def test_expert_parallel_share(T, k, E, eb, ee, N, K, group, pair, pairs):
    """Weights of the local experts only, with as many rows as fall to them,
    every pair on them, or every pair on one of them."""
    note(f"{config(T * k, E, ee - eb, True, N, K, group, pair)} pairs={pairs}")
    g = _gen(T + N)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if pairs == "local":
        idx = eb + idx % (ee - eb)
    elif pairs == "one expert":
        idx[:] = ee - 1
    idx = idx.cuda()
    m = X.sort_pairs(idx, E, eb, ee)
    P = int(m.offsets[E])
    w = [_weights(g, ee - eb, N, K, group, True, "bf16") for _ in range(2 if pair else 1)]
    up = w[1] if pair else None
    x = _randn(g, (T, K), "bf16")
    out = torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = X.expert_matvec_int4(x, w[0], m, w_up=up, from_tokens=True, out=out)
    assert torch.isnan(got[P:]).all()
    pr = m.pair_of_row[:P].long()
    ref, tol = _product_ref(x.double()[pr // k], idx.reshape(-1)[pr].long() - eb, w[0], up, "bf16")
    _close(got[:P], ref, tol, "local rows")
