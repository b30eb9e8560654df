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


def test_outputs_apart_from_gates_maps_and_weights():
    """An output over the gates, the map or the weights of its own call is
    refused, one right behind them in the same buffer is not."""
    T, k, E, d = 64, 2, 4, 32
    g = _gen(31)
    m = X.sort_pairs(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda(), E)

    def beside(t, shape, dtype):
        """(t again in a buffer of its own, an output over its last 16 bytes, one right behind it)"""
        n = -(-t.nbytes // 16) * 16
        size = torch.empty(shape, dtype=dtype).nbytes
        raw = torch.zeros(n + size, dtype=torch.uint8, device="cuda")
        raw[:t.nbytes] = t.contiguous().reshape(-1).view(torch.uint8)
        view = lambda at, like, s: raw[at:at + like].view(dtype if s is shape else t.dtype).view(s)
        return view(0, t.nbytes, t.shape), view(n - 16, size, shape), view(n, size, shape)

    def check(t, shape, dtype, call):
        t2, over, behind = beside(t, shape, dtype)
        with pytest.raises(ValueError, match="overlap"):
            call(t2, over)
        want = call(t2, None)
        got = call(t2, behind)
        assert got.data_ptr() == behind.data_ptr() and torch.equal(got, want)

    f32 = torch.float32
    x, y, gate = _randn(g, (T, d)), _randn(g, (T * k, d)), torch.rand((T, k), generator=g).cuda()
    named = lambda **o: X.PairMap(m.T, m.k, m.E, 0, E, **{**dict(
        counts=m.counts, offsets=m.offsets, row_of_pair=m.row_of_pair, pair_of_row=m.pair_of_row), **o})
    for op, src, shape in ((X.permute_rows, x, (T * k, d)), (X.unpermute_rows, y, (T, d)),
                           (lambda *a, **o: X.unpermute_rows_backward(*a, **o)[0], x, (T * k, d))):
        check(gate, shape, f32, lambda t, o: op(src, m, gate=t, out=o))
        check(m.row_of_pair, shape, f32, lambda t, o: op(src, named(row_of_pair=t), gate=gate, out=o))
    bf = torch.bfloat16
    w = [_weights(g, E, d, 64, 32, True, "bf16") for _ in range(2)]
    xb, out = _randn(g, (T, 64), "bf16"), (T * k, d)
    call = lambda o, a=w[0], b=w[1], mm=m: X.expert_matvec_int4(xb, a, mm, w_up=b, from_tokens=True, out=o)
    check(m.pair_of_row, out, bf, lambda t, o: call(o, mm=named(pair_of_row=t)))
    check(m.offsets, out, bf, lambda t, o: call(o, mm=named(offsets=t)))
    for name in ("codes", "scales", "zeros"):
        for i in range(2):
            def with_array(t, o):
                ws = list(w)
                ws[i] = X.Int4Weights(**{**dict(codes=w[i].codes, scales=w[i].scales, zeros=w[i].zeros), name: t})
                return call(o, *ws)
            check(getattr(w[i], name), out, bf, with_array)


def test_a_map_whose_array_was_changed_in_place_is_refused():
    """The 4-bit product reads offsets and, from token rows, pairs: neither is
    followed once it is shorter than the map says."""
    g = _gen(8)
    idx = torch.randint(0, 4, (6, 2), generator=g, dtype=torch.int32).cuda()
    w, x, rows = _weights(g, 4, 16, 64, 32, False, "bf16"), _randn(g, (6, 64), "bf16"), _randn(g, (12, 64), "bf16")
    for name in ("offsets", "pair_of_row"):
        m = X.sort_pairs(idx, 4)
        want = X.expert_matvec_int4(rows, w, m)
        getattr(m, name).data = getattr(m, name)[:3].clone()
        with pytest.raises(ValueError, match=name):
            X.expert_matvec_int4(x, w, m, from_tokens=True)
        if name == "pair_of_row":   # not read where x holds the sorted rows
            assert torch.equal(X.expert_matvec_int4(rows, w, m), want)


def test_lost_gradients_are_refused():
    """Rows, gates, scales and outputs that require a gradient while gradients
    are recorded; not under no_grad, detached, or in the _backward functions,
    whose results are no one's to differentiate."""
    T, k, E, d = 5, 2, 3, 32
    g = _gen(9)
    m = X.sort_pairs(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda(), E)
    x, y, gate = _randn(g, (T, d)), _randn(g, (T * k, d)), torch.rand((T, k), generator=g).cuda()
    w, xb = _weights(g, E, 16, d, 32, False, "bf16"), _randn(g, (T, d), "bf16")
    grad = lambda t: t.detach().clone().requires_grad_()
    wg = X.Int4Weights(w.codes, grad(w.scales))
    buf = lambda: torch.zeros(T * k, d, device="cuda")
    for call in (lambda: X.permute_rows(grad(x), m, out=buf()),
                 lambda: X.permute_rows(x, m, gate=grad(gate), out=buf()), lambda: X.permute_rows(x, m, out=grad(buf())),
                 lambda: X.unpermute_rows(grad(y), m), lambda: X.unpermute_rows(y, m, gate=grad(gate)),
                 lambda: X.expert_matvec_int4(grad(xb), w, m, from_tokens=True),
                 lambda: X.expert_matvec_int4(xb, wg, m, from_tokens=True),
                 lambda: X.expert_matvec_int4(xb, w, m, w_up=wg, from_tokens=True)):
        with pytest.raises(RuntimeError, match="autograd"):
            call()
        with torch.no_grad():
            call()
    want = X.unpermute_rows(y, m, gate=gate)
    assert torch.equal(X.unpermute_rows(grad(y).detach(), m, gate=grad(gate).detach()), want)
    dx, dgate = X.permute_rows_backward(grad(y), m, gate=grad(gate), x=grad(x))
    assert torch.equal(dx, want) and not dx.requires_grad and not dgate.requires_grad
    X.unpermute_rows_backward(grad(x), m, gate=grad(gate), y=grad(y))
    X.quantize_int4(grad(xb), 32)


def test_weights_moved_from_the_cpu():
    w = _weights(_gen(4), 1, 48, 128, 32, True, "bf16")
    x = _randn(_gen(5), (3, 128), "bf16")
    there = w.to("cpu")
    with pytest.raises(ValueError, match="devices"):
        X.expert_matvec_int4(x, there)
    assert torch.equal(X.expert_matvec_int4(x, there.to("cuda")), X.expert_matvec_int4(x, w))


@pytest.mark.parametrize("rows", [1, 8, 32])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_an_outlier_on_weights_of_zero(rows, dt):
    """An x of 6e4 among x of 1, on weights whose code is their zero point,
    adds nothing to the result and leaves no more than the bound of the two
    sums that cancel, 2^-24 s |x| (32 + q + z) a step."""
    N, K, G, at = 96, 1024, 128, 777
    w = _weights(_gen(21), 1, N, K, G, True, dt)
    zero, byte = w.zeros[0, :, at // G], w.codes[0, :, at // 2]
    byte.copy_((byte & 15) | (zero << 4))           # element 777 lies in the high nibble
    x = _randn(_gen(22), (rows, K), dt)
    x[:, at] = 6e4
    ref, tol = _product_ref(x.double(), torch.zeros(rows, dtype=torch.long, device="cuda"), w, None, dt)
    without = x.clone()
    without[:, at] = 0
    assert torch.equal(ref, _product_ref(without.double(), torch.zeros(rows, dtype=torch.long, device="cuda"), w, None,
                                         dt)[0])
    _close(X.expert_matvec_int4(x, w), ref, tol, "with the outlier")
