"""The head norm and rotation on the GPU against the plain 64-bit form.

Error bounds, derived from the arithmetic.  With u half a step of the type
(2^-11 f16, 2^-8 bf16) and d the head dimension:
  * a value is exact when loaded; the sum of d squares is off by a factor of at
    most 1 + (d + 2) 2^-24, its root by half of that, and the division, the
    root and the two products with the norm and the weight by 2^-24 each or
    a little more: y is off by (d / 2 + 16) 2^-24 of itself
  * an angle is formed in f64 (three roundings: the frequency's turns, their
    constant, the product: 2^-51 of the angle), reduced exactly, and rounded to
    f32 as a half turn or less (2^-25 half turns: 2^-23 radians); sine and
    cosine add 2^-22: delta = 2^-21 + 2^-50 |angle|
  * out = c y_a -+ s y_b: (|y_a| + |y_b|) |rotary_scale| (delta + (d / 2 + 20) 2^-24)
  * one rounding to the type: u |out|, and 2^-25 below f16's normal range
    (bf16: 2^-134)
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_attention_lightning_indexer_amd as li  # noqa: E402
from oracle import rope as plain  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f16": 2.0**-11, "bf16": 2.0**-8}
LEAST = {"f16": 2.0**-25, "bf16": 2.0**-134}


def check(got, x, weight, positions, inv, axes, eps, interleaved, scale, kind):
    """got and x on the GPU, the rest in NumPy."""
    d = x.shape[-1]
    out, reach, angle = plain.norm_rope(x.double().cpu().numpy(), weight, positions, inv, axes, eps, interleaved, scale)
    delta = 2.0**-21 + 2.0**-50 * np.abs(angle).max(initial=0.0)
    bound = reach * (delta + (d / 2 + 20) * 2.0**-24) + UNIT[kind] * np.abs(out) + LEAST[kind]
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(out))
    fine = ~np.isnan(out)
    assert (np.abs(g - out)[fine] <= bound[fine]).all(), float((np.abs(g - out)[fine] / bound[fine]).max())


def frequencies(m, base=10000.0):
    return (base ** -(np.arange(m) / max(m, 1))).astype(np.float32)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n,hq,hk,d,m,axes,interleaved", [
    (1, 1, 1, 8, 4, 1, False), (1, 64, 8, 128, 64, 1, False), (3, 5, 2, 24, 12, 1, True), (7, 3, 1, 16, 0, 1, False),
    (33, 16, 16, 80, 40, 3, False), (5, 7, 3, 72, 36, 2, False), (9, 4, 4, 72, 16, 4, True), (4, 1, 0, 256, 128, 4, False),
    (65, 6, 2, 96, 20, 1, False), (17, 12, 4, 192, 96, 1, True), (130, 2, 1, 32, 8, 2, True), (11, 33, 5, 64, 32, 1, False),
    (2, 9, 1, 248, 124, 1, True), (2, 3, 2, 248, 124, 1, False), (19, 8, 8, 40, 20, 1, False), (6, 200, 3, 128, 32, 1, False),
    (3, 7, 2, 128, 16, 1, True), (3, 7, 2, 128, 32, 2, True), (3, 7, 2, 128, 48, 1, True), (5, 3, 1, 256, 72, 4, True),
    (5, 3, 1, 72, 20, 1, True), (5, 3, 1, 40, 12, 2, True), (2, 2, 2, 8, 4, 1, True), (2, 2, 2, 16, 8, 1, True),
    (4100, 2, 1, 64, 32, 1, False), (4097, 9, 2, 48, 24, 3, True),
])
def test_against_the_plain_form(kind, n, hq, hk, d, m, axes, interleaved):
    rng = np.random.default_rng(n * 1000 + d + m)
    q, k = (dev(rng.standard_normal((n, max(h, 1), d)) * np.exp2(rng.integers(-6, 6, (n, max(h, 1), 1))), DTYPE[kind])
            for h in (hq, hk))
    wq, wk = 1 + 0.3 * rng.standard_normal((2, d)).astype(np.float32)
    wk = dev(wk, DTYPE[kind])                       # one weight in f32, one of the rows' type
    positions = rng.integers(-40, 200000, (axes, n))
    inv = frequencies(m)
    axis = rng.integers(0, axes, m).tolist()
    pos = dev(positions) if n % 2 else dev(positions).int()
    got_q, got_k = li.norm_rope(q, k if hk else None, pos if axes > 1 else pos[0], dev(inv), dev(wq), wk if hk else None,
                                eps=1e-5, axes=axis if axes > 1 else None, interleaved=interleaved, rotary_scale=1.25)
    check(got_q, q, wq.astype(np.float64), positions, inv, axis, 1e-5, interleaved, 1.25, kind)
    if hk:
        check(got_k, k, wk.double().cpu().numpy(), positions, inv, axis, 1e-5, interleaved, 1.25, kind)
    else:
        assert got_k is None


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slices_of_one_projection_in_place(kind, interleaved):
    """q and k as slices of a fused projection, written back to it; v and the rest keep their bytes."""
    rng = np.random.default_rng(5)
    n, hq, hk, d, m = 37, 6, 2, 128, 48
    rows = dev(rng.standard_normal((n, (hq + 2 * hk) * d + 8)), DTYPE[kind])
    before = rows.clone()
    q, k = rows[:, :hq * d].view(n, hq, d), rows[:, hq * d:(hq + hk) * d].view(n, hk, d)
    positions, inv = rng.integers(0, 5000, (1, n)), frequencies(m)
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    out = li.norm_rope(q, k, dev(positions[0]), dev(inv), dev(w), None, interleaved=interleaved, q_out=q, k_out=k)
    assert out[0] is q and out[1] is k
    old_q, old_k = before[:, :hq * d].view(n, hq, d), before[:, hq * d:(hq + hk) * d].view(n, hk, d)
    check(q, old_q, w.astype(np.float64), positions, inv, [0] * m, 1e-6, interleaved, 1.0, kind)
    check(k, old_k, None, positions, inv, [0] * m, 1e-6, interleaved, 1.0, kind)
    assert torch.equal(rows[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_other_strides():
    """Head-major rows, and outputs of yet another order with room between them."""
    rng = np.random.default_rng(6)
    n, h, d, m = 19, 5, 96, 48
    q = dev(rng.standard_normal((h, n, d)), torch.float16).transpose(0, 1)
    k = dev(rng.standard_normal((n, h, 2 * d)), torch.float16)[..., d:]
    q_out = torch.full((n, h + 1, d + 8), 7.0, dtype=torch.float16, device=DEV)
    k_out = torch.full((h, n, d), 7.0, dtype=torch.float16, device=DEV).transpose(0, 1)
    positions, inv = rng.integers(0, 900, (1, n)), frequencies(m)
    li.norm_rope(q, k, dev(positions[0]), dev(inv), q_out=q_out[:, 1:, 8:], k_out=k_out)
    check(q_out[:, 1:, 8:], q, None, positions, inv, [0] * m, 0, False, 1.0, "f16")
    check(k_out, k, None, positions, inv, [0] * m, 0, False, 1.0, "f16")
    assert (q_out[:, 0] == 7).all() and (q_out[:, :, :8] == 7).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_far_positions(kind):
    """Angles of positions past 2^20 and 2^40, where a product in 32 bits has no digit left."""
    rng = np.random.default_rng(7)
    n, d, m = 24, 64, 32
    q = dev(rng.standard_normal((n, 2, d)), DTYPE[kind])
    inv = frequencies(m, 500.0)
    positions = np.concatenate([rng.integers(2**20, 2**31, n - 4), [2**31 - 1, -2**31, 2**24 + 1, 2**25 + 1]])[None]
    for p in (dev(positions), dev(positions).int()):
        got, _ = li.norm_rope(q, None, p[0], dev(inv))
        check(got, q, None, positions, inv, [0] * m, 0, False, 1.0, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_extreme_rows(kind):
    """Rows of zeros, of the type's largest and smallest values, with infinities and NaN: each by itself."""
    d, m = 128, 64
    top = float(torch.finfo(DTYPE[kind]).max)
    x = torch.randn((9, 2, d), generator=torch.Generator().manual_seed(3)).to(DTYPE[kind])
    x[1, 0] = 0
    x[2, 1] = top
    x[3, 0] *= float(torch.finfo(DTYPE[kind]).tiny)
    x[4, 0, 5] = float("inf")
    x[5, 1, 77] = float("nan")
    x[6, 0, ::2] = -top
    x = x.to(DEV)
    positions, inv = np.arange(9)[None] * 321, frequencies(m)
    w = np.linspace(0.5, 1.5, d).astype(np.float32)
    for weight in (w, None):
        got, _ = li.norm_rope(x, None, dev(positions[0]), dev(inv), None if weight is None else dev(w), eps=1e-6)
        keep = [0, 1, 3, 7, 8] + ([2, 6] if weight is not None else [])
        check(got[keep], x[keep], None if weight is None else w.astype(np.float64), positions[:, keep], inv, [0] * m,
              1e-6, False, 1.0, kind)
        # the other head of a row with infinities or NaN is untouched by them
        clean = x.clone()
        clean[4:6] = torch.nan_to_num(clean[4:6], nan=0.0, posinf=0.0)
        same, _ = li.norm_rope(clean, None, dev(positions[0]), dev(inv), None if weight is None else dev(w), eps=1e-6)
        assert torch.equal(got[4, 1], same[4, 1]) and torch.equal(got[5, 0], same[5, 0])
        if weight is not None:
            assert got[5, 1].isnan().all()
            turned_with_inf = [5, 5 + m]             # inf / inf
            assert got[4, 0][turned_with_inf].isnan().all()


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_rows_whose_squares_leave_the_range(eps):
    """bf16 rows of sizes from 2^-120 to 2^120 side by side: their squares are past f32's range on both sides."""
    n, d, m = 25, 128, 64
    rng = np.random.default_rng(21)
    x = rng.standard_normal((n, 3, d)) * np.exp2(np.linspace(-120, 120, 3 * n).reshape(3, n).T[..., None])
    q = dev(x, torch.bfloat16)
    positions, inv = rng.integers(0, 9000, (1, n)), frequencies(m)
    w = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    got, _ = li.norm_rope(q, None, dev(positions[0]), dev(inv), dev(w), eps=eps)
    check(got, q, w.astype(np.float64), positions, inv, [0] * m, float(np.float32(eps)), False, 1.0, "bf16")


@pytest.mark.parametrize("size,scale", [(-131, 0), (-128, -20), (-48, 100), (-60, 120), (100, -90), (40, 80)])
def test_rows_and_weights_far_apart(size, scale):
    """bf16 rows down to subnormal values, with weights whose product with 1 / sqrt(mean) leaves f32's range."""
    n, d, m = 20, 64, 32
    rng = np.random.default_rng(22)
    q = dev(rng.standard_normal((n, 2, d)) * 2.0**size, torch.bfloat16)
    positions, inv = rng.integers(0, 9000, (1, n)), frequencies(m)
    w = ((1 + 0.2 * rng.standard_normal(d)) * 2.0**scale).astype(np.float32)
    got, _ = li.norm_rope(q, None, dev(positions[0]), dev(inv), dev(w), eps=0.0)
    check(got, q, w.astype(np.float64), positions, inv, [0] * m, 0.0, False, 1.0, "bf16")


def test_a_weight_norms_and_none_does_not():
    """No weight, no frequency: the rows pass bit for bit; weights of one and eps 0 make unit mean squares."""
    x = torch.randn((5, 3, 40), device=DEV).half()
    pos, inv = torch.arange(5, device=DEV), torch.empty(0, device=DEV)
    got, _ = li.norm_rope(x, None, pos, inv)
    assert torch.equal(got, x)
    got, _ = li.norm_rope(x, None, pos, inv, torch.ones(40, device=DEV), eps=0.0)
    assert ((got.double() ** 2).mean(-1) - 1).abs().max() < 2.0**-9


def test_rotations_add_up():
    """Position 0 turns nothing; scores of rotated rows depend on the distance alone."""
    n, d, m = 64, 128, 64
    q = torch.randn((1, 1, d), device=DEV).bfloat16().expand(n, 1, d).contiguous()
    k = torch.randn((1, 1, d), device=DEV).bfloat16().expand(n, 1, d).contiguous()
    inv = dev(frequencies(m))
    zero, _ = li.norm_rope(q, None, torch.zeros(n, dtype=torch.long, device=DEV), inv)
    assert torch.equal(zero, q)
    at = torch.arange(n, device=DEV) * 1000
    a, b = li.norm_rope(q, k, at, inv)
    z = (a.double() * b.double()).sum(-1)
    exact = (q.double() * k.double()).sum(-1)
    # |a . b| of a pair's halves is at most the product of their lengths, which turning keeps; each value is rounded
    # once (2^-8 of it), the sums of products of rounded values are exact to 2^-50
    size = (torch.hypot(*q.double().chunk(2, -1)) * torch.hypot(*k.double().chunk(2, -1))).sum(-1)
    assert ((z - exact).abs() <= size * (2 * 2.0**-8 + 2.0**-15)).all()


def test_a_stream_and_a_graph():
    """Another stream than the current one's work, and replays of a captured call against eager ones."""
    rng = np.random.default_rng(9)
    q, k = (torch.randn((50, h, 64), device=DEV).half() for h in (8, 2))
    w, inv = torch.rand(64, device=DEV), dev(frequencies(32))
    pos = dev(rng.integers(0, 9000, 50))
    want = li.norm_rope(q, k, pos, inv, w, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = li.norm_rope(q, k, pos, inv, w, w)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(q), torch.empty_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        li.norm_rope(q, k, pos, inv, w, w, q_out=out[0], k_out=out[1])
    for step in range(4):
        q.normal_()
        pos += step
        want = li.norm_rope(q, k, pos, inv, w, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), step


def test_empty_and_refused():
    q = torch.randn((4, 3, 64), device=DEV).half()
    k, pos, inv = q[:, :1], torch.arange(4, device=DEV), torch.rand(32, device=DEV)
    none = li.norm_rope(q[:0], k[:0], pos[:0], inv)
    assert none[0].shape == (0, 3, 64) and none[1].shape == (0, 1, 64)
    for error, call in [
        (TypeError, lambda: li.norm_rope(q.float(), k, pos, inv)),
        (TypeError, lambda: li.norm_rope(q, k.bfloat16(), pos, inv)),
        (ValueError, lambda: li.norm_rope(q, k[:3], pos, inv)),
        (ValueError, lambda: li.norm_rope(q, k, pos[:3], inv)),
        (TypeError, lambda: li.norm_rope(q, k, pos.float(), inv)),
        (ValueError, lambda: li.norm_rope(q, k, pos, inv, axes=[0] * 32)),
        (ValueError, lambda: li.norm_rope(q, k, pos[None], inv, axes=[0] * 31)),
        (li.IndexerError, lambda: li.norm_rope(q, k, pos[None], inv, axes=[1] * 32)),
        (li.IndexerError, lambda: li.norm_rope(q, k, pos, torch.rand(36, device=DEV))),
        (li.IndexerError, lambda: li.norm_rope(q[..., :60], k[..., :60], pos, inv)),
        (ValueError, lambda: li.norm_rope(q.transpose(1, 2), None, pos, inv)),
        (ValueError, lambda: li.norm_rope(q, k, pos, inv, torch.ones(32, device=DEV))),
        (TypeError, lambda: li.norm_rope(q, k, pos, inv, torch.ones(64, device=DEV).bfloat16())),
        (ValueError, lambda: li.norm_rope(q, None, pos, inv, None, torch.ones(64, device=DEV))),
        (ValueError, lambda: li.norm_rope(q.cpu(), k, pos, inv)),
        (ValueError, lambda: li.norm_rope(q, k, pos.cpu(), inv)),
        (TypeError, lambda: li.norm_rope(q, k, pos, inv.double())),
    ]:
        with pytest.raises(error):
            call()
