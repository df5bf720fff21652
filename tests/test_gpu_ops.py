"""The stand-alone operators on the GPU against their definitions in 64 bits.

Tolerances.  A result that is rounded once to a type t may be off by
eps(t)/2 of its value (plus half of t's smallest step near zero).  An fp32 sum
of n terms in any order is within n * 2^-24 of the sum of the terms' magnitudes
when each addition rounds to nearest; the tensor core's additions may cut off
instead, 2^-23 each.  Quantisation, sorting and copies are exact.
"""
import numpy as np
import pytest

from tests import _gpu as G
from tests import _ops_ref as ref

pytestmark = pytest.mark.gpu

TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def dt(name):
    t = G.torch()
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}[name]


def rounding(name, value):
    """Half a step of a type at `value`."""
    return G.torch().finfo(dt(name)).eps / 2 * np.abs(value) + TINY[name] / 2


def f64(x):
    return x.detach().cpu().double().numpy()


def randn(shape, seed, dtype="f32", scale=1.0):
    t = G.torch()
    g = t.Generator().manual_seed(seed)
    return (t.randn(shape, generator=g) * scale).to(dt(dtype)).cuda()


def placed(x, pad, shift):
    """The same 2-D values in a buffer with `pad` more elements a row, from element `shift` on."""
    t = G.torch()
    n, H = x.shape
    buf = t.zeros(shift + n * (H + pad), dtype=x.dtype, device=x.device)
    v = buf[shift:].view(n, H + pad)[:, :H]
    v.copy_(x)
    return v


def ids_of(T, k, E, seed, low=0, high=None):
    t = G.torch()
    g = t.Generator().manual_seed(seed)
    return t.randint(low, E if high is None else high, (T, k), generator=g, dtype=t.int32).cuda()


# ----------------------------------------------------------------------- sort
@pytest.mark.parametrize("T, k, E, low, high", [
    (1, 1, 1, 0, 1), (1, 8, 64, 0, 64), (3, 32, 1024, 0, 1024), (33, 8, 64, -1, 66), (257, 5, 7, 0, 7),
    (1000, 6, 257, -3, 260), (4097, 4, 1024, 0, 1024), (8192, 10, 512, 0, 514), (70001, 3, 100, -1, 100),
    (50, 2, 8, -5, 0), (50, 2, 8, 8, 20), (999, 7, 16, 3, 4),
])
def test_sort_tokens(T, k, E, low, high):
    F = G.library()
    ids = ids_of(T, k, E, T + k, low, high)
    r = F.sort_tokens(ids, E)
    for name, want in zip(("counts", "offsets", "perm", "inv"), ref.sort_pairs(ids.cpu().numpy(), E)):
        assert np.array_equal(r[name].cpu().numpy(), want), name


def test_sort_of_no_tokens_and_of_extreme_ids():
    t, F = G.torch(), G.library()
    r = F.sort_tokens(t.empty((0, 3), dtype=t.int32, device="cuda"), 5)
    assert r["counts"].tolist() == [0] * 5 and r["offsets"].tolist() == [0] * 6 and r["inv"].shape == (0, 3)
    ids = t.tensor([[2147483647, -2147483648], [4, 4], [5, 0]], dtype=t.int32, device="cuda")
    r = F.sort_tokens(ids, 5)
    assert r["inv"].tolist() == [[-1, -1], [1, 2], [-1, 0]] and r["perm"].tolist() == [5, 2, 3, -1, -1, -1]


# ------------------------------------------------------- dispatch and combine
ROWS = [  # T, k, E, sinks, H, pad, shift
    (1, 1, 1, 0, 1, 0, 0), (2, 3, 4, 1, 7, 0, 0), (5, 8, 16, 0, 64, 0, 0), (33, 8, 64, 2, 2048, 0, 0),
    (64, 2, 8, 1, 100, 4, 0), (17, 6, 32, 0, 255, 1, 1), (9, 4, 8, 0, 264, 8, 8), (300, 10, 128, 3, 520, 0, 0),
    (12, 32, 40, 0, 2047, 0, 3), (7, 5, 9, 9, 4100, 0, 0),
]


def _rows_case(T, k, E, sinks, seed):
    ids = ids_of(T, k, E, seed, 0, E + sinks)
    return G.library().sort_tokens(ids, E)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16", "u8"])
@pytest.mark.parametrize("case", ROWS)
def test_dispatch_copies_and_leaves_other_rows(case, dtype):
    t, F = G.torch(), G.library()
    T, k, E, sinks, H, pad, shift = case
    inv = _rows_case(T, k, E, sinks, 1)["inv"]
    x = randn((T, H), 2)
    x = (x * 50).to(t.uint8) if dtype == "u8" else x.to(dt(dtype))
    x = placed(x, pad, shift)
    for rows in {T * k, max(1, T * k - 3)}:               # a capacity below what is needed drops the rest
        out = placed(t.full((rows, H), 77, dtype=x.dtype, device="cuda"), pad, shift)
        got = F.dispatch(x, inv, out=out)
        assert got is out
        want = ref.dispatch(f64(x), inv.cpu().numpy(), np.full((rows, H), 77.0))
        assert np.array_equal(f64(out), want)
    fresh = F.dispatch(x, inv)
    used = inv[inv >= 0].long()
    assert t.equal(fresh[used], x[t.nonzero(inv >= 0)[:, 0]])


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("case", ROWS)
def test_dispatch_backward(case, dtype):
    F = G.library()
    T, k, E, sinks, H, pad, shift = case
    inv = _rows_case(T, k, E, sinks, 3)["inv"]
    dxs = placed(randn((T * k, H), 4, dtype), pad, shift)
    dx = F.dispatch_backward(dxs, inv)
    want, mag = ref.combine(f64(dxs), inv.cpu().numpy(), np.ones((T, k)))
    assert np.all(np.abs(f64(dx) - want) <= k * 2.0 ** -24 * mag + rounding(dtype, want) * (1 + k * 2.0 ** -24))


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("f16", "f16"), ("bf16", "f32"),
                                   ("f16", "bf16")])
@pytest.mark.parametrize("case", ROWS)
def test_combine_and_its_gradients(case, types):
    t, F = G.torch(), G.library()
    T, k, E, sinks, H, pad, shift = case
    ti, to = types
    inv = _rows_case(T, k, E, sinks, 5)["inv"]
    ys = placed(randn((T * k, H), 6, ti), pad, shift)
    gates = randn((T, k), 7).abs()
    iv, yd, gd = inv.cpu().numpy(), f64(ys), f64(gates)
    y = F.combine(ys, inv, gates, out_dtype=dt(to))
    want, mag = ref.combine(yd, iv, gd)
    # k products and additions, one multiply-add each: n = k roundings
    assert y.dtype == dt(to)
    assert np.all(np.abs(f64(y) - want) <= k * 2.0 ** -24 * mag + rounding(to, want) * (1 + k * 2.0 ** -24))
    plain = F.combine(ys, inv, out_dtype=dt(to))
    assert t.equal(plain, F.combine(ys, inv, t.ones_like(gates), out_dtype=dt(to)))
    dy = placed(randn((T, H), 8, to), pad, shift)
    before = placed(randn((T * k, H), 9, ti), pad, shift)
    out = before.clone()
    dys, dg = F.combine_backward(dy, ys, inv, gates, out=out)
    w_dys, w_dg, s_dg = ref.combine_backward(f64(dy), yd, iv, gd, f64(before))
    # gate * dy is one fp32 rounding before that to the type
    assert np.all(np.abs(f64(dys) - w_dys) <= rounding(ti, w_dys) * (1 + 2.0 ** -23) + 2.0 ** -24 * np.abs(w_dys))
    unnamed = np.setdiff1d(np.arange(T * k), iv[iv >= 0])
    assert np.array_equal(f64(dys)[unnamed], f64(before)[unnamed])
    assert np.all(np.abs(f64(dg) - w_dg) <= H * 2.0 ** -24 * s_dg + TINY["f32"])
    assert np.all(f64(dg)[iv < 0] == 0)


EVEN = [  # T, k, E, sinks, H, pad, shift: rows that start and end on pairs, and some that do not quite
    (11, 6, 16, 1, 2046, 0, 0), (9, 3, 8, 0, 258, 2, 2), (5, 8, 16, 0, 34, 0, 1), (4, 2, 4, 0, 256, 0, 2),
    (6, 5, 8, 1, 254, 1, 0), (3, 1, 2, 0, 2, 0, 0), (200, 4, 16, 0, 98, 0, 2),
]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("case", EVEN)
def test_rows_of_pairs(case, types):
    test_combine_and_its_gradients(case, types)
    test_dispatch_backward(case, types[0])
    test_dispatch_copies_and_leaves_other_rows(case, types[0])


def test_combine_gradient_against_differences():
    """Directional differences of <dy, combine(ys, gates)> in 64 bits."""
    F = G.library()
    T, k, E, H = 23, 4, 9, 96
    inv = _rows_case(T, k, E, 2, 11)["inv"]
    ys, gates, dy = randn((T * k, H), 12), randn((T, k), 13), randn((T, H), 14)
    dys, dg = F.combine_backward(dy, ys, inv, gates, out=G.torch().zeros_like(ys))
    iv = inv.cpu().numpy()
    rng = np.random.default_rng(0)

    def loss(a, b):
        return float((f64(dy) * ref.combine(a, iv, b)[0]).sum())

    u, v, h = rng.standard_normal(ys.shape), rng.standard_normal(gates.shape), 1e-3
    got_y, got_g = float((f64(dys) * u).sum()), float((f64(dg) * v).sum())
    # the loss is linear in each: central differences are exact up to 64-bit rounding (~1e-16 / h of the loss's
    # terms); dys and dg carry fp32 roundings: 2^-24 of each element, and of H terms
    near_y = (loss(f64(ys) + h * u, f64(gates)) - loss(f64(ys) - h * u, f64(gates))) / (2 * h)
    near_g = (loss(f64(ys), f64(gates) + h * v) - loss(f64(ys), f64(gates) - h * v)) / (2 * h)
    size = float(np.abs(f64(dy)).sum() * np.abs(f64(ys)).max() * np.abs(f64(gates)).max())
    assert abs(got_y - near_y) <= 2.0 ** -23 * np.abs(f64(dys) * u).sum() + 1e-12 * size
    s_dg = ref.combine_backward(f64(dy), f64(ys), iv, f64(gates), f64(ys))[2]
    assert abs(got_g - near_g) <= H * 2.0 ** -24 * (s_dg * np.abs(v)).sum() + 1e-12 * size


def test_dispatch_gradient_against_differences():
    F = G.library()
    T, k, E, H = 19, 3, 8, 40
    inv = _rows_case(T, k, E, 1, 15)["inv"]
    dxs = randn((T * k, H), 16)
    dx = F.dispatch_backward(dxs, inv)
    iv = inv.cpu().numpy()
    x, u, h = f64(randn((T, H), 17)), f64(randn((T, H), 18)), 1e-3

    def loss(a):
        return float((f64(dxs) * ref.dispatch(a, iv, np.zeros((T * k, H)))).sum())

    near = (loss(x + h * u) - loss(x - h * u)) / (2 * h)
    mag = ref.combine(f64(dxs), iv, np.ones((T, k)))[1]
    size = float(np.abs(f64(dxs)).sum() * np.abs(x).max())
    assert abs(float((f64(dx) * u).sum()) - near) <= (k + 1) * 2.0 ** -24 * (mag * np.abs(u)).sum() + 1e-12 * size


def test_dropped_pairs_and_unnamed_rows_do_not_leak():
    t, F = G.torch(), G.library()
    nan = float("nan")
    inv = t.tensor([[0, -1], [-1, -1], [2, 9], [-7, 1]], dtype=t.int32, device="cuda")   # 9 is past the rows
    ys = randn((4, 72), 19)
    ys[3] = nan                                             # named by nobody
    gates = t.tensor([[.5, nan], [nan, float("inf")], [.25, nan], [nan, 2.0]], device="cuda")
    y = F.combine(ys, inv, gates)
    assert t.isfinite(y).all() and (y[1] == 0).all()
    assert t.equal(y[0], .5 * ys[0]) and t.equal(y[2], .25 * ys[2]) and t.equal(y[3], 2 * ys[1])
    dy = randn((4, 72), 20)
    dy[1] = nan                                             # a token with no pair left
    out = t.full_like(ys, 5.0)
    dys, dg = F.combine_backward(dy, ys, inv, gates, out=out)
    assert t.isfinite(dys).all() and (dys[3] == 5).all() and t.isfinite(dg).all()
    assert (dg[1] == 0).all() and dg[0, 1] == 0 and dg[2, 1] == 0 and dg[3, 0] == 0
    dx = F.dispatch_backward(ys, inv)
    assert t.isfinite(dx).all() and (dx[1] == 0).all()
    xs = t.full((4, 72), 5.0, device="cuda")
    F.dispatch(dy, inv, out=xs)
    assert (xs[3] == 5).all() and t.isfinite(xs).all()


def test_partial_gradients_of_combine():
    """dys alone (ys not read) and dgates alone, through the C entry point."""
    t, F = G.torch(), G.library()
    T, k, H = 6, 2, 40
    inv = _rows_case(T, k, 4, 0, 21)["inv"]
    ys, dy, gates = randn((T * k, H), 22), randn((T, H), 23), randn((T, k), 24)
    dys, dg = F.combine_backward(dy, ys, inv, gates)
    s = t.cuda.current_stream().cuda_stream
    a, b = t.zeros_like(dys), t.zeros_like(dg)
    L = F.lib()
    assert L.moe_combine_backward(dy.data_ptr(), 0, H, None, 0, H, T * k, T, k, H, inv.data_ptr(), gates.data_ptr(),
                                  a.data_ptr(), H, None, s) == 0
    assert L.moe_combine_backward(dy.data_ptr(), 0, H, ys.data_ptr(), 0, H, T * k, T, k, H, inv.data_ptr(),
                                  gates.data_ptr(), None, H, b.data_ptr(), s) == 0
    assert t.equal(a, dys) and t.equal(b, dg)


# ----------------------------------------------------------------- quantise
def _hard_rows(n, K, seed):
    """Values of many sizes, on borders between codes, zeros and subnormals among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, K)) * 2.0 ** rng.integers(-12, 12, (n, 1))
    grid = rng.choice([0, .25, .5, .75, 1, 1.25, 1.75, 2.5, 3.5, 5, 6, 7], (n, K)) * rng.choice([-1, 1], (n, K))
    d = rng.choice([1, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875], (n, K // 16)) * 2.0 ** rng.integers(-4, 4, (n, K // 16))
    on = grid * np.repeat(d, 16, axis=1)
    x = np.where(rng.random((n, 1)) < 0.5, x, on)
    x[rng.random((n, K)) < 0.05] = 0
    if n > 2:
        x[1] = 0
        x[2, :K // 2] = 0
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n, K, per, pad, shift", [
    (1, 32, 1, 0, 0), (3, 64, 1, 0, 0), (8, 2048, 1, 0, 0), (257, 96, 1, 0, 0), (5, 4128, 1, 8, 8), (4, 544, 1, 3, 1),
    (2, 32800, 1, 0, 0), (64, 256, 16, 0, 0), (6, 160, 2, 0, 0), (1024, 2048, 1024, 0, 0), (12, 96, 4, 2, 2),
    (700, 1024, 350, 0, 0), (64, 256, 16, 16, 0), (8, 128, 8, 0, 1), (600, 1312, 2, 0, 0), (1200, 1024, 8, 0, 0), (48, 4096, 16, 0, 0),
])
def test_quantize_is_exact(dtype, fmt, n, K, per, pad, shift):
    t, F = G.torch(), G.library()
    x = placed(t.from_numpy(_hard_rows(n, K, n + K)).to(dt(dtype)).cuda(), pad, shift)
    q = F.fp4_quantize(x, fmt, rows_per_scale=per)
    codes, scales, Gs, vals = ref.quantize(f64(x), fmt, per)
    assert np.array_equal(q.scales.cpu().numpy(), scales.reshape(n, -1))
    if fmt == "nvfp4":
        assert np.array_equal(f64(q.global_scale), Gs)
    got = ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), Gs, fmt, per)
    assert np.array_equal(got, vals)
    assert np.array_equal(f64(F.fp4_dequantize(q)), vals)
    back = F.fp4_dequantize(q, dtype=t.bfloat16)
    assert np.array_equal(f64(back), f64(t.from_numpy(vals).float().to(t.bfloat16)))
    again = F.FP4Tensor(*(None if p is None else t.empty_like(p) for p in q[:3]), fmt)
    assert F.fp4_quantize(x, fmt, per, out=again) is again
    assert all(a is None or t.equal(a, b) for a, b in zip(again[:3], q[:3]))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("per, pad", [(1, 0), (4, 0), (4, 16), (8, 1)])
def test_quantize_at_the_ends_of_the_range(fmt, per, pad):
    """The largest and smallest floats, infinities, NaN; blocks that are not finite become NaN alone."""
    t, F = G.torch(), G.library()
    x = np.zeros((8, 128), dtype=np.float32)
    x[0] = np.finfo(np.float32).max
    x[1, ::3] = 2.0 ** -149
    x[2, 5] = 2.0 ** -126
    x[3] = np.linspace(-1, 1, 128)
    x[3, 40] = np.nan
    x[4] = np.linspace(-3, 3, 128)
    x[4, 70], x[4, 90] = np.inf, -np.inf
    x[5] = np.nan
    x[6, :64] = 1e-30
    x[6, 64:] = 1e30
    x[7] = -0.0
    q = F.fp4_quantize(placed(t.from_numpy(x).cuda(), pad, 0), fmt, rows_per_scale=per)
    codes, scales, Gs, vals = ref.quantize(x.astype(np.float64), fmt, per)
    assert np.array_equal(q.scales.cpu().numpy(), scales.reshape(8, -1))
    if fmt == "nvfp4":
        assert np.array_equal(f64(q.global_scale), Gs)
    with np.errstate(over="ignore"):
        want = vals.astype(np.float32).astype(np.float64)
    assert np.array_equal(f64(F.fp4_dequantize(q)), want, equal_nan=True)


def test_quantize_matrices_at_once():
    """A 3-D tensor: one global scale a matrix, as three calls would give."""
    t, F = G.torch(), G.library()
    w = randn((3, 40, 96), 30, "bf16", 0.02)
    w[1] *= 100
    q = F.fp4_quantize(w, "nvfp4")
    assert q.codes.shape == (3, 40, 48) and q.scales.shape == (3, 40, 6) and q.global_scale.shape == (3,)
    for e in range(3):
        one = F.fp4_quantize(w[e], "nvfp4", rows_per_scale=40)
        assert t.equal(q.codes[e], one.codes) and t.equal(q.scales[e], one.scales)
        assert q.global_scale[e] == one.global_scale[0]
    assert F.fp4_dequantize(q).shape == w.shape
    first = F.fp4_quantize(w[:, :1], "nvfp4")              # one row of each matrix: a row stride of 40 rows
    for e in range(3):
        one = F.fp4_quantize(w[e, :1], "nvfp4")
        assert t.equal(first.codes[e], one.codes) and first.global_scale[e] == one.global_scale[0]
    with pytest.raises(F.MoEError):
        F.fp4_quantize(w[:, :2], "nvfp4")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_dequantize_every_code(fmt):
    t, F = G.torch(), G.library()
    block = ref.BLOCK[fmt]
    codes = np.tile(np.arange(256, dtype=np.uint8), block // 2)[: 256 * block // 2].reshape(256, block // 2)
    if block == 16:                                        # K must be a multiple of 32: two blocks a row
        codes = np.concatenate([codes, codes], 1)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], codes.shape[1] * 2 // block, axis=1)
    Gs = np.full(256, 0.375, dtype=np.float32) if fmt == "nvfp4" else None
    q = F.FP4Tensor(t.from_numpy(codes).cuda(), t.from_numpy(scales).cuda(),
                    None if Gs is None else t.from_numpy(Gs).cuda(), fmt)
    with np.errstate(over="ignore"):
        want = ref.values(codes, scales, Gs, fmt).astype(np.float32)
    assert np.array_equal(F.fp4_dequantize(q).cpu().numpy(), want, equal_nan=True)


# ------------------------------------------------------------------- product
def _operands(fmt, rows, E, N, K, seed):
    """Random codes and scales of a few octaves (every code, every mantissa), on the GPU."""
    t, F = G.torch(), G.library()
    rng = np.random.default_rng(seed)

    def one(lead, per):
        codes = rng.integers(0, 256, lead + (K // 2,), dtype=np.uint8)
        nb = lead + (K // ref.BLOCK[fmt],)
        scales = rng.integers(124, 131, nb, dtype=np.uint8) if fmt == "mxfp4" else rng.integers(40, 72, nb, dtype=np.uint8)
        n = int(np.prod(lead)) // per
        g = None if fmt == "mxfp4" else t.from_numpy(rng.uniform(0.5, 2, n).astype(np.float32)).cuda()
        return F.FP4Tensor(t.from_numpy(codes).cuda(), t.from_numpy(scales).cuda(), g, fmt)

    return one((rows,), 1), one((E, N), N)


def _wide(q, per):
    c, s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    g = None if q.global_scale is None else q.global_scale.cpu().numpy()
    return ref.values(c.reshape(-1, c.shape[-1]), s.reshape(-1, s.shape[-1]), g, q.fmt, per)


def _check_product(x, w, offsets, y0, y, out):
    N, K = w.codes.shape[-2], 2 * w.codes.shape[-1]
    E = w.codes.shape[0]
    off = [0, x.codes.shape[0]] if offsets is None else offsets.tolist()
    want, mag = ref.matmul(_wide(x, 1), _wide(w, N).reshape(E, N, K), off, f64(y0))
    # products are exact; K additions that may cut off; the two scales' products round twice
    tol = (K * 2.0 ** -23 + 2.0 ** -23) * mag * (1 + 2.0 ** -20) + rounding(out, want) * (1 + 2.0 ** -10)
    err = np.abs(f64(y) - want)
    assert np.all(err <= tol), f"worst {np.max(err - tol)} at {np.unravel_index(np.argmax(err - tol), err.shape)}"
    a, b = off[0], off[-1]
    keep = np.r_[0:a, b:want.shape[0]]
    assert np.array_equal(f64(y)[keep], f64(y0)[keep])


DENSE = [(1, 1, 32), (1, 4096, 4096), (2, 127, 96), (7, 128, 256), (16, 130, 288), (17, 256, 512), (33, 64, 2048),
         (65, 384, 1056), (128, 129, 160), (129, 256, 320), (300, 200, 1024), (1000, 512, 768), (3, 2048, 8224),
         (1, 300, 2560), (2, 256, 3584), (16, 512, 1536), (5, 128, 5632), (9, 130, 6720), (4, 64, 2304)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows, N, K", DENSE)
def test_dense_product(fmt, rows, N, K):
    t, F = G.torch(), G.library()
    x, w = _operands(fmt, rows, 1, N, K, rows + N + K)
    for out in ("f32", "bf16", "f16"):
        if out == "f16" and K > 1024:
            continue                                       # sums pass fp16's range
        y = F.fp4_matmul(x, w, out_dtype=dt(out))
        _check_product(x, w, None, t.zeros_like(y), y, out)
    flat = F.FP4Tensor(w.codes[0], w.scales[0], w.global_scale, fmt)
    assert t.equal(F.fp4_matmul(x, flat, out_dtype=dt("f32")), F.fp4_matmul(x, w, out_dtype=dt("f32")))


GROUPED = [  # segment lengths, rows behind, N, K
    ([1], 0, 64, 64), ([0, 1, 0], 2, 128, 256), ([3, 0, 17, 16, 0, 1], 0, 200, 512), ([40, 5, 130, 0, 64], 3, 256, 288),
    ([256, 1, 129, 300], 0, 129, 1024), ([0, 0], 5, 128, 64), ([2] * 64, 0, 512, 2048), ([1] * 100 + [0] * 24, 1, 130, 96),
    ([0] * 1000 + [7] + [0] * 23, 0, 128, 128), ([700], 9, 320, 256), ([20, 45, 0, 31, 40, 33] * 10, 2, 400, 288),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("lens, behind, N, K", GROUPED)
def test_grouped_product(fmt, lens, behind, N, K):
    t, F = G.torch(), G.library()
    rows, E = sum(lens) + behind, len(lens)
    x, w = _operands(fmt, rows, E, N, K, rows + N + K)
    off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
    for out, pad, shift in (("f32", 0, 0), ("bf16", 3, 1), ("f32", 8, 4)):
        y0 = placed(randn((rows, N), 1, out), pad, shift)
        y = placed(y0, pad, shift)
        assert F.fp4_matmul(x, w, off, out=y) is y
        _check_product(x, w, off, y0, y, out)
        again = placed(y0, pad, shift)
        F.fp4_matmul(x, w, off, out=again)
        assert t.equal(y, again)


WIDE = [  # many rows: segment lengths, rows behind, N, K
    ([1300], 0, 4000, 288), ([2561], 3, 2100, 1024), ([700, 0, 257, 256, 1, 95, 300], 5, 3328, 1056),
    ([90, 33, 161, 128, 129, 255] * 6, 0, 513, 2048), ([150, 20, 400, 60] * 5, 2, 1280, 4096),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("lens, behind, N, K", WIDE)
def test_product_of_many_rows(fmt, lens, behind, N, K):
    t, F = G.torch(), G.library()
    rows, E = sum(lens) + behind, len(lens)
    x, w = _operands(fmt, rows, E, N, K, rows + N + K)
    off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
    for out, pad, shift in (("f32", 0, 0), ("bf16", 0, 0), ("bf16", 3, 1), ("bf16", 8, 8)):
        y0 = placed(randn((rows, N), 1, out), pad, shift)
        y = placed(y0, pad, shift)
        F.fp4_matmul(x, w, off, out=y)
        _check_product(x, w, off, y0, y, out)
        again = placed(y0, pad, shift)
        F.fp4_matmul(x, w, off, out=again)
        assert t.equal(y, again)


SHARED = [  # K shared by clusters of 8, 4 and 2, some with nothing to do, and the sizes beside them
    ([16], 0, 128, 256), ([2], 0, 64, 32), ([16], 0, 1920, 2048), ([16], 0, 2048, 2048), ([64], 0, 500, 4096),
    ([17], 0, 1024, 8192), ([200], 0, 100, 4064), ([1], 0, 2048, 4096), ([150], 0, 1024, 2048), ([130], 0, 1024, 1024),
    ([33], 0, 10000, 288), ([16], 0, 16384, 512), ([8], 0, 8192, 512), ([1], 0, 8192, 256), ([1], 0, 128, 768),
    ([40, 5, 33], 2, 300, 2304), ([0, 100, 0, 0, 17], 1, 130, 4608), ([1] * 9, 0, 1000, 544),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("lens, behind, N, K", SHARED)
def test_product_whose_k_is_shared(fmt, lens, behind, N, K):
    t, F = G.torch(), G.library()
    rows, E = sum(lens) + behind, len(lens)
    x, w = _operands(fmt, rows, E, N, K, rows + N + K)
    off = None if E == 1 else t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
    for out, pad, shift in (("f32", 0, 0), ("bf16", 3, 1)):
        y0 = placed(randn((rows, N), 1, out), pad, shift)
        y = placed(y0, pad, shift)
        F.fp4_matmul(x, w, off, out=y)
        _check_product(x, w, off, y0, y, out)
        again = placed(y0, pad, shift)
        F.fp4_matmul(x, w, off, out=again)
        assert t.equal(y, again)


def test_grouped_product_of_a_first_row_past_zero():
    """offsets[0] > 0: the rows before the first segment stay as they are too."""
    t, F = G.torch(), G.library()
    x, w = _operands("nvfp4", 50, 3, 136, 160, 3)
    off = t.tensor([5, 20, 20, 45], dtype=t.int32, device="cuda")
    y0 = randn((50, 136), 2)
    y = y0.clone()
    F.fp4_matmul(x, w, off, out=y)
    _check_product(x, w, off, y0, y, "f32")


def test_offsets_out_of_range_are_cut_to_the_rows():
    t, F = G.torch(), G.library()
    x, w = _operands("mxfp4", 20, 3, 64, 64, 4)
    y0 = randn((20, 64), 3)
    wild, cut = ([-9, 6, 15, 1 << 30], [0, 6, 15, 20])
    ys = []
    for off in (wild, cut):
        y = y0.clone()
        F.fp4_matmul(x, w, t.tensor(off, dtype=t.int32, device="cuda"), out=y)
        ys.append(y)
    assert t.equal(*ys)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_product_of_scales_that_are_not_aligned(fmt, shift):
    t, F = G.torch(), G.library()
    for rows, N, K in ((20, 130, 512), (5, 64, 128), (1200, 3900, 256)):
        x, w = _operands(fmt, rows, 1, N, K, 5)

        def moved(s):
            buf = t.empty(s.numel() + shift, dtype=t.uint8, device="cuda")
            buf[shift:].copy_(s.flatten())
            return buf[shift:].view(s.shape)

        y = F.fp4_matmul(F.FP4Tensor(x.codes, moved(x.scales), x.global_scale, fmt),
                         F.FP4Tensor(w.codes, moved(w.scales), w.global_scale, fmt), out_dtype=dt("f32"))
        assert t.equal(y, F.fp4_matmul(x, w, out_dtype=dt("f32")))
        _check_product(x, w, None, t.zeros_like(y), y, "f32")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_nan_blocks_stay_in_their_rows(fmt):
    """A NaN scale in a row of x is that row of y, one in a row of w that column, one
    behind the segments nothing."""
    t, F = G.torch(), G.library()
    x, w = _operands(fmt, 40, 2, 72, 256, 6)
    nan = 255 if fmt == "mxfp4" else 127
    off = t.tensor([0, 17, 38], dtype=t.int32, device="cuda")
    clean = F.fp4_matmul(x, w, off, out=t.zeros((40, 72), device="cuda"))
    x.scales[16, 1] = nan
    x.scales[39, 0] = nan
    w.scales[1, 5, 2] = nan
    y = F.fp4_matmul(x, w, off, out=t.zeros((40, 72), device="cuda"))
    hit = t.zeros((40, 72), dtype=t.bool, device="cuda")
    hit[16] = True
    hit[17:38, 5] = True
    assert t.isnan(y[hit]).all() and t.equal(y[~hit], clean[~hit])


# ------------------------------------------------------- streams, graphs, use
def _path(F, x, ids, gates, w1, w2, E, fmt):
    t = G.torch()
    r = F.sort_tokens(ids, E)
    q = F.fp4_quantize(x, fmt)
    parts = [F.dispatch(p, r["inv"]) for p in (q.codes, q.scales)]
    gs = None if q.global_scale is None else F.dispatch(q.global_scale[:, None], r["inv"])[:, 0]
    a = F.fp4_matmul(F.FP4Tensor(*parts, gs, fmt), w1, r["offsets"], out_dtype=t.float32)
    gate, up = a.chunk(2, dim=1)
    h = t.nn.functional.silu(gate) * up
    ys = F.fp4_matmul(F.fp4_quantize(h, fmt), w2, r["offsets"], out_dtype=t.float32)
    return F.combine(ys, r["inv"], gates, out_dtype=t.bfloat16), ys, r


def _path_inputs(fmt, T, H, inter, E, k, seed=40):
    F = G.library()
    w1 = F.fp4_quantize(randn((E, 2 * inter, H), seed, "bf16", 0.05), fmt)
    w2 = F.fp4_quantize(randn((E, H, inter), seed + 1, "bf16", 0.05), fmt)
    return randn((T, H), seed + 2, "bf16"), ids_of(T, k, E, seed + 3), randn((T, k), seed + 4).abs(), w1, w2


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_graph_replays_the_path_and_streams_do_not_mix(fmt):
    t, F = G.torch(), G.library()
    E, k, H, inter = 16, 4, 512, 256
    x, ids, gates, w1, w2 = _path_inputs(fmt, 60, H, inter, E, k)
    want = _path(F, x, ids, gates, w1, w2, E, fmt)[0].clone()
    x2, ids2, gates2 = randn(x.shape, 50, "bf16"), ids_of(60, k, E, 51), randn(gates.shape, 52).abs()
    want2 = _path(F, x2, ids2, gates2, w1, w2, E, fmt)[0].clone()
    bufs = [x.clone(), ids.clone(), gates.clone()]
    graphs, outs = [], []
    for _ in range(2):                                     # two graphs over the same inputs share no workspace
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            outs.append(_path(F, *bufs, w1, w2, E, fmt)[0])
        graphs.append(g)
    side = [t.cuda.Stream(), t.cuda.Stream()]
    for inputs, expect in (((x2, ids2, gates2), want2), ((x, ids, gates), want)):
        for b, v in zip(bufs, inputs):
            b.copy_(v)
        t.cuda.synchronize()
        for rep in range(3):
            for g, s in zip(graphs, side):
                with t.cuda.stream(s):
                    g.replay()
        t.cuda.synchronize()
        assert t.equal(outs[0], expect) and t.equal(outs[1], expect)
    # calls given a stream, two at once
    t.cuda.synchronize()
    got = []
    for s, (a, i, gt) in zip(side, ((x, ids, gates), (x2, ids2, gates2))):
        r = F.sort_tokens(i, E, stream=s)
        xs = F.dispatch(a, r["inv"], stream=s)
        got.append((F.combine(xs, r["inv"], gt, stream=s.cuda_stream), r, a, gt))
    t.cuda.synchronize()
    for y, r, a, gt in got:
        assert t.equal(y, F.combine(F.dispatch(a, r["inv"]), r["inv"], gt))


def test_calls_with_no_rows():
    t, F = G.torch(), G.library()
    for fmt in ("mxfp4", "nvfp4"):
        q = F.fp4_quantize(t.empty((0, 64), device="cuda"), fmt)
        assert q.codes.shape == (0, 32) and F.fp4_dequantize(q).shape == (0, 64)
        w = F.fp4_quantize(randn((8, 64), 1), fmt, rows_per_scale=8)
        assert F.fp4_matmul(q, w).shape == (0, 8)
        three = F.fp4_quantize(t.empty((3, 0, 64), device="cuda"), fmt)
        assert three.codes.shape == (3, 0, 32)
    none = t.empty((0, 4), dtype=t.int32, device="cuda")
    x = t.empty((0, 24), device="cuda")
    assert F.dispatch(x, none).shape == (0, 24) and F.combine(x, none).shape == (0, 24)
    assert F.dispatch_backward(x, none).shape == (0, 24)
    dys, dg = F.combine_backward(x, x, none)
    assert dys.shape == (0, 24) and dg.shape == (0, 4)
    # tokens, but no row: every pair is dropped
    inv = t.full((5, 4), -1, dtype=t.int32, device="cuda")
    assert F.dispatch(randn((5, 24), 2), inv, rows=0).shape == (0, 24)
    assert (F.combine(x, inv) == 0).all() and (F.dispatch_backward(x, inv) == 0).all()
    dys, dg = F.combine_backward(randn((5, 24), 3), x, inv)
    assert dys.shape == (0, 24) and (dg == 0).all()


def test_a_call_whose_tensors_are_not_on_the_current_device(monkeypatch):
    """The detour that such a call takes: its first attempt finds another device current."""
    t, F = G.torch(), G.library()
    F.fp4_quantize                                         # loads the operators
    from fp4_expert_layer_b200 import ops
    x = randn((6, 64), 4, "bf16")
    want = F.fp4_quantize(x)
    real, told = ops._ops, []

    class AnotherDeviceAtFirst:
        @staticmethod
        def fp4_quantize(*args):
            told.append(t.cuda.current_device())
            return None if len(told) == 1 else real.fp4_quantize(*args)

    monkeypatch.setattr(ops, "_ops", AnotherDeviceAtFirst)
    got = F.fp4_quantize(x)
    assert told == [0, 0] and t.equal(got.codes, want.codes) and t.equal(got.scales, want.scales)


def test_wide_products_on_two_streams_at_once():
    """Two products that each fill the GPU, in flight together, many times over."""
    t, F = G.torch(), G.library()
    E, N, K = 8, 1536, 1024
    work = []
    for i in range(2):
        x, w = _operands("nvfp4", 1500, E, N, K, 90 + i)
        off = t.tensor(np.linspace(0, 1500, E + 1).astype(np.int32), device="cuda")
        work.append((x, w, off, F.fp4_matmul(x, w, off)))
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    got = [[F.fp4_matmul(x, w, off, stream=s) for s, (x, w, off, _) in zip(streams, work)] for _ in range(20)]
    t.cuda.synchronize()
    for pair in got:
        for y, (_, _, _, want) in zip(pair, work):
            assert t.equal(y, want)


FIRST_CALL = r"""
import torch as t
import fp4_expert_layer_b200 as F
x = t.randn(40, 256, device="cuda").bfloat16()
w = t.randn(64, 256, device="cuda").bfloat16()
ids = t.randint(0, 4, (40, 2), dtype=t.int32, device="cuda")
def path():
    r = F.sort_tokens(ids, 4)
    y = F.fp4_matmul(F.fp4_quantize(x, "nvfp4"), F.fp4_quantize(w, "nvfp4", rows_per_scale=64))
    xs = F.dispatch(y, r["inv"])
    return F.combine(xs, r["inv"])
g = t.cuda.CUDAGraph()
with t.cuda.graph(g):
    got = path()
g.replay()
t.cuda.synchronize()
assert t.equal(got, path()) and t.isfinite(got).all() and got.abs().max() > 0
print("first call captured")
"""


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    G.library()
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=600,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]


def test_more_than_2_31_elements():
    """Element offsets that pass 32 bits: the last rows against calls on those rows alone."""
    t, F = G.torch(), G.library()
    T, H, tail = 270_000, 8192, 300                        # 2.2e9 elements, 4.4 GB in bf16
    x = t.randn((T, H), device="cuda", dtype=t.bfloat16)
    inv = t.arange(T - 1, -1, -1, dtype=t.int32, device="cuda").view(T, 1)
    xs = F.dispatch(x, inv)
    assert t.equal(xs[:tail], x[-tail:].flip(0)) and t.equal(xs[-tail:], x[:tail].flip(0))
    back = F.combine(xs, inv, t.full((T, 1), 2.0, device="cuda"))
    assert t.equal(back[-tail:], 2 * x[-tail:]) and t.equal(back[:tail], 2 * x[:tail])
    dys, dg = F.combine_backward(x, back, inv, out=xs)
    assert t.equal(dys[:tail], x[-tail:].flip(0))
    term = x[-tail:].double() * back[:tail].flip(0).double()
    off = dg[-tail:, 0].double() - term.sum(1)
    assert bool((off.abs() <= H * 2.0 ** -24 * term.abs().sum(1)).all())
    del back, dys, xs
    for fmt in ("mxfp4", "nvfp4"):
        q, last = F.fp4_quantize(x, fmt), F.fp4_quantize(x[-tail:], fmt)
        assert all(a is None or t.equal(a[-tail:], b) for a, b in zip(q[:3], last[:3]))
        assert t.equal(F.fp4_dequantize(q, dtype=t.bfloat16)[-tail:], F.fp4_dequantize(last, dtype=t.bfloat16))
    one = F.fp4_quantize(x, "nvfp4", rows_per_scale=T)
    assert t.equal(one.global_scale[0], q.global_scale.max())
    del x, q, last, one
    x, w = _operands("mxfp4", 550_000, 1, 4104, 32, 95)
    y = F.fp4_matmul(x, w)
    last = F.FP4Tensor(x.codes[-tail:].clone(), x.scales[-tail:].clone(), None, "mxfp4")
    assert t.equal(y[-tail:], F.fp4_matmul(last, w))


def test_quantize_and_long_sort_in_a_graph():
    """The forms of several launches: each replay starts its counts and scales anew."""
    t, F = G.torch(), G.library()
    E, k = 300, 8
    x = t.empty((3, 600, 1024), dtype=t.bfloat16, device="cuda")
    ids = t.empty((4000, k), dtype=t.int32, device="cuda")
    inputs = [(randn(x.shape, 64 + i, "bf16", s), ids_of(4000, k, E, 66 + i, -1, E + 1)) for i, s in
              enumerate((50.0, 0.01))]
    x.copy_(inputs[0][0])
    ids.copy_(inputs[0][1])
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        q, r = F.fp4_quantize(x, "nvfp4"), F.sort_tokens(ids, E)
    for a, i in inputs + inputs[:1]:
        x.copy_(a)
        ids.copy_(i)
        g.replay()
        t.cuda.synchronize()
        want, order = F.fp4_quantize(a, "nvfp4"), F.sort_tokens(i, E)
        assert all(t.equal(m, n) for m, n in zip(q[:3], want[:3]))
        assert all(t.equal(r[n], order[n]) for n in order)


def test_backward_in_a_graph():
    t, F = G.torch(), G.library()
    T, k, E, H = 40, 3, 8, 136
    inv = _rows_case(T, k, E, 1, 60)["inv"]
    ys, dy, gates = randn((T * k, H), 61), randn((T, H), 62), randn((T, k), 63)
    keep = t.zeros_like(ys)
    dys, dg = F.combine_backward(dy, ys, inv, gates, out=keep.clone())
    dx = F.dispatch_backward(ys, inv)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        dys2, dg2 = F.combine_backward(dy, ys, inv, gates, out=keep)
        dx2 = F.dispatch_backward(ys, inv)
    g.replay()
    t.cuda.synchronize()
    assert t.equal(dys, dys2) and t.equal(dg, dg2) and t.equal(dx, dx2)


def test_path_equals_the_layers_own_a4_forward():
    """Route, sort, quantise, dispatch, product, SwiGLU, quantise, product, combine:
    the layer's A4 forward on the same weights, which fp4_quantize made.  Near a
    border the two forms of silu can pick neighbouring codes of h; the tolerance is
    the one the layer's own A4 test has for that."""
    import synth
    t, F = G.torch(), G.library()
    from tests import _cases as cs
    import oracle
    wl = synth.custom_workload(512, 256, 16, 4)
    lw = synth.make_layer(wl, seed=70)
    E, H, inter = 16, 512, 256
    mats = [randn((E, *s), 71 + i, "bf16", 0.05) for i, s in enumerate(((inter, H), (inter, H), (H, inter)))]
    q = [F.fp4_quantize(m, "mxfp4") for m in mats]
    for m in range(3):
        lw.codes[m] = q[m].codes.cpu().numpy()
        lw.scales[m] = q[m].scales.cpu().numpy()
    L = oracle.Layer.from_weights(lw, numerics="a4")
    x_bits, _ = cs.tokens_with_margin(L, wl, 130, stream=5)
    layer = G.make_layer(lw, n_slots=E, max_tokens=130, numerics="a4")
    y_layer, r = G.run(layer, x_bits)
    layer.close()
    x = G.to_device(x_bits)
    ids = t.empty((130, 4), dtype=t.int32, device="cuda")
    gates = t.empty((130, 4), dtype=t.float32, device="cuda")
    F._lib.route_topk_noalloc(x, t.from_numpy(lw.router_w).cuda(),
                              None if lw.router_bias is None else t.from_numpy(lw.router_bias).cuda(), 4, ids, gates)
    w1 = F.FP4Tensor(t.cat([q[0].codes, q[1].codes], 1), t.cat([q[0].scales, q[1].scales], 1), None, "mxfp4")
    y, _, s = _path(F, x, ids, gates, w1, q[2], E, "mxfp4")
    assert np.array_equal(s["offsets"].cpu().numpy(), r["offsets"])
    assert np.array_equal(s["inv"].cpu().numpy().reshape(-1), r["inv"])
    y32 = F.combine(_, s["inv"], gates)
    G.check_output(y32.cpu().numpy(), y_layer)
    y_ref, *_r = L.forward(x_bits)
    G.check_output(y32.cpu().numpy(), y_ref)


def test_binding_refusals_on_the_gpu():
    t, F = G.torch(), G.library()
    x, w = _operands("nvfp4", 8, 2, 64, 64, 80)
    off = t.tensor([0, 4, 8], dtype=t.int32, device="cuda")
    xb = randn((8, 64), 1, "bf16")
    inv = t.zeros((8, 2), dtype=t.int32, device="cuda")
    bad = [
        lambda: F.fp4_matmul(x, w),                                           # groups without offsets
        lambda: F.fp4_matmul(x, w, off.long()),
        lambda: F.fp4_matmul(x, w, off[:2]),
        lambda: F.fp4_matmul(x, w, off.cpu()),
        lambda: F.fp4_matmul(x, w, off, out_dtype=t.float64),
        lambda: F.fp4_matmul(x, w, off, out=t.empty((8, 63), device="cuda")),
        lambda: F.fp4_matmul(x._replace(fmt="mxfp4"), w, off),
        lambda: F.fp4_matmul(x._replace(global_scale=None), w, off),
        lambda: F.fp4_matmul(x._replace(scales=x.scales[:, :2]), w, off),
        lambda: F.fp4_matmul(x._replace(codes=x.codes.t()), w, off),
        lambda: F.fp4_quantize(xb, "fp8"),
        lambda: F.fp4_quantize(xb.long()),
        lambda: F.fp4_quantize(xb[:, :40]),
        lambda: F.fp4_quantize(xb.t()),
        lambda: F.fp4_quantize(xb, "nvfp4", rows_per_scale=3),
        lambda: F.fp4_quantize(xb[:1].expand(8, 64)),                         # rows that are one row
        lambda: F.fp4_quantize(xb, "nvfp4", out=x._replace(fmt="mxfp4", global_scale=None)),
        lambda: F.sort_tokens(inv.long(), 4),
        lambda: F.sort_tokens(inv, 0),
        lambda: F.sort_tokens(inv, 1025),
        lambda: F.dispatch(xb, inv[:4]),
        lambda: F.dispatch(xb.double(), inv),
        lambda: F.dispatch(xb, inv.t()),
        lambda: F.dispatch(xb, inv.cpu()),
        lambda: F.combine(xb, inv, t.ones((8, 3), device="cuda")),
        lambda: F.combine(xb, inv, t.ones((8, 2), device="cuda").half()),
        lambda: F.combine(xb.view(t.uint8), inv),
        lambda: F.combine_backward(xb, xb[:, :32], inv),
        lambda: F.dispatch_backward(xb, inv, out=t.empty((8, 64), device="cuda")),
        lambda: F.dispatch(xb, inv, stream=t.cuda.Stream(), out=t.empty((16, 64))),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(F.MoEError) as ei:
            call()
        assert ei.value.status == 1, i


# ------------------------------------------------- products after a wait that gave up
def _give_up(F, stream=None):
    s = G.torch().cuda.current_stream() if stream is None else stream
    assert F.lib().moe_debug_give_up(0, s.cuda_stream) == 0


def _reported_once(F, call):
    with pytest.raises(F.MoEError) as ei:
        call()
    assert ei.value.status == 5 and "gave up" in str(ei.value)
    return call()


def _small_products():
    """One of each kernel: K shared by a cluster, weights streamed, CTA pairs."""
    t, F = G.torch(), G.library()
    out = []
    for i, (lens, N, K) in enumerate((([3], 256, 2048), ([2] * 80, 256, 256), ([300, 80], 512, 512))):
        x, w = _operands("nvfp4", sum(lens), len(lens), N, K, 200 + i)
        off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
        out.append((x, w, off, F.fp4_matmul(x, w, off)))
    return out


def test_a_wait_that_gave_up_is_reported_once():
    t, F = G.torch(), G.library()
    for x, w, off, want in _small_products():
        _give_up(F)
        t.cuda.synchronize()
        y = t.full_like(want, 7.0)
        with pytest.raises(F.MoEError) as ei:
            F.fp4_matmul(x, w, off, out=y)
        assert ei.value.status == 5 and "gave up" in str(ei.value)
        t.cuda.synchronize()
        assert (y == 7).all()                              # the refused call did nothing
        assert t.equal(F.fp4_matmul(x, w, off), want)
    for _ in range(2):                                     # two failures, one report
        _give_up(F)
    t.cuda.synchronize()
    assert t.equal(_reported_once(F, lambda: F.fp4_matmul(x, w, off)), want)


def test_a_failure_reported_inside_a_capture():
    """The refused call adds no node; the capture goes on, and its replays are right."""
    t, F = G.torch(), G.library()
    for x, w, off, want in _small_products():
        y = t.zeros_like(want)
        _give_up(F)
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            _reported_once(F, lambda: F.fp4_matmul(x, w, off, out=y))
        assert t.equal(F.fp4_matmul(x, w, off), want)      # before any replay
        g.replay()
        t.cuda.synchronize()
        assert t.equal(y, want)


def test_a_failure_ends_no_other_product():
    """Products beside it on another stream, and replayed after it, are right."""
    t, F = G.torch(), G.library()
    side = t.cuda.Stream()
    for x, w, off, want in _small_products():
        y = t.zeros_like(want)
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            F.fp4_matmul(x, w, off, out=y)
        t.cuda.synchronize()
        _give_up(F, side)                                  # a millisecond on the side stream
        for _ in range(3):                                 # the first replay beside it, the others after it
            y.zero_()
            g.replay()
            t.cuda.synchronize()
            assert t.equal(y, want)
        with t.cuda.stream(side):
            again = _reported_once(F, lambda: F.fp4_matmul(x, w, off))
        t.cuda.synchronize()
        assert t.equal(again, want)


def test_a_program_that_only_replays_asks_with_no_rows():
    t, F = G.torch(), G.library()
    _, w, off, _ = _small_products()[2]
    none = F.fp4_quantize(t.empty((0, 512), device="cuda"), "nvfp4")
    assert F.fp4_matmul(none, w, off).shape == (0, 512)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        _give_up(F)
    for _ in range(2):
        g.replay()
        t.cuda.synchronize()
        assert _reported_once(F, lambda: F.fp4_matmul(none, w, off)).shape == (0, 512)


# ---------------------------------------------- global scales far from one another
FAR = [  # x's scale, w's scale: their product leaves fp32's range, or its normal numbers, where y does not
    (1.3 * 2.0 ** -70, 1.7 * 2.0 ** -75), (1.1 * 2.0 ** -75, 1.9 * 2.0 ** -80), (1.9 * 2.0 ** -66, 1.7 * 2.0 ** -62),
    (-1.7 * 2.0 ** -90, 1.3 * 2.0 ** -50), (1.5 * 2.0 ** 60, 1.3 * 2.0 ** -140), (1.3 * 2.0 ** 100, 1.7 * 2.0 ** -120),
]
FAR_SIZES = [  # each kernel of the product: K shared, weights streamed, pairs with and without whole rows
    ([3], 256, 2048, 0), ([20, 0, 13], 130, 512, 0), ([2] * 80, 256, 256, 0), ([300, 70], 512, 512, 0), ([300, 70], 515, 512, 1),
]


@pytest.mark.parametrize("lens, N, K, pad", FAR_SIZES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_global_scales_meet_the_sum_one_by_one(lens, N, K, pad, out):
    t, F = G.torch(), G.library()
    rows, E = sum(lens), len(lens)
    x, w = _operands("nvfp4", rows, E, N, K, 300 + N)
    rng = np.random.default_rng(N)
    for q in (x, w):                                       # block scales up to the largest: sums near 2^25
        q.scales.copy_(t.from_numpy(rng.integers(112, 127, tuple(q.scales.shape), dtype=np.uint8)))
    off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
    for xg, wg in FAR:
        far = t.arange(rows, device="cuda") % 3 != 1       # ordinary rows among them in every tile
        x.global_scale.copy_(t.where(far, t.full((rows,), xg, device="cuda"), t.full((rows,), 2.0 ** -3 / abs(wg), device="cuda")
                                     if 2.0 ** -3 / abs(wg) < 3e38 else t.full((rows,), 2.0 ** 100, device="cuda")))
        w.global_scale.fill_(wg)
        y = placed(t.zeros((rows, N), dtype=dt(out), device="cuda"), pad, pad)
        F.fp4_matmul(x, w, off, out=y)
        _check_product(x, w, off, t.zeros_like(y), y, out)


@pytest.mark.parametrize("lens, N, K, pad", FAR_SIZES)
def test_a_sum_of_zero_is_zero_at_any_global_scale(lens, N, K, pad):
    """And a sum that is not stays infinite of its sign where the value passes the range."""
    t, F = G.torch(), G.library()
    rows, E = sum(lens), len(lens)
    x, w = _operands("nvfp4", rows, E, N, K, 400 + N)
    x.codes[::2] = 0
    w.codes[:, 1::2] = 0
    x.global_scale.fill_(2.0 ** 70)
    w.global_scale.fill_(2.0 ** 80)
    off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
    y = F.fp4_matmul(x, w, off, out_dtype=t.float32)
    zero = t.zeros((rows, N), dtype=t.bool, device="cuda")
    zero[::2] = True
    zero[:, 1::2] = True
    assert (y[zero] == 0).all()
    one = x._replace(global_scale=t.ones_like(x.global_scale)), w._replace(global_scale=t.ones_like(w.global_scale))
    sign = t.sign(F.fp4_matmul(*one, off, out_dtype=t.float32))
    assert t.equal(y[sign != 0], sign[sign != 0] * float("inf"))


@pytest.mark.parametrize("K", [1 << 30, (1 << 30) - 32])
def test_product_of_the_longest_rows(K):
    """Half a gigabyte of codes a row: what lies at the far end counts, and nothing twice."""
    t, F = G.torch(), G.library()
    codes = t.zeros((3, K // 2), dtype=t.uint8, device="cuda")
    scales = t.full((3, K // 32), 127, dtype=t.uint8, device="cuda")
    codes[0, -16:] = 0x22                                  # 32 ones in the last block
    codes[0, 0] = 0x07                                     # and 6 in front
    codes[1, -16:] = 0x44                                  # twos
    codes[1, 0] = 0x02
    codes[2, K // 4] = 0x22                                # elements that the row of x does not have
    scales[0, -1] = 128
    scales[1, -1] = 129
    x = F.FP4Tensor(codes[:1], scales[:1], None, "mxfp4")
    y = F.fp4_matmul(x, F.FP4Tensor(codes[1:], scales[1:], None, "mxfp4"), out_dtype=t.float32)
    assert y.tolist() == [[6 + 32 * 2 * (2 * 4), 0]]


# ------------------------------------------------ values at any global scale
def _nearest(value, name):
    """value (float64 products of a short number and an fp32 one: exact) rounded once to a type."""
    t = G.torch()
    f = t.finfo(dt(name))
    m, e = np.frexp(value)
    low = int(np.log2(f.smallest_normal)) + 1              # exponent (as frexp counts) of the smallest normal number
    bits = int(round(-np.log2(f.eps))) + 1
    step = np.ldexp(1.0, np.maximum(e, low) - bits)
    r = np.round(value / step) * step                      # ties to even; the quotient is exact
    return np.where(np.abs(r) > f.max, np.copysign(np.inf, r), r)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_dequantize_rounds_once_at_any_global_scale(out):
    """Every code and every scale code with global scales of 24 digits, from subnormal to near the end of the range."""
    t, F = G.torch(), G.library()
    rng = np.random.default_rng(7)
    Gs = np.concatenate([rng.uniform(0.5, 2, 300), rng.uniform(0.5, 2, 300) * 2.0 ** rng.integers(-148, 127, 300),
                         -rng.uniform(0.5, 2, 20), 2.0 ** rng.integers(-100, 100, 20), [0.0]]).astype(np.float32)
    # a product that lies next to a border of bf16 or of f16: found by trying last digits
    near = np.float32(1.5) + np.arange(64, dtype=np.float32) * np.float32(2.0 ** -23)
    Gs = np.concatenate([Gs, near, near + np.float32(2.0 ** -8), near + np.float32(2.0 ** -11)])
    n = Gs.size
    codes = np.tile(np.arange(256, dtype=np.uint8), 127 * 8 // 256 + 1)[:127 * 8]
    codes = np.stack([np.roll(codes, 3 * i) for i in range(n)])
    codes = np.concatenate([codes, codes[:, :8]], 1)       # 128 blocks of 16: every finite scale, and 0 again
    scales = np.tile(np.r_[np.arange(127), 0].astype(np.uint8), (n, 1))
    scales[1::2] |= 128                                    # the entry point takes signs too
    q = F.FP4Tensor(t.from_numpy(codes).cuda(), t.from_numpy(scales).cuda(), t.from_numpy(Gs).cuda(), "nvfp4")
    want = _nearest(ref.values(codes, scales, Gs, "nvfp4"), out)
    got = f64(F.fp4_dequantize(q, dtype=dt(out)))
    bad = got != want
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {got[bad][:4]} {want[bad][:4]}"
    # one scale for all rows, of a tensor with three axes, into the caller's own rows
    for g in Gs[[0, 301, 5]]:
        one = F.FP4Tensor(q.codes.view(1, n, -1), q.scales.view(1, n, -1), t.tensor([g], device="cuda"), "nvfp4")
        want = _nearest(ref.values(codes, scales, np.array([g]), "nvfp4", n), out)
        assert np.array_equal(f64(F.fp4_dequantize(one, dtype=dt(out)))[0], want)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_mxfp4_values_past_a_types_range(out):
    """Scale code 254 is 2^127: 4 and 6 of it are infinite, as a rounding of any number past the range is."""
    t, F = G.torch(), G.library()
    codes = np.tile(np.arange(256, dtype=np.uint8), (255, 1))[:, :256]
    scales = np.repeat(np.arange(255, dtype=np.uint8)[:, None], 512 // 32, axis=1)
    q = F.FP4Tensor(t.from_numpy(codes).cuda(), t.from_numpy(scales).cuda(), None, "mxfp4")
    assert np.array_equal(f64(F.fp4_dequantize(q, dtype=dt(out))), _nearest(ref.values(codes, scales, None, "mxfp4"), out))


# ------------------------------------------------------------- autograd's records
def _writes():
    """Each call that takes `out`: (call, outputs whose memory it writes)."""
    t, F = G.torch(), G.library()
    inv = t.arange(8, dtype=t.int32, device="cuda").view(4, 2)
    x, ys, dy = randn((4, 64), 1), randn((8, 64), 2), randn((4, 64), 3)
    xq, wq = _operands("nvfp4", 4, 1, 8, 64, 5)
    q = F.FP4Tensor(t.empty_like(xq.codes), t.empty_like(xq.scales), t.empty_like(xq.global_scale), "nvfp4")
    new = lambda *shape: t.zeros(shape, device="cuda")
    return {
        "fp4_quantize": (lambda out, **kw: F.fp4_quantize(x, "nvfp4", out=q, **kw), q[:3]),
        "fp4_dequantize": (lambda out, **kw: F.fp4_dequantize(xq, out=out, **kw), [new(4, 64)]),
        "fp4_matmul": (lambda out, **kw: F.fp4_matmul(xq, wq, out=out, **kw), [new(4, 8)]),
        "dispatch": (lambda out, **kw: F.dispatch(x, inv, out=out, **kw), [new(8, 64)]),
        "dispatch_backward": (lambda out, **kw: F.dispatch_backward(ys, inv, out=out, **kw), [new(4, 64)]),
        "combine": (lambda out, **kw: F.combine(ys, inv, out=out, **kw), [new(4, 64)]),
        "combine_backward": (lambda out, **kw: F.combine_backward(dy, ys, inv, out=out, **kw), [new(8, 64)]),
    }


@pytest.mark.parametrize("name", ["fp4_quantize", "fp4_dequantize", "fp4_matmul", "dispatch", "dispatch_backward", "combine",
                                  "combine_backward"])
def test_a_written_out_moves_its_version(name):
    """What autograd goes by when a tensor that it saved has been overwritten."""
    t = G.torch()
    call, outs = _writes()[name]
    before = [o._version for o in outs]
    call(outs[0])
    assert all(o._version > v for o, v in zip(outs, before))
    middle = [o._version for o in outs]
    call(outs[0], stream=t.cuda.current_stream())
    assert all(o._version > v for o, v in zip(outs, middle))
    if name != "fp4_quantize":                             # the squares' gradient needs the values that are gone
        leaf = t.ones_like(outs[0], requires_grad=True)
        loss = (leaf * outs[0]).sum()
        call(outs[0])
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    with t.inference_mode():                               # tensors without a version are written as ever
        call_in, outs_in = _writes()[name]
        call_in(outs_in[0])
    call_in(outs_in[0])


@pytest.mark.parametrize("name", ["fp4_dequantize", "fp4_matmul", "dispatch", "dispatch_backward", "combine",
                                  "combine_backward"])
def test_an_out_that_records_a_graph_is_refused(name):
    """As torch's own out= refuses it; not where nothing is recorded."""
    t, F = G.torch(), G.library()
    call, (out,) = _writes()[name]
    leaf = out.requires_grad_()
    for o in (leaf, leaf * 2):
        kept = o.detach().clone()
        with pytest.raises(F.MoEError) as ei:
            call(o)
        assert ei.value.status == 1 and "out requires grad" in str(ei.value)
        assert t.equal(o.detach(), kept)
        with t.no_grad():
            call(o)
        assert not t.equal(o.detach(), kept)


def _detached_calls():
    """Each call whose result is a number times an input: (call, that input, the function's name)."""
    t, F = G.torch(), G.library()
    inv = t.arange(8, dtype=t.int32, device="cuda").view(4, 2)
    x, ys, dy, gates = randn((4, 64), 1), randn((8, 64), 2), randn((4, 64), 3), randn((4, 2), 4)
    xq, wq = _operands("nvfp4", 4, 1, 8, 64, 5)
    scaled = lambda q: lambda g: q._replace(global_scale=g)
    return [
        (lambda v: F.dispatch(v, inv), x, "dispatch"), (lambda v: F.dispatch_backward(v, inv), ys, "dispatch_backward"),
        (lambda v: F.combine(v, inv, gates), ys, "combine"), (lambda v: F.combine(ys, inv, v), gates, "combine"),
        (lambda v: F.combine_backward(v, ys, inv, gates), dy, "combine_backward"),
        (lambda v: F.combine_backward(dy, v, inv, gates), ys, "combine_backward"),
        (lambda v: F.combine_backward(dy, ys, inv, v), gates, "combine_backward"),
        (lambda v: F.fp4_dequantize(scaled(xq)(v)), xq.global_scale, "fp4_dequantize"),
        (lambda v: F.fp4_matmul(scaled(xq)(v), wq), xq.global_scale, "fp4_matmul"),
        (lambda v: F.fp4_matmul(xq, scaled(wq)(v)), wq.global_scale, "fp4_matmul"),
    ]


def test_an_input_whose_gradient_is_not_recorded_is_warned_of():
    """The result is what it was, detached; no warning where nothing would be recorded anyway."""
    import warnings
    t, F = G.torch(), G.library()
    first = lambda r: r[0] if isinstance(r, tuple) else r
    for call, v, name in _detached_calls():
        want = first(call(v))
        leaf = v.clone().requires_grad_()
        with pytest.warns(UserWarning, match=f"{name}: .* requires grad"):
            got = first(call(leaf))
        assert t.equal(got, want) and not got.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with t.no_grad():
                assert t.equal(first(call(leaf)), want)
            assert t.equal(first(call(leaf.detach())), want)
            with pytest.raises(UserWarning):               # a program may make errors of them
                call(leaf)
    with warnings.catch_warnings():                        # codes have no gradient: quantising a parameter is no mistake
        warnings.simplefilter("error")
        F.fp4_quantize(t.nn.Parameter(randn((8, 64), 6)), "nvfp4")


def test_gradients_called_within_a_function_of_ones_own():
    """combine and dispatch as torch.autograd.Functions: the calls inside them are not warned of."""
    import warnings
    t, F = G.torch(), G.library()
    T, k, E, H = 9, 3, 5, 64
    inv = _rows_case(T, k, E, 1, 7)["inv"]

    class Dispatch(t.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return F.dispatch(x, inv, out=x.new_zeros(T * k, H))

        @staticmethod
        def backward(ctx, d):
            return F.dispatch_backward(d.contiguous(), inv)

    class Combine(t.autograd.Function):
        @staticmethod
        def forward(ctx, ys, gates):
            ctx.save_for_backward(ys, gates)
            return F.combine(ys, inv, gates)

        @staticmethod
        def backward(ctx, d):
            ys, gates = ctx.saved_tensors
            return F.combine_backward(d.contiguous(), ys, inv, gates, out=t.zeros_like(ys))

    x, gates, dy = randn((T, H), 8).requires_grad_(), randn((T, k), 9).requires_grad_(), randn((T, H), 10)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        y = Combine.apply(Dispatch.apply(x).square(), gates)
        y.backward(dy)
    iv = inv.cpu().numpy()
    xs = ref.dispatch(f64(x), iv, np.zeros((T * k, H)))
    dys, dg, mag = ref.combine_backward(f64(dy), xs ** 2, iv, f64(gates), np.zeros((T * k, H)))
    dx, dmag = ref.combine(2 * xs * dys, iv, np.ones((T, k)))
    # three fp32 roundings of xs^2 and its gradient, and the sums' own
    assert np.all(np.abs(f64(gates.grad) - dg) <= (H + 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -20) + TINY["f32"])
    assert np.all(np.abs(f64(x.grad) - dx) <= (k + 4) * 2.0 ** -24 * dmag * (1 + 2.0 ** -20) + TINY["f32"])


def test_a_wait_for_a_long_item_has_a_longer_limit():
    """4 us a stage, ten times what one takes: no row that the product accepts is given up on."""
    t, F = G.torch(), G.library()
    _, w, off, _ = _small_products()[2]
    none = F.fp4_quantize(t.empty((0, 512), device="cuda"), "nvfp4")
    took = []
    for stages in (0, 50000):
        a, b = t.cuda.Event(enable_timing=True), t.cuda.Event(enable_timing=True)
        a.record()
        assert F.lib().moe_debug_give_up(stages, t.cuda.current_stream().cuda_stream) == 0
        b.record()
        t.cuda.synchronize()
        took.append(a.elapsed_time(b))
        _reported_once(F, lambda: F.fp4_matmul(none, w, off))
    # the limit is a time of the GPU's own clock, read every 256 polls: not before it, and soon after
    assert 0.99 <= took[0] < 100 and 200 <= took[1] < 400, took
    assert F.lib().moe_debug_give_up(-1, None) == 1 and F.lib().moe_debug_give_up(250001, None) == 1


@pytest.mark.parametrize("out, pad", [("f32", 0), ("bf16", 0), ("bf16", 3)])
@pytest.mark.parametrize("which", ["every third", "chunks", "one"])
def test_distant_scales_in_tiles_of_many_rows(which, out, pad):
    """Both ends of the accumulators, several items a pair, chunks with and without such rows."""
    t, F = G.torch(), G.library()
    lens, N, K = [1300, 0, 257, 256, 1, 95, 900], 2100, 288
    rows, E = sum(lens), len(lens)
    x, w = _operands("nvfp4", rows, E, N, K, 500)
    rng = np.random.default_rng(5)
    for q in (x, w):
        q.scales.copy_(t.from_numpy(rng.integers(112, 127, tuple(q.scales.shape), dtype=np.uint8)))
    r = t.arange(rows, device="cuda")
    far = {"every third": r % 3 == 0, "chunks": r % 64 < 32, "one": r == 1400}[which]
    w.global_scale.fill_(1.9 * 2.0 ** -80)
    x.global_scale.copy_(t.where(far, 1.1 * 2.0 ** -75, 1.3 * 2.0 ** 70))
    off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
    y0 = randn((rows, N), 1, out)
    y = placed(y0, pad, 0)
    F.fp4_matmul(x, w, off, out=y)
    _check_product(x, w, off, y0, y, out)
    again = placed(y0, pad, 0)
    F.fp4_matmul(x, w, off, out=again)
    assert t.equal(y, again)


@pytest.mark.parametrize("out, pad, shift", [("bf16", 8, 8), ("bf16", 3, 1), ("f16", 8, 0), ("f16", 1, 1), ("f32", 3, 1)])
def test_dequantize_rounds_once_into_rows_at_any_element(out, pad, shift):
    t, F = G.torch(), G.library()
    n, K = 700, 544
    rng = np.random.default_rng(9)
    codes = rng.integers(0, 256, (n, K // 2), dtype=np.uint8)
    scales = rng.integers(0, 127, (n, K // 16), dtype=np.uint8)
    Gs = (rng.uniform(0.5, 2, n) * 2.0 ** rng.integers(-20, 6, n)).astype(np.float32)
    # on a border of bf16, and of f16, but for the last digits: 1.5 (1 + 2^-8) / 1.5 and the like
    Gs[::5] = np.float32(1 + 2.0 ** -8) + np.float32(2.0 ** -23) * rng.integers(-2, 3, Gs[::5].size).astype(np.float32)
    Gs[1::5] = np.float32(1 + 2.0 ** -11) + np.float32(2.0 ** -23) * rng.integers(-2, 3, Gs[1::5].size).astype(np.float32)
    q = F.FP4Tensor(t.from_numpy(codes).cuda(), t.from_numpy(scales).cuda(), t.from_numpy(Gs).cuda(), "nvfp4")
    o = placed(t.full((n, K), 7.0, dtype=dt(out), device="cuda"), pad, shift)
    F.fp4_dequantize(q, out=o)
    assert np.array_equal(f64(o), _nearest(ref.values(codes, scales, Gs, "nvfp4"), out))
    if pad:
        whole = t.as_strided(o, (n - 1, pad), (K + pad, 1), o.storage_offset() + K)
        assert (whole == 0).all()                          # what lies between the rows is not touched
