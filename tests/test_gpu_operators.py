"""GPU parity of layer norm, gradient clipping and the 4-bit expert FFN against their float64
definitions.

Tolerances.  u = 2^-24 is half a step of float32; an output rounded to bf16 is off by at most 2^-8 of
its value more.  A sum of n values is off by at most (its longest chain of additions) * u * (the sum
of the magnitudes): a row of H elements is summed by at least 64 lanes and joined in at most 16
further steps, so its chain is at most H / 64 + 16; sums over rows are bounded by the number of rows
and joins, in any order.
"""
import numpy as np
import pytest
import torch

import balanced_token_dispatch_moonep_amd as M
from balanced_token_dispatch_moonep_amd.layer import GradClipper, MoonEPLayer, W4Experts
import oracle as O
from oracle import around as A
import workload as W

from gpu_util import DEV, say, i32, f32, bf16_from_bits, f64_of, rel_fro

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32


def _half(dtype):
    return 2.0 ** -8 if dtype == BF else U


def _rows(rows, H, dtype, seed, scale=1.0, offset=0.3):
    rng = np.random.default_rng(seed)
    x = scale * (rng.standard_normal((rows, H)) * (0.5 + rng.random(H)) + offset)
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)


def _params(H, seed):
    rng = np.random.default_rng(seed + 1)
    return f32(1 + 0.2 * rng.standard_normal(H)), f32(0.3 * rng.standard_normal(H))


def _norm_dims(rows, H, dtype, R=1, accum=False):
    return M.Dims.make(R, R, 0, rows // R, 1, H, f32_rows=dtype == F32, grad_accum=accum)


def _far(got, want, tol, what):
    d = np.abs(got - want)
    worst = float((d / np.maximum(tol, 1e-300)).max()) if d.size else 0.0
    say(f"  {what}: {worst:.3f} of its tolerance")
    assert np.isfinite(got).all() and (d <= tol).all(), what


def _check_norm(rows, H, dtype, weight=True, bias=True, seed=0, scale=1.0, offset=0.3):
    say("norm", rows, H, dtype, weight, bias, seed)
    x = _rows(rows, H, dtype, seed, scale, offset)
    w, b = _params(H, seed)
    w, b = w if weight else None, b if bias else None
    y = torch.full((1, rows, H), -7.0, dtype=dtype, device=DEV)
    mean, rstd = (torch.full((rows,), -7.0, device=DEV) for _ in range(2))
    M.moonep_layer_norm(_norm_dims(rows, H, dtype), x[None], w, b, EPS, y, mean, rstd)
    torch.cuda.synchronize()
    xs = f64_of(x)
    ws = None if w is None else f64_of(w)
    ry, rm, rr = A.layer_norm(xs, ws, None if b is None else f64_of(b), EPS)
    chain = H / 64 + 16
    dm = (chain * np.abs(xs).mean(1) + np.abs(rm)) * U
    # squares of (x - m): the mean's own error enters squared; a rounding each for difference and square,
    # then eps, root and quotient
    dr = rr * ((chain + 8) * U + (rr * dm) ** 2)
    _far(f64_of(mean), rm, dm, "mean")
    _far(f64_of(rstd), rr, dr, "rstd")
    n = (xs - rm[:, None]) * rr[:, None]
    dn = rr[:, None] * dm[:, None] + np.abs(n) * (dr / rr + 3 * U)[:, None]
    aw = 1.0 if ws is None else np.abs(ws)
    tol = aw * dn + 2 * U * (np.abs(n) * aw + np.abs(ry)) + _half(dtype) * np.abs(ry)
    _far(f64_of(y[0]), ry, tol * (1 + 1e-2), "y")


SHAPES = [(1, 8), (1, 7168), (3, 16), (5, 24), (64, 128), (7, 504), (9, 512), (3, 520), (33, 1000), (2, 1024),
          (5, 1032), (6, 2048), (7, 2056), (3, 4096), (4, 4104), (3, 8192), (5, 8200), (2, 16384), (3, 16392),
          (2, 32768), (2, 32776), (1, 100000), (1000, 64), (515, 328)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,H", SHAPES)
def test_norm(rows, H, dtype):
    _check_norm(rows, H, dtype)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("H", [72, 7168, 40000])
def test_norm_without_parameters(H, weight, bias):
    _check_norm(4, H, BF, weight, bias, seed=3)


def test_norm_buffers_side_by_side():
    """Inputs and outputs cut out of one buffer with nothing between them."""
    rows, H = 5, 64
    n = rows * H
    buf = torch.full((4 * n + 64,), 7.0, device=DEV)
    x, y, dx, dy = (buf[i * n:(i + 1) * n].view(1, rows, H) for i in range(4))
    xs, ds = _rows(rows, H, F32, 15), _rows(rows, H, F32, 16)
    x.copy_(xs), dy.copy_(ds)
    w, b = _params(H, 15)
    mean, rstd, dw, db = (torch.empty(k, device=DEV) for k in (rows, rows, H, H))
    d = _norm_dims(rows, H, F32)
    ws = torch.empty(M.moonep_layer_norm_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    M.moonep_layer_norm(d, x, w, b, EPS, y, mean, rstd)
    M.moonep_layer_norm_backward(d, dy, x, w, mean, rstd, dx, dw, db, ws)
    alone = [torch.empty(1, rows, H, device=DEV) for _ in range(2)]
    M.moonep_layer_norm(d, xs[None], w, b, EPS, alone[0])
    M.moonep_layer_norm_backward(d, ds[None], xs[None], w, mean, rstd, alone[1], None, None)
    assert torch.equal(y, alone[0]) and torch.equal(dx, alone[1])
    assert torch.equal(x[0], xs) and torch.equal(dy[0], ds) and bool((buf[4 * n:] == 7.0).all())
    with pytest.raises(M.MoonEPError):
        M.moonep_layer_norm(d, x, w, b, EPS, x)
    with pytest.raises(M.MoonEPError):
        M.moonep_layer_norm_backward(d, dy, x, w, mean, rstd, dy, None, None)


def test_norm_far_from_zero():
    """A mean a thousand times the spread: the variance is that of the centred row."""
    for dtype in (F32, BF):
        _check_norm(5, 4096, dtype, seed=4, offset=1000.0)
    _check_norm(5, 4096, F32, seed=4, scale=1e15)
    _check_norm(5, 4096, F32, seed=4, scale=1e-3)


def test_norm_constant_and_broken_rows():
    rows, H = 6, 264
    x = _rows(rows, H, F32, 5)
    x[1] = 3.0
    x[2, 17] = float("nan")
    x[4, 200] = float("inf")
    w, b = _params(H, 5)
    y = torch.zeros(1, rows, H, device=DEV)
    M.moonep_layer_norm(_norm_dims(rows, H, F32), x[None], w, b, EPS, y)
    assert torch.equal(y[0, 1], b)
    assert torch.isnan(y[0, 2]).all() and torch.isnan(y[0, 4]).all()
    for r in (0, 3, 5):
        alone = torch.zeros(1, 1, H, device=DEV)
        M.moonep_layer_norm(_norm_dims(1, H, F32), x[r][None, None], w, b, EPS, alone)
        assert torch.equal(alone[0, 0], y[0, r])


def _check_backward(rows, H, dtype, weight=True, seed=0, accum=False, want=(True, True)):
    say("norm backward", rows, H, dtype, weight, seed, accum, want)
    x, dy = _rows(rows, H, dtype, seed), _rows(rows, H, dtype, seed + 50, scale=1e-2, offset=0.1)
    w = _params(H, seed)[0] if weight else None
    xs, ds = f64_of(x), f64_of(dy)
    _, m, r = A.layer_norm(xs, None, None, EPS)
    mean, rstd = f32(m), f32(r)
    dx = torch.full((1, rows, H), -7.0, dtype=dtype, device=DEV)
    dw, db = (torch.full((H,), 0.25, device=DEV) if k else None for k in want)
    d = _norm_dims(rows, H, dtype, accum=accum)
    ws = torch.full((M.moonep_layer_norm_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
    M.moonep_layer_norm_backward(d, dy[None], x[None], w, mean, rstd, dx, dw, db, ws if any(want) else None)
    torch.cuda.synchronize()
    m, r = f64_of(mean), f64_of(rstd)
    ws64 = None if w is None else f64_of(w)
    rx, rw, rb = A.layer_norm_backward(ds, xs, ws64, m, r)
    n = (xs - m[:, None]) * r[:, None]
    g = ds if w is None else ds * ws64
    chain = H / 64 + 16
    c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    dc1, dc2 = (chain + 2) * U * a1, (chain + 5) * U * a2
    tol = r[:, None] * (dc1 + np.abs(n) * dc2 + 4 * U * (np.abs(g) + np.abs(c1) + 2 * np.abs(n * c2))) \
        + 2 * U * np.abs(rx) + _half(dtype) * np.abs(rx)
    _far(f64_of(dx[0]), rx, tol * (1 + 1e-2), "dx")
    base = 0.25 if accum else 0.0
    for got, ref, mass, what in ((dw, rw, np.abs(ds * n).sum(0), "dweight"), (db, rb, np.abs(ds).sum(0), "dbias")):
        if got is not None:
            _far(f64_of(got), base + ref, (rows + 16) * U * mass + 2 * U * (base + np.abs(ref)), what)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,H", SHAPES)
def test_norm_backward(rows, H, dtype):
    _check_backward(rows, H, dtype)


@pytest.mark.parametrize("rows,H", [(5, 72), (300, 2048), (17, 7168), (3, 40000)])
def test_norm_backward_options(rows, H):
    _check_backward(rows, H, BF, weight=False, seed=1)
    _check_backward(rows, H, BF, accum=True, seed=2)
    for want in ((True, False), (False, True), (False, False)):
        _check_backward(rows, H, F32, want=want, seed=3, accum=True)


def test_norm_backward_many_rows():
    _check_backward(20011, 136, BF, seed=4)
    _check_backward(3001, 1024, F32, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,H", [(700, 2056), (520, 4104), (515, 5120), (300, 8200), (257, 12288), (513, 16384)])
def test_norm_backward_several_rows_a_workgroup(rows, H, dtype):
    _check_backward(rows, H, dtype, seed=6)
    _check_backward(rows, H, dtype, weight=False, seed=7, accum=True)


def test_norm_backward_of_an_infinite_weight():
    """The last columns' weights are infinite and their dy is not zero: c1 is infinite in each row, and
    the other columns' sums over rows stay finite."""
    rows, H = 300, 8200
    for dtype in (BF, F32):
        x, dy = _rows(rows, H, dtype, 8), _rows(rows, H, dtype, 58)
        dy[:, -1] = 1.0
        w = torch.ones(H, device=DEV)
        w[-1] = float("inf")
        xs, ds = f64_of(x), f64_of(dy)
        _, m, r = A.layer_norm(xs, None, None, EPS)
        d = _norm_dims(rows, H, dtype)
        ws = torch.full((M.moonep_layer_norm_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
        dx, dw, db = torch.empty_like(x[None]), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
        M.moonep_layer_norm_backward(d, dy[None], x[None], w, f32(m), f32(r), dx, dw, db, ws)
        torch.cuda.synchronize()
        assert not np.isfinite(f64_of(dx)).any()
        _far(f64_of(db), ds.sum(0), (rows + 16) * U * np.abs(ds).sum(0) + 2 * U * np.abs(ds.sum(0)), "dbias")
        assert torch.isfinite(dw).all()


def test_norm_gradient_against_differences():
    """dx, dweight and dbias predict how the library's own forward changes, in float32.

    The loss sum(y dy) along a direction v, at +-h: central differences of the forward's outputs.  The
    forward is off by at most 30 u of max|y| an element, so the difference quotient by
    30 u |dy|_1 max|y| / h; the third-order term is below 20 h^2 |dy|_1 for rows of unit spread."""
    rows, H, h = 4, 256, 2.0 ** -7
    rng = np.random.default_rng(6)
    x, dy = _rows(rows, H, F32, 6), f32(rng.standard_normal((rows, H)))
    w, b = _params(H, 6)
    d = _norm_dims(rows, H, F32)
    y = torch.empty(1, rows, H, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)

    def loss(x, w, b):
        M.moonep_layer_norm(d, x[None], w, b, EPS, y, mean, rstd)
        return float((y[0].double() * dy.double()).sum())

    loss(x, w, b)
    big = float(y.abs().max())
    dx, dw, db = torch.empty_like(y), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(M.moonep_layer_norm_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    M.moonep_layer_norm_backward(d, dy[None], x[None], w, mean, rstd, dx, dw, db, ws)
    mass = float(dy.abs().sum())
    for name, at, grad in (("x", x, dx[0]), ("w", w, dw), ("b", b, db)):
        v = f32(rng.choice([-1.0, 1.0], tuple(at.shape)))
        args = dict(x=x, w=w, b=b)
        up = loss(**{**args, name: at + h * v})
        down = loss(**{**args, name: at - h * v})
        want = (up - down) / (2 * h)
        got = float((grad.double() * v.double()).sum())
        tol = mass * (30 * U * big / h + 20 * h * h * 0.05)
        say("  along", name, got, want, "tolerance", tol)
        assert abs(got - want) <= tol


# ----------------------------------------------------------------------------
# gradient norm and clipping
# ----------------------------------------------------------------------------

def _grads(lengths, dtypes, seed, scale=1e-2):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy((scale * rng.standard_normal(n)).astype(np.float32)).to(t).to(DEV)
            for n, t in zip(lengths, dtypes)]


def _norm_of(gl):
    ws = torch.full((M.moonep_grad_norm_workspace_bytes(gl),), 255, dtype=torch.uint8, device=DEV)
    norm = torch.full((1,), -7.0, device=DEV)
    M.moonep_grad_norm(gl, ws, norm)
    return norm


LISTS = {
    "one": [1], "few": [3, 8, 5], "empty among": [0, 17, 0, 1000], "odd": [4095, 4097, 16383, 16384, 16385, 7],
    "long": [1_500_001], "many": list(range(1, 401)), "tables": [64] * 161 + [100_003] * 2 + [0] * 170 + [33],
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed"])
def test_clip(name, types):
    lengths = LISTS[name]
    say("clip", name, types)
    t = [{"f32": F32, "bf16": BF, "mixed": (F32, BF)[i % 2]}[types] for i in range(len(lengths))]
    grads = _grads(lengths, t, 7)
    before = [f64_of(g) for g in grads]
    exact = A.grad_norm(before)
    gl = M.GradList(grads)
    norm = _norm_of(gl)
    assert abs(float(norm) - exact) <= exact * U * 1.01
    M.moonep_grad_clip(gl, norm, exact * 2)                  # small enough: as they were
    for g, v in zip(grads, before):
        np.testing.assert_array_equal(f64_of(g), v)
    M.moonep_grad_clip(gl, norm, np.float32(exact * 0.3))
    c = float(np.float32(exact * 0.3)) / exact
    for g, v in zip(grads, before):
        # norm, quotient and product: a rounding each; then the type's own
        tol = np.abs(v * c) * (3.01 * U + (2.0 ** -8 if g.dtype == BF else 0.0))
        assert (np.abs(f64_of(g) - v * c) <= tol).all()


def test_clip_shapes_and_neighbours():
    """Gradients of any shape, cut out of one buffer: what lies between them stays."""
    buf = torch.full((4096,), 3.0, device=DEV)
    a, b = buf[4:4 + 35].view(5, 7), buf[1024:1024 + 1500].view(3, 500)
    gl = M.GradList([b, a])
    norm = _norm_of(gl)
    want = 3.0 * np.sqrt(35 + 1500)
    assert abs(float(norm) - want) <= want * U * 1.01
    M.moonep_grad_clip(gl, norm, 0.0)
    host = buf.cpu().numpy()
    assert not host[4:39].any() and not host[1024:2524].any()
    assert (host[:4] == 3).all() and (host[39:1024] == 3).all() and (host[2524:] == 3).all()


def test_norm_range():
    """Squares that float32 cannot hold."""
    for v in (1e30, 1e-30):
        g = torch.full((1000,), v, device=DEV)
        want = float(g[0]) * np.sqrt(1000)
        assert abs(float(_norm_of(M.GradList([g]))) - want) <= want * U * 1.01
    g = torch.full((9,), 1e-42, device=DEV)                  # below the smallest normal: steps of 2^-149
    assert abs(float(_norm_of(M.GradList([g]))) - 3 * float(g[0])) <= 2.0 ** -149


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size,most", [(1e38, 1.0), (1e38, 1e-5), (1e30, 1e-12), (1e20, 1e-18), (1e38, 1e-38)])
def test_clip_by_a_factor_that_float32_holds_badly(size, most, dtype):
    """max_norm / norm below the smallest normal float32: its steps of 2^-149 are large beside it.  The
    clipped values are off by a rounding each of norm, quotient and product, and by half a step of 2^-149
    (bf16: 2^-133) where they are below the smallest normal themselves."""
    g = f32([size, -size / 2, size / 3, 0.0, size / 1000]).to(dtype)
    v = f64_of(g)
    gl = M.GradList([g])
    norm = _norm_of(gl)
    M.moonep_grad_clip(gl, norm, most)
    want = v * (float(np.float32(most)) / A.grad_norm([v]))
    tol = np.abs(want) * (3.01 * U + (2.0 ** -8 if dtype == BF else 0.0)) + 2.0 ** (-134 if dtype == BF else -150) * 1.01
    _far(f64_of(g), want, tol, "clipped")


def test_clip_not_finite():
    g = f32([1.0, -2.0, np.inf, 0.0])
    gl = M.GradList([g])
    norm = _norm_of(gl)
    assert np.isinf(float(norm))
    M.moonep_grad_clip(gl, norm, 1.0)
    np.testing.assert_array_equal(g.cpu().numpy(), [0.0, -0.0, np.nan, 0.0])
    h = f32([1.0, np.nan])
    gl = M.GradList([h])
    norm = _norm_of(gl)
    assert np.isnan(float(norm))
    M.moonep_grad_clip(gl, norm, 1.0)
    assert torch.isnan(h).all()
    z = torch.zeros(5, device=DEV)
    gl = M.GradList([z])
    norm = _norm_of(gl)
    M.moonep_grad_clip(gl, norm, 0.0)                        # 0 <= 0: as they were
    assert float(norm) == 0.0 and not z.any()
    M.moonep_grad_clip(gl, norm, float("inf"))


def test_grad_list_empty_and_refusals():
    gl = M.GradList([])
    norm = _norm_of(gl)
    assert float(norm) == 0.0
    M.moonep_grad_clip(gl, norm, 1.0)
    gl = M.GradList([torch.zeros(0, device=DEV)])
    assert float(_norm_of(gl)) == 0.0
    g = torch.zeros(64, device=DEV)
    with pytest.raises(M.MoonEPError):
        M.moonep_grad_clip(M.GradList([g, g[16:32]]), norm, 1.0)
    with pytest.raises(M.MoonEPError):
        _norm_of(M.GradList([g[1:]]))
    with pytest.raises(ValueError, match="contiguous"):
        M.GradList([g.view(8, 8).t()])
    h = torch.zeros(64, device=DEV)
    gl = M.GradList([h])
    assert float(_norm_of(gl)) == 0.0
    h.data = torch.ones(64, device=DEV)                      # other memory of the same size is followed
    assert float(_norm_of(gl)) == 8.0
    h.data = torch.ones(32, device=DEV)
    with pytest.raises(ValueError, match="changed"):
        _norm_of(gl)
    h.data = torch.ones(8, 8, device=DEV).t()[:, ::2].reshape(32).expand(2, 32)[:, :32]
    with pytest.raises(ValueError, match="changed"):
        _norm_of(gl)


@pytest.mark.parametrize("change", [lambda t: t.bfloat16(), lambda t: t.cpu(), lambda t: t[:16],
                                    lambda t: t.view(torch.int32)], ids=["type", "host", "part", "type in place"])
def test_grad_list_refuses_a_changed_tensor(change):
    """Neither call launches anything: the tensors and the norm stay as they were."""
    g, h = torch.ones(64, device=DEV), torch.full((5,), 2.0, device=DEV)
    gl = M.GradList([g, h])
    ws = torch.empty(M.moonep_grad_norm_workspace_bytes(gl), dtype=torch.uint8, device=DEV)
    norm = torch.full((1,), 100.0, device=DEV)
    g.data = change(g.data)
    now = g.detach().clone()
    with pytest.raises(ValueError, match="changed"):
        M.moonep_grad_norm(gl, ws, norm)
    with pytest.raises(ValueError, match="changed"):
        M.moonep_grad_clip(gl, norm, 1.0)
    assert torch.equal(g, now) and float(norm) == 100.0 and bool((h == 2.0).all())


# ----------------------------------------------------------------------------
# 4-bit weights
# ----------------------------------------------------------------------------

def _bits(values):
    return W.bf16_bits(np.asarray(values, np.float32))


def _quantized(bits):
    """(codes, scales) tensors of the library for bf16 bits [E, Kin, N]."""
    E, Kin, N = bits.shape
    codes = torch.full((E, M.moonep_w4_code_bytes(Kin, N)), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((E, M.moonep_w4_scale_bytes(Kin, N)), 77, dtype=torch.uint8, device=DEV)
    M.moonep_quantize_w4(bf16_from_bits(bits), codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("E,Kin,N", [(1, 32, 32), (2, 96, 64), (1, 160, 320), (1, 544, 32), (1, 1152, 96)])
def test_quantize_matches_definition(E, Kin, N):
    say("quantize", E, Kin, N)
    rng = np.random.default_rng(Kin + N)
    w = rng.standard_normal((E, Kin, N)) * 10.0 ** rng.uniform(-4, 2, (E, 1, N))
    w[:, :, 1] = 0.0
    w[:, 5, 2] = 1e30
    codes, scales = _quantized(_bits(w))
    for e in range(E):
        c, s = A.pack_w4(*A.quantize_w4(W.bf16_to_f32(_bits(w))[e]))
        np.testing.assert_array_equal(scales[e].cpu().numpy(), s)
        np.testing.assert_array_equal(codes[e].cpu().numpy(), c)


def test_quantize_every_bf16():
    """Every bf16 value in a group whose largest value is 1.75, 1 or itself; ties, signs of zero,
    subnormals, infinities and NaN among them."""
    every = np.arange(65536, dtype=np.uint16)
    for top in (0x3FE0, 0x3F80, 0):
        bits = np.zeros((1, 32, 65536), np.uint16)
        bits[0, 3] = every
        bits[0, 9] = top
        bits[0, 20] = every ^ 0x8000
        codes, scales = _quantized(bits)
        got_c = codes[0].cpu().numpy().reshape(4096, 1, 4, 16, 16)[:, 0, 0]       # [tile, column, byte]
        got_s = scales[0].cpu().numpy().reshape(4096, 1, 4, 16, 4)[:, 0, 0, :, 0].reshape(-1)
        v = np.abs(W.bf16_to_f32(every).astype(np.float64))
        t = float(W.bf16_to_f32(np.array([top], np.uint16))[0])
        fine = np.isfinite(v)
        m = np.maximum(np.where(fine, v, 1.0), t)
        e = np.maximum(np.where(m > 0, np.frexp(m)[1] - 3, -126), -126)
        np.testing.assert_array_equal(got_s, np.where(fine, e + 127, 255))
        a = v[fine] / 2.0 ** e[fine]
        d = np.abs(a[:, None] - A.E2M1[None])
        near = d == d.min(1, keepdims=True)
        even = near & (np.arange(8) % 2 == 0)[None]
        want = np.where(near.sum(1) > 1, even.argmax(1), near.argmax(1))
        sign = (every[fine] >> 15).astype(np.int64)
        c = got_c.reshape(65536, 16)
        np.testing.assert_array_equal((c[:, 1] >> 4)[fine], want | sign << 3)     # value 3
        np.testing.assert_array_equal((c[:, 10] & 15)[fine], want | (1 - sign) << 3)   # value 20
        assert not c[~fine].any()


def _ffn_case(T, K, E, H, I, seed, R=1, masked=(), outside=False):
    rng = np.random.default_rng(seed)
    topk = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    gates = rng.random((T, K)).astype(np.float32)
    for t in masked:
        topk[t] = -1
        gates[t] = np.nan                                    # of a pair that names no expert
    if outside:
        topk[0, 0], topk[-1, -1] = E, -2147483648
    x = _bits(rng.standard_normal((T, H)))
    w13, w2 = _bits(0.1 * rng.standard_normal((E, H, 2 * I))), _bits(0.1 * rng.standard_normal((E, I, H)))
    return topk, gates, x, w13, w2


def _packed(w):
    return _quantized(w)


def _values(w):
    return np.stack([A.w4_values(*A.quantize_w4(m)) for m in W.bf16_to_f32(w)])


def _run_ffn(topk, gates, x, p13, p2, E, H, I, R=1, ws=None, out=None):
    T, K = topk.shape
    d = M.Dims.make(R, E, 0, T // R, K, H, I)
    if ws is None:
        ws = torch.full((M.moonep_w4_ffn_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
    if out is None:
        out = torch.full((R, T // R, H), -7.0, dtype=BF, device=DEV)
    M.moonep_w4_ffn(d, i32(topk.reshape(R, T // R, K)), f32(gates.reshape(R, T // R, K)),
                    bf16_from_bits(x.reshape(R, T // R, H)), *p13, *p2, ws, out)
    return out.reshape(T, H)


def _check_ffn(T, K, E, H, I, seed=0, R=1, **kw):
    say("ffn", T, K, E, H, I, seed, R, kw)
    topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, seed, **kw)
    out = _run_ffn(topk, gates, x, _packed(w13), _packed(w2), E, H, I, R)
    torch.cuda.synchronize()
    ref, off = A.w4_ffn(W.bf16_to_f32(x), topk, gates, _values(w13), _values(w2))
    _far(f64_of(out), ref, off + 2.0 ** -8 * np.abs(ref) * (1 + 1e-2), "out")
    for t in kw.get("masked", ()):
        assert not out[t].any()


# one token and many; experts with no, few, 8, 16, 17 and more than 64 rows; sizes that end in the
# first, second and third group of a block of 128, and in a block that is not a multiple of four
@pytest.mark.parametrize("T,K,E,H,I", [
    (1, 1, 1, 32, 32), (1, 2, 4, 64, 96), (2, 2, 4, 128, 64), (3, 1, 2, 160, 32), (8, 1, 1, 96, 64),
    (9, 1, 1, 96, 64), (16, 1, 1, 128, 128), (17, 1, 1, 160, 96), (33, 2, 2, 192, 64), (65, 1, 1, 64, 32),
    (130, 2, 3, 96, 96), (5, 2, 16, 320, 192), (24, 4, 8, 288, 224), (7, 8, 8, 544, 160), (40, 3, 5, 640, 32),
    (1, 8, 32, 1056, 544), (200, 16, 16, 32, 32), (32, 2, 64, 32, 512), (33, 1, 64, 64, 512), (64, 1, 2, 160, 96),
])
def test_ffn(T, K, E, H, I):
    _check_ffn(T, K, E, H, I, seed=T + H)


# both sides of what decides between the ways of a call: 64 and 65 pairs, H of 1024 and 4096 and more,
# pairs times I of 49152 and more
@pytest.mark.parametrize("T,K,E,H,I", [
    (8, 8, 32, 1024, 96), (8, 8, 32, 1056, 96), (13, 5, 32, 1056, 96), (16, 4, 4, 4096, 64), (16, 4, 4, 4128, 64),
    (16, 3, 16, 96, 1024), (17, 3, 16, 96, 1024), (3, 1, 2, 8224, 32),
])
def test_ffn_ways(T, K, E, H, I):
    _check_ffn(T, K, E, H, I, seed=T + H)


@pytest.mark.parametrize("E", [511, 512])
@pytest.mark.parametrize("used", [2, 5, 9])
def test_ffn_chunks(E, used):
    """Up to 200 rows an expert, of 511 experts of 32 (in chunks of 32 rows) and of 512 (of 64)."""
    topk, gates, x, w13, w2 = _ffn_case(200, 2, E, 96, 32, seed=used)
    topk = topk % used * 37
    out = _run_ffn(topk, gates, x, _packed(w13), _packed(w2), E, 96, 32)
    torch.cuda.synchronize()
    ref, off = A.w4_ffn(W.bf16_to_f32(x), topk, gates, _values(w13), _values(w2))
    _far(f64_of(out), ref, off + 2.0 ** -8 * np.abs(ref) * (1 + 1e-2), "out")


@pytest.mark.parametrize("R", [2, 4])
def test_ffn_ranks(R):
    _check_ffn(8, 2, 6, 128, 64, seed=1, R=R)


@pytest.mark.parametrize("T,masked", [(1, (0,)), (6, (0, 5)), (20, tuple(range(1, 20)))])
def test_ffn_ended_sequences(T, masked):
    _check_ffn(T, 3, 7, 160, 64, seed=2, masked=masked)


def test_ffn_ids_outside():
    _check_ffn(12, 2, 4, 96, 64, seed=3, outside=True)


def test_ffn_same_expert_twice():
    topk, gates, x, w13, w2 = _ffn_case(4, 2, 3, 64, 64, 4)
    topk[:, 1] = topk[:, 0]
    out = _run_ffn(topk, gates, x, _packed(w13), _packed(w2), 3, 64, 64)
    ref, off = A.w4_ffn(W.bf16_to_f32(x), topk, gates, _values(w13), _values(w2))
    _far(f64_of(out), ref, off + 2.0 ** -8 * np.abs(ref) * (1 + 1e-2), "out")


def test_ffn_most_pairs():
    """The largest number of pairs, on a small expert each."""
    _check_ffn(1024, 8, 64, 32, 32, seed=5)
    d = M.Dims.make(1, 64, 0, 1025, 8, 32, 32)
    with pytest.raises(M.MoonEPError):
        M.moonep_w4_ffn_workspace_bytes(d)


@pytest.mark.parametrize("T", [21, 70])
def test_ffn_rows_do_not_mix(T):
    """A NaN, an infinity or a poisoned weight group reaches its own tokens only; and a token's result
    does not depend on the others of its batch (21: few pairs, 70: many)."""
    K, E, H, I = 2, 5, 160, 96
    topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, 6)
    p13, p2 = _packed(w13), _packed(w2)
    clean = _run_ffn(topk, gates, x, p13, p2, E, H, I)
    bad = x.copy()
    bad[4, 3] = 0x7FC0
    bad[9, 150] = 0x7F80
    out = _run_ffn(topk, gates, bad, p13, p2, E, H, I)
    assert torch.isnan(out[4]).all() and not torch.isfinite(out[9]).any()
    for t in range(T):
        if t not in (4, 9):
            assert torch.equal(out[t], clean[t])
    turn = np.random.default_rng(1).permutation(T)           # other neighbours, the same products in the same order
    turned = _run_ffn(topk[turn], gates[turn], x[turn], p13, p2, E, H, I)
    assert torch.equal(turned, clean[torch.from_numpy(turn).to(DEV)])
    w2 = w2.copy()
    w2[2, 40, 7] = 0x7F80
    out = _run_ffn(topk, gates, x, p13, _packed(w2), E, H, I)
    hit = (topk == 2).any(1)
    assert torch.isnan(out[torch.from_numpy(hit).to(DEV), 7]).all()
    out[:, 7] = clean[:, 7]
    assert torch.equal(out, clean)


def test_ffn_batch_does_not_matter_within_a_way():
    """A token has the same bits in every call of few pairs, and in every one of more."""
    K, E, H, I = 2, 5, 1056, 96
    topk, gates, x, w13, w2 = _ffn_case(90, K, E, H, I, 8)
    p13, p2 = _packed(w13), _packed(w2)
    for whole, parts in ((90, (33, 40, 61)), (32, (1, 5, 17, 31))):
        want = _run_ffn(topk[:whole], gates[:whole], x[:whole], p13, p2, E, H, I)
        for T in parts:
            assert torch.equal(_run_ffn(topk[:T], gates[:T], x[:T], p13, p2, E, H, I), want[:T])


# ----------------------------------------------------------------------------
# wide experts, from their codes
# ----------------------------------------------------------------------------

def _random_packed(E, Kin, N, gen):
    """Random codes [E, Kin, N], scale bytes [E, Kin/32, N] and the two in the header's layout."""
    codes = torch.randint(0, 16, (E, Kin, N), dtype=torch.uint8, device=DEV, generator=gen)
    scales = torch.randint(118, 122, (E, Kin // 32, N), dtype=torch.uint8, device=DEV, generator=gen)
    kb, sb, nb = -(-Kin // 128), -(-Kin // 512), N // 16
    c = torch.nn.functional.pad(codes, (0, 0, 0, kb * 128 - Kin)).view(E, kb, 4, 16, 2, nb, 16)
    c = (c[:, :, :, :, 0] | c[:, :, :, :, 1] << 4).permute(0, 4, 1, 2, 5, 3)
    s = torch.nn.functional.pad(scales, (0, 0, 0, sb * 16 - Kin // 32), value=127).view(E, sb, 4, 4, nb, 16)
    s = s.permute(0, 4, 1, 3, 5, 2)
    return codes, scales, (c.reshape(E, -1).contiguous(), s.reshape(E, -1).contiguous())


def _values64(codes, scales):
    """One matrix in float64 on the GPU."""
    table = torch.tensor(np.concatenate([A.E2M1, -A.E2M1]), device=DEV)
    v = table[codes.int()].view(scales.shape[0], 32, -1) * torch.exp2(scales.double() - 127).unsqueeze(1)
    return v.view(codes.shape)


def test_random_packed_is_the_headers_layout():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(40)
    for Kin, N in ((160, 32), (576, 64)):
        codes, scales, (c, s) = _random_packed(2, Kin, N, gen)
        for e in range(2):
            wc, wsc = A.pack_w4(codes[e].cpu().numpy(), scales[e].cpu().numpy())
            np.testing.assert_array_equal(c[e].cpu().numpy(), wc)
            np.testing.assert_array_equal(s[e].cpu().numpy(), wsc)
            got = A.w4_values(codes[e].cpu().numpy(), scales[e].cpu().numpy())
            np.testing.assert_array_equal(_values64(codes[e], scales[e]).cpu().numpy(), got)


# Few pairs of wide experts and both sides of what decides about them (H over 4096, at most 32 pairs, at most
# two an expert, more than 49152 pairs times I), 8 to 100 rows an expert, and experts wider than their input.
@pytest.mark.parametrize("T,K,E,H,I", [
    (4, 8, 16, 4128, 2048), (5, 8, 16, 4128, 2048), (2, 13, 13, 4128, 2048), (3, 13, 13, 4128, 2048),
    (16, 2, 4, 4128, 2048), (4, 8, 16, 4096, 2048), (1, 8, 8, 7168, 2048), (8, 8, 8, 7168, 2048),
    (100, 4, 4, 7168, 2048), (1, 2, 2, 4096, 14336), (2, 2, 2, 4096, 14336), (4, 2, 4, 2880, 2880),
    (1, 1, 2, 512, 32768),
])
def test_ffn_wide(T, K, E, H, I):
    """Against float64.  A matrix instruction adds 32 products to the sum, in at most 33 steps that are off
    by a step of float32 each (2 u: cut or rounded), and a sum has a 32nd of its length in instructions,
    then at most 8 waves' parts: chains of n / 32 + 48.  The activation: |silu'| < 1.1, eight roundings,
    and two bf16 terms of 16 bits together."""
    say("ffn wide", T, K, E, H, I)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T * 1000 + H + I)
    c13, s13, p13 = _random_packed(E, H, 2 * I, gen)
    c2, s2, p2 = _random_packed(E, I, H, gen)
    rng = np.random.default_rng(T + I)
    topk = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    gates, x = rng.random((T, K)).astype(np.float32), _bits(rng.standard_normal((T, H)) * 0.25)
    got = _run_ffn(topk, gates, x, p13, p2, E, H, I).double()
    xs, gs, ids = bf16_from_bits(x).double(), f32(gates).double(), i32(topk)
    out, off, mass = (torch.zeros(T, H, dtype=torch.float64, device=DEV) for _ in range(3))
    n1, n2 = (H / 32 + 48) * 2 * U, (2 * I / 32 + 48) * 2 * U
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        w = _values64(c13[e], s13[e])
        gu, dgu = xs[t] @ w, n1 * (xs[t].abs() @ w.abs())
        g, v = gu[:, :I], gu[:, I:]
        s = g * torch.sigmoid(g)
        a = s * v
        da = 1.1 * dgu[:, :I] * (v.abs() + dgu[:, I:]) + s.abs() * dgu[:, I:] + a.abs() * (8 * U + 2.0 ** -15)
        w = _values64(c2[e], s2[e])
        y, dy = a @ w, da @ w.abs() + n2 * ((a.abs() + da) @ w.abs())
        share = gs[t, k, None]
        out.index_add_(0, t, share * y)
        off.index_add_(0, t, share * dy)
        mass.index_add_(0, t, share * (y.abs() + dy))
    tol = off + (K + 1) * U * mass + 2.0 ** -8 * out.abs() * (1 + 1e-2)
    _far(got.cpu().numpy(), out.cpu().numpy(), tol.cpu().numpy(), "out")


def test_ffn_deterministic_and_streams():
    T, K, E, H, I = 50, 4, 6, 256, 128
    topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, 7)
    p13, p2 = _packed(w13), _packed(w2)
    first = _run_ffn(topk, gates, x, p13, p2, E, H, I)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:                                        # two calls at once, scratch of their own
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(_run_ffn(topk, gates, x, p13, p2, E, H, I))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


# ----------------------------------------------------------------------------
# offsets past 32 bits
# ----------------------------------------------------------------------------

def test_norm_past_32_bits():
    """More than 2^31 elements: the last rows are what they are alone."""
    H = 8192
    rows = (1 << 31) // H + 3
    x, dy = (torch.empty(1, rows, H, dtype=BF, device=DEV).normal_() for _ in range(2))
    w, b = _params(H, 30)
    y = torch.empty_like(x)
    mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (rows, rows, H, H))
    d = _norm_dims(rows, H, BF)
    ws = torch.empty(M.moonep_layer_norm_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    M.moonep_layer_norm(d, x, w, b, EPS, y, mean, rstd)
    small = _norm_dims(5, H, BF)
    part = torch.empty(1, 5, H, dtype=BF, device=DEV)
    M.moonep_layer_norm(small, x[:, -5:].clone(), w, b, EPS, part)
    assert torch.equal(part, y[:, -5:])
    M.moonep_layer_norm_backward(d, dy, x, w, mean, rstd, y, dw, db, ws)
    M.moonep_layer_norm_backward(small, dy[:, -5:].clone(), x[:, -5:].clone(), w, mean[-5:].clone(), rstd[-5:].clone(),
                                 part, None, None)
    assert torch.equal(part, y[:, -5:])
    ref = torch.zeros(H, dtype=torch.float64, device=DEV)
    mass = torch.zeros(H, dtype=torch.float64, device=DEV)
    for at in range(0, rows, 1 << 15):
        block = dy[0, at:at + (1 << 15)].double()
        ref += block.sum(0)
        mass += block.abs().sum(0)
    # at most `rows` additions follow one another (and far fewer do)
    assert bool(((db.double() - ref).abs() <= rows * U * mass).all())


def test_clip_past_32_bits():
    n = (1 << 31) + 5
    g = torch.full((n,), 2.0 ** -10, device=DEV)
    gl = M.GradList([g])
    norm = _norm_of(gl)
    want = np.sqrt(float(n)) * 2.0 ** -10
    assert abs(float(norm) - want) <= want * U * 1.01
    M.moonep_grad_clip(gl, norm, float(norm) / 4)            # an exact quarter
    for part in (g[:7], g[n // 2:n // 2 + 7], g[-7:]):
        assert torch.equal(part, torch.full((7,), 2.0 ** -12, device=DEV))


@pytest.mark.parametrize("T", [1, 40])
def test_ffn_past_32_bits(T):
    """Codes of more than 2^32 bytes: the last experts give what they give alone."""
    E, K, H, I = 320, 2, 7168, 2048
    gen = torch.Generator(device=DEV)
    gen.manual_seed(31)
    packed = []
    for kin, n in ((H, 2 * I), (I, H)):
        packed.append(torch.randint(0, 256, (E, M.moonep_w4_code_bytes(kin, n)), dtype=torch.uint8, device=DEV, generator=gen))
        packed.append(torch.full((E, M.moonep_w4_scale_bytes(kin, n)), 120, dtype=torch.uint8, device=DEV))
    assert packed[0].numel() > 1 << 32
    rng = np.random.default_rng(32)
    topk = np.stack([rng.permutation([0, E - 1]) for _ in range(T)]).astype(np.int32)
    gates, x = rng.random((T, K)).astype(np.float32), _bits(rng.standard_normal((T, H)))
    out = _run_ffn(topk, gates, x, packed[:2], packed[2:], E, H, I)
    few = [p[[0, E - 1]].contiguous() for p in packed]
    alone = _run_ffn(np.minimum(topk, 1), gates, x, few[:2], few[2:], 2, H, I)
    assert torch.isfinite(out).all() and torch.equal(out, alone)


# ----------------------------------------------------------------------------
# a step of them together
# ----------------------------------------------------------------------------

CFG = W.Config("around", R=4, E=16, B=4, S=96, K=2, H=256, I=128, dtype="bf16", lam=1.0, seed=3)


def _layer(cfg, training, accum=False):
    topk, gates, _ = W.routing_for(cfg)
    w13f, w2f = W.expert_weights_np(cfg.E, cfg.H, cfg.I, cfg.seed)
    d = M.Dims.make(cfg.R, cfg.E, cfg.B, cfg.S, cfg.K, cfg.H, cfg.I, training=training, grad_accum=accum)
    w, b = _params(cfg.H, 8)
    layer = MoonEPLayer(d, w13=bf16_from_bits(_bits(w13f)), w2=bf16_from_bits(_bits(w2f)), training=training,
                        norm_weight=w, norm_bias=b)
    return layer, topk, gates, _bits(w13f), _bits(w2f)


def test_training_step():
    """norm -> layer -> backward -> the norm's backward -> clipping, against the oracles.  2e-2 is the
    bound of the layer's own tests (bf16 products and rows)."""
    cfg = CFG
    layer, topk, gates, wb13, wb2 = _layer(cfg, True)
    x = _rows(cfg.R * cfg.S, cfg.H, BF, 9).reshape(cfg.R, cfg.S, cfg.H)
    doutb = W.grad_rows(cfg.R, cfg.S, cfg.H, cfg.seed, "bf16")
    g = f32(gates)
    out = layer.forward(x, i32(topk), g)
    dx = layer.backward(bf16_from_bits(doutb), g)
    torch.cuda.synchronize()
    xs = f64_of(x).reshape(-1, cfg.H)
    ny, m, r = A.layer_norm(xs, f64_of(layer.norm_weight), f64_of(layer.norm_bias), layer.norm_eps)
    nb = _bits(ny).reshape(cfg.R, cfg.S, cfg.H)
    ref = O.moe_direct(nb, topk, gates, wb13, wb2)
    assert rel_fro(f64_of(out), ref) <= 2e-2
    rdn, rw13, rw2 = O.moe_direct_backward(nb, topk, gates, wb13, wb2, doutb)[:3]
    rdx, rdw, rdb = A.layer_norm_backward(rdn.reshape(-1, cfg.H), xs, f64_of(layer.norm_weight), m, r)
    assert rel_fro(f64_of(dx).reshape(-1, cfg.H), rdx) <= 2e-2
    assert rel_fro(f64_of(layer.dnorm_weight), rdw) <= 2e-2 and rel_fro(f64_of(layer.dnorm_bias), rdb) <= 2e-2
    assert rel_fro(f64_of(layer.dw13), rw13) <= 2e-2 and rel_fro(f64_of(layer.dw2), rw2) <= 2e-2

    before = [f64_of(v) for v in layer.grads()]
    assert len(before) == 4
    exact = A.grad_norm(before)
    norm = GradClipper([layer]).clip(0.5 * exact)
    assert abs(float(norm) - exact) <= exact * U * 1.01
    for v, old in zip(layer.grads(), before):
        assert (np.abs(f64_of(v) - 0.5 * old) <= np.abs(old) * 0.5 * 4.01 * U).all()


def test_training_step_router_reads_the_norm_and_accumulates():
    layer, topk, gates, _, _ = _layer(CFG, True, accum=True)
    plain, _, _, _, _ = _layer(CFG, True)
    x = _rows(CFG.R * CFG.S, CFG.H, BF, 10).reshape(CFG.R, CFG.S, CFG.H)
    dout = bf16_from_bits(W.grad_rows(CFG.R, CFG.S, CFG.H, 1, "bf16"))
    tk, g = i32(topk), f32(gates)
    n = layer.norm(x)                                        # what the router reads
    a = layer.forward(n, tk, g).clone()
    b = plain.forward(x, tk, g)
    assert torch.equal(a, b)
    layer.backward(dout, g)
    plain.backward(dout, g)
    for u, v in zip(layer.grads(), plain.grads()):
        assert torch.equal(u, v)
    layer.forward(x, tk, g)
    layer.backward(dout, g)
    for u, v in zip(layer.grads()[2:], plain.grads()[2:]):
        assert torch.equal(u, v + v)


def test_decoding_follows_the_layer():
    """The decoder's tokens are those of the 4-bit definition on the normed rows, and near the bf16
    layer's: 4-bit weights are off by at most a quarter of their value or of their group's smallest
    step, about 11% in the mean square for normal weights; three matrices deep."""
    cfg = CFG
    layer, topk, gates, wb13, wb2 = _layer(cfg, False)
    x = _rows(cfg.R * cfg.S, cfg.H, BF, 11)
    full = layer.forward(x.reshape(cfg.R, cfg.S, cfg.H), i32(topk), f32(gates)).reshape(-1, cfg.H)
    T = 24
    dec = layer.decoder(max_tokens=32)
    out = dec.forward(x[:T], i32(topk.reshape(-1, cfg.K)[:T]), f32(gates.reshape(-1, cfg.K)[:T])).clone()
    normed = dec.norm(x[:T])
    assert torch.equal(normed, layer.normed.reshape(-1, cfg.H)[:T])
    again = dec.forward(normed, i32(topk.reshape(-1, cfg.K)[:T]), f32(gates.reshape(-1, cfg.K)[:T]))
    assert torch.equal(again, out)
    ref, off = A.w4_ffn(f64_of(normed), topk.reshape(-1, cfg.K)[:T], gates.reshape(-1, cfg.K)[:T], _values(wb13),
                        _values(wb2))
    _far(f64_of(out), ref, off + 2.0 ** -8 * np.abs(ref) * (1 + 1e-2), "out")
    assert rel_fro(f64_of(out), f64_of(full)[:T]) <= 0.3
    with pytest.raises(ValueError, match="tokens"):
        dec.forward(x[:33], i32(topk.reshape(-1, cfg.K)[:33]), f32(gates.reshape(-1, cfg.K)[:33]))


def test_decoding_normed_rows_in_parts():
    """The normed rows in two calls, as a copy, and over themselves.  All calls are of few pairs, whose
    sums do not depend on the batch: the same bits."""
    layer, topk, gates, _, _ = _layer(CFG, False)
    T, K = 24, CFG.K
    x, tk, g = _rows(T, CFG.H, BF, 13), i32(topk.reshape(-1, K)[:T]), f32(gates.reshape(-1, K)[:T])
    dec = layer.decoder(max_tokens=32)
    want = dec.forward(x, tk, g).clone()
    n = dec.norm(x)
    parts = [dec.forward(n[lo:hi], tk[lo:hi], g[lo:hi]).clone() for lo, hi in ((0, 9), (9, T))]
    assert torch.equal(torch.cat(parts), want)
    assert torch.equal(dec.forward(n.clone(), tk, g, normed=True), want)
    with pytest.raises(ValueError, match="norm"):
        dec.norm(n[9:])


def test_layer_copy_of_normed_rows():
    """A copy of the normed rows gives the output and the gradients of the rows themselves."""
    layer, topk, gates, _, _ = _layer(CFG, True)
    plain, _, _, _, _ = _layer(CFG, True)
    x = _rows(CFG.R * CFG.S, CFG.H, BF, 14).reshape(CFG.R, CFG.S, CFG.H)
    dout = bf16_from_bits(W.grad_rows(CFG.R, CFG.S, CFG.H, 2, "bf16"))
    tk, g = i32(topk), f32(gates)
    with pytest.raises(ValueError, match="norm"):
        layer.forward(x, tk, g, normed=True)
    copy = layer.norm(x).clone()
    assert torch.equal(layer.forward(copy, tk, g, normed=True), plain.forward(x, tk, g))
    assert torch.equal(layer.backward(dout, g), plain.backward(dout, g))
    for u, v in zip(layer.grads(), plain.grads()):
        assert torch.equal(u, v)


def test_captured_steps():
    """A decode step and a clipped gradient in one graph, replayed with new inputs and with eager work
    between the replays; two graphs share the scratch and run one after another."""
    layer, topk, gates, _, _ = _layer(CFG, False)
    T, K, H = 8, CFG.K, CFG.H
    dec = layer.decoder(max_tokens=T)
    xs = [_rows(T, H, BF, 20 + i) for i in range(4)]
    tks = [i32(topk.reshape(-1, K)[8 * i:8 * i + T]) for i in range(4)]
    gs = [f32(gates.reshape(-1, K)[8 * i:8 * i + T]) for i in range(4)]
    grad = _grads([5000, 31], [F32, BF], 21)
    gl = M.GradList(grad)
    gws = torch.empty(M.moonep_grad_norm_workspace_bytes(gl), dtype=torch.uint8, device=DEV)
    norm = torch.zeros(1, device=DEV)
    nd = _norm_dims(T, H, BF)
    nws = torch.empty(M.moonep_layer_norm_workspace_bytes(nd), dtype=torch.uint8, device=DEV)
    mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (T, T, H, H))
    y, dx = (torch.empty(1, T, H, dtype=BF, device=DEV) for _ in range(2))

    def step(x, tk, g):
        out = dec.forward(x, tk, g)
        M.moonep_layer_norm(nd, x[None], layer.norm_weight, layer.norm_bias, EPS, y, mean, rstd)
        M.moonep_layer_norm_backward(nd, out[None], x[None], layer.norm_weight, mean, rstd, dx, dw, db, nws)
        M.moonep_grad_norm(gl, gws, norm)
        M.moonep_grad_clip(gl, norm, 0.05)
        return [out, y, dx, dw, db, norm, *grad]

    x, tk, g = xs[0].clone(), tks[0].clone(), gs[0].clone()
    fresh = [v.clone() for v in grad]

    def reset(i):
        x.copy_(xs[i]), tk.copy_(tks[i]), g.copy_(gs[i])
        for v, f in zip(grad, fresh):
            v.copy_(f * (i + 1))

    want = []
    for i in range(4):
        reset(i)
        want.append([v.clone() for v in step(x, tk, g)])
    graphs = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(x, tk, g)
        graphs.append((graph, got))
    for rep in range(2):
        for i in range(4):
            say("  replay", rep, i)
            reset(i)
            graph, got = graphs[(rep + i) % 2]
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want[i]):
                assert torch.equal(a, b)


def test_launches_go_to_the_stream_given():
    """Each call, given a stream that is being captured while another is current: all its launches are in
    the graph, in order, and none ran before the replay."""
    T, K, E, H, I = 6, 2, 3, 64, 64
    topk, gates, x, w13, w2 = _ffn_case(40, K, E, H, I, 9)
    rows = _rows(T, H, F32, 17)[None]
    dy = _rows(T, H, F32, 18)[None]
    w, b = _params(H, 17)
    nd = _norm_dims(T, H, F32)
    y, dx = torch.zeros_like(rows), torch.zeros_like(rows)
    mean, rstd, dw, db = (torch.zeros(n, device=DEV) for n in (T, T, H, H))
    nws = torch.zeros(M.moonep_layer_norm_workspace_bytes(nd), dtype=torch.uint8, device=DEV)
    gl = M.GradList([dx, dw, db])
    gws, norm = torch.zeros(M.moonep_grad_norm_workspace_bytes(gl), dtype=torch.uint8, device=DEV), torch.zeros(1, device=DEV)
    packed = [torch.zeros((E, f(k, n)), dtype=torch.uint8, device=DEV) for k, n in ((H, 2 * I), (I, H))
              for f in (M.moonep_w4_code_bytes, M.moonep_w4_scale_bytes)]
    weights = bf16_from_bits(w13), bf16_from_bits(w2)
    few = (M.Dims.make(1, E, 0, T, K, H, I), T)
    many = (M.Dims.make(1, E, 0, 40, K, H, I), 40)
    tk, g, xr = i32(topk), f32(gates), bf16_from_bits(x)
    ffn = [(d, tk[None, :n], g[None, :n], xr[None, :n],
            torch.zeros(M.moonep_w4_ffn_workspace_bytes(d), dtype=torch.uint8, device=DEV),
            torch.zeros(1, n, H, dtype=BF, device=DEV)) for d, n in (few, many)]
    outs = [y, mean, rstd, dx, dw, db, norm, *packed, ffn[0][5], ffn[1][5]]

    def calls(stream):
        M.moonep_layer_norm(nd, rows, w, b, EPS, y, mean, rstd, stream=stream)
        M.moonep_layer_norm_backward(nd, dy, rows, w, mean, rstd, dx, dw, db, nws, stream=stream)
        M.moonep_grad_norm(gl, gws, norm, stream=stream)
        M.moonep_grad_clip(gl, norm, 1e-3, stream=stream)
        M.moonep_quantize_w4(weights[0], *packed[:2], stream=stream)
        M.moonep_quantize_w4(weights[1], *packed[2:], stream=stream)
        for d, ids, gate, xs, ws, out in ffn:
            M.moonep_w4_ffn(d, ids, gate, xs, *packed, ws, out, stream=stream)

    calls(None)
    torch.cuda.synchronize()
    want = [v.clone() for v in outs]
    assert all(bool(v.bool().any()) for v in want)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for v in outs:
        v.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            calls(side)
    torch.cuda.synchronize()
    assert not any(bool(v.bool().any()) for v in outs)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for v, ref in zip(outs, want):
            assert torch.equal(v, ref)
            v.zero_()


def test_another_stream_waits_for_nothing():
    """Work goes to the stream given, in its order."""
    rows, H = 64, 7168
    x = _rows(rows, H, BF, 12)[None]
    w, b = _params(H, 12)
    y = torch.zeros_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    M.moonep_layer_norm(_norm_dims(rows, H, BF), x, w, b, EPS, y, stream=s)
    s.synchronize()
    z = torch.zeros_like(x)
    M.moonep_layer_norm(_norm_dims(rows, H, BF), x, w, b, EPS, z)
    assert torch.equal(y, z)
