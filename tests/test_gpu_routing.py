"""GPU parity of routing, sorting by expert, the weighted combine's gradient and the 8-bit experts against
their float64 definitions.

Tolerances.  u = 2^-24 is half a step of float32; an output rounded to bf16 is off by at most 2^-8 of its value
more.  The bounds of gates and gradients come with the definitions, which count the roundings of a float32
evaluation.  The 8-bit experts round their activation to codes, where a value next to a border may take
either: the definition bounds that too.  Few pairs, and tiles of 64 rows, widen codes to bf16 and add in float32;
the 8-bit matrix instruction of larger tiles keeps a sum of 64 products to 2^-16 of their magnitudes (measured 2^-15.8 at
most over sums of one instruction, 2^-16 and less over longer ones): 2^-15 here.  Tiles store an expert's outputs in
float16: 11 significant bits, so half a step is at most 2^-11 of the value.
"""
import numpy as np
import pytest
import torch

import balanced_token_dispatch_moonep_amd as M
from balanced_token_dispatch_moonep_amd.layer import Fp8Experts, GradClipper, MoonEPLayer, Router
import oracle as O
from oracle import routing as G
import workload as W

from gpu_util import DEV, say, i32, f32, bf16_from_bits, f64_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
MODES = {"softmax": M.ROUTE_SOFTMAX, "softmax_all": M.ROUTE_SOFTMAX_ALL, "sigmoid": M.ROUTE_SIGMOID}


def _near(got, want, tol, what):
    d = np.abs(got - want)
    worst = float((d / np.maximum(tol, 1e-300)).max()) if d.size else 0.0
    say(f"  {what}: {worst:.3f} of its tolerance")
    assert np.isfinite(got).all() and (d <= tol).all(), what


# ----------------------------------------------------------------------------
# router
# ----------------------------------------------------------------------------

def _logits(T, E, dtype, seed, masked=()):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((2 * rng.standard_normal((T, E))).astype(np.float32)).to(dtype)
    z[rng.random((T, E)) < 0.05] = -float("inf")
    for t in masked:
        z[t] = -float("inf")
    return z.to(DEV)


def _route(z, bias, K, mode, scale=1.0, R=1):
    T, E = z.shape
    d = M.Dims.make(R, E, 0, T // R, K, 8)
    topk = torch.full((R, T // R, K), -7, dtype=torch.int32, device=DEV)
    gates = torch.full((R, T // R, K), -7.0, device=DEV)
    M.moonep_route(d, z.reshape(R, T // R, E), bias, topk, gates, MODES[mode], scale)
    return topk.reshape(T, K), gates.reshape(T, K)


# experts that fill a row's 16 lanes once, partly, and up to 64 times; sizes that loads of four do not divide
SIZES = [(1, 1, 1), (3, 2, 2), (17, 7, 3), (5, 16, 16), (16, 63, 4), (33, 64, 8), (2, 66, 5), (9, 128, 2), (7, 130, 16),
         (50, 256, 8), (11, 257, 6), (4, 512, 10), (3, 516, 1), (6, 1024, 16), (2, 1023, 9)]


@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("mode", MODES)
def test_route(mode, dtype, bias):
    for n, (T, E, K) in enumerate(SIZES):
        say("route", mode, dtype, bias, T, E, K)
        z = _logits(T, E, dtype, n, masked=(0,) if T > 2 else ())
        b = np.random.default_rng(n + 50).standard_normal(E).astype(np.float32) if bias else None
        if bias and E > 4:
            b[E // 2] = -np.inf
        ids, gates = _route(z, f32(b) if bias else None, K, mode, 1.5)
        want, ref, tol = G.route(z.double().cpu().numpy(), b, K, mode, 1.5)
        np.testing.assert_array_equal(ids.cpu().numpy(), want)
        _near(gates.double().cpu().numpy(), ref, tol, "gates")


# more rows than get a wave each: 16 lanes a row, which hold 4 to 64 elements each
@pytest.mark.parametrize("E,K", [(5, 3), (64, 8), (65, 2), (128, 16), (250, 8), (256, 8), (256, 9), (400, 5), (512, 16), (1000, 4),
                                 (1023, 16)])
def test_route_many_rows(E, K):
    T = 4100
    rows = [0, 1, 2, 3, 1000, 4095, 4096, 4097, 4099]
    for mode in MODES:
        for bias in (False, True):
            dtype = BF if bias else F32
            z = _logits(T, E, dtype, E, masked=(1,))
            b = np.random.default_rng(E).standard_normal(E).astype(np.float32) if bias else None
            ids, gates = _route(z, f32(b) if bias else None, K, mode, 0.5)
            zs, got = z[rows].double().cpu().numpy(), ids.cpu().numpy()
            want, ref, tol = G.route(zs, b, K, mode, 0.5)
            np.testing.assert_array_equal(got[rows], want)
            _near(gates[rows].double().cpu().numpy(), ref, tol, "gates")
            dg = torch.randn(T, K, generator=torch.Generator().manual_seed(E)).to(DEV)
            dz = _route_backward(dg, z, ids, mode, 0.5)
            ref, tol = G.route_backward(dg[rows].cpu().numpy(), zs, got[rows], mode, 0.5)
            if dtype == BF:
                tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            _near(dz[rows].double().cpu().numpy(), ref, tol, "dlogits")


def test_route_ties_go_to_the_lower_id():
    rng = np.random.default_rng(1)
    for E, K in ((5, 3), (64, 16), (200, 8), (1001, 16)):
        z = rng.integers(-2, 3, (40, E)).astype(np.float32)
        z[z == 0] = np.where(rng.random((z == 0).sum()) < 0.5, 0.0, -0.0)    # zeros of both signs are one value
        for bias in (None, rng.integers(0, 2, E).astype(np.float32)):
            for dtype in (F32, BF):
                want = G.route(z, bias, K, "softmax")[0]
                for copies in (1, 110):                      # 64 lanes a row, and 16
                    ids, _ = _route(torch.from_numpy(z).to(dtype).to(DEV).repeat(copies, 1), None if bias is None else f32(bias),
                                    K, "softmax")
                    np.testing.assert_array_equal(ids.cpu().numpy(), np.tile(want, (copies, 1)))


def test_route_bias_next_to_a_border():
    """Sums that float32 would round to one value are told apart."""
    z = np.array([[1.0, 1.0 + 2.0 ** -23, 1.0]], np.float32)
    ids, _ = _route(f32(z), f32([1024.0, 1024.0, 1024.0]), 3, "softmax")
    assert ids.tolist() == [[1, 0, 2]]
    # sigmoids that are one float32
    z = np.array([[18.0, 18.5, 19.0]], np.float32)
    ids, _ = _route(f32(z), f32([0.0, 0.0, 0.0]), 3, "sigmoid")
    assert ids.tolist() == [[2, 1, 0]]


@pytest.mark.parametrize("K", [1, 8, 16])
@pytest.mark.parametrize("E", [64, 256, 1000])
def test_route_order_of_all_values(E, K):
    """Values of every kind, many of them in one lane: NaN of either sign first, then infinity, down to the smallest
    numbers of either sign; 64 lanes a row, and 16."""
    bits = np.array([0x7fc00000, 0xffc00001, 0x7f800000, 0x7f7fffff, 0x3f800001, 0x3f800000, 0x00800000, 0x00000002, 0x00000001,
                     0, 0x80000000, 0x80000001, 0x80800000, 0xbf800000, 0xff7fffff, 0xff800000], np.uint32)
    rng = np.random.default_rng(E + K)
    z = np.full((30, E), -np.inf, np.float32)
    for t in range(30):
        n = rng.integers(0, 24)
        at = rng.permutation(E)[:n] if t % 2 else rng.permutation(min(E, 256))[:n] // 4 * 4       # of one lane or two
        z[t, at] = rng.choice(bits, len(at)).view(np.float32)
    key = np.where(np.isnan(z), 4e38, np.where(z == np.inf, 3.9e38, z.astype(np.float64)))
    order = np.argsort(-key, axis=1, kind="stable")[:, :K]
    want = np.where(np.take_along_axis(z, order, 1) == -np.inf, -1, order)
    for copies in (1, 140):
        for bias in (None, np.zeros(E, np.float32)):
            ids, _ = _route(f32(np.tile(z, (copies, 1))), None if bias is None else f32(bias), K, "softmax")
            np.testing.assert_array_equal(ids.cpu().numpy(), np.tile(want, (copies, 1)))


@pytest.mark.parametrize("mode", MODES)
def test_route_not_finite(mode):
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[0.0, nan, 1.0, 2.0], [-inf, 3.0, -inf, -inf], [-inf] * 4, [0.0, inf, 1.0, 2.0], [1.0, 2.0, 3.0, 4.0],
                      [-300.0, -400.0, -310.0, -500.0], [3e38, -3e38, 1.0, 2.0]], device=DEV)
    ids, gates = _route(z, None, 2, mode)
    assert ids.tolist() == [[1, 3], [1, -1], [-1, -1], [1, 3], [3, 2], [0, 2], [0, 3]]
    g = gates.cpu()
    assert torch.isnan(g[0]).all()                           # a NaN among the picked, and ranked first
    assert g[1, 1] == 0 and g[2].tolist() == [0.0, 0.0]
    if mode != "softmax_all":
        assert g[1, 0] == 1
        # sigmoids that underflow as numbers, not as shares
        np.testing.assert_allclose(g[5].double().numpy(), np.exp([0.0, -10.0]) / (1 + np.exp(-10)), rtol=64 * U)
    if mode == "sigmoid":
        np.testing.assert_allclose(g[3].double().numpy(), [1 / (1 + 1 / (1 + np.exp(-2))), 1 - 1 / (1 + 1 / (1 + np.exp(-2)))],
                                   rtol=32 * U)
    else:
        assert torch.isnan(g[3]).all() and g[6].tolist() == [1.0, 0.0]
    ids, _ = _route(z, torch.tensor([nan, 0.0, 0.0, 0.0], device=DEV), 2, mode)
    assert ids.tolist() == [[0, 1], [1, -1], [-1, -1], [0, 1], [0, 3], [0, 2], [0, 3]]


def test_route_ranks_and_rows():
    """[R, S, E] rows are one list; a row does not depend on the others."""
    z = _logits(24, 40, F32, 5)
    ids, gates = _route(z, None, 4, "softmax")
    for R in (2, 8):
        a, b = _route(z, None, 4, "softmax", R=R)
        assert torch.equal(a, ids) and torch.equal(b, gates)
    for t in (0, 13, 23):
        a, b = _route(z[t:t + 1].clone(), None, 4, "softmax")
        assert torch.equal(a[0], ids[t]) and torch.equal(b[0], gates[t])


def _route_backward(dg, z, ids, mode, scale):
    T, E = z.shape
    d = M.Dims.make(1, E, 0, T, ids.shape[1], 8)
    out = torch.full((1, T, E), -7.0, dtype=z.dtype, device=DEV)
    M.moonep_route_backward(d, dg[None], z[None], ids[None], out, MODES[mode], scale)
    return out[0]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("mode", MODES)
def test_route_backward(mode, dtype):
    for n, (T, E, K) in enumerate(SIZES):
        say("route backward", mode, dtype, T, E, K)
        rng = np.random.default_rng(n + 70)
        z = _logits(T, E, dtype, n, masked=(0,) if T > 2 else ())
        ids = _route(z, None, K, mode)[0].cpu().numpy()
        dg = rng.standard_normal((T, K)).astype(np.float32)
        dg[ids < 0] = np.nan                                 # of a pick that is none
        if T > 3 and K > 1:
            ids[1, 0], dg[1, 0] = E, np.inf
            ids[2, 1] = -2147483648
            dg[2, 1] = np.nan
        got = _route_backward(f32(dg), z, i32(ids), mode, -1.5)
        ref, tol = G.route_backward(dg, z.double().cpu().numpy(), ids, mode, -1.5)
        if dtype == BF:
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        _near(got.double().cpu().numpy(), ref, tol, "dlogits")


@pytest.mark.parametrize("mode", MODES)
def test_route_backward_same_id_twice(mode):
    z = _logits(6, 20, F32, 9)
    z[z == -float("inf")] = 0.5
    ids = np.array([[3, 3, 7], [5, 5, 5], [0, 1, 0], [19, 2, 19], [4, -1, 4], [8, 8, 20]], np.int32)
    dg = np.random.default_rng(8).standard_normal((6, 3)).astype(np.float32)
    got = _route_backward(f32(dg), z, i32(ids), mode, 1.0)
    ref, tol = G.route_backward(dg, z.double().cpu().numpy(), ids, mode)
    _near(got.double().cpu().numpy(), ref, tol, "dlogits")


@pytest.mark.parametrize("mode", MODES)
def test_route_gradient_against_differences(mode):
    """The kernel's gradient against differences of the kernel's gates.  A share's third derivative along one
    logit is below 1, so central differences of h are off by h^2 / 6, and by the gates' own 64 u / h."""
    T, E, K, h = 12, 24, 4, 2.0 ** -5
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(DEV)
    ids, _ = _route(z, None, K, mode)
    # picks stay picked under a step of h: lifted by a bias, which moves no gate
    dg = torch.randn(T, K, generator=torch.Generator().manual_seed(3)).to(DEV)
    got = _route_backward(dg, z, ids, mode, 1.0)
    for t in range(T):
        bias = torch.zeros(E, device=DEV)
        bias[ids[t].long()] = 100.0
        rows = z[t].repeat(2 * E, 1)
        i = torch.arange(E, device=DEV)
        rows[i, i] += h
        rows[E + i, i] -= h
        k2, g2 = _route(rows, bias, K, mode)
        weight = torch.zeros(E, device=DEV)
        weight[ids[t].long()] = dg[t]
        loss = (weight[k2.long()].double() * g2.double()).sum(1)
        want = (loss[:E] - loss[E:]) / (2 * h)
        tol = dg[t].abs().double().sum() * (h * h / 6 + 64 * U / h)
        assert float((got[t].double() - want).abs().max()) <= float(tol)


# ----------------------------------------------------------------------------
# rows without a plan
# ----------------------------------------------------------------------------

def _sort(topk, E, R=1, pair=True):
    T, K = topk.shape
    d = M.Dims.make(R, E, 0, T // R, K, 8)
    ws = torch.full((M.moonep_sort_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)
    dest = torch.full((R, T // R, K), -7, dtype=torch.int32, device=DEV)
    pairs = torch.full((T * K,), -7, dtype=torch.int32, device=DEV) if pair else None
    M.moonep_sort(d, i32(topk.reshape(R, T // R, K)), ws, offsets, dest, pairs)
    return offsets, dest.reshape(T, K), pairs


def _check_sort(topk, E, **kw):
    offsets, dest, pair = _sort(topk, E, **kw)
    flat = topk.reshape(-1).astype(np.int64)
    on = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(on, flat, E), kind="stable")
    n = int(on.sum())
    want = np.full(flat.size, -1, np.int32)
    want[order[:n]] = np.arange(n)
    np.testing.assert_array_equal(dest.cpu().numpy().reshape(-1), want)
    np.testing.assert_array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.bincount(flat[on], minlength=E).cumsum()]))
    if pair is not None:
        got = pair.cpu().numpy()
        np.testing.assert_array_equal(got[:n], order[:n])
        assert (got[n:] == -7).all()                         # behind the last row: left as they were


# one workgroup's rounds and waves, its limit of 2048 pairs, several parts of 1024 and (over 65536 pairs) 2048, the last of
# them short
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 256), (63, 1, 5), (64, 1, 5), (65, 1, 5), (128, 8, 256), (511, 1, 3),
                                   (513, 1, 3), (512, 8, 1024), (4096, 1, 2), (4097, 1, 500), (1024, 8, 1024), (8193, 1, 7), (4097, 2, 1), (1250, 10, 33), (20011, 15, 1024),
                                   (2048, 1, 6), (2049, 1, 6), (16384, 4, 300), (16385, 4, 300),
                                   (262144, 4, 256), (70000, 16, 1000)])
def test_sort(T, K, E):
    say("sort", T, K, E)
    rng = np.random.default_rng(T + E)
    topk = rng.integers(0, E, (T, K)).astype(np.int32)      # an id may repeat
    _check_sort(topk, E)
    topk[rng.random((T, K)) < 0.3] = -1
    topk[rng.random((T, K)) < 0.05] = E
    topk[0, 0] = -2147483648
    _check_sort(topk, E, pair=False)
    _check_sort(np.where(rng.random((T, K)) < 0.9, E - 1, topk), E)          # almost all to one


def test_sort_without_rows_and_ranks():
    for T in (1, 3000, 9000):
        offsets, dest, pair = _sort(np.full((T, 2), -1, np.int32), 6)
        assert not offsets.any() and (dest == -1).all() and (pair == -7).all()
    topk = np.random.default_rng(0).integers(-1, 9, (96, 3)).astype(np.int32)
    for R in (2, 8, 32):
        _check_sort(topk, 9, R=R)


def test_sort_past_a_million_pairs():
    """Parts of more than 2048 pairs."""
    topk = np.random.default_rng(3).integers(-1, 300, (600011, 2)).astype(np.int32)
    _check_sort(topk, 300)


def _rows(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _check_combine_backward(T, K, H, dtype, seed, weights=True, dy=True, dgates=True):
    say("combine backward", T, K, H, dtype, seed, weights, dy, dgates)
    rng = np.random.default_rng(seed)
    topk = rng.integers(-1, 6, (T, K)).astype(np.int32)
    dest = _sort(topk, 6)[1]
    d = M.Dims.make(1, 6, 0, T, K, H, f32_rows=dtype == F32)
    y, dout = _rows((T * K, H), dtype, seed), _rows((1, T, H), dtype, seed + 1)
    gates = f32(rng.standard_normal((1, T, K))) if weights else None
    got = torch.full((T * K, H), -7.0, dtype=dtype, device=DEV) if dy else None
    dg = torch.full((1, T, K), -7.0, device=DEV) if dgates else None
    M.moonep_combine_backward(d, dest[None], y if dgates else None, gates, dout, got, dg)
    if dy:                                                   # the bits of a dispatch with the gates as scale
        want = torch.full((T * K, H), -7.0, dtype=dtype, device=DEV)
        M.moonep_dispatch(d, dest[None], dout, gates, want)
        assert torch.equal(got, want)
    if dgates:
        _, ref, tol = G.combine_backward(dest.cpu().numpy(), y.double().cpu().numpy(), None,
                                         dout[0].double().cpu().numpy())
        _near(dg[0].double().cpu().numpy(), ref, tol, "dgates")


# rows of 4 and 14 vectors a lane at a time, on both sides of each, and longer ones
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("H", [8, 72, 512, 520, 1024, 1032, 2048, 3584, 3592, 4096, 4104, 7168, 7176, 16384])
def test_combine_backward(H, dtype):
    _check_combine_backward(7, 3, H, dtype, H)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,K,H", [(1, 1, 64), (5, 16, 264), (130, 8, 1088), (3, 2, 8200)])
def test_combine_backward_options(T, K, H, dtype):
    for kw in (dict(weights=False), dict(dy=False), dict(dgates=False), dict(weights=False, dgates=False)):
        _check_combine_backward(T, K, H, dtype, T + H, **kw)


def test_combine_backward_keeps_to_its_rows():
    """NaN rows that no dest names are not read into anything, infinities stay in their pair."""
    T, K, H = 4, 2, 264
    dest = torch.tensor([[[0, 1], [-1, 2], [3, -1], [-1, -1]]], dtype=torch.int32, device=DEV)
    y, dout = _rows((T * K, H), BF, 1), _rows((1, T, H), BF, 2)
    y[4:] = float("nan")
    y[2, 5] = float("inf")
    gates = torch.full((1, T, K), float("nan"), device=DEV)
    gates[0, 0] = 0.5
    d = M.Dims.make(1, 6, 0, T, K, H)
    dy, dg = torch.full((T * K, H), -7.0, dtype=BF, device=DEV), torch.full((1, T, K), -7.0, device=DEV)
    M.moonep_combine_backward(d, dest, y, gates, dout, dy, dg)
    assert (dy[4:] == -7).all() and torch.isnan(dy[2:4]).all() and torch.isfinite(dy[:2]).all()
    g = dg[0].cpu()
    assert torch.isfinite(g[0]).all() and g[1, 0] == 0 and torch.isinf(g[1, 1]) and torch.isfinite(g[2, 0])
    assert g[2, 1] == 0 and g[3].tolist() == [0.0, 0.0]


def test_combine_backward_past_32_bits():
    T, K, H = 150001, 2, 7168                                # more than 2^31 elements of y
    d = M.Dims.make(1, 2, 0, T, K, H)
    dest = torch.arange(T * K, dtype=torch.int32, device=DEV).flip(0).reshape(1, T, K).contiguous()
    y, dout = (torch.empty(s, dtype=BF, device=DEV).normal_() for s in ((T * K, H), (1, T, H)))
    gates = torch.rand(1, T, K, device=DEV)
    dy, dg = torch.empty_like(y), torch.empty(1, T, K, device=DEV)
    M.moonep_combine_backward(d, dest, y, gates, dout, dy, dg)
    small = M.Dims.make(1, 2, 0, 3, K, H)
    for lo in (0, T - 3):                                    # rows at the far end, and at the beginning
        rows = dest[0, lo:lo + 3].reshape(-1).long()
        sy, sdy, sdg = y[rows].clone(), torch.empty(6, H, dtype=BF, device=DEV), torch.empty(1, 3, K, device=DEV)
        at = torch.arange(6, dtype=torch.int32, device=DEV).reshape(1, 3, K)
        M.moonep_combine_backward(small, at, sy, gates[:, lo:lo + 3].clone(), dout[:, lo:lo + 3].clone(), sdy, sdg)
        assert torch.equal(dy[rows], sdy) and torch.equal(dg[:, lo:lo + 3], sdg)


def test_rows_there_and_back():
    """Sort, dispatch, experts that scale, combine, and the gradient of all that against its formula."""
    T, K, E, H = 300, 3, 40, 136                             # 40 experts of one rank, some pairs dropped
    rng = np.random.default_rng(11)
    topk = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    topk[rng.random((T, K)) < 0.2] = -1
    offsets, dest, pair = _sort(topk, E)
    d = M.Dims.make(1, E, 0, T, K, H, f32_rows=True)
    x, dout = _rows((1, T, H), F32, 1), _rows((1, T, H), F32, 2)
    gates = f32(rng.random((1, T, K)))
    recv = torch.full((T * K, H), -7.0, device=DEV)
    M.moonep_dispatch(d, dest[None], x, None, recv)
    n = int(offsets[-1])
    assert torch.equal(recv[:n], x[0, (pair[:n] // K).long()]) and (recv[n:] == -7).all()
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), offsets.diff().long())
    y = torch.full((T * K, H), float("nan"), device=DEV)
    y[:n] = recv[:n] * (2.0 ** (expert % 5).float())[:, None]
    out = torch.empty_like(x)
    M.moonep_combine(d, dest[None], y, gates, out)
    on = torch.from_numpy(topk >= 0).to(DEV)
    s = torch.where(on, 2.0 ** (i32(topk) % 5).float(), torch.zeros((), device=DEV)).double()
    share = (gates[0].double() * s).sum(1, keepdim=True)
    tol = 2 * K * U * (gates[0].double() * s).abs().sum(1, keepdim=True) * x[0].abs().double()
    assert bool(((out[0].double() - share * x[0].double()).abs() <= tol).all())
    dy, dg, dx = torch.zeros_like(y), torch.empty_like(gates), torch.empty_like(x)
    M.moonep_combine_backward(d, dest[None], y, gates, dout, dy, dg)
    dy[:n] *= (2.0 ** (expert % 5).float())[:, None]
    M.moonep_combine(d, dest[None], dy, None, dx)
    assert bool(((dx[0].double() - share * dout[0].double()).abs() <=
                 3 * K * U * (gates[0].double() * s).abs().sum(1, keepdim=True) * dout[0].abs().double()).all())
    want = s * (x[0].double() * dout[0].double()).sum(1, keepdim=True)
    assert bool(((dg[0].double() - want).abs() <= (H / 64 + 20) * U * s * (x[0] * dout[0]).abs().double().sum(1, keepdim=True)).all())


# ----------------------------------------------------------------------------
# 8-bit weights
# ----------------------------------------------------------------------------

def _bits(values):
    return W.bf16_bits(np.asarray(values, np.float32))


def _quantized(bits):
    E, Kin, N = bits.shape
    codes = torch.full((E, M.moonep_fp8_code_bytes(Kin, N)), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((E, M.moonep_fp8_scale_bytes(Kin, N)), 77, dtype=torch.uint8, device=DEV)
    M.moonep_quantize_fp8(bf16_from_bits(bits), codes, scales)
    torch.cuda.synchronize()
    return codes, scales


@pytest.mark.parametrize("E,Kin,N", [(1, 32, 32), (2, 96, 64), (1, 160, 320), (3, 128, 128), (1, 544, 32), (1, 1152, 96)])
def test_quantize_matches_definition(E, Kin, N):
    say("quantize", E, Kin, N)
    rng = np.random.default_rng(Kin + N)
    w = rng.standard_normal((E, Kin, N)) * 10.0 ** rng.uniform(-3, 2, (E, Kin // 32, N // 32)).repeat(32, 1).repeat(32, 2)
    w[:, :32, :32] = 0.0
    w[:, 5, 2] = 1e-38
    w[-1, Kin - 1, N - 1] = 1e30
    codes, scales = _quantized(_bits(w))
    for e in range(E):
        c, s = G.pack_fp8(*G.quantize_fp8(W.bf16_to_f32(_bits(w))[e]))
        np.testing.assert_array_equal(scales[e].cpu().numpy(), s)
        np.testing.assert_array_equal(codes[e].cpu().numpy(), c)


def test_quantize_every_bf16():
    """Every bf16 value, 128 of them a block: whole binades, ties, subnormals, infinities and NaN among them;
    and beside a larger value in its block, from its own size up."""
    every = np.arange(65536, dtype=np.uint16)
    bits = np.zeros((1, 128, 512 * 128), np.uint16)
    bits[0, 3] = every
    bits[0, 100] = every ^ 0x8000
    codes, scales = _quantized(bits)
    codes = codes[0].cpu().numpy().reshape(2048, 8, 32, 16)
    scales = scales[0].cpu().numpy().reshape(512, 4)
    v = W.bf16_to_f32(every).astype(np.float64).reshape(512, 128)
    for b in range(512):
        c, s = G.quantize_fp8(np.stack([v[b], -v[b]]))
        assert scales[b].tolist() == [s[0, 0], 127, 127, 127]
        got = codes[4 * b:4 * b + 4].transpose(1, 3, 0, 2).reshape(128, 128)
        if not np.isfinite(v[b]).all():
            assert ((got & 127) == 127).all()
            continue
        np.testing.assert_array_equal(got[3], c[0])
        np.testing.assert_array_equal(got[100], c[1])
        assert not got[[0, 2, 4, 99, 127]].any()


def _ffn_case(T, K, E, H, I, seed, masked=(), outside=False):
    rng = np.random.default_rng(seed)
    topk = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    gates = rng.random((T, K)).astype(np.float32)
    for t in masked:
        topk[t] = -1
        gates[t] = np.nan                                    # of a pair that names no expert
    if outside:
        topk[0, 0], topk[-1, -1] = E, -2147483648
    x = _bits(rng.standard_normal((T, H)) * 2.0 ** rng.integers(-3, 4, (T, 1)))
    w13, w2 = _bits(0.1 * rng.standard_normal((E, H, 2 * I))), _bits(0.1 * rng.standard_normal((E, I, H)))
    return topk, gates, x, w13, w2


def _values(w):
    return np.stack([G.fp8_values(*G.quantize_fp8(m)) for m in W.bf16_to_f32(w)])


def _run_ffn(topk, gates, x, p13, p2, E, H, I, R=1):
    T, K = topk.shape
    d = M.Dims.make(R, E, 0, T // R, K, H, I)
    ws = torch.full((M.moonep_fp8_ffn_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((R, T // R, H), -7.0, dtype=BF, device=DEV)
    M.moonep_fp8_ffn(d, i32(topk.reshape(R, T // R, K)), f32(gates.reshape(R, T // R, K)),
                     bf16_from_bits(x.reshape(R, T // R, H)), *p13, *p2, ws, out)
    return out.reshape(T, H)


def _way(T, K, E, H):
    """(which kernels take a call, what its bound counts)."""
    if T <= 8 and T * K <= 64 and H <= 8192:
        return "few", {}
    if T * K < 36 * E:
        return "tiles of 64", dict(keep=2.0 ** -11)
    return f"tiles of {128 if T * K < 192 * E else 256}", dict(unit=2.0 ** -15, keep=2.0 ** -11)


def _check_ffn(T, K, E, H, I, seed=0, R=1, **kw):
    way, more = _way(T, K, E, H)
    say("ffn", T, K, E, H, I, seed, R, kw, way)
    topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, seed, **kw)
    out = _run_ffn(topk, gates, x, _quantized(w13), _quantized(w2), E, H, I, R)
    torch.cuda.synchronize()
    ref, off = G.fp8_ffn(W.bf16_to_f32(x), topk, gates, _values(w13), _values(w2), **more)
    _near(f64_of(out), ref, off + 2.0 ** -8 * (np.abs(ref) + off), "out")
    for t in kw.get("masked", ()):
        assert not out[t].any()


# few pairs: one token to eight, fewer and more pairs than experts, one block of input values and several, on
# both sides of the longest rows; tiles of 64: experts with no, few, 31, 32, 33, 64, 65 and more rows; sizes
# that end inside a block of 128, in one block and in several, and more than 16 blocks
@pytest.mark.parametrize("T,K,E,H,I", [
    (1, 1, 1, 32, 32), (1, 2, 4, 64, 96), (2, 2, 4, 128, 64), (3, 1, 2, 160, 32), (8, 1, 1, 96, 64), (8, 8, 40, 256, 160),
    (8, 8, 16, 288, 128), (4, 16, 16, 416, 64), (5, 2, 16, 320, 192), (7, 8, 8, 544, 160), (1, 8, 32, 1056, 544),
    (3, 1, 2, 2208, 32), (2, 2, 2, 64, 2080), (2, 1, 2, 8192, 32), (2, 1, 2, 8224, 32), (1, 1, 1, 64, 4128),
    (9, 1, 1, 96, 64), (8, 9, 9, 96, 64), (31, 1, 1, 128, 128), (32, 1, 1, 160, 96), (33, 1, 1, 192, 64),
    (35, 1, 1, 64, 32), (64, 1, 2, 2208, 32), (70, 2, 4, 96, 96), (24, 4, 8, 288, 224), (200, 16, 128, 32, 32),
    (65, 1, 2, 96, 2080), (12, 2, 3, 256, 1056),
])
def test_ffn_few_rows(T, K, E, H, I):
    _check_ffn(T, K, E, H, I, seed=T + H)


# tiles of 128 rows (36 to 191 pairs an expert) and of 256, sorted with the rounding and in launches of their own: one in part and several, experts without rows;
# one, two, three and more stages of 128 input values, 16 and 17 and more than 32 of them; columns that end
# inside a tile of 256 and inside a block of 128
@pytest.mark.parametrize("T,K,E,H,I", [
    (36, 1, 1, 32, 32), (48, 1, 1, 32, 32), (64, 2, 2, 128, 64), (127, 1, 1, 160, 96), (128, 1, 1, 288, 128), (129, 1, 1, 384, 160),
    (191, 1, 1, 512, 320), (192, 1, 1, 96, 64), (255, 1, 1, 128, 128), (256, 1, 1, 160, 288), (257, 1, 1, 288, 32),
    (600, 2, 3, 320, 96), (100, 3, 5, 416, 192), (70, 2, 2, 2048, 32), (70, 2, 2, 2080, 32), (200, 1, 1, 2208, 64),
    (60, 1, 1, 4256, 32), (200, 1, 1, 64, 2112), (64, 1, 1, 96, 4128), (700, 1, 2, 544, 32), (1100, 2, 20, 64, 32), (2100, 2, 3, 64, 32),
])
def test_ffn_tiles(T, K, E, H, I):
    _check_ffn(T, K, E, H, I, seed=T + H)


@pytest.mark.parametrize("T", [8, 40, 120, 480])
def test_ffn_ranks_and_ids(T):
    for R in (2, 4):
        _check_ffn(T, 2, 4, 128, 64, seed=1, R=R)
    _check_ffn(T, 2, 4, 160, 64, seed=2, masked=(0, T // 2, T - 1))
    _check_ffn(T, 2, 4, 160, 64, seed=3, masked=tuple(range(1, T)))
    _check_ffn(T, 2, 4, 160, 64, seed=4, masked=tuple(range(T)))
    _check_ffn(T, 2, 4, 96, 32, seed=5, outside=True)


@pytest.mark.parametrize("T,K", [(8, 5), (9, 2), (100, 2), (300, 2), (800, 2)])
def test_ffn_uneven_and_repeated(T, K):
    """All pairs to one of many experts, which each token names twice or more."""
    E, H, I = 6, 96, 160
    topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, 6)
    topk[:] = 4
    topk[T // 3, 0] = 1
    p = _quantized(w13), _quantized(w2)
    out = _run_ffn(topk, gates, x, *p, E, H, I)
    _, more = _way(T, K, E, H)
    ref, off = G.fp8_ffn(W.bf16_to_f32(x), topk, gates, _values(w13), _values(w2), **more)
    _near(f64_of(out), ref, off + 2.0 ** -8 * (np.abs(ref) + off), "out")


# what is computed where, exactly: one value a row, large gates (silu(g) = g), one value a column of w2, each
# block of 128 of its own size, so that every sum has one term and every rounding is exact
@pytest.mark.parametrize("T,E,H,I", [(8, 3, 416, 224), (6, 5, 2208, 544), (20, 5, 416, 224), (40, 3, 2208, 544),
                                     (300, 3, 416, 224), (150, 2, 2208, 544), (1100, 3, 416, 544), (500, 1, 2208, 352),
                                     (260, 1, 4256, 32)])
def test_ffn_exact(T, E, H, I):
    say("exact", T, E, H, I)
    rng = np.random.default_rng(T + H)
    blocks = lambda n, lo, hi: np.repeat(2.0 ** rng.integers(lo, hi, -(-n // 128)), 128)[:n]
    at, val = rng.integers(0, H, T), rng.choice([1.0, 1.5, 2.0, 3.5], T) * 2.0 ** rng.integers(0, 3, T)
    x = np.zeros((T, H))
    x[np.arange(T), at] = val
    gate = 64 * blocks(H, 0, 3)[:, None] * np.ones((E, 1, I))
    up = rng.choice([-2.0, -1.0, 0.0, 1.0, 1.5], (E, H, I)) * blocks(H, -2, 3)[:, None] * blocks(I, -4, 4)
    w2 = np.zeros((E, I, H))
    for e in range(E):
        w2[e, rng.integers(0, I, H), np.arange(H)] = rng.choice([-1.0, 1.0, 1.25], H)
    w2 *= blocks(I, -3, 3)[:, None] * blocks(H, -3, 3)
    topk = rng.integers(-1, E, (T, 1)).astype(np.int32)
    w13 = np.concatenate([gate, up], 2)
    out = _run_ffn(topk, np.ones((T, 1), np.float32), _bits(x), _quantized(_bits(w13)), _quantized(_bits(w2)), E, H, I)
    want = np.zeros((T, H))
    for t in range(T):
        e = topk[t, 0]
        if e >= 0:
            a = G.round_rows((val[t] * gate[e, at[t]] * (val[t] * up[e, at[t]]))[None])[0]
            want[t] = a @ w2[e]
    np.testing.assert_array_equal(f64_of(out), W.bf16_to_f32(_bits(want)))


@pytest.mark.parametrize("T", [8, 12, 300, 700])
def test_ffn_rows_do_not_mix(T):
    """A token with NaN or infinities changes no other; NaN gates count only where an expert is named."""
    E, K, H, I = 3, 2, 160, 64
    topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, 8)
    p = _quantized(w13), _quantized(w2)
    want = _run_ffn(topk, gates, x, *p, E, H, I)
    bad = x.copy()
    bad[3, 5], bad[T - 1, 150] = 0x7FC0, 0x7F80
    got = _run_ffn(topk, gates, bad, *p, E, H, I)
    fine = np.setdiff1d(np.arange(T), [3, T - 1])
    assert torch.equal(got[fine], want[fine]) and torch.isnan(got[[3, T - 1]]).all()
    gates[5, 0] = np.nan
    topk[6, 1] = -1
    gates[6, 1] = np.nan
    got = _run_ffn(topk, gates, x, *p, E, H, I)
    assert torch.isnan(got[5]).all() and torch.isfinite(got[6]).all()


def test_ffn_broken_weights():
    """A block of weights with a NaN reaches the outputs of its expert only."""
    E, K, H, I = 3, 1, 256, 160
    for T in (7, 9, 200, 600):
        topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, 8)
        want = _run_ffn(topk, gates, x, _quantized(w13), _quantized(w2), E, H, I)
        w2[1, 130, 200] = 0x7F80
        got = _run_ffn(topk, gates, x, _quantized(w13), _quantized(w2), E, H, I)
        of = topk[:, 0] == 1
        assert torch.equal(got[~of], want[~of]) and torch.equal(got[of][:, :128], want[of][:, :128])
        assert torch.isnan(got[of][:, 128:]).all()


def test_ffn_batch_does_not_matter_within_a_way():
    """A token's bits: in calls of few pairs, in tiles of 64 rows, and in those of 128 and 256."""
    E, K, H, I = 4, 2, 416, 160
    topk, gates, x, w13, w2 = _ffn_case(900, K, E, H, I, 12)
    p = _quantized(w13), _quantized(w2)
    run = lambda lo, hi: _run_ffn(topk[lo:hi], gates[lo:hi], x[lo:hi], *p, E, H, I)
    few = run(0, 8)
    for lo, hi in ((0, 1), (2, 7), (7, 8)):
        assert torch.equal(run(lo, hi), few[lo:hi])
    some = run(0, 71)
    for lo, hi in ((0, 9), (7, 40), (60, 71)):
        assert torch.equal(run(lo, hi), some[lo:hi])
    many = run(0, 900)
    for lo, hi in ((0, 72), (100, 450), (300, 899)):
        assert torch.equal(run(lo, hi), many[lo:hi])


def test_ffn_deterministic_and_streams():
    E, K, H, I = 4, 3, 256, 128
    for T in (7, 30, 150, 400):
        topk, gates, x, w13, w2 = _ffn_case(T, K, E, H, I, 7)
        p = _quantized(w13), _quantized(w2)
        first = _run_ffn(topk, gates, x, *p, E, H, I)
        torch.cuda.synchronize()
        outs = []
        for s in [torch.cuda.Stream() for _ in range(2)]:    # two calls at once, scratch of their own
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                outs.append(_run_ffn(topk, gates, x, *p, E, H, I))
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, first)


@pytest.mark.parametrize("T", [1, 30, 7700])
def test_ffn_past_32_bits(T):
    """Codes of more than 2^32 bytes: the last experts give what they give alone."""
    E, K, H, I = 160, 2, 7168, 2048
    gen = torch.Generator(device=DEV)
    gen.manual_seed(31)
    packed = []
    for kin, n in ((H, 2 * I), (I, H)):
        codes = torch.randint(0, 256, (E, M.moonep_fp8_code_bytes(kin, n)), dtype=torch.uint8, device=DEV, generator=gen)
        codes &= 0xBF                                        # no NaN, nothing of 2^1 and more
        packed += [codes, torch.full((E, M.moonep_fp8_scale_bytes(kin, n)), 121, dtype=torch.uint8, device=DEV)]
    assert packed[0].numel() > 1 << 32
    rng = np.random.default_rng(32)
    topk = np.stack([rng.permutation([0, E - 1]) for _ in range(T)]).astype(np.int32)
    gates, x = rng.random((T, K)).astype(np.float32), _bits(rng.standard_normal((T, H)))
    out = _run_ffn(topk, gates, x, packed[:2], packed[2:], E, H, I)
    few = [p[[0, E - 1]].contiguous() for p in packed]
    alone = _run_ffn(np.minimum(topk, 1), gates, x, few[:2], few[2:], 2, H, I)   # the same way by T, K and E
    assert torch.isfinite(out).all() and bool(out.any())
    assert torch.equal(out, alone)


def test_ffn_rows_past_32_bits():
    """Rows of x past 2^31 bytes in 8 bits, and more than 2^31 elements of outputs."""
    T, E, H, I = 320003, 1, 7168, 32
    x = torch.empty(1, T, H, dtype=BF, device=DEV).normal_()
    rng = np.random.default_rng(4)
    p = [*_quantized(_bits(0.1 * rng.standard_normal((E, H, 2 * I)))), *_quantized(_bits(0.1 * rng.standard_normal((E, I, H))))]
    def run(rows):
        n = rows.shape[1]
        d = M.Dims.make(1, E, 0, n, 1, H, I)
        ws = torch.empty(M.moonep_fp8_ffn_workspace_bytes(d), dtype=torch.uint8, device=DEV)
        out = torch.empty(1, n, H, dtype=BF, device=DEV)
        M.moonep_fp8_ffn(d, torch.zeros(1, n, 1, dtype=torch.int32, device=DEV), torch.ones(1, n, 1, device=DEV), rows, *p,
                         ws, out)
        return out
    out = run(x)
    assert torch.equal(out[:, -60:], run(x[:, -60:].clone())) and torch.equal(out[:, :60], run(x[:, :60].clone()))


# ----------------------------------------------------------------------------
# a step of them together
# ----------------------------------------------------------------------------

CFG = W.Config("routed", R=4, E=16, B=4, S=96, K=2, H=256, I=128, dtype="bf16", lam=1.0, seed=5)


def _layer(cfg, **kw):
    w13, w2 = W.expert_weights_np(cfg.E, cfg.H, cfg.I, cfg.seed)
    d = M.Dims.make(cfg.R, cfg.E, cfg.B, cfg.S, cfg.K, cfg.H, cfg.I, training=kw.get("training", False))
    return MoonEPLayer(d, bf16_from_bits(_bits(w13)), bf16_from_bits(_bits(w2)), **kw), _bits(w13), _bits(w2)


@pytest.mark.parametrize("mode", MODES)
def test_training_step_with_a_router(mode):
    """Router, layer, and both backward passes: gates' and logits' gradients against the plan-free layer."""
    cfg = CFG
    layer, b13, b2 = _layer(cfg, training=True, gate_grad=True)
    plain, _, _ = _layer(cfg, training=True)
    router = Router(layer.d, MODES[mode], scale=1.5, training=True)
    z = f32(np.random.default_rng(1).standard_normal((cfg.R, cfg.S, cfg.E)))
    x, dout = _rows((cfg.R, cfg.S, cfg.H), BF, 1), _rows((cfg.R, cfg.S, cfg.H), BF, 2)
    topk, gates = router.forward(z)
    out = layer.forward(x, topk, gates)
    assert torch.equal(out, plain.forward(x, topk, gates))
    dx = layer.backward(dout, gates)
    assert torch.equal(dx, plain.backward(dout, gates))      # the gates' gradient changes nothing else
    assert torch.equal(layer.dw13, plain.dw13) and torch.equal(layer.dw2, plain.dw2)
    dlogits = router.backward(layer.dgates)
    # dg = <dout, y> of the y that the layer holds
    tk, g = topk.cpu().numpy().reshape(-1, cfg.K), gates.double().cpu().numpy().reshape(-1, cfg.K)
    dest = layer.dest.cpu().numpy().reshape(-1, cfg.K)
    _, dg, tol = G.combine_backward(dest, layer.y.double().cpu().numpy(), None, dout.double().cpu().numpy().reshape(-1, cfg.H))
    _near(layer.dgates.double().cpu().numpy().reshape(-1, cfg.K), dg, tol, "dgates")
    # and that y is the experts' own: 2e-2 is the layer's tolerance for products of bf16 rows
    w13, w2 = W.bf16_to_f32(b13).astype(np.float64), W.bf16_to_f32(b2).astype(np.float64)
    xd, dd = x.double().cpu().numpy().reshape(-1, cfg.H), dout.double().cpu().numpy().reshape(-1, cfg.H)
    for t in range(0, len(xd), 37):
        for k in range(cfg.K):
            gu = xd[t] @ w13[tk[t, k]]
            a, u = gu[:cfg.I], gu[cfg.I:]
            y = (a / (1 + np.exp(-a)) * u) @ w2[tk[t, k]]
            assert abs(dg[t, k] - dd[t] @ y) <= 2e-2 * np.linalg.norm(dd[t]) * np.linalg.norm(y)
    got = layer.dgates.double().cpu().numpy().reshape(-1, cfg.K)
    ref, tol = G.route_backward(got, z.double().cpu().numpy().reshape(-1, cfg.E), tk, mode, 1.5)
    _near(dlogits.double().cpu().numpy().reshape(-1, cfg.E), ref, tol, "dlogits")
    norm = GradClipper([layer]).clip(1e-3)
    assert float(norm) > 1e-3


def test_serving_in_8_bits():
    """Prompts and decoded tokens by one set of experts: what the call gives, with the norm in front, from one
    scratch, and near the bf16 layer."""
    cfg = CFG
    w, b = f32(1 + 0.1 * np.random.default_rng(1).standard_normal(cfg.H)), f32(np.zeros(cfg.H))
    layer, b13, b2 = _layer(cfg, norm_weight=w, norm_bias=b)
    T = cfg.R * cfg.S
    dec = layer.decoder(T * 8, bits=8)
    assert isinstance(dec, Fp8Experts)
    router = Router(M.Dims.make(1, cfg.E, 0, T, cfg.K, 8), M.ROUTE_SIGMOID)
    x = _rows((T, cfg.H), BF, 3)
    topk, gates = (v[0] for v in router.forward(f32(np.random.default_rng(2).standard_normal((1, T, cfg.E)))))
    want = layer.forward(x.reshape(cfg.R, cfg.S, cfg.H), topk.reshape(cfg.R, cfg.S, cfg.K),
                         gates.reshape(cfg.R, cfg.S, cfg.K)).reshape(T, cfg.H).clone()
    normed = layer.normed.reshape(T, cfg.H)
    p = _quantized(b13), _quantized(b2)
    for n in (1, 5, 96, T):
        out = dec.forward(x[:n], topk[:n], gates[:n]).clone()
        alone = _run_ffn(topk[:n].cpu().numpy(), gates[:n].cpu().numpy(), normed[:n].view(torch.int16).cpu().numpy().view(np.uint16),
                         *p, cfg.E, cfg.H, cfg.I)
        assert torch.equal(out, alone)
        # four roundings to 4 bits of mantissa, 2^-4 / sqrt(3) each at most: x, w13, act, w2
        assert float((out.double() - want[:n].double()).norm() / want[:n].double().norm()) < 4 * 2.0 ** -4 / 3 ** 0.5
    many = dec.forward(x.repeat(8, 1), topk.repeat(8, 1), gates.repeat(8, 1)).clone()
    assert torch.equal(many[:T], many[-T:])
    part = dec.forward(x[3:7], topk[3:7], gates[3:7])        # ids and gates that begin between 16-byte addresses
    assert torch.equal(part, dec.forward(x[3:7].clone(), topk[3:7].clone(), gates[3:7].clone()))
    with pytest.raises(ValueError, match="tokens"):
        dec.forward(x.repeat(9, 1), topk.repeat(9, 1), gates.repeat(9, 1))


def test_captured_steps():
    """Routing, sorting, the combine's gradient and the 8-bit experts in graphs that share their buffers, replayed
    with new inputs and with eager work between the replays."""
    T, K, E, H, I = 120, 2, 4, 160, 96
    _, _, _, w13, w2 = _ffn_case(1, K, E, H, I, 3)
    experts = Fp8Experts(bf16_from_bits(w13), bf16_from_bits(w2), K, T)
    d = M.Dims.make(1, E, 0, T, K, H)
    router = Router(d, M.ROUTE_SOFTMAX_ALL, training=True)
    ws = torch.empty(M.moonep_sort_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    offsets, dest = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(1, T, K, dtype=torch.int32, device=DEV)
    recv, dy = (torch.zeros(T * K, H, dtype=BF, device=DEV) for _ in range(2))
    dg = torch.empty(1, T, K, device=DEV)
    z, x = torch.empty(1, T, E, device=DEV), torch.empty(T, H, dtype=BF, device=DEV)

    def step():
        topk, gates = router.forward(z)
        out = experts.forward(x, topk[0], gates[0])
        few = experts.forward(x[:5], topk[0, :5], gates[0, :5]).clone()
        out = experts.forward(x, topk[0], gates[0])
        M.moonep_sort(d, topk, ws, offsets, dest)
        M.moonep_dispatch(d, dest, x[None], None, recv)
        M.moonep_combine_backward(d, dest, recv, gates, out[None], dy, dg)
        return [topk, gates, out, few, offsets, dest, recv, dy, dg, router.backward(dg)]

    def reset(i):
        z.copy_(_rows((1, T, E), F32, 40 + i)), x.copy_(_rows((T, H), BF, 50 + i))

    want = []
    for i in range(4):
        reset(i)
        want.append([v.clone() for v in step()])
    graphs, side = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
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
    T, K, E, H, I = 4200, 2, 3, 64, 64
    _, _, x, w13, w2 = _ffn_case(T, K, E, H, I, 9)
    z, xr, weights = _rows((1, T, E), F32, 1), bf16_from_bits(x), (bf16_from_bits(w13), bf16_from_bits(w2))
    d = M.Dims.make(1, E, 0, T, K, H, I)
    topk, dest = (torch.zeros(1, T, K, dtype=torch.int32, device=DEV) for _ in range(2))
    gates, dg = (torch.zeros(1, T, K, device=DEV) for _ in range(2))
    dz, offsets = torch.zeros_like(z), torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    pair = torch.zeros(T * K, dtype=torch.int32, device=DEV)
    ws = torch.zeros(M.moonep_sort_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    packed = [torch.zeros((E, f(k, n)), dtype=torch.uint8, device=DEV) for k, n in ((H, 2 * I), (I, H))
              for f in (M.moonep_fp8_code_bytes, M.moonep_fp8_scale_bytes)]
    recv, dy = (torch.zeros(T * K, H, dtype=BF, device=DEV) for _ in range(2))
    ffn = []
    for n in (6, 100, T):
        dn = M.Dims.make(1, E, 0, n, K, H, I)
        ffn.append((dn, n, torch.zeros(M.moonep_fp8_ffn_workspace_bytes(dn), dtype=torch.uint8, device=DEV),
                    torch.zeros(1, n, H, dtype=BF, device=DEV)))
    outs = [topk, dest, gates, dg, dz, offsets, pair, *packed, recv, dy, *(f[3] for f in ffn)]

    def calls(stream):
        M.moonep_route(d, z, None, topk, gates, stream=stream)
        M.moonep_sort(d, topk, ws, offsets, dest, pair, stream=stream)
        M.moonep_dispatch(d, dest, xr[None], None, recv, stream=stream)
        M.moonep_combine_backward(d, dest, recv, gates, xr[None], dy, dg, stream=stream)
        M.moonep_route_backward(d, dg, z, topk, dz, stream=stream)
        M.moonep_quantize_fp8(weights[0], *packed[:2], stream=stream)
        M.moonep_quantize_fp8(weights[1], *packed[2:], stream=stream)
        for dn, n, w, out in ffn:
            M.moonep_fp8_ffn(dn, topk[:, :n], gates[:, :n], xr[None, :n], *packed, w, out, stream=stream)

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


# ----------------------------------------------------------------------------
# masked experts, borders of codes, and workgroups that take several tiles
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("E,K,T", [(4, 4, 6), (70, 16, 30), (256, 8, 4200), (1000, 3, 4200)])
def test_route_bias_masks_whatever_the_logit(E, K, T, mode):
    """A bias of -inf takes an expert out, also one whose logit is NaN or infinite."""
    say("masked by the bias", mode, E, K, T)
    rng = np.random.default_rng(E)
    z = (2 * rng.standard_normal((T, E))).astype(np.float32)
    b = rng.standard_normal(E).astype(np.float32)
    off = rng.permutation(E)[:E // 2]
    b[off] = -np.inf
    bad = np.array([np.nan, np.inf, -np.inf, 3e38, 0.0, -np.nan], np.float32)
    z[:, off] = bad[rng.integers(0, 6, (T, len(off)))]
    ids, gates = _route(f32(z), f32(b), K, mode)
    z[:, off] = -np.inf                                      # picked as if the logits were
    some = np.unique(np.r_[:min(T, 40), max(T - 40, 0):T])
    want, ref, tol = G.route(z[some], b, K, mode)
    np.testing.assert_array_equal(ids.cpu().numpy()[some], want)
    if mode != "softmax_all":                                # whose gates are made of every logit
        _near(gates.double().cpu().numpy()[some], ref, tol, "gates")


def _next_to_borders(rng, a, k, n=1 << 21):
    """Gates and ups (g, u) of 128 columns, each a sum of three codes over 1, 16 and 256: the first has the largest
    silu(g) u, and as many as there are lie so close to the border between two codes that an exponential of -g log2(e)
    rounded to float32 takes the other one, but 10 roundings of float32 away from it.  Codes [128, 3] of both, and how many
    those are."""
    small = np.array([*range(16), *range(16, 32, 2), *range(32, 64, 4)], np.float64)
    g3 = np.stack([np.full(n, float(a)), rng.choice(small, n), rng.choice(small, n)], 1)
    u3 = np.stack([rng.choice(np.arange(8.0, 15.0), n), rng.choice(small[:24], n), rng.choice(small[:24], n)], 1) * 2.0 ** k
    g3[0], u3[0] = (a, 0, 0), (15 * 2.0 ** k, 30 * 2.0 ** k, 30 * 2.0 ** k)
    parts = np.array([1, 2.0 ** -4, 2.0 ** -8])
    g, u = -(g3 @ parts), u3 @ parts
    v = np.abs(g / (1 + np.exp(-g)) * u)
    m = v / 2.0 ** np.floor(np.log2(v))                      # borders: 1 + odd sixteenths
    border = 1 + (2 * np.clip(np.floor((m - 1) * 8), 0, 7) + 1) / 16
    r = m / border - 1
    t = (-g).astype(np.float32) * np.float32(np.log2(np.e))  # what a float32 product makes of the exponent
    shift = (t.astype(np.float64) + g * np.log2(np.e)) * np.log(2)
    clear = np.abs(r) > 10 * U
    clear &= np.abs(m - 1) > 2.0 ** -8                       # a power of two has borders of two distances
    other = clear & (np.sign(r - shift) != np.sign(r)) & (np.abs(r - shift) > 8 * U)
    other[0] = False
    at = np.flatnonzero(other)[:100]
    rest = np.flatnonzero(clear & ~other & (np.abs(r) > 2.0 ** -10))
    at = np.concatenate([[0], at, rest[rest > 0][:127 - len(at)]])
    assert 448 / 256 * 0.99 > m[0] > 1.01 and (v[at[1:]] < v[0]).all() and (v[at] > v[0] / 2.0 ** 13).all()
    return -g3[at], u3[at], int(other[at].sum())


@pytest.mark.parametrize("T", [6, 24, 60, 240])
def test_ffn_activation_next_to_borders(T):
    """silu(g) u within 8 roundings of float32 for gates far below zero, in every way of a call: values closer than
    2^-18 to the border between two codes, and farther than 10 roundings from it, get the code of their own side.  Every
    product before and behind the activation is exact."""
    say("activation", T)
    rng = np.random.default_rng(77)
    levels = [(48, 70), (52, 76), (56, 82), (60, 87), (64, 93), (72, 105)]
    H, I, nb = 128 * len(levels), 128, len(levels)
    w13, x = np.zeros((1, H, 2 * I)), np.zeros((T, H))
    want, near = np.zeros((nb, I)), 0
    for b, (a, k) in enumerate(levels):
        g3, u3, n = _next_to_borders(rng, a, k)
        rows = b * 128 + rng.permutation(128)[:3]
        w13[0, rows, :I], w13[0, rows, I:] = g3.T, u3.T
        x[b::nb, rows] = 1, 2.0 ** -4, 2.0 ** -8
        g, u = (c @ np.array([1, 2.0 ** -4, 2.0 ** -8]) for c in (g3, u3))
        want[b] = G.round_rows((g / (1 + np.exp(-g)) * u)[None])[0]
        near += n
    assert near > 50
    w2 = np.zeros((1, I, H))
    w2[0, np.arange(I), np.arange(I)] = 1
    np.testing.assert_array_equal(_values(_bits(w13)), w13)  # held exactly in 8 bits
    p = _quantized(_bits(w13)), _quantized(_bits(w2))
    out = f64_of(_run_ffn(np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32), _bits(x), *p, 1, H, I))
    assert not out[:, I:].any()
    np.testing.assert_array_equal(out[:, :I], want[np.arange(T) % nb])


@pytest.mark.parametrize("T", [6, 24, 60, 240])
def test_ffn_gates_of_any_size(T):
    """Gates up to the largest numbers of either sign: silu(g) is g or next to nothing; one that overflows is a block of NaN."""
    say("large gates", T)
    H, I = 384, 128
    sizes = np.array([88, 96, 104, 120, 144, 240]), np.array([1, 1.75, 1.5, 1.125]) * 2.0 ** 127
    w13, x, want = np.zeros((1, H, 2 * I)), np.zeros((T, H)), np.zeros((2, I))
    for b in range(2):
        g = np.resize(np.concatenate([sizes[b], -sizes[b]]), I)
        w13[0, 128 * b + 5, :I], w13[0, 128 * b + 5, I:] = g, (1, 2.0 ** -100)[b]
        x[b::3, 128 * b + 5] = 1
        want[b] = G.round_rows((np.maximum(g, 0) * (1, 2.0 ** -100)[b])[None])[0]
    w13[0, 300, 7], w13[0, 301, 7], w13[0, 300, I + 7] = 2.0 ** 127, 2.0 ** 127, 1
    x[2::3, 300:302] = 1                                     # a gate of 2^128 in float32
    w2 = np.zeros((1, I, H))
    w2[0, np.arange(I), np.arange(I)] = 1
    p = _quantized(_bits(w13)), _quantized(_bits(w2))
    out = f64_of(_run_ffn(np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32), _bits(x), *p, 1, H, I))
    for b in range(2):
        assert (out[b::3, :I] == want[b]).all() and not out[b::3, I:].any()
    assert np.isnan(out[2::3]).all()


def _exact_many(topk, E, H, I, seed):
    """The call's output and the definition's, bit for bit, for many experts: as in test_ffn_exact one value a row, one a
    column of w2 and large gates, so that every sum of a product has one term; gates that are powers of two, and a token's
    pairs added in k order in float32."""
    T, K = topk.shape
    rng = np.random.default_rng(seed)
    blocks = lambda n, lo, hi: np.repeat(2.0 ** rng.integers(lo, hi, -(-n // 128)), 128)[:n].astype(np.float32)
    pick = lambda values, *shape: np.array(values, np.float32)[rng.integers(0, len(values), shape, dtype=np.int8)]
    at, val = rng.integers(0, H, T), pick([1, 1.5, 2, 3.5], T) * 2.0 ** rng.integers(0, 3, T)
    x = np.zeros((T, H), np.float32)
    x[np.arange(T), at] = val
    w13 = np.empty((E, H, 2 * I), np.float32)
    gate = 64 * blocks(H, 0, 3)
    w13[:, :, :I] = gate[:, None]
    w13[:, :, I:] = pick([-2, -1, 0, 1, 1.5], E, H, I) * (blocks(H, -2, 3)[:, None] * blocks(I, -4, 4))
    from_i, w2_value = rng.integers(0, I, (E, H)), pick([-1, 1, 1.25], E, H) * blocks(H, -3, 3)
    w2 = np.zeros((E, I, H), np.float32)
    w2_value = w2_value * blocks(I, -3, 3)[from_i]
    np.put_along_axis(w2, from_i[:, None], w2_value[:, None], 1)
    gates = pick([0.25, 0.5, 1, 2], T, K)
    want = np.zeros((T, H), np.float32)
    for k in range(K):
        on = np.flatnonzero((topk[:, k] >= 0) & (topk[:, k] < E))
        e = topk[on, k]
        a = (val[on] * gate[at[on]])[:, None] * (val[on][:, None] * w13[e, at[on], I:])
        y = np.take_along_axis(G.round_rows(a), from_i[e], 1) * w2_value[e]
        want[on] += (gates[on, k, None] * y).astype(np.float32)
    out = _run_ffn(topk, gates, _bits(x), _quantized(_bits(w13)), _quantized(_bits(w2)), E, H, I)
    return f64_of(out), W.bf16_to_f32(_bits(want))


def _tiles(topk, E, H, I):
    """Tiles of the two products of a call, and the rows of one."""
    n = np.bincount(topk[(topk >= 0) & (topk < E)], minlength=E)
    rows = 64 if topk.size < 36 * E else 128 if topk.size < 192 * E else 256
    runs = int((-(-n // rows)).sum())
    return runs * -(-I // 128), runs * -(-H // 256), rows, n


# More tiles than workgroups in both products, of more stages than the ring holds: each workgroup goes on to further tiles,
# full ones and those that end early, in rows and in columns, after each other.
@pytest.mark.parametrize("E,H,I,rows,sizes", [
    (128, 544, 416, 64, (128, 64, 65, 100, 3, 1, 0, 2, 3, 3, 4, 2)),
    (64, 800, 544, 128, (128, 256, 1, 140, 129, 40, 0, 127)),
    (56, 800, 544, 256, (256, 512, 1, 300, 257, 30, 0, 255)),
])
def test_ffn_exact_many_tiles(E, H, I, rows, sizes):
    rng = np.random.default_rng(E)
    topk = np.concatenate([np.full(sizes[e % len(sizes)], e) for e in range(E)] + [np.full(50, -1)])
    topk = rng.permutation(topk).astype(np.int32)[:, None]
    up, down, of, n = _tiles(topk, E, H, I)
    say("exact, many tiles", len(topk), E, H, I, up, down, of)
    assert of == rows and up > 300 and down > 256 and (n == rows).any() and (n % rows > 0).any()
    assert -(-H // 128) > 3 and -(-I // 128) > 3 and H >= 512 and H % 256
    got, want = _exact_many(topk, E, H, I, E)
    np.testing.assert_array_equal(got, want)


# the join of 4096 tokens and more, seven pieces of 512 columns a wave: several pairs a token, some without an expert, rows
# of less than a piece, of several, and of more than seven
@pytest.mark.parametrize("T,K,E,H,I", [(4096, 3, 5, 64, 32), (4099, 8, 40, 1056, 32), (4097, 2, 3, 3616, 32)])
def test_ffn_exact_joins_of_many_tokens(T, K, E, H, I):
    say("exact, joins", T, K, E, H, I)
    rng = np.random.default_rng(H)
    topk = rng.integers(-1, E + 1, (T, K)).astype(np.int32)  # an id may repeat
    topk[T // 2] = -1
    got, want = _exact_many(topk, E, H, I, H)
    np.testing.assert_array_equal(got, want)
    assert not got[T // 2].any()
