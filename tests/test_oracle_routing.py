"""The float64 definitions of routing, the weighted combine's gradient and the 8-bit experts, pinned: gradients
against differences, codes against torch's own 8-bit type, the layout against the header's formula."""
import numpy as np
import pytest

from oracle import routing as G

MODES = ("softmax", "softmax_all", "sigmoid")


def test_route_by_hand():
    z = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, gates, _ = G.route(z, None, 2, "softmax", 3.0)
    assert ids.tolist() == [[1, 2]]
    np.testing.assert_allclose(gates, [[2.0, 1.0]])
    _, gates, _ = G.route(z, None, 2, "softmax_all")
    np.testing.assert_allclose(gates, [[0.5, 0.25]])
    ids, gates, _ = G.route(z, None, 2, "sigmoid")
    s = np.array([4 / 5, 2 / 3])
    np.testing.assert_allclose(gates, [s / s.sum()])
    # a bias moves the choice and no gate; ties go to the lower id; -inf is never picked
    ids, gates, _ = G.route(z, np.array([9.0, 0, 0, 9.0]), 2, "softmax_all")
    assert ids.tolist() == [[0, 3]]
    np.testing.assert_allclose(gates, [[1 / 8, 1 / 8]])
    z[0, [0, 1]] = -np.inf
    ids, gates, _ = G.route(z, np.array([9.0, 0, 0, -np.inf]), 3, "softmax")
    assert ids.tolist() == [[2, -1, -1]] and gates.tolist() == [[1.0, 0.0, 0.0]]


@pytest.mark.parametrize("mode", MODES)
def test_route_gradient_against_differences(mode):
    rng = np.random.default_rng(3)
    T, E, K = 4, 7, 3
    z, dg = rng.standard_normal((T, E)), rng.standard_normal((T, K))
    ids, _, _ = G.route(z, None, K, mode)
    ids[2, 1] = -1

    def loss(z):
        return sum(float(2.5 * (G._shares(z[t], ids[t], mode)[0] * dg[t]).sum()) for t in range(T))

    got, _ = G.route_backward(dg, z, ids, mode, 2.5)
    want = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[i] += 1e-5
        down[i] -= 1e-5
        want[i] = (loss(up) - loss(down)) / 2e-5
    np.testing.assert_allclose(got, want, rtol=0, atol=1e-8)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4)
    T, K, H, E = 5, 2, 6, 3
    topk = rng.integers(-1, E, (T, K))
    offsets, dest, pair = G.sort_pairs(topk, E)
    assert offsets[-1] == (topk >= 0).sum() == len(pair)
    np.testing.assert_array_equal(dest.reshape(-1)[pair], np.arange(len(pair)))
    assert all((np.diff(pair[offsets[e]:offsets[e + 1]]) > 0).all() for e in range(E))
    y, gates, dout = rng.standard_normal((T * K, H)), rng.random((T, K)), rng.standard_normal((T, H))

    def loss(y, gates):
        return sum(float(gates[t, k] * y[dest[t, k]] @ dout[t]) for t in range(T) for k in range(K) if dest[t, k] >= 0)

    dy, dg, _ = G.combine_backward(dest, y, gates, dout)
    for v, got in ((gates, dg), (y, None)):
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + 1e-3
            up = loss(y, gates)
            v[i] = keep - 1e-3
            want = (up - loss(y, gates)) / 2e-3
            v[i] = keep
            have = got[i] if got is not None else dy[i[0]][i[1]] if i[0] in dy else 0.0
            assert abs(have - want) < 1e-10


def test_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(G.e4m3(), t)
    rng = np.random.default_rng(5)
    a = np.concatenate([rng.uniform(-448, 448, 5000), 2.0 ** rng.uniform(-12, 8, 5000), G.e4m3()[:126],
                        (G.e4m3()[:126] + G.e4m3()[1:127]) / 2, [0.0, -0.0, 448.0]]).astype(np.float32)
    want = torch.from_numpy(a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(G._nearest(a), want)


def test_quantize_fp8_scales():
    w = np.zeros((160, 160))
    w[0, 0], w[3, 130], w[129, 2] = 448.0, 449.0, 1e-30
    codes, scales = G.quantize_fp8(w)
    assert scales.tolist() == [[127, 128], [int(np.floor(np.log2(1e-30))) - 8 + 127, 1]]
    assert codes[0, 0] == 126 and G.fp8_values(codes, scales)[3, 130] == 448.0    # 224.5 rounds to 224
    w[5, 5] = np.inf
    codes, scales = G.quantize_fp8(w)
    assert (codes[:128, :128] == 127).all() and scales[0, 0] == 127 and not codes[128:, :128].all()


def test_pack_fp8_is_the_headers_layout():
    rng = np.random.default_rng(0)
    Kin, N = 160, 192
    codes = rng.integers(0, 256, (Kin, N)).astype(np.uint8)
    scales = rng.integers(1, 255, (2, 2)).astype(np.uint8)
    cb, sb = G.pack_fp8(codes, scales)
    assert cb.size == N * 2 * 128 and sb.size == 2 * 4
    for k, n in [(0, 0), (15, 31), (16, 32), (127, 47), (128, 3), (159, 191)]:
        assert cb[((n // 32 * 2 + k // 128) * 8 + k % 128 // 16) * 512 + n % 32 * 16 + k % 16] == codes[k, n]
    assert sb.tolist() == [scales[0, 0], scales[1, 0], 127, 127, scales[0, 1], scales[1, 1], 127, 127]
    assert not cb.reshape(N // 32, 2, 8, 32, 16)[:, 1, 2:].any()                 # past Kin


def test_round_rows_bound():
    """Values that the bound allows to be off stay inside what it says."""
    rng = np.random.default_rng(6)
    a = rng.standard_normal((20, 200))
    off = 1e-3 * rng.random((20, 200))
    q, far = G.round_rows(a, off)
    for _ in range(50):
        moved = G.round_rows(a + off * rng.uniform(-1, 1, a.shape))
        assert (np.abs(moved - q) <= far).all()
    assert (far == 0).mean() > 0.5


def test_ffn_against_the_float_layer():
    """With weights and rows that 8 bits hold exactly, and activations rounded, the FFN is the bf16 layer's."""
    import oracle as O
    import workload as W
    rng = np.random.default_rng(1)
    T, K, E, H, I = 6, 2, 4, 64, 32
    w13, w2 = (rng.choice([-1.0, -0.5, 0.0, 0.5, 1.5], s) / 8 for s in ((E, H, 2 * I), (E, I, H)))
    topk = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    gates = rng.random((T, K)).astype(np.float32)
    x = rng.choice([-2.0, -1.0, 0.0, 0.75, 3.0], (T, H))
    want = O.moe_direct(W.bf16_bits(x.astype(np.float32))[None], topk[None], gates[None],
                        W.bf16_bits(w13.astype(np.float32)), W.bf16_bits(w2.astype(np.float32)))[0]
    got, off = G.fp8_ffn(x, topk, gates, w13, w2)
    # the rounded activation: half a step of 2^-4 each, some 2^-5 together
    assert np.linalg.norm(got - want) < 0.04 * np.linalg.norm(want) and off.shape == got.shape
    assert not G.fp8_ffn(x, np.full((T, K), -1), gates, w13, w2)[0].any()
