"""The float64 definitions of the operators round the layer, pinned: gradients against differences,
4-bit codes against a direct search and their layout against the header's formula."""
import numpy as np
import pytest

from oracle import around as A


@pytest.mark.parametrize("rows,H", [(1, 8), (3, 24), (5, 40)])
def test_norm_gradient_against_differences(rows, H):
    rng = np.random.default_rng(rows * 100 + H)
    x, dy = rng.standard_normal((rows, H)), rng.standard_normal((rows, H))
    w, b = 1 + 0.1 * rng.standard_normal(H), rng.standard_normal(H)
    eps = 1e-5

    def loss(x, w, b):
        return float((A.layer_norm(x, w, b, eps)[0] * dy).sum())

    _, mean, rstd = A.layer_norm(x, w, b, eps)
    grads = A.layer_norm_backward(dy, x, w, mean, rstd)
    h = 1e-5
    for v, got in zip((x, w, b), grads):
        want = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + h
            up = loss(x, w, b)
            v[i] = keep - h
            want[i] = (up - loss(x, w, b)) / (2 * h)
            v[i] = keep
        # central differences: h^2 times the third derivative, and 1e-16 / h of rounding
        np.testing.assert_allclose(got, want, rtol=0, atol=1e-7 * max(1.0, np.abs(want).max()))


def test_quantize_values():
    w = np.zeros((64, 1))
    w[:16, 0] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.3, 0.2, -6.5, 4.0, 0.0, -0.0, 6.0]
    codes, scales = A.quantize_w4(w)
    assert scales[0, 0] == 127 and scales[1, 0] == 1     # the largest is 7 = 1.75 * 2^2; a zero group
    got = A.w4_values(codes, scales)[:16, 0]
    np.testing.assert_array_equal(got, [0, 1, 1, 2, 2, 4, 4, 6, 0, -0.5, 0, -6, 4, 0, 0, 6])
    assert codes[8, 0] == 8 and codes[14, 0] == 8        # signs stay
    w[3, 0] = np.inf
    codes, scales = A.quantize_w4(w)
    assert scales[0, 0] == 255 and np.isnan(A.w4_values(codes, scales)[:32]).all()


def test_pack_is_the_headers_layout():
    rng = np.random.default_rng(0)
    Kin, N = 160, 48
    codes = rng.integers(0, 16, (Kin, N)).astype(np.uint8)
    scales = rng.integers(1, 255, (Kin // 32, N)).astype(np.uint8)
    cb, sb = A.pack_w4(codes, scales)
    assert cb.size == N * 2 * 64 and sb.size == N * 1 * 16
    for k, n in [(0, 0), (31, 15), (32, 16), (127, 47), (128, 3), (159, 20)]:
        at = (((n // 16 * 2 + k // 128) * 4 + k % 128 // 32) * 16 + n % 16) * 16 + k % 32 // 2
        assert (cb[at] >> (4 * (k % 2))) & 15 == codes[k, n]
        at = (((n // 16) * 4 + k // 32 % 4) * 16 + n % 16) * 4 + k // 128
        assert sb[at] == scales[k // 32, n]
    assert not cb.reshape(N // 16, 2, 4, 16, 16)[:, 1, 1:].any()                 # past Kin
    assert (sb.reshape(N // 16, 4, 16, 4)[:, 1:, :, 1:] == 127).all()


def test_ffn_against_the_float_layer():
    """With weights that 4 bits hold exactly, the FFN is the one of the bf16 layer's oracle."""
    import oracle as O
    import workload as W
    rng = np.random.default_rng(1)
    T, K, E, H, I = 6, 2, 4, 64, 32
    w13, w2 = (rng.choice([-1.0, -0.5, 0.0, 0.5, 1.5], s) / 8 for s in ((E, H, 2 * I), (E, I, H)))
    topk = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    gates = rng.random((T, K)).astype(np.float32)
    xb = W.bf16_bits(rng.standard_normal((1, T, H)).astype(np.float32))
    want = O.moe_direct(xb, topk[None], gates[None], W.bf16_bits(w13.astype(np.float32)),
                        W.bf16_bits(w2.astype(np.float32)))[0]
    got, _ = A.w4_ffn(W.bf16_to_f32(xb)[0], topk, gates, w13, w2)
    np.testing.assert_allclose(got, want, rtol=1e-10, atol=1e-12)


def test_ffn_skips_ids_outside():
    w13, w2 = np.ones((2, 32, 64)), np.ones((2, 32, 32))
    x = np.ones((1, 32))
    out, _ = A.w4_ffn(x, np.array([[-1, 2]]), np.array([[np.nan, 1.0]]), w13, w2)
    assert not out.any()
