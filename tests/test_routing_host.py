"""Routing, sorting and the 8-bit experts without a GPU: sizes, and everything that is refused on the host before a
launch."""
import ctypes
import os
import re

import pytest

import balanced_token_dispatch_moonep_amd as M

EINVAL, EALIGN, ENOTSUP = -1, -2, -4
VP = ctypes.c_void_p
FAR = 1 << 44                        # buffers that are far from each other


def _dims(**kw):
    base = dict(R=1, E=32, B=0, S=8, K=8, H=7168, I=2048)
    base.update(kw)
    return M.Dims.make(**base)


def _caller(fn, names, lead=()):
    """call(d, lead values, name=address or None): every buffer aligned and far from the others but for those named."""
    def call(d, *values, **kw):
        args = [kw.get(n, (i + 1) * FAR) for i, n in enumerate(names)]
        return getattr(M.lib, fn)(ctypes.byref(d) if d else None, *(values or lead),
                                  *(None if a is None else VP(a) for a in args), None)
    return call


route = _caller("moonep_route", ("logits", "bias", "topk", "gates"), (0, 1.0))
route_backward = _caller("moonep_route_backward", ("dgates", "logits", "topk", "dlogits"), (0, 1.0))
sort = _caller("moonep_sort", ("topk", "ws", "offsets", "dest", "pair"))
combine_backward = _caller("moonep_combine_backward", ("dest", "y", "gates", "dout", "dy", "dgates"))
ffn = _caller("moonep_fp8_ffn", ("topk", "gates", "x", "c13", "s13", "c2", "s2", "ws", "out"))


@pytest.mark.parametrize("call,names", [(route, ("logits", "topk", "gates")),
                                        (route_backward, ("dgates", "logits", "topk", "dlogits")),
                                        (sort, ("topk", "ws", "offsets", "dest")),
                                        (combine_backward, ("dest", "y", "dout")),
                                        (ffn, ("topk", "gates", "x", "c13", "s13", "c2", "s2", "ws", "out"))])
def test_null_and_misaligned(call, names):
    assert call(None) == EINVAL
    for n in names:
        assert call(_dims(), **{n: None}) == EINVAL
        assert call(_dims(), **{n: FAR * 50 + 4}) == EALIGN


def test_optional_pointers_are_aligned():
    assert route(_dims(), bias=4) == EALIGN and sort(_dims(), pair=4) == EALIGN
    for n in ("gates", "dy", "dgates"):
        assert combine_backward(_dims(), **{n: 4}) == EALIGN
    assert combine_backward(_dims(), dy=None, dgates=None) == EINVAL


@pytest.mark.parametrize("call", [route, route_backward])
def test_route_refuses(call):
    for bad in (dict(E=0), dict(E=1025, K=1), dict(K=0), dict(K=17), dict(E=4), dict(S=0), dict(R=0), dict(R=65),
                dict(S=1 << 28)):
        assert call(_dims(**bad)) == EINVAL
    for mode in (3, 19, 32, 1 << 31):
        assert call(_dims(), mode, 1.0) == EINVAL
    for scale in (float("inf"), float("-inf"), float("nan")):
        assert call(_dims(), 0, scale) == EINVAL
    bad = _dims()
    bad.flags = 1024
    assert call(bad) == EINVAL
    # H, I, B and ranks that own unequal shares are not looked at: the next thing refused is the pointer
    assert call(_dims(H=0, I=-3, B=1000, R=3, E=1024), topk=FAR * 50 + 4) == EALIGN


def test_more_rows_than_a_launch_has_lanes():
    for call in (route, route_backward):
        assert call(_dims(S=(1 << 27) + 1, K=1)) == ENOTSUP
        assert call(_dims(S=1 << 27, K=1), topk=FAR * 50 + 4) == EALIGN
    assert combine_backward(_dims(S=(1 << 25) + 1, K=1)) == ENOTSUP
    assert combine_backward(_dims(S=1 << 25, K=1), dest=FAR * 50 + 4) == EALIGN


def test_route_refuses_overlap():
    d = _dims(S=64)                                          # picks: 2048 bytes; logits: 8192
    assert route(d, topk=FAR + 8192 - 16) == EINVAL          # the logits' end
    assert route(d, gates=FAR * 3 + 2048 - 16) == EINVAL     # topk's
    assert route(d, gates=FAR * 2 + 112) == EINVAL           # the bias's
    assert route_backward(d, dlogits=FAR * 2 + 8192 - 16) == EINVAL
    assert route_backward(d, dlogits=FAR * 3 - 8192 + 16) == EINVAL
    # bf16 logits are half as long
    assert route(d, 16, 1.0, topk=FAR + 4096 - 16) == EINVAL
    assert route(d, 16, 1.0, topk=FAR + 4096, gates=4) == EALIGN


def test_sort_refuses():
    for bad in (dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(S=0), dict(R=65), dict(S=1 << 28)):
        assert M.lib.moonep_sort_workspace_bytes(ctypes.byref(_dims(**bad))) == 0
        assert sort(_dims(**bad)) == EINVAL
    d = _dims(S=64)
    assert sort(d, dest=FAR + 2048 - 16) == EINVAL           # topk's end
    assert sort(d, pair=FAR * 4 + 2032) == EINVAL            # dest's
    assert sort(d, offsets=FAR * 2) == EINVAL                # the scratch
    assert sort(_dims(E=3, K=16, H=0, R=5), topk=FAR * 50 + 4) == EALIGN      # more picks than experts: ids may repeat


def test_sort_workspace():
    size = lambda **kw: M.moonep_sort_workspace_bytes(_dims(**kw))
    assert size() == size(S=256) == 256                      # one workgroup keeps all of it
    assert size(S=1025) == 1280 and 9 * 32 * 4 == 1152       # nine parts of 1024 pairs, in whole 256 bytes
    assert size(S=1025, E=31) == 1280                        # an even number of experts
    assert size(S=8192) == size(S=8193) == 64 * 32 * 4       # parts of 2048 pairs: 33, and room for 64 smaller ones
    assert size(S=1 << 26, K=16, E=1024) == 256 * 1024 * 4   # the most parts


def test_combine_backward_refuses():
    for bad in (dict(H=12), dict(H=0), dict(K=0), dict(K=17), dict(S=0), dict(R=0), dict(S=1 << 28)):
        assert combine_backward(_dims(**bad)) == EINVAL
    d = _dims(S=4, K=2, H=1024)                              # rows 2048 bytes, 8 of them
    assert combine_backward(d, dy=FAR * 2 + 8 * 2048 - 16) == EINVAL          # y's end
    assert combine_backward(d, dy=FAR * 4 + 4 * 2048 - 16) == EINVAL          # dout's
    assert combine_backward(d, dgates=FAR * 3 + 16) == EINVAL                 # the gates
    assert combine_backward(d, dgates=FAR * 5 + 8 * 2048 - 16) == EINVAL      # dy
    assert combine_backward(_dims(S=4, K=2, H=1024, f32_rows=True), dy=FAR * 2 + 8 * 4096 - 16) == EINVAL
    # experts are not looked at
    assert combine_backward(_dims(E=0, R=3), dest=FAR * 50 + 4) == EALIGN


def test_rows_without_a_plan():
    """Dispatch and combine look at R, S, K, H and the row type: rows that moonep_sort placed have no ranks."""
    for e in (0, 5, 256, 5000):
        d = _dims(E=e)
        assert M.lib.moonep_dispatch(ctypes.byref(d), VP(4), VP(FAR), None, VP(FAR * 2), None) == EALIGN
        assert M.lib.moonep_combine(ctypes.byref(d), VP(4), VP(FAR), None, VP(FAR * 2), None) == EALIGN
    for bad in (dict(R=0), dict(K=0), dict(K=17), dict(S=0), dict(H=4), dict(S=1 << 28)):
        assert M.lib.moonep_dispatch(ctypes.byref(_dims(**bad)), VP(4), VP(FAR), None, VP(FAR * 2), None) == EINVAL


def test_fp8_sizes():
    assert M.moonep_fp8_code_bytes(32, 32) == 4096 and M.moonep_fp8_scale_bytes(32, 32) == 4
    assert M.moonep_fp8_code_bytes(160, 96) == 3 * 2 * 4096 and M.moonep_fp8_scale_bytes(160, 160) == 8
    assert M.moonep_fp8_scale_bytes(640, 128) == 8           # five blocks, padded to eight
    assert M.moonep_fp8_code_bytes(7168, 4096) == 7168 * 4096
    for kin, n, code in ((0, 32, EINVAL), (32, -32, EINVAL), (33, 32, ENOTSUP), (32, 40, ENOTSUP), (1 << 21, 32, ENOTSUP)):
        assert M.lib.moonep_fp8_code_bytes(kin, n) == M.lib.moonep_fp8_scale_bytes(kin, n) == 0
        for f in (M.moonep_fp8_code_bytes, M.moonep_fp8_scale_bytes):
            with pytest.raises(M.MoonEPError) as e:
                f(kin, n)
            assert e.value.code == code


def test_quantize_refuses():
    def call(E=2, Kin=64, N=96, w=FAR, c=2 * FAR, s=3 * FAR):
        return M.lib.moonep_quantize_fp8(E, Kin, N, *(None if a is None else VP(a) for a in (w, c, s)), None)

    assert call(E=0) == call(E=1025) == call(Kin=0) == call(N=0) == EINVAL
    assert call(Kin=48) == call(N=100) == ENOTSUP
    for n in "wcs":
        assert call(**{n: None}) == EINVAL and call(**{n: FAR * 9 + 8}) == EALIGN
    assert call(c=FAR + 2 * 64 * 96 * 2 - 16) == EINVAL      # w's end
    assert call(s=2 * FAR + 2 * 3 * 4096 - 16) == EINVAL     # the codes'


def test_ffn_refuses():
    for bad in (dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(K=33), dict(S=0), dict(R=65), dict(H=0), dict(I=0)):
        assert ffn(_dims(**bad)) == EINVAL
    for bad in (dict(H=7176), dict(I=40), dict(f32_rows=True), dict(S=(1 << 19) + 1)):
        assert ffn(_dims(**bad)) == ENOTSUP
        with pytest.raises(M.MoonEPError) as e:
            M.moonep_fp8_ffn_workspace_bytes(_dims(**bad))
        assert e.value.code == ENOTSUP
    # rows of x that 32-bit offsets do not reach
    assert ffn(_dims(S=1 << 19, K=1, H=8192)) == ENOTSUP
    d = _dims(S=2, K=2, E=4, H=64, I=32)
    ws = M.moonep_fp8_ffn_workspace_bytes(d)
    at = {n: (i + 1) * FAR for i, n in enumerate(("topk", "gates", "x", "c13", "s13", "c2", "s2", "ws", "out"))}
    assert ffn(d, out=at["x"]) == EINVAL and ffn(d, out=at["ws"] + ws - 16) == EINVAL
    for n in ("topk", "gates", "x", "c13", "s13", "c2", "s2"):
        assert ffn(d, ws=at[n]) == EINVAL


def test_ffn_workspace_serves_smaller_calls():
    """Whatever way a call takes: few pairs, tiles of 64, 128 or 256 rows, one workgroup's sort or several."""
    for E, K, H, I in ((4, 2, 64, 32), (32, 8, 1024, 512), (256, 8, 7168, 2048), (1, 1, 96, 2048)):
        last = 0
        for T in (1, 2, 5, 8, 9, 20, 47, 48, 90, 100, 191, 192, 193, 300, 700, 1023, 1024, 1025, 1600, 6000, 6200, 30000, 131072,
                  131200, 140000):
            n = M.moonep_fp8_ffn_workspace_bytes(_dims(S=T, E=E, K=K, H=H, I=I))
            assert n >= last
            last = n


def test_constants_match_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moonep.h")).read()
    found = dict(re.findall(r"#define MOONEP_([A-Z0-9_]+) +\(?([0-9 <]+)\)?", text))
    assert eval(found["FP8_MAX_PAIRS"]) == M.FP8_MAX_PAIRS
    assert [int(found[n]) for n in ("ROUTE_SOFTMAX", "ROUTE_SOFTMAX_ALL", "ROUTE_SIGMOID", "ROUTE_BF16")] == \
        [M.ROUTE_SOFTMAX, M.ROUTE_SOFTMAX_ALL, M.ROUTE_SIGMOID, M._ROUTE_BF16]


def test_binding_refuses(monkeypatch):
    """Types, shapes and modes, on host tensors that pass for the GPU's."""
    torch = pytest.importorskip("torch")
    real = M._ptr

    def ptr(t, name, dtype=None, shape=None, numel=None, optional=False):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        for what, want, got in (("dtype", dtype, t is not None and t.dtype), ("shape", shape, t is not None and tuple(t.shape))):
            if t is not None and want is not None and want != got:
                raise ValueError(f"{name} must have {what} {want}")
        return 0 if t is not None else real(t, name, optional=optional)

    monkeypatch.setattr(M, "_ptr", ptr)
    d = M.Dims.make(1, 4, 0, 3, 2, 32, 32)
    z, ids, g = torch.zeros(1, 3, 4), torch.zeros(1, 3, 2, dtype=torch.int32), torch.zeros(1, 3, 2)
    for bad in (z.double(), z.half(), z[:, :2], z.int()):
        with pytest.raises(ValueError):
            M.moonep_route(d, bad, None, ids, g, stream=0)
    with pytest.raises(ValueError, match="mode"):
        M.moonep_route(d, z, None, ids, g, mode=3, stream=0)
    with pytest.raises(ValueError, match="bias"):
        M.moonep_route(d, z, torch.zeros(5), ids, g, stream=0)
    with pytest.raises(ValueError, match="dlogits"):
        M.moonep_route_backward(d, g, z.bfloat16(), ids, z, stream=0)
    with pytest.raises(ValueError, match="required"):
        M.moonep_combine_backward(d, ids, None, g, torch.zeros(1, 3, 32).bfloat16(), None, g, stream=0)
    with pytest.raises(ValueError, match="shape"):
        M.moonep_quantize_fp8(torch.zeros(32, 32).bfloat16(), None, None, stream=0)


def test_layer_refuses():
    torch = pytest.importorskip("torch")
    from balanced_token_dispatch_moonep_amd import layer as L
    d = M.Dims.make(1, 4, 0, 3, 2, 32, 0)
    for kw in (dict(training=True), dict()):
        with pytest.raises(ValueError, match="gradient of the gates"):
            L.MoonEPLayer(d, device="cpu", gate_grad=True, **kw)
    layer = L.MoonEPLayer(d, device="cpu")
    with pytest.raises(ValueError, match="nothing to decode"):
        layer.decoder(4, bits=8)
    layer.d = M.Dims.make(1, 4, 0, 3, 2, 32, 32)
    with pytest.raises(ValueError, match="4 or 8"):
        layer.decoder(4, bits=16)
    r = L.Router(d, device="cpu")
    with pytest.raises(ValueError, match="training"):
        r.backward(torch.zeros(1, 3, 2))
    with pytest.raises(ValueError, match="forward"):
        L.Router(d, training=True, device="cpu").backward(torch.zeros(1, 3, 2))


def test_rows_of_more_tokens_than_a_launch_has_waves():
    """A wave a token, and in the staged calls a wave a (token, k) pair; lanes are counted in 32 bits.  Every call has a
    misaligned pointer, so that nothing is enqueued where the sizes pass."""
    most = (1 << 26) - 4
    for fn, names, rows in (("moonep_dispatch", ("dest", "src", "scale", "recv"), 1),
                            ("moonep_combine", ("dest", "y", "gates", "out"), 1),
                            ("moonep_dispatch_staged", ("dest", "src", "scale", "stage", "recv"), 8),
                            ("moonep_combine_staged", ("dest", "y", "gates", "stage", "out"), 8)):
        call = _caller(fn, names)
        for n, code in ((most // rows, EALIGN), (most // rows + 1, ENOTSUP), (1 << 26, ENOTSUP)):
            assert call(_dims(S=n, K=rows, H=8), dest=FAR * 50 + 4) == code
