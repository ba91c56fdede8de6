"""The operators round the layer without a GPU: sizes, and everything that is refused on the host
before a launch."""
import ctypes

import pytest

import balanced_token_dispatch_moonep_amd as M

EINVAL, EALIGN, ENOTSUP = -1, -2, -4
VP = ctypes.c_void_p
G, MIS = VP(0x10000), VP(0x10004)


def _dims(**kw):
    base = dict(R=1, E=32, B=0, S=8, K=8, H=7168, I=2048)
    base.update(kw)
    return M.Dims.make(**base)


def _norm(d, x=G, w=G, b=G, eps=1e-5, y=G, mean=G, rstd=G):
    return M.lib.moonep_layer_norm(ctypes.byref(d) if d else None, x, w, b, eps, y, mean, rstd, None)


def test_norm_refuses():
    d = _dims()
    assert _norm(None) == EINVAL
    assert _norm(_dims(H=1004)) == EINVAL
    assert _norm(_dims(S=0)) == EINVAL
    assert _norm(d, x=None) == EINVAL and _norm(d, y=None) == EINVAL
    for eps in (-1e-5, float("nan"), float("inf")):
        assert _norm(d, eps=eps) == EINVAL
    assert _norm(d, mean=None) == EINVAL and _norm(d, rstd=None) == EINVAL
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        assert _norm(d, **{name: MIS}) == EALIGN


def test_norm_backward_refuses():
    d = _dims()
    names = ("dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias", "ws")

    def call(d=d, **kw):
        a = [kw.get(n, G) for n in names]
        return M.lib.moonep_layer_norm_backward(ctypes.byref(d), *a, None)

    assert call(_dims(H=12)) == EINVAL
    for n in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert call(**{n: None}) == EINVAL
    assert call(ws=None, dweight=None) == EINVAL
    for n in names:
        assert call(**{n: MIS}) == EALIGN


def test_norm_dims_that_count():
    """Only R, S, H and the row type: the planner's limits on experts, K and B are not the norm's."""
    want = M.moonep_layer_norm_workspace_bytes(_dims())
    for other in (dict(E=256), dict(E=0), dict(E=5000), dict(K=0), dict(K=64), dict(B=100), dict(I=-1)):
        assert M.moonep_layer_norm_workspace_bytes(_dims(**other)) == want
        assert _norm(_dims(**other), x=None) == EINVAL and _norm(_dims(**other), x=MIS) == EALIGN
    assert M.moonep_layer_norm_workspace_bytes(_dims(R=3)) == M.moonep_layer_norm_workspace_bytes(_dims(S=24))
    # the most rows (of 8 bf16 each, 17 GB)
    assert M.moonep_layer_norm_workspace_bytes(_dims(S=1 << 30, H=8)) > 0
    for bad in (dict(R=0), dict(R=65), dict(S=0), dict(S=-5), dict(H=0), dict(H=-8), dict(H=12), dict(R=2, S=1 << 30)):
        assert M.lib.moonep_layer_norm_workspace_bytes(ctypes.byref(_dims(**bad))) == 0
        assert _norm(_dims(**bad), x=MIS) == EINVAL
    bad = _dims()
    bad.flags = 1024
    assert _norm(bad, x=MIS) == EINVAL


def test_norm_refuses_overlap():
    """64 rows of 1024 bf16, 131072 bytes, each buffer far from the others but for those named."""
    d = _dims(S=64, H=1024)
    at = {n: VP((i + 1) << 20) for i, n in enumerate(("x", "w", "b", "y", "mean", "rstd"))}
    end = 64 * 1024 * 2
    for y in (1 << 20, (1 << 20) + end - 16, (1 << 20) - end + 16):       # all of x, its end, its beginning
        assert _norm(d, **{**at, "y": VP(y)}) == EINVAL
    assert _norm(d, **{**at, "y": VP((2 << 20) - end + 16)}) == EINVAL     # the weight
    assert _norm(d, **{**at, "mean": VP((4 << 20) + end - 16)}) == EINVAL  # y's end
    assert _norm(d, **{**at, "rstd": VP((5 << 20) + 240)}) == EINVAL       # the means' end


def test_norm_backward_refuses_overlap():
    d = _dims(S=64, H=1024)
    names = ("dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias", "ws")
    at = {n: (i + 1) << 22 for i, n in enumerate(names)}
    end = 64 * 1024 * 2

    def call(**kw):
        return M.lib.moonep_layer_norm_backward(ctypes.byref(d), *(VP({**at, **kw}[n]) for n in names), None)

    for over in ("dy", "x"):
        for off in (0, end - 16, 16 - end):
            assert call(dx=at[over] + off) == EINVAL
    assert call(dweight=at["weight"]) == EINVAL
    assert call(dbias=at["dweight"] + 4096 - 16) == EINVAL
    assert call(ws=at["x"] + end - 16) == EINVAL
    assert call(ws=at["mean"] + 64) == EINVAL
    assert call(ws=at["dx"] + end - 16) == EINVAL
    assert call(dweight=at["ws"]) == EINVAL


def test_norm_workspace():
    one, many = (M.moonep_layer_norm_workspace_bytes(_dims(S=s)) for s in (1, 1 << 15))
    assert 2 * 7168 * 4 <= one < many < 64 << 20
    assert M.lib.moonep_layer_norm_workspace_bytes(ctypes.byref(_dims(H=4))) == 0
    assert M.lib.moonep_layer_norm_workspace_bytes(None) == 0


def _grads(at, numel, dtype):
    n = len(at)
    return n, (VP * n)(*at), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtype)


def test_grad_norm_refuses():
    f = M.lib.moonep_grad_norm
    assert f(-1, None, None, None, G, G, None) == EINVAL
    assert f(1, None, None, None, G, G, None) == EINVAL
    ok = ([0x10000, 0x20000], [100, 100], [0, 1])
    assert f(*_grads(*ok), None, G, None) == EINVAL
    assert f(*_grads(*ok), G, None, None) == EINVAL
    assert f(*_grads(*ok), MIS, G, None) == EALIGN
    assert f(*_grads(*ok), G, MIS, None) == EALIGN
    assert f(*_grads([0x10000, None], [100, 100], [0, 1]), G, G, None) == EINVAL
    assert f(*_grads([0x10000, 0x20002], [100, 100], [0, 1]), G, G, None) == EALIGN
    assert f(*_grads([0x10000, 0x20000], [100, -1], [0, 1]), G, G, None) == EINVAL
    assert f(*_grads([0x10000, 0x20000], [100, 1 << 41], [0, 1]), G, G, None) == EINVAL
    assert f(*_grads([0x10000, 0x20000], [100, 100], [0, 2]), G, G, None) == EINVAL
    assert M.lib.moonep_grad_norm_workspace_bytes(-1) == 0
    assert 0 < M.lib.moonep_grad_norm_workspace_bytes(0) <= M.lib.moonep_grad_norm_workspace_bytes(1000)


def test_grad_clip_refuses():
    f = M.lib.moonep_grad_clip
    ok = ([0x10000, 0x20000], [100, 100], [0, 1])
    for most in (-1.0, float("nan")):
        assert f(*_grads(*ok), G, most, None) == EINVAL
    assert f(*_grads(*ok), None, 1.0, None) == EINVAL
    assert f(*_grads(*ok), MIS, 1.0, None) == EALIGN
    # shared memory: the same gradient twice, one that reaches into another (in either order)
    assert f(*_grads([0x10000, 0x10000], [100, 100], [0, 0]), G, 1.0, None) == EINVAL
    assert f(*_grads([0x10000, 0x10190 - 16], [100, 4], [0, 0]), G, 1.0, None) == EINVAL
    assert f(*_grads([0x20000, 0x10000], [4, 0x4001], [1, 0]), G, 1.0, None) == EINVAL
    assert f(*_grads([0x30000, 0x20000, 0x10000], [4, 0x8001, 4], [1, 1, 0]), G, 1.0, None) == EINVAL


def test_grads_apart_from_norm_and_scratch():
    """100 float32 (400 bytes) and 100 bf16 (200 bytes); what a call writes or goes by lies elsewhere."""
    norm, clip = M.lib.moonep_grad_norm, M.lib.moonep_grad_clip
    g = _grads([0x100000, 0x200000], [100, 100], [0, 1])
    far, ws = VP(0x300000), VP(0x400000)
    for at in (0x100000, 0x100000 + 384, 0x200000, 0x200000 + 192):
        assert norm(*g, ws, VP(at), None) == EINVAL
        assert norm(*g, VP(at), far, None) == EINVAL
        assert clip(*g, VP(at), 1.0, None) == EINVAL
    size = M.lib.moonep_grad_norm_workspace_bytes(2)
    assert norm(*g, VP(0x100000 - size + 16), far, None) == EINVAL


def test_w4_sizes():
    assert M.moonep_w4_code_bytes(7168, 4096) == 7168 * 4096 // 2
    assert M.moonep_w4_scale_bytes(7168, 4096) == 7168 * 4096 // 32
    assert M.moonep_w4_code_bytes(160, 96) == 96 * 2 * 64
    assert M.moonep_w4_scale_bytes(160, 96) == 96 * 16
    for kin, n in ((0, 32), (33, 32), (32, 16), (-32, 32), (32, 0), (16, 32)):
        assert M.lib.moonep_w4_code_bytes(kin, n) == 0 and M.lib.moonep_w4_scale_bytes(kin, n) == 0
        with pytest.raises(M.MoonEPError):
            M.moonep_w4_code_bytes(kin, n)


def test_refused_sizes_say_why():
    """A size that the call would not support is ENOTSUP, one that is none is EINVAL."""
    def code(f, *a):
        with pytest.raises(M.MoonEPError) as e:
            f(*a)
        return e.value.code

    for f in (M.moonep_w4_code_bytes, M.moonep_w4_scale_bytes):
        assert code(f, 72, 64) == code(f, 64, 16) == ENOTSUP
        assert code(f, 0, 64) == code(f, 64, -32) == EINVAL
    for bad in (dict(H=7176), dict(I=2056), dict(f32_rows=True), dict(S=1025)):
        assert code(M.moonep_w4_ffn_workspace_bytes, _dims(**bad)) == ENOTSUP
    for bad in (dict(S=0), dict(K=0), dict(E=2000)):
        assert code(M.moonep_w4_ffn_workspace_bytes, _dims(**bad)) == EINVAL
    assert code(M.moonep_layer_norm_workspace_bytes, _dims(H=4)) == EINVAL
    assert code(M.moonep_plan_workspace_bytes, _dims(E=0)) == EINVAL


def test_quantize_refuses():
    f = M.lib.moonep_quantize_w4
    for e, kin, n in ((0, 64, 64), (1025, 64, 64), (1, 0, 64), (1, 64, -1)):
        assert f(e, kin, n, G, G, G, None) == EINVAL
    assert f(1, 72, 64, G, G, G, None) == ENOTSUP
    for i in range(3):
        a = [G, G, G]
        a[i] = None
        assert f(1, 64, 64, *a, None) == EINVAL
        a[i] = MIS
        assert f(1, 64, 64, *a, None) == EALIGN


def test_ffn_refuses():
    def call(d, **kw):
        a = [kw.get(str(i), G) for i in range(9)]
        return M.lib.moonep_w4_ffn(ctypes.byref(d) if d else None, *a, None)

    assert call(None) == EINVAL
    for bad in (dict(R=0), dict(S=0), dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(E=4, K=5), dict(I=0)):
        assert call(_dims(**bad)) == EINVAL
        assert M.lib.moonep_w4_ffn_workspace_bytes(ctypes.byref(_dims(**bad))) == 0
    bad = _dims()
    bad.flags = 1024
    assert call(bad) == EINVAL
    for bad in (dict(H=7176), dict(I=2056), dict(f32_rows=True), dict(S=1025)):
        assert call(_dims(**bad)) == ENOTSUP
    for i in range(9):
        assert call(_dims(), **{str(i): None}) == EINVAL
        assert call(_dims(), **{str(i): MIS}) == EALIGN
    # the planner's limit of 64 home experts a rank is not this call's
    assert M.moonep_w4_ffn_workspace_bytes(_dims(E=256, S=1)) > 0
    assert M.W4_MAX_PAIRS == 8192


@pytest.mark.parametrize("E,K,H,I", [(32, 8, 7168, 2048), (8, 4, 1024, 512), (1, 1, 32, 32), (64, 2, 32, 512), (256, 8, 64, 32)])
def test_ffn_workspace_serves_smaller_batches(E, K, H, I):
    """A decoder's scratch for its largest batch serves the smaller ones."""
    sizes = [M.moonep_w4_ffn_workspace_bytes(_dims(E=E, K=K, H=H, I=I, S=s)) for s in range(1, 8192 // K + 1, 3)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert all(n % 256 == 0 and n > 0 for n in sizes)


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    d = M.Dims.make(1, 1, 0, 4, 1, 64)
    x, w, u = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.moonep_layer_norm(d, x, w, w, 1e-5, x, stream=0)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.GradList([w])
    with pytest.raises(TypeError):
        M.GradList([1.0])
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        M.GradList([u])
    with pytest.raises(ValueError, match="GPU tensor"):
        M.moonep_quantize_w4(torch.zeros(1, 32, 32, dtype=torch.bfloat16), u, u, stream=0)


def test_new_constants_match_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moonep.h")).read()
    found = dict(re.findall(r"#define MOONEP_([A-Z0-9_]+) (\d+)\n", text))
    assert int(found["W4_MAX_PAIRS"]) == M.W4_MAX_PAIRS
    assert (int(found["GRAD_F32"]), int(found["GRAD_BF16"])) == (0, 1)


CHANGES = {
    "type": lambda t, torch: t.bfloat16(),
    "type at the same address": lambda t, torch: t.view(torch.int32),
    "type and length at the same address": lambda t, torch: t.view(torch.bfloat16)[:64],
    "part at the same address": lambda t, torch: t[:16],
    "one element, repeated": lambda t, torch: t[:1].expand(64),
    "other order": lambda t, torch: t.view(8, 8).t(),
}


@pytest.mark.parametrize("name", [*CHANGES, "resized"])
def test_grad_list_refuses_a_changed_tensor(monkeypatch, name):
    """Whatever the kernels take for granted of a tensor is looked at in each call, at an old address
    too.  Host tensors stand for the GPU's; nothing is launched."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(M, "_ptr", lambda t, *a, **k: t.data_ptr())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    g, h = torch.zeros(64), torch.zeros(3)
    gl = M.GradList([h, g])
    n, at, numel, dtype = gl._arrays()
    assert (n, list(at), list(numel), list(dtype)) == (2, [h.data_ptr(), g.data_ptr()], [3, 64], [0, 0])
    g.data = torch.zeros(64)                                 # other memory of the same form is followed
    assert list(gl._arrays()[1]) == [h.data_ptr(), g.data_ptr()]
    keep = g.data
    if name == "resized":
        g.resize_(16)
    else:
        g.data = CHANGES[name](keep, torch)
    with pytest.raises(ValueError, match="changed"):
        gl._arrays()
    with pytest.raises(ValueError, match="changed"):         # and stays refused
        gl._arrays()
    g.data = keep if name != "resized" else torch.zeros(64)
    assert list(gl._arrays()[1]) == [h.data_ptr(), g.data_ptr()]


@pytest.fixture
def host_layer(monkeypatch):
    """The layer module on host tensors: the norm doubles rows and counts them, the experts and the
    dispatch copy them."""
    torch = pytest.importorskip("torch")
    from balanced_token_dispatch_moonep_amd import layer as L
    normed = []

    def norm(d, x, w, b, eps, y, mean=None, rstd=None):
        normed.append(x.clone())
        y.copy_(2 * x)

    monkeypatch.setattr(L, "moonep_layer_norm", norm)
    monkeypatch.setattr(L, "moonep_quantize_w4", lambda *a: None)
    monkeypatch.setattr(L, "moonep_w4_ffn", lambda d, topk, gates, x, a, b, c, e, ws, out: out.copy_(x))
    monkeypatch.setattr(L, "moonep_plan", lambda *a: None)
    monkeypatch.setattr(L, "moonep_dispatch", lambda d, dest, x, s, recv: recv.copy_(x.reshape(recv.shape)))
    monkeypatch.setattr(L, "moonep_combine", lambda d, dest, y, g, out: out.copy_(y.reshape(out.shape)))
    return torch, L, normed


def test_decoder_norms_rows_once(host_layer):
    """What norm() returned, whole or in parts, is not normed again; neither is a copy that says so."""
    torch, L, seen = host_layer
    H, T = 32, 6
    w = torch.zeros(2, H, 64, dtype=torch.bfloat16), torch.zeros(2, 32, H, dtype=torch.bfloat16)
    dec = L.W4Experts(*w, K=1, max_tokens=8, norm_weight=torch.ones(H))
    x = torch.arange(T * H).reshape(T, H).bfloat16()
    topk, gates = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1)
    want = dec.forward(x, topk, gates).clone()
    assert torch.equal(want, 2 * x) and len(seen) == 1
    n = dec.norm(x)
    for lo, hi in ((0, T), (0, 2), (2, T), (5, 6)):
        assert torch.equal(dec.forward(n[lo:hi], topk[lo:hi], gates[lo:hi]), want[lo:hi])
    assert len(seen) == 2
    assert torch.equal(dec.forward(n.clone(), topk, gates, normed=True), want) and len(seen) == 2
    assert torch.equal(dec.forward(n.clone(), topk, gates), 4 * x)       # rows that only happen to be normed
    for rows in (n, n[2:]):                                              # over the rows that it reads
        with pytest.raises(ValueError, match="norm"):
            dec.norm(rows)


def test_layer_norms_rows_once(host_layer):
    torch, L, seen = host_layer
    d = M.Dims.make(2, 2, 0, 3, 1, 16)
    x = torch.arange(96).reshape(2, 3, 16).bfloat16()
    layer = L.MoonEPLayer(d, device="cpu", training=True, norm_weight=torch.ones(16))
    with pytest.raises(ValueError, match="norm"):            # its backward would have no rows to go to
        layer.forward(x.clone(), None, None, normed=True)
    want = layer.forward(x, None, None).clone()
    assert torch.equal(want, 2 * x) and len(seen) == 1
    n = layer.norm(x)
    assert torch.equal(layer.forward(n, None, None), want)
    assert torch.equal(layer.forward(n.clone(), None, None, normed=True), want)
    assert len(seen) == 2 and layer.x is x
    with pytest.raises(ValueError, match="norm"):
        layer.norm(n)
    assert torch.equal(layer.forward(x + 1, None, None), 2 * (x + 1)) and len(seen) == 3
