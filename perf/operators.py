"""The operators round the MoE layer, as cases to measure: each with a plain form and the library's call.

* layer norm, forward (``moonep_layer_norm``) and backward (``moonep_layer_norm_backward``);
* the global norm of many gradients and clipping by it (``moonep_grad_norm``, ``moonep_grad_clip``);
* the experts' SwiGLU FFN for decoded tokens, weights in 4 bits (``moonep_w4_ffn``).

``own`` chooses between the two: false computes the plain form in elementary torch operations,
true calls the library.  ``prepare`` makes the same inputs for both.
"""
import math

import torch

own = False

EPS = 1e-5
#: The values of the eight e2m1 magnitudes (1 sign, 2 exponent, 1 mantissa bit).
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 32


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # the norm in front of the layer for one decoded token: launch latency
        dict(name="norm one token", op="norm", rows=1, H=7168, dtype="bf16"),
        # the norm of one training step's rows (8 ranks of 4096 tokens)
        dict(name="norm training rows", op="norm", rows=32768, H=7168, dtype="bf16"),
        # its gradient for a small float32 layer with a ragged number of rows
        dict(name="norm gradient ragged", op="norm_backward", rows=333, H=576, dtype="f32"),
        # its gradient of one training step's rows
        dict(name="norm gradient training", op="norm_backward", rows=32768, H=7168, dtype="bf16"),
        # many small gradients of mixed lengths and types, as of norms, biases and routers
        dict(name="clip many small", op="clip", tensors=60, largest=50021, bf16=20),
        # a few larger ones, as of a small layer's experts
        dict(name="clip small layer", op="clip", tensors=6, largest=2621440, bf16=0),
        # the expert gradients of eight experts, float32
        dict(name="clip experts", op="clip", tensors=2, largest=234881024, bf16=0),
        # a small layer's experts, a few ragged tokens
        dict(name="experts small", op="ffn", T=5, K=2, E=16, H=320, I=192, masked=1),
        # one token over the home experts of one rank
        dict(name="experts one token", op="ffn", T=1, K=8, E=32, H=7168, I=2048, masked=0),
        # a batch of eight sequences, one of them ended
        dict(name="experts 8 tokens", op="ffn", T=8, K=8, E=32, H=7168, I=2048, masked=1),
        # a large decode batch: every expert is read, about 16 rows each
        dict(name="experts 64 tokens", op="ffn", T=64, K=8, E=32, H=7168, I=2048, masked=3),
        # the largest decode batch
        dict(name="experts 128 tokens", op="ffn", T=128, K=8, E=32, H=7168, I=2048, masked=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_backward", "clip", "ffn", "ffn"))
    if op in ("norm", "norm_backward"):
        H = 8 * _log(rng, 1, 2048)
        rows = _log(rng, 1, min(65536, 32768 * 7168 // (2 * H)))
        return dict(op=op, rows=rows, H=H, dtype=rng.choice(("bf16", "bf16", "f32")))
    if op == "clip":
        n = _log(rng, 1, 60)
        return dict(op=op, tensors=n, largest=_log(rng, 16, 200_000_000 // n), bf16=rng.randint(0, n))
    H, I = 32 * _log(rng, 2, 224), 32 * _log(rng, 1, 64)
    E = rng.choice((4, 8, 16, 32))
    K = rng.randint(1, min(E, 8))
    T = _log(rng, 1, 100)
    return dict(op=op, T=T, K=K, E=E, H=H, I=I, masked=rng.randint(0, min(3, T - 1)))


def _numels(case):
    """Lengths from the largest down, by halves and odd remainders: experts', routers' and norms' gradients."""
    n, big = case["tensors"], case["largest"]
    if n == 2:
        return [big, big // 2]
    return [max(1, int(big * 0.8 ** i) - (i % 3) * (i > 0)) for i in range(n)]


# ----------------------------------------------------------------------------
# 4-bit weights: quantised in groups of 32 along the input direction, laid out for the kernels
# ----------------------------------------------------------------------------

def _quantise(w):
    """[E, Kin, N] values -> codes [E, Kin, N] (uint8, sign in bit 3) and scale exponents
    [E, Kin/32, N] (uint8, biased by 127): OCP MX FP4, scale 2^(floor(log2 max) - 2)."""
    E, Kin, N = w.shape
    w = w.float().reshape(E, Kin // GROUP, GROUP, N)
    top = w.abs().amax(2)
    exp = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.full_like(top, -126).int()).clamp(-126, 127)
    a = torch.ldexp(w.abs(), -exp.unsqueeze(2))
    code = torch.zeros(a.shape, dtype=torch.uint8, device=w.device)
    # halfway values go to the even code
    code += a > 0.25
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code |= torch.signbit(w).to(torch.uint8) << 3
    return code.reshape(E, Kin, N), (exp + 127).to(torch.uint8)


def _lay_out(code, scale):
    """The library's layout.  Codes [E][N/16][Kin/128][4 groups][16 columns][32 codes], two a byte,
    the first in the low half; scales [E][N/16][Kin/512][4 groups][16 columns][4 blocks of 128]."""
    E, Kin, N = code.shape
    kb, nb = -(-Kin // 128), N // 16
    sb = -(-kb // 4)
    c = torch.nn.functional.pad(code, (0, 0, 0, kb * 128 - Kin))
    c = c.reshape(E, kb, 4, GROUP, nb, 16).permute(0, 4, 1, 2, 5, 3).contiguous()
    c = c[..., 0::2] | (c[..., 1::2] << 4)
    s = torch.nn.functional.pad(scale, (0, 0, 0, sb * 16 - Kin // GROUP), value=127)
    s = s.reshape(E, sb, 4, 4, nb, 16).permute(0, 4, 1, 3, 5, 2).contiguous()
    return c.reshape(E, -1), s.reshape(E, -1)


def _weights(codes, scales, Kin, N):
    """float32 [n, Kin, N] from codes [n, ...] and scales [n, ...] in the library's layout."""
    n, kb, nb = codes.shape[0], -(-Kin // 128), N // 16
    sb = -(-kb // 4)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(n, nb, kb, 4, 16, GROUP)
    s = scales.reshape(n, nb, sb, 4, 16, 4).permute(0, 1, 2, 5, 3, 4).reshape(n, nb, sb * 4, 4, 16)[:, :, :kb]
    w = table[c.int()] * torch.exp2(s.float() - 127).unsqueeze(-1)
    return w.permute(0, 2, 3, 5, 1, 4).reshape(n, kb * 128, N)[:, :Kin]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _hidden(rows, H, gen):
    """Hidden rows of a residual stream: channels of unequal size and offset, a few of them large."""
    size = 0.5 + torch.rand(H, generator=gen, device="cuda")
    size[:: max(1, H // 5)] *= 12
    offset = 0.3 * torch.randn(H, generator=gen, device="cuda")
    return torch.randn(rows, H, generator=gen, device="cuda") * size + offset


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] in ("norm", "norm_backward"):
        rows, H, t = case["rows"], case["H"], _dtype(case)
        s["x"] = _hidden(rows, H, gen).to(t).reshape(1, rows, H)
        s["weight"] = 1 + 0.1 * randn(H)
        s["bias"] = 0.1 * randn(H)
        s["y"] = torch.empty_like(s["x"])
        s["mean"], s["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
        if case["op"] == "norm_backward":
            s["dy"] = (1e-2 * randn(1, rows, H)).to(t)
            x = s["x"].reshape(rows, H).float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["dweight"], s["dbias"] = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    elif case["op"] == "clip":
        lengths = _numels(case)
        s["grads"] = [1e-3 * randn(n) for n in lengths]
        for i in range(case["bf16"]):
            s["grads"][-1 - i] = s["grads"][-1 - i].bfloat16()
        s["norm"] = torch.empty(1, device="cuda")
        s["limit"] = 0.5e-3 * math.sqrt(sum(lengths))      # about half the norm
    else:
        T, K, E, H, I = (case[k] for k in "TKEHI")
        s["x"] = randn(1, T, H).bfloat16()
        # the experts that a skewed router picks: all of a token's differ
        z = randn(T, E) - 0.3 * torch.log(torch.arange(1, E + 1, device="cuda"))
        top, ids = z.topk(K, dim=1)
        ids = ids.int()
        gates = torch.softmax(top, dim=1)
        if case["masked"]:                                  # ended sequences: no experts
            ids[T - case["masked"]:] = -1
        s["topk"], s["gates"] = ids.reshape(1, T, K), gates.reshape(1, T, K).contiguous()
        s["w13"], s["w13_scale"] = _lay_out(*_quantise((0.02 * randn(E, H, 2 * I)).bfloat16()))
        s["w2"], s["w2_scale"] = _lay_out(*_quantise((0.02 * randn(E, I, H)).bfloat16()))
        s["out"] = torch.empty(1, T, H, dtype=torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _norm_plain(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    y = c * rstd * s["weight"] + s["bias"]
    return dict(y=y.to(s["x"].dtype), mean=mean.reshape(-1), rstd=rstd.reshape(-1))


def _norm_backward_plain(s):
    H = s["x"].shape[-1]
    x, dy = s["x"].reshape(-1, H).float(), s["dy"].reshape(-1, H).float()
    r = s["rstd"][:, None]
    n = (x - s["mean"][:, None]) * r
    g = dy * s["weight"]
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype).reshape(s["x"].shape), dweight=(dy * n).sum(0), dbias=dy.sum(0))


def _clip_plain(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt().float().reshape(1)
    c = torch.clamp(s["limit"] / norm, max=1.0)
    for g in s["grads"]:
        g.copy_(g.float() * c)
    return dict(norm=norm, grads=s["grads"])


def _ffn_plain(s):
    T, K, E, H, I = (s["case"][k] for k in "TKEHI")
    x = s["x"].reshape(T, H).float()
    ids, gates = s["topk"].reshape(-1).long(), s["gates"].reshape(-1)
    gates = torch.where(ids >= 0, gates, torch.zeros_like(gates))
    ids = ids.clamp(min=0)
    if T * K <= E:          # the weights of each pair's expert
        rows, of = x.repeat_interleave(K, 0).unsqueeze(1), ids
    else:                   # every expert, for every token
        rows, of = x.unsqueeze(0).expand(E, T, H), slice(None)
    gu = torch.matmul(rows, _weights(s["w13"][of], s["w13_scale"][of], H, 2 * I))
    g, u = gu[..., :I], gu[..., I:]
    y = torch.matmul(g / (1 + torch.exp(-g)) * u, _weights(s["w2"][of], s["w2_scale"][of], I, H))
    if T * K <= E:
        out = (y.reshape(T, K, H) * gates.reshape(T, K, 1)).sum(1)
    else:
        share = torch.zeros(T, E, device="cuda").scatter_add_(1, ids.reshape(T, K), gates.reshape(T, K))
        out = (y * share.t().unsqueeze(-1)).sum(0)
    return out.bfloat16().reshape(1, T, H)


def _kept(s, name, make):
    """What a program makes once and keeps: workspaces, and the list of its gradients."""
    if name not in s:
        s[name] = make()
    return s[name]


def _run_own(s):
    import balanced_token_dispatch_moonep_amd as M

    def room(size):
        return lambda: torch.empty(size(), dtype=torch.uint8, device="cuda")

    case, op = s["case"], s["case"]["op"]
    if op in ("norm", "norm_backward"):
        d = _kept(s, "dims", lambda: M.Dims.make(1, 1, 0, case["rows"], 1, case["H"], f32_rows=case["dtype"] == "f32"))
        if op == "norm":
            M.moonep_layer_norm(d, s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"], s["rstd"])
            return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
        ws = _kept(s, "ws", room(lambda: M.moonep_layer_norm_workspace_bytes(d)))
        M.moonep_layer_norm_backward(d, s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["y"], s["dweight"],
                                     s["dbias"], ws)
        return dict(dx=s["y"], dweight=s["dweight"], dbias=s["dbias"])
    if op == "clip":
        grads = _kept(s, "list", lambda: M.GradList(s["grads"]))
        ws = _kept(s, "ws", room(lambda: M.moonep_grad_norm_workspace_bytes(grads)))
        M.moonep_grad_norm(grads, ws, s["norm"])
        M.moonep_grad_clip(grads, s["norm"], s["limit"])
        return dict(norm=s["norm"], grads=s["grads"])
    d = _kept(s, "dims", lambda: M.Dims.make(1, case["E"], 0, case["T"], case["K"], case["H"], case["I"]))
    ws = _kept(s, "ws", room(lambda: M.moonep_w4_ffn_workspace_bytes(d)))
    M.moonep_w4_ffn(d, s["topk"], s["gates"], s["x"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], ws, s["out"])
    return s["out"]


def run(state):
    if own:
        r = _run_own(state)
    else:
        r = dict(norm=_norm_plain, norm_backward=_norm_backward_plain, clip=_clip_plain,
                 ffn=_ffn_plain)[state["case"]["op"]](state)
    if state["case"]["op"] == "clip":
        # gradients are clipped in place, so the next pass asks for a little less: it clips again
        state["limit"] *= 0.995
    return r


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "norm_backward"):
        n, b = case["rows"] * case["H"], 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "norm":
            return dict(bytes=2 * b * n + 8 * case["H"] + 8 * case["rows"], flops=8 * n)
        return dict(bytes=3 * b * n + 12 * case["H"] + 8 * case["rows"], flops=14 * n)
    if case["op"] == "clip":
        lengths = _numels(case)
        b = sum(n * (2 if i >= len(lengths) - case["bf16"] else 4) for i, n in enumerate(lengths))
        return dict(bytes=3 * b + 4, flops=3 * sum(lengths))    # read for the norm, read and written to clip
    T, K, E, H, I = (case[k] for k in "TKEHI")
    pairs = (T - case["masked"]) * K
    read = E * (1 - (1 - K / E) ** (T - case["masked"]))        # experts that tokens pick, expected
    return dict(bytes=read * 3 * H * I * (1 / 2 + 1 / 32) + 4 * T * H + 8 * T * K, flops=6 * H * I * pairs)


# ----------------------------------------------------------------------------
# the definitions, in 64 bits
# ----------------------------------------------------------------------------

def _exact_weight(codes, scales, Kin, N):
    """One expert's [Kin, N] in 64 bits, each code found by its place in the layout."""
    dev = codes.device
    k = torch.arange(Kin, device=dev)[:, None]
    n = torch.arange(N, device=dev)[None, :]
    kb, sb = (Kin + 127) // 128, (Kin + 511) // 512
    lane = (k % 128 // 32) * 16 + n % 16
    at = (((n // 16) * kb + k // 128) * 64 + lane) * 16 + k % 32 // 2
    v = (codes[at].int() >> (4 * (k % 2))) & 15
    mag, top = v & 1, v >> 1 & 3
    value = torch.where(top > 0, (1 + 0.5 * mag.double()) * torch.exp2(top.double() - 1), 0.5 * mag.double())
    value = torch.where(v >= 8, -value, value)
    e = scales[(((n // 16) * sb + k // 512) * 64 + lane) * 4 + k // 128 % 4].double()
    return value * torch.exp2(e - 127)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + EPS) * s["weight"].double() + s["bias"].double()
        return dict(y=y, mean=mean.reshape(-1), rstd=1 / torch.sqrt(var + EPS).reshape(-1))
    if case["op"] == "norm_backward":
        # through the row's two statistics, step by step by the chain rule
        rows, H = case["rows"], case["H"]
        x, dy, w = s["x"].reshape(rows, H).double(), s["dy"].reshape(rows, H).double(), s["weight"].double()
        sigma = torch.sqrt(torch.var(x, dim=1, correction=0, keepdim=True) + EPS)
        c = x - x.mean(1, keepdim=True)
        dn = dy * w
        dsigma = -(dn * c).sum(1, keepdim=True) / sigma.square()
        dc = dn / sigma + dsigma * c / (H * sigma)
        dx = dc - dc.sum(1, keepdim=True) / H
        return dict(dx=dx.reshape(s["x"].shape), dweight=(dy * c / sigma).sum(0), dbias=dy.sum(0))
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
        c = min(1.0, s["limit"] / norm)
        return dict(norm=torch.tensor([norm], dtype=torch.float64), grads=[g.double() * c for g in s["grads"]])
    T, K, E, H, I = (case[k] for k in "TKEHI")
    x, out = s["x"].reshape(T, H).double(), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    ids, gates = s["topk"].reshape(T, K), s["gates"].reshape(T, K).double()
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        gu = x[t] @ _exact_weight(s["w13"][e], s["w13_scale"][e], H, 2 * I)
        a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        out.index_add_(0, t, gates[t, k, None] * (a @ _exact_weight(s["w2"][e], s["w2_scale"][e], I, H)))
    return out.reshape(1, T, H)
