"""Routing, sorting and 8-bit experts, as cases to measure: each with a plain form and the library's call.

* the router's top K with its gates, forward (``moonep_route``) and backward (``moonep_route_backward``);
* tokens sorted by expert (``moonep_sort``), for dispatch and combine without a plan;
* the gradient of the weighted combine, for rows and for gates (``moonep_combine_backward``);
* the experts' SwiGLU FFN in 8-bit floating point, a scale for each block of 128 (``moonep_fp8_ffn``).

``own`` chooses between the two: false computes the plain form in elementary torch operations,
true calls the library.  ``prepare`` makes the same inputs for both.
"""
import math

import torch

own = False

BLOCK = 128
NONE = -7               # what the buffers hold where an operator writes nothing


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decoded token: launch latency; sigmoid gates, a bias that balances the experts
        dict(name="route one token", op="route", T=1, E=256, K=8, mode="sigmoid", bias=True, dtype="f32", masked=0),
        # the rows of one training step (8 ranks of 4096 tokens)
        dict(name="route training rows", op="route", T=32768, E=256, K=8, mode="softmax", bias=False, dtype="f32",
             masked=0),
        # gradient of gates over all experts, bf16 logits, a ragged batch with padding
        dict(name="route gradient ragged", op="route_backward", T=4099, E=160, K=6, mode="softmax_all", bias=False,
             dtype="bf16", masked=35),
        # a decode batch, three of its sequences ended
        dict(name="sort decode batch", op="sort", T=128, E=256, K=8, masked=3),
        # the pairs of one training step
        dict(name="sort training pairs", op="sort", T=32768, E=256, K=8, masked=0),
        # a small float32 layer, ragged, some pairs dropped
        dict(name="combine gradient ragged", op="combine_backward", T=333, E=16, K=3, H=576, dtype="f32", masked=20),
        # one rank's tokens of a training step
        dict(name="combine gradient training", op="combine_backward", T=4096, E=256, K=8, H=7168, dtype="bf16",
             masked=0),
        # a small layer's experts, a few ragged tokens
        dict(name="fp8 experts small", op="ffn", T=5, K=2, E=16, H=320, I=192, masked=1),
        # one token over the home experts of one rank
        dict(name="fp8 experts one token", op="ffn", T=1, K=8, E=32, H=7168, I=2048, masked=0),
        # a decode batch: every expert is read, about 16 rows each
        dict(name="fp8 experts 64 tokens", op="ffn", T=64, K=8, E=32, H=7168, I=2048, masked=3),
        # a short prompt, or a large decode batch: about 128 rows an expert
        dict(name="fp8 experts 512 tokens", op="ffn", T=512, K=8, E=32, H=7168, I=2048, masked=0),
        # a batch of prompts: about 2000 rows an expert
        dict(name="fp8 experts prompt", op="ffn", T=8192, K=8, E=32, H=7168, I=2048, masked=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_backward", "sort", "combine_backward", "ffn", "ffn", "ffn"))
    if op in ("route", "route_backward"):
        E = _log(rng, 2, 512)
        T = _log(rng, 1, 65536)
        mode = rng.choice(("softmax", "softmax_all", "sigmoid"))
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(E, 16)), mode=mode, bias=rng.random() < 0.5,
                    dtype=rng.choice(("f32", "bf16")), masked=rng.randint(0, T // 8))
    if op == "sort":
        E = _log(rng, 1, 1024)
        T = _log(rng, 1, 65536)
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(E, 16)), masked=rng.randint(0, T // 2))
    if op == "combine_backward":
        H = 8 * _log(rng, 1, 1024)
        K = rng.randint(1, 8)
        T = _log(rng, 1, min(16384, 4096 * 8 * 7168 // (2 * H * K)))
        return dict(op=op, T=T, E=rng.choice((8, 64, 256)), K=K, H=H, dtype=rng.choice(("bf16", "bf16", "f32")),
                    masked=rng.randint(0, T // 2))
    H, I = 32 * _log(rng, 2, 224), 32 * _log(rng, 1, 64)
    E = rng.choice((4, 8, 16, 32))
    K = rng.randint(1, min(E, 8))
    T = _log(rng, 1, 6000)
    return dict(op=op, T=T, K=K, E=E, H=H, I=I, masked=rng.randint(0, T // 4))


# ----------------------------------------------------------------------------
# 8-bit values: e4m3 with a power of two for each block of 128, the smallest that brings the block's
# largest magnitude to at most 448
# ----------------------------------------------------------------------------

def _exponent(top):
    """Exponents (int32) of the scales of blocks whose largest magnitudes are given."""
    m, e = torch.frexp(top)
    return torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -126)).clamp(min=-126)


def _codes(x, exp):
    return torch.ldexp(x, -exp).to(torch.float8_e4m3fn)


def _rounded_rows(x):
    """Rows of float32 [n, K] as the values that their 8 bits stand for: a scale for 128 along the row."""
    n, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % BLOCK)).reshape(n, -1, BLOCK)
    exp = _exponent(x.abs().amax(2, keepdim=True))
    return torch.ldexp(_codes(x, exp).float(), exp).reshape(n, -1)[:, :K].contiguous()


def _quantise(w):
    """[Kin, N] -> e4m3 [kb * 128, N] (bytes) and scale bytes [kb, nb], blocks of 128 x 128, both padded."""
    Kin, N = w.shape
    w = torch.nn.functional.pad(w.float(), (0, -N % BLOCK, 0, -Kin % BLOCK))
    kb, nb = w.shape[0] // BLOCK, w.shape[1] // BLOCK
    w = w.reshape(kb, BLOCK, nb, BLOCK)
    exp = _exponent(w.abs().amax((1, 3), keepdim=True))
    code = _codes(w, exp).reshape(kb * BLOCK, nb * BLOCK)[:, :N]
    return code.view(torch.uint8), (exp.reshape(kb, nb) + 127).to(torch.uint8)


def _lay_out(code, scale):
    """The library's layout.  Codes [N/32][kb][8 pieces][32 columns][16 bytes along Kin]; scales
    [nb][kb, padded to a multiple of 4 with 127]."""
    K, N = code.shape
    c = code.reshape(K // BLOCK, 8, 16, N // 32, 32).permute(3, 0, 1, 4, 2).contiguous()
    s = torch.nn.functional.pad(scale.t(), (0, -scale.shape[0] % 4), value=127).contiguous()
    return c.reshape(-1), s.reshape(-1)


def _weights(codes, scales, Kin, N):
    """float32 [Kin, N] from one matrix in the library's layout."""
    kb, nb = -(-Kin // BLOCK), -(-N // BLOCK)
    c = codes.view(torch.float8_e4m3fn).float().reshape(N // 32, kb, 8, 32, 16).permute(1, 2, 4, 0, 3)
    c = c.reshape(kb, BLOCK, N)
    s = torch.exp2(scales.reshape(nb, -1)[:, :kb].t().float() - 127)
    return (c * s.repeat_interleave(BLOCK, 1)[:, None, :N]).reshape(kb * BLOCK, N)[:Kin]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _picks(T, E, K, masked, gen):
    """Distinct experts of each token from a skewed router; the last `masked` tokens have none."""
    z = torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-30).log_().neg_().log_().neg_()
    z -= 0.3 * torch.log(torch.arange(1, E + 1, device="cuda"))
    ids = z.topk(K, dim=1)[1].int()
    if masked:
        ids[T - masked:] = -1
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    op, T, E, K = case["op"], case["T"], case["E"], case["K"]
    s = dict(case=case)
    if op in ("route", "route_backward"):
        z = randn(T, E) - 0.3 * torch.log(torch.arange(1, E + 1, device="cuda"))
        if case["masked"]:                                  # padding has no experts
            z[T - case["masked"]:] = -math.inf
        s["logits"] = z.to(_dtype(case)).reshape(1, T, E)
        s["bias"] = 0.1 * randn(E) if case["bias"] else None
        s["scale"] = 2.5 if case["mode"] == "sigmoid" else 1.0
        s["topk"] = torch.empty(1, T, K, dtype=torch.int32, device="cuda")
        s["gates"] = torch.empty(1, T, K, device="cuda")
        if op == "route_backward":
            s["topk"] = _route_plain(s)["topk"]
            s["dgates"] = randn(1, T, K)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    ids = _picks(T, E, K, case["masked"], gen)
    if op == "sort":
        s["topk"] = ids.reshape(1, T, K)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["dest"] = torch.empty(1, T, K, dtype=torch.int32, device="cuda")
        s["pair"] = torch.full((T * K,), NONE, dtype=torch.int32, device="cuda")
        return s
    gates = torch.softmax(randn(T, K), dim=1).reshape(1, T, K)
    if op == "combine_backward":
        H, t = case["H"], _dtype(case)
        s["topk"], s["gates"] = ids.reshape(1, T, K), gates
        s["dest"] = _sort_plain(s)["dest"]
        s["y"], s["dout"] = randn(T * K, H, dtype=t), randn(1, T, H, dtype=t)
        s["dy"] = torch.full((T * K, H), 0.0, dtype=t, device="cuda")
        s["dgates"] = torch.empty_like(gates)
        return s
    H, I = case["H"], case["I"]
    s["x"] = (randn(T, H) * (0.5 + torch.rand(H, generator=gen, device="cuda"))).bfloat16().reshape(1, T, H)
    s["topk"], s["gates"] = ids.reshape(1, T, K), gates
    for name, kin, n in (("w13", H, 2 * I), ("w2", I, H)):
        packed = [_lay_out(*_quantise((0.02 * randn(kin, n)).bfloat16())) for _ in range(E)]
        s[name], s[name + "_scale"] = (torch.stack(v) for v in zip(*packed))
    s["out"] = torch.empty(1, T, H, dtype=torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _route_plain(s):
    K, mode = s["case"]["K"], s["case"]["mode"]
    z = s["logits"].double()
    key = z
    if s["bias"] is not None:
        key = (1 / (1 + torch.exp(-z)) if mode == "sigmoid" else z) + s["bias"].double()
    # descending, ties to the lower id
    top, ids = (v[..., :K].contiguous() for v in torch.sort(key, dim=-1, descending=True, stable=True))
    none = top == -math.inf
    if s["bias"] is not None:
        none |= torch.gather(z, -1, ids) == -math.inf
    picked = torch.gather(z, -1, ids).masked_fill(none, -math.inf)
    if mode == "sigmoid":
        g = 1 / (1 + torch.exp(-picked))
        gates = g / g.sum(-1, keepdim=True)
    else:
        m = z.amax(-1, keepdim=True)
        total = torch.exp((z if mode == "softmax_all" else picked) - m).sum(-1, keepdim=True)
        gates = torch.exp(picked - m) / total
    gates = (s["scale"] * gates).masked_fill(none, 0.0)
    return dict(topk=ids.int().masked_fill(none, -1), gates=gates.float())


def _route_backward_plain(s):
    mode, ids = s["case"]["mode"], s["topk"].long()
    z, dg = s["logits"].float(), s["dgates"].masked_fill(ids < 0, 0.0)
    picked = torch.gather(z, -1, ids.clamp(min=0)).masked_fill(ids < 0, -math.inf)
    m = picked.amax(-1, keepdim=True).clamp(min=-3e38)
    if mode == "sigmoid":
        g = 1 / (1 + torch.exp(-picked))
        p = (g / g.sum(-1, keepdim=True)).masked_fill(ids < 0, 0.0)
        d = p * (1 - g) * (dg - (p * dg).sum(-1, keepdim=True))
    elif mode == "softmax":
        p = torch.exp(picked - m)
        p = (p / p.sum(-1, keepdim=True)).masked_fill(ids < 0, 0.0)
        d = p * (dg - (p * dg).sum(-1, keepdim=True))
    else:
        m = z.amax(-1, keepdim=True).clamp(min=-3e38)
        every = torch.exp(z - m)
        every = (every / every.sum(-1, keepdim=True)).nan_to_num(0.0)
        p = torch.gather(every, -1, ids.clamp(min=0)).masked_fill(ids < 0, 0.0)
        d = p * dg
    dz = torch.zeros_like(z).scatter_add_(-1, ids.clamp(min=0), d)
    if mode == "softmax_all":
        dz -= every * d.sum(-1, keepdim=True)
    return dict(dlogits=(s["scale"] * dz).to(s["logits"].dtype))


def _sort_plain(s):
    E, ids = s["case"]["E"], s["topk"].reshape(-1).long()
    key = torch.where(ids < 0, E, ids)
    order = torch.sort(key, stable=True)[1].int()
    offsets = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0).int()
    offsets = torch.nn.functional.pad(offsets, (1, 0))
    dest = torch.empty_like(order)
    dest[order.long()] = torch.arange(len(order), dtype=torch.int32, device="cuda")
    dest = torch.where(ids < 0, -1, dest)
    pair = torch.where(torch.arange(len(order), device="cuda") < offsets[E], order, NONE)
    return dict(offsets=offsets, dest=dest.reshape(s["topk"].shape), pair=pair)


def _combine_backward_plain(s):
    T, H = s["case"]["T"], s["case"]["H"]
    dest, gates = s["dest"].reshape(T, -1).long(), s["gates"].reshape(T, -1)
    dout = s["dout"].reshape(T, H).float()
    dy, dgates = s["dy"], torch.zeros_like(gates)
    for k in range(dest.shape[1]):
        here = dest[:, k] >= 0
        row = dest[:, k].clamp(min=0)
        dgates[:, k] = (dout * s["y"][row].float()).sum(1).masked_fill(~here, 0.0)
        d = (gates[:, k, None] * dout).to(dy.dtype)
        if s["case"]["masked"]:
            dy = torch.cat((dy, dy[:1]))                        # a last row takes what is dropped
            dy[torch.where(here, row, len(s["dy"]))] = d
            dy = dy[: len(s["dy"])]
        else:
            dy[row] = d
    return dict(dy=dy, dgates=dgates.reshape(s["gates"].shape))


def _ffn_plain(s):
    T, K, E, H, I = (s["case"][k] for k in "TKEHI")
    x = _rounded_rows(s["x"].reshape(T, H).float())
    ids = s["topk"].reshape(-1)
    out = torch.zeros(T, H, device="cuda")
    order = torch.sort(ids, stable=True)[1]
    counts = torch.bincount(ids + 1, minlength=E + 1).tolist()
    begin, y = counts[0], torch.zeros(T * K, H, device="cuda")
    for e in range(E):
        pairs = order[begin:begin + counts[e + 1]]
        begin += len(pairs)
        if not len(pairs):
            continue
        gu = torch.matmul(x[pairs // K], _weights(s["w13"][e], s["w13_scale"][e], H, 2 * I))
        g, u = gu[:, :I], gu[:, I:]
        a = _rounded_rows(g / (1 + torch.exp(-g)) * u)
        y[pairs] = torch.matmul(a, _weights(s["w2"][e], s["w2_scale"][e], I, H))
    for k in range(K):
        out += s["gates"].reshape(T, K)[:, k, None] * y.reshape(T, K, H)[:, k]
    return out.bfloat16().reshape(1, T, H)


def _kept(s, name, make):
    """What a program makes once and keeps: dims and workspaces."""
    if name not in s:
        s[name] = make()
    return s[name]


def _run_own(s):
    import balanced_token_dispatch_moonep_amd as M

    def room(size):
        return lambda: torch.empty(size(), dtype=torch.uint8, device="cuda")

    case, op = s["case"], s["case"]["op"]
    T, E, K = case["T"], case["E"], case["K"]
    d = _kept(s, "dims", lambda: M.Dims.make(1, E, 0, T, K, case.get("H", 8), case.get("I", 0),
                                             f32_rows=op == "combine_backward" and case["dtype"] == "f32"))
    if op in ("route", "route_backward"):
        mode = dict(softmax=M.ROUTE_SOFTMAX, softmax_all=M.ROUTE_SOFTMAX_ALL, sigmoid=M.ROUTE_SIGMOID)[case["mode"]]
        if op == "route":
            M.moonep_route(d, s["logits"], s["bias"], s["topk"], s["gates"], mode, s["scale"])
            return dict(topk=s["topk"], gates=s["gates"])
        M.moonep_route_backward(d, s["dgates"], s["logits"], s["topk"], s["dlogits"], mode, s["scale"])
        return dict(dlogits=s["dlogits"])
    if op == "sort":
        ws = _kept(s, "ws", room(lambda: M.moonep_sort_workspace_bytes(d)))
        M.moonep_sort(d, s["topk"], ws, s["offsets"], s["dest"], s["pair"])
        return dict(offsets=s["offsets"], dest=s["dest"], pair=s["pair"])
    if op == "combine_backward":
        M.moonep_combine_backward(d, s["dest"], s["y"], s["gates"], s["dout"], s["dy"], s["dgates"])
        return dict(dy=s["dy"], dgates=s["dgates"])
    ws = _kept(s, "ws", room(lambda: M.moonep_fp8_ffn_workspace_bytes(d)))
    M.moonep_fp8_ffn(d, s["topk"], s["gates"], s["x"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], ws, s["out"])
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    return dict(route=_route_plain, route_backward=_route_backward_plain, sort=_sort_plain,
                combine_backward=_combine_backward_plain, ffn=_ffn_plain)[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    T, E, K, live = case["T"], case["E"], case["K"], case["T"] - case["masked"]
    if case["op"] in ("route", "route_backward"):
        b = T * E * (2 if case["dtype"] == "bf16" else 4)
        if case["op"] == "route":
            return dict(bytes=b + 8 * T * K + (4 * E if case["bias"] else 0), flops=T * E * 8)
        # only the gates over all experts need every logit
        read = b if case["mode"] == "softmax_all" else T * K * (2 if case["dtype"] == "bf16" else 4)
        return dict(bytes=b + read + 8 * T * K, flops=T * E * 4)
    if case["op"] == "sort":
        return dict(bytes=8 * T * K + 4 * live * K + 4 * (E + 1), flops=T * K * 4)
    if case["op"] == "combine_backward":
        b, H = 2 if case["dtype"] == "bf16" else 4, case["H"]
        return dict(bytes=b * H * (T + 2 * live * K) + 12 * T * K, flops=3 * live * K * H)
    H, I = case["H"], case["I"]
    read = E * (1 - (1 - K / E) ** live)        # experts that tokens pick, expected
    return dict(bytes=read * 3 * H * I * (1 + 1 / 16384) + 4 * T * H + 8 * T * K, flops=6 * H * I * live * K)


# ----------------------------------------------------------------------------
# the definitions, in 64 bits
# ----------------------------------------------------------------------------

def _exact_round(v):
    """What e4m3 makes of float64 values: steps of 2^-9 below 2^-6, else eight a power of two; halves to even."""
    e = (torch.frexp(v)[1] - 1).clamp(min=-6)
    step = torch.exp2((e - 3).double())
    return torch.round(v / step) * step


def _exact_rows(x):
    """Block by block along the row, by the smallest power of two that 448 of hold the largest."""
    out = torch.empty_like(x)
    for k in range(0, x.shape[1], BLOCK):
        b = x[:, k:k + BLOCK]
        top = b.abs().amax(1, keepdim=True)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 8
        e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(min=-126)
        out[:, k:k + BLOCK] = _exact_round(b / torch.exp2(e)) * torch.exp2(e)
    return out


def _exact_weight(codes, scales, Kin, N):
    """One matrix [Kin, N] in 64 bits, each code found by its place in the layout."""
    k = torch.arange(Kin, device=codes.device)[:, None]
    n = torch.arange(N, device=codes.device)[None, :]
    kb = (Kin + BLOCK - 1) // BLOCK
    v = codes[((n // 32) * kb + k // BLOCK) * 4096 + (k % BLOCK // 16) * 512 + (n % 32) * 16 + k % 16].int()
    e, m = v >> 3 & 15, (v & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 512)
    s = scales[(n // BLOCK) * (-(-kb // 4) * 4) + k // BLOCK].double()
    return torch.where(v >= 128, -mag, mag) * torch.exp2(s - 127)


def _exact_gates(z, ids, mode, scale):
    """Gates of the picked logits z [T, E] float64; ids < 0 have none."""
    at = ids.long().clamp(min=0)
    none = ids < 0
    if mode == "softmax_all":
        g = torch.gather(torch.softmax(z, -1), -1, at)
    else:
        w = torch.nn.functional.logsigmoid(z) if mode == "sigmoid" else z
        g = torch.softmax(torch.gather(w, -1, at).masked_fill(none, -math.inf), -1)
    return scale * g.masked_fill(none, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    T, E, K, op = case["T"], case["E"], case["K"], case["op"]
    if op in ("route", "route_backward"):
        z = s["logits"].reshape(T, E).double()
        if op == "route":
            key = torch.sigmoid(z) if case["mode"] == "sigmoid" else z.clone()
            key = (key + s["bias"].double() if case["bias"] else z).masked_fill(z == -math.inf, -math.inf)
            ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
            index = torch.arange(E, device="cuda")
            for k in range(K):
                top = key.amax(1, keepdim=True)
                best = torch.where(key == top, index, E).amin(1, keepdim=True)
                ids[:, k] = torch.where(top == -math.inf, -1, best)[:, 0]
                key.scatter_(1, best, -math.inf)
            gates = _exact_gates(z, ids, case["mode"], s["scale"])
            return dict(topk=ids.reshape(1, T, K), gates=gates.reshape(1, T, K))
        with torch.enable_grad():       # the gradient of the gates' own definition
            ids = s["topk"].reshape(T, K)
            fine = z.clamp(min=-1e4).requires_grad_(True)
            gates = _exact_gates(fine, ids, case["mode"], s["scale"])
            dz, = torch.autograd.grad(gates, fine, s["dgates"].reshape(T, K).double())
        return dict(dlogits=dz.nan_to_num(0.0).reshape(1, T, E))
    if op == "sort":
        # counting, expert by expert
        ids = s["topk"].reshape(-1)
        offsets, dest, pair = [0], torch.full_like(ids, -1), torch.full_like(ids, NONE)
        for e in range(E):
            p = (ids == e).nonzero()[:, 0].int()
            dest[p.long()] = offsets[-1] + torch.arange(len(p), dtype=torch.int32, device="cuda")
            pair[offsets[-1]:offsets[-1] + len(p)] = p
            offsets.append(offsets[-1] + len(p))
        return dict(offsets=torch.tensor(offsets, dtype=torch.int32), dest=dest.reshape(1, T, K), pair=pair)
    if op == "combine_backward":
        H = case["H"]
        dy = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
        dgates = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        t, k = (s["dest"][0] >= 0).nonzero(as_tuple=True)
        for i in range(0, len(t), 65536):
            ti, ki = t[i:i + 65536], k[i:i + 65536]
            row, d = s["dest"][0, ti, ki].long(), s["dout"][0, ti].double()
            dy[row] = s["gates"][0, ti, ki, None].double() * d
            dgates[ti, ki] = torch.linalg.vecdot(d, s["y"][row].double())
        return dict(dy=dy, dgates=dgates.reshape(1, T, K))
    H, I = case["H"], case["I"]
    x = _exact_rows(s["x"].reshape(T, H).double())
    ids, gates = s["topk"].reshape(T, K), s["gates"].reshape(T, K).double()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        gu = x[t] @ _exact_weight(s["w13"][e], s["w13_scale"][e], H, 2 * I)
        a = _exact_rows(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
        out.index_add_(0, t, gates[t, k, None] * (a @ _exact_weight(s["w2"][e], s["w2_scale"][e], I, H)))
    return out.reshape(1, T, H)
