"""Cases and plain forms of the operators on block-scaled 8-bit floating point (fp8):
quantising activation rows and weights and reading them back, the linear layer on
them, products grouped by expert (plain and gated), routing by scores, and the expert
layer that runs all of them.

fp8: e4m3 codes (bias 7, largest 448, no infinities) under fp32 scales.  An activation
scale belongs to 128 consecutive k of a row and is kept k-block-major, (ceil(K/128),
rows); a weight scale belongs to 128 rows by 128 k, (ceil(N/128), ceil(K/128)).  Blocks
at the end may be shorter.  With A = max(absmax, 448 * 2^-126) of a block the scale is
A / 448 and the codes are e4m3(448 y / A) to nearest, ties to even (the unrounded ratio
to the block's largest, so that ties are ties); a block that holds a NaN or an infinity
has the scale NaN and codes 0.  With a Hadamard rotation the rows are first transformed
per group of g values (signs, fast Walsh-Hadamard butterflies of distance 1, 2, 4, ...
in fp32, times 1/sqrt(g), signs).

Routing: an expert's score is the softmax over all experts or the sigmoid of its logit;
its choice value is the score plus a bias.  Experts lie in groups of equal size; a
group's value is its largest choice value, or the sum of its two largest.  The best
top_groups groups are kept, then the best k experts in them, ties to the lower index.
Weights are the scores (not the choice values), over their sum if renormalized, times
a factor.  -inf and NaN logits are never taken.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# What 8-bit codes made within a pass lead to is returned in 16 bits: the roundings before
# them move one value in a million over a code's border.
READ = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.bfloat16}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # the activations of a decode batch, rotated in groups of 64
        dict(name="quantize decode", op="quantize", M=32, K=3840, g=64, dtype="bf16"),
        # the activations of a long prompt before a down projection, not rotated
        dict(name="quantize prefill", op="quantize", M=8192, K=10240, g=0, dtype="bf16"),
        # a layer's weights, laid out when a model is loaded
        dict(name="quantize weights", op="weights", N=10240, K=3840, g=64, dtype="f32"),
        # one token through a projection: latency
        dict(name="linear one token", op="linear", M=1, K=3840, N=3840, g=64, dtype="bf16", bias=True),
        # a ragged batch, widths that no tile divides, single-precision activations, no rotation
        dict(name="linear ragged f32", op="linear", M=333, K=5392, N=7161, g=0, dtype="f32", bias=False),
        # prefill
        dict(name="linear prefill", op="linear", M=8192, K=3840, N=3840, g=0, dtype="bf16", bias=True),
        # a decode batch's rows over the experts: a few rows each, weights are the cost
        dict(name="grouped decode", op="grouped", T=32, k=4, E=32, K=3840, N=2560, skew=1.0, dtype="bf16", bias=True),
        # a prompt's rows over the experts through the gated up projection: ragged groups
        dict(name="gated prefill", op="gated", T=4099, k=4, E=32, K=3840, F=1280, skew=1.5, dtype="bf16", bias=False),
        # routing of a decode batch: softmax, no groups
        dict(name="route decode", op="route", T=32, E=128, k=8, groups=1, top_groups=1, best=1, scores="softmax",
             bias=False, renorm=True, scale=1.0, skew=1.0, dtype="bf16"),
        # routing of a prompt: sigmoid scores, a bias for balance, groups
        dict(name="route prefill", op="route", T=8192, E=256, k=8, groups=8, top_groups=4, best=2, scores="sigmoid",
             bias=True, renorm=True, scale=2.5, skew=1.0, dtype="f32"),
        # the whole expert layer: a small decode batch, and a prompt
        dict(name="experts decode", op="experts", T=16, k=4, E=32, K=3840, F=1280, groups=4, top_groups=2, best=2,
             scores="sigmoid", bias=True, renorm=True, scale=2.5, skew=1.0, g=0, dtype="bf16"),
        dict(name="experts prefill", op="experts", T=8192, k=4, E=32, K=3840, F=1280, groups=4, top_groups=2, best=2,
             scores="sigmoid", bias=True, renorm=True, scale=2.5, skew=1.0, g=64, dtype="bf16"),
    ]


def _size(rng, lo, hi, step=1):
    """A size of [lo, hi], a multiple of step, spread over the logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi:
            return v


def _routing(rng, E, k):
    """How a token's k of E experts are chosen; E is a multiple of 4."""
    groups = rng.choice([1, 1] + [n for n in (2, 4, 8, 16) if E % n == 0 and E // n >= 2])
    low = -(-k // (E // groups))   # groups that hold k experts
    scores = rng.choice(["softmax", "sigmoid"])
    return dict(groups=groups, top_groups=rng.randint(low, groups), best=rng.choice([1, 2]), scores=scores,
                bias=rng.random() < 0.6, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))


def draw(rng):
    op = rng.choice(["quantize", "weights", "linear", "linear", "grouped", "gated", "route", "route", "experts",
                     "experts"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    g = rng.choice([0, 0, 16, 32, 64, 128, 256])
    step = max(16, g)
    if op == "quantize":
        return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, step, 10240, step), g=g, dtype=dtype)
    if op == "linear":
        return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, step, 10240, step), N=_size(rng, 16, 3840), g=g,
                    dtype=dtype, bias=rng.random() < 0.5)
    if op == "weights":
        return dict(op=op, N=_size(rng, 16, 10240), K=_size(rng, step, 3840, step), g=g, dtype=dtype)
    skew = round(rng.uniform(0.0, 2.0), 2)
    if op == "route":
        E = _size(rng, 4, 512, 4)
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=_size(rng, 1, 8192), E=E, k=k, skew=skew, dtype=dtype, **_routing(rng, E, k))
    # rows, experts and widths together stay below the largest listed case
    E = _size(rng, 4, 48, 4)
    k = rng.randint(1, min(8, E))
    T = _size(rng, 1, 32768 // k if k > 4 else 8192)
    if op == "grouped":
        return dict(op=op, T=T, k=k, E=E, K=_size(rng, 16, 3840, 16), N=_size(rng, 16, 2560), skew=skew, dtype=dtype,
                    bias=rng.random() < 0.5)
    if op == "gated":
        return dict(op=op, T=T, k=k, E=E, K=_size(rng, 16, 3840, 16), F=_size(rng, 128, 1280, 128), skew=skew,
                    dtype=rng.choice(["bf16", "f16"]), bias=rng.random() < 0.5)
    return dict(op=op, T=T, k=k, E=E, K=_size(rng, max(64, step), 3840, step), F=_size(rng, 128, 1280, 128), skew=skew,
                g=g, dtype=rng.choice(["bf16", "f16"]), **_routing(rng, E, k))


def work(case):
    op, xb = case["op"], 4 if case["dtype"] == "f32" else 2
    act, wt = 1 + 4 / 128, 1 + 4 / 16384   # bytes of an fp8 value with its scale
    if op in ("quantize", "weights"):
        n, f = case["K"] * case["M" if op == "quantize" else "N"], act if op == "quantize" else wt
        # in, codes and scales out, in again, values out
        return dict(bytes=n * (xb + 2 + 2 * f), flops=n * (math.log2(case["g"]) if case["g"] else 1))
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return dict(bytes=M * K * xb + N * K * wt + M * N * 2, flops=2 * M * N * K)
    T, k, E = case["T"], case["k"], case["E"]
    if op == "route":
        return dict(bytes=T * E * xb + T * k * 16 + 8 * E, flops=T * E * 8)
    R, live, K = T * k, min(E, T * k), case["K"]
    if op == "grouped":
        N = case["N"]
        return dict(bytes=T * K * act + live * N * K * wt + R * N * xb, flops=2 * R * N * K)
    F = case["F"]
    if op == "gated":
        # the values go out in fp8, come in again and leave in 16 bits
        return dict(bytes=T * K * act + live * 2 * F * K * wt + R * F * (2 * act + xb), flops=4 * R * F * K)
    return dict(bytes=2 * T * K * xb + T * E * 4 + live * 3 * F * K * wt, flops=6 * R * K * F)


# ---- the plain forms: elementary operations in 32 bits -----------------------

def _rotate(x, g, sign_in, sign_out):
    """Rows of x (fp32) times diag(sign_in) H_g diag(sign_out) / sqrt(g) per group of g."""
    if not g:
        return x
    v = x.reshape(-1, g) * sign_in
    d = 1
    while d < g:
        v = v.reshape(-1, g // (2 * d), 2, d)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), 2)
        d *= 2
    v = v.reshape(-1, g) * torch.tensor(1.0 / math.sqrt(g), dtype=torch.float32, device=x.device) * sign_out
    return v.reshape(x.shape)


def _codes(b, amax):
    """(e4m3 codes, scales) of blocks b with the largest magnitudes amax (fp32, broadcastable)."""
    bad = ~(amax < math.inf)
    top = amax.clamp(min=448 * 2.0 ** -126)
    c = torch.where(bad, 0.0, b * 448 / top).to(torch.float8_e4m3fn)
    return c, torch.where(bad, math.nan, top / 448)


def _quantize(y):
    """fp32 rows -> (codes (rows, K), scales (blocks, rows))."""
    K = y.shape[-1]
    b = torch.nn.functional.pad(y, (0, -K % 128)).reshape(y.shape[0], -1, 128)
    c, s = _codes(b, b.abs().amax(-1, keepdim=True))
    return c.reshape(y.shape[0], -1)[:, :K].contiguous(), s.squeeze(-1).t().contiguous()


def _quantize_weights(w):
    """fp32 (..., N, K) -> (codes (..., N, K), scales (..., blocks of N, blocks of K))."""
    N, K = w.shape[-2:]
    p = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    b = p.reshape(*w.shape[:-2], p.shape[-2] // 128, 128, p.shape[-1] // 128, 128)
    c, s = _codes(b, b.abs().amax((-3, -1), keepdim=True))
    return c.reshape(p.shape)[..., :N, :K].contiguous(), s.squeeze(-1).squeeze(-2).contiguous()


def _values(codes, scales):
    """(rows, K) codes, (blocks, rows) scales -> the fp32 values they stand for."""
    return codes.float() * scales.t().repeat_interleave(128, 1)[:, :codes.shape[1]]


def _weight_values(codes, scales):
    N, K = codes.shape[-2:]
    return codes.float() * scales.repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]


def _route(logits, c, bias):
    """Scores and choices in 64 bits: two that are close must not change places."""
    T, E = logits.shape
    k, G, device = c["k"], c["groups"], logits.device
    l = logits.double()
    live = l > -math.inf
    if c["scores"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        top = torch.where(live, l, -math.inf).amax(1, keepdim=True)
        e = torch.where(live, torch.where(l == top, 1.0, torch.exp(l - top)), 0.0)
        s = e / e.sum(1, keepdim=True)
    s = torch.where(live, s, 0.0)
    value = s if bias is None else s + bias.double()
    order = torch.where(live, l if bias is None else value, -math.inf)   # without a bias the scores' order is the logits'
    if G > 1:
        of = order if c["best"] == 1 else torch.where(live, value, -math.inf)
        two = torch.sort(of.reshape(T, G, E // G), dim=2, descending=True)[0][:, :, :c["best"]]
        worth = torch.where(two[:, :, 0] > -math.inf, torch.where(two > -math.inf, two, 0.0).sum(2), -math.inf)
        kept = torch.sort(worth, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        member = torch.zeros(T, G, dtype=torch.bool, device=device)
        member[torch.arange(T, device=device).unsqueeze(1), kept] = True
        order = torch.where(member.repeat_interleave(E // G, 1), order, -math.inf)
    val, idx = torch.sort(order, dim=1, descending=True, stable=True)
    idx, taken = idx[:, :k], val[:, :k] > -math.inf
    w = torch.where(taken, s.gather(1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    w = (w * c["scale"]).float()
    experts = torch.where(taken, idx, -1).to(torch.int32)
    key = torch.where(taken, idx, E).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=device).scatter_add(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
    perm = torch.sort(key, stable=True)[1]
    at = torch.arange(T * k, device=device)
    routed = at < offsets[E]
    rows = torch.where(routed, perm // k, -1).to(torch.int32)
    pos = torch.empty_like(perm)
    pos[perm] = torch.where(routed, at, -1)
    return dict(weights=w, experts=experts, rows=rows, pos=pos.reshape(T, k).to(torch.int32), offsets=offsets)


def _grouped(a, w, offsets, rows, cap):
    """a[rows[i]] times the transpose of w[e] for offsets[e] <= i < offsets[e+1]: every
    expert's rows in a slab of `cap`, one batched product."""
    E = w.shape[0]
    i = torch.arange(rows.numel(), device=a.device)
    e = (i.unsqueeze(1) >= offsets[1:].unsqueeze(0)).sum(1)
    live = e < E
    slot = torch.where(live, e * cap + i - offsets[e.clamp(max=E - 1)], E * cap)
    x = a.new_zeros(E * cap + 1, a.shape[1])
    x[slot] = torch.where(live.unsqueeze(1), a[rows.clamp(min=0)], 0)
    y = torch.bmm(x[:-1].reshape(E, cap, -1), w.transpose(1, 2).contiguous()).reshape(E * cap, -1)
    return torch.where(live.unsqueeze(1), y[slot.clamp(max=E * cap - 1)], 0), e.clamp(max=E - 1), live


# ---- inputs ------------------------------------------------------------------

def _activations(rows, K, dtype, gen):
    """Normal rows with one channel in a hundred twenty times as large."""
    x = torch.randn(rows, K, device="cuda", generator=gen)
    x *= torch.where(torch.rand(K, device="cuda", generator=gen) < 0.01, 20.0, 1.0)
    return x.to(DTYPES[dtype])


def _weights(shape, gen):
    return _quantize_weights(torch.randn(*shape, device="cuda", generator=gen) * shape[-1] ** -0.5)


def _logits(case, gen, dtype):
    """Normal logits; experts differ in popularity by `skew`; one token in sixteen has masked
    experts, and every 61st token is padding, with nothing left."""
    T, E = case["T"], case["E"]
    l = torch.randn(T, E, device="cuda", generator=gen) + case["skew"] * torch.randn(E, device="cuda", generator=gen)
    t = torch.arange(T, device="cuda").unsqueeze(1)
    l = torch.where((t % 16 == 5) & (torch.rand(T, E, device="cuda", generator=gen) < 0.5), -math.inf, l)
    return torch.where(t % 61 == 60, -math.inf, l).to(DTYPES[dtype])


PLAIN_ROUTING = dict(groups=1, top_groups=1, best=1, scores="softmax", renorm=True, scale=1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], case["dtype"]
    s = dict(case=dict(case))
    if case.get("g"):
        for name in ("sign_in", "sign_out"):
            s[name] = (torch.randint(0, 2, (case["g"],), device="cuda", generator=gen) * 2 - 1).to(torch.int8)
    if op in ("quantize", "linear"):
        s["x"] = _activations(case["M"], case["K"], dtype, gen)
        if op == "linear":
            s["w"] = _weights((case["N"], case["K"]), gen)
            s["bias"] = torch.randn(case["N"], device="cuda", generator=gen).to(DTYPES[dtype]) if case["bias"] else None
        return s
    if op == "weights":
        s["x"] = (torch.randn(case["N"], case["K"], device="cuda", generator=gen) * case["K"] ** -0.5).to(DTYPES[dtype])
        return s
    E = case["E"]
    s["logits"] = _logits(case, gen, dtype if op == "route" else "f32")
    # what balancing has added to the experts' choice values
    s["balance"] = 0.1 * torch.randn(E, device="cuda", generator=gen) if op in ("route", "experts") and case["bias"] else None
    if op == "route":
        return s
    K = case["K"]
    r = _route(s["logits"], case if op == "experts" else dict(PLAIN_ROUTING, k=case["k"]), s["balance"])
    # rows a batched plain product has to make room for, per expert
    s["cap"] = max(1, int((r["offsets"][1:] - r["offsets"][:-1]).max()))
    if op == "experts":
        s["x"] = _activations(case["T"], K, dtype, gen)
        s["w13"] = _weights((E, 2 * case["F"], K), gen)
        s["w2"] = _weights((E, K, case["F"]), gen)
        return s
    N = case["N"] if op == "grouped" else 2 * case["F"]
    s["a"] = _quantize(_activations(case["T"], K, dtype, gen).float())
    s["w"] = _weights((E, N, K), gen)
    s["bias"] = torch.randn(E, N, device="cuda", generator=gen).to(DTYPES[dtype]) if case["bias"] else None
    s["offsets"], s["rows"] = r["offsets"], r["rows"]
    return s


# ---- one pass ----------------------------------------------------------------

def _run_own(s):
    import bit_quantized_linear_rotate_amd as w4
    c = s["case"]
    op, dtype = c["op"], DTYPES[c["dtype"]]
    h = w4.Hadamard(c["g"], s["sign_in"], s["sign_out"]) if c.get("g") else None
    if op == "quantize":
        codes, scales = w4.w8a8_quantize_fp8(s["x"], h)
        return w4.w8a8_dequantize_fp8(codes, scales, READ[c["dtype"]])
    if op == "weights":
        codes, scales = w4.w8a8_quantize_weights_fp8(s["x"], h)
        return w4.w8a8_dequantize_weights_fp8(codes, scales, READ[c["dtype"]])
    if op == "linear":
        return w4.w8a8_linear_fp8(s["x"], *s["w"], h=h, bias=s["bias"], out_dtype=READ[c["dtype"]])
    if op == "grouped":
        return w4.w8a8_grouped_gemm_fp8(*s["a"], *s["w"], s["offsets"], rows=s["rows"], bias=s["bias"], out_dtype=dtype)
    if op == "gated":
        codes, scales = w4.w8a8_grouped_gated_fp8(*s["a"], *s["w"], s["offsets"], rows=s["rows"], bias=s["bias"])
        return w4.w8a8_dequantize_fp8(codes, scales, dtype)
    routing = dict(scores=c["scores"], bias=s["balance"], groups=c["groups"], top_groups=c["top_groups"],
                   group_best=c["best"], renormalize=c["renorm"], scale=c["scale"])
    if op == "route":
        weights, experts, rows, pos, offsets = w4.w4a4_route_experts_scored(s["logits"], c["k"], **routing)
        return dict(weights=weights, experts=experts, rows=rows, pos=pos, offsets=offsets)
    return w4.w8a8_experts_fp8(s["x"], s["logits"], c["k"], *s["w13"], *s["w2"], h=h, **routing)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, dtype = c["op"], DTYPES[c["dtype"]]
    if op == "route":
        return _route(s["logits"], c, s["balance"])
    if op in ("grouped", "gated"):
        y, e, live = _grouped(_values(*s["a"]), _weight_values(*s["w"]), s["offsets"], s["rows"], s["cap"])
        if s["bias"] is not None:
            y = torch.where(live.unsqueeze(1), y + s["bias"].float()[e], 0)
        if op == "grouped":
            return y.to(dtype)
        gate, up = y[:, :c["F"]], y[:, c["F"]:]
        return _values(*_quantize(gate / (1 + torch.exp(-gate)) * up)).to(dtype)
    y = _rotate(s["x"].float(), c["g"], s.get("sign_in"), s.get("sign_out"))
    if op == "weights":
        return _weight_values(*_quantize_weights(y)).to(READ[c["dtype"]])
    a = _values(*_quantize(y))
    if op == "quantize":
        return a.to(READ[c["dtype"]])
    if op == "linear":
        y = a @ _weight_values(*s["w"]).t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(READ[c["dtype"]])
    r = _route(s["logits"], c, s["balance"])
    F = c["F"]
    y, _, _ = _grouped(a, _weight_values(*s["w13"]), r["offsets"], r["rows"], s["cap"])
    gate, up = y[:, :F], y[:, F:]
    act = _values(*_quantize(gate / (1 + torch.exp(-gate)) * up))
    y, _, _ = _grouped(act, _weight_values(*s["w2"]), r["offsets"], torch.arange(act.shape[0], device=act.device),
                       s["cap"])
    picked = torch.where((r["pos"] >= 0).unsqueeze(2), y[r["pos"].clamp(min=0)], 0)
    return (picked * r["weights"].unsqueeze(2)).sum(1).to(dtype)


# ---- the definition in 64 bits -----------------------------------------------

def _exact_e4m3(v):
    """The e4m3 value nearest to v (float64), the even one on a tie."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -6))     # 2^(e - 1) <= |v| < 2^e
    step = torch.ldexp(torch.ones_like(v), e - 4)         # eight steps to a power of two
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_blocks(y, rows):
    """The fp8 value of every element of y (float64) with one scale per `rows` x 128."""
    out = torch.empty_like(y)
    for k0 in range(0, y.shape[1], 128):
        b = y[:, k0:k0 + 128]
        amax = b.abs().amax(1)
        pad = torch.nn.functional.pad(amax, (0, -amax.numel() % rows))
        amax = pad.reshape(-1, rows).amax(1).repeat_interleave(rows)[:amax.numel()].unsqueeze(1)
        amax = amax.clamp(min=448 * 2.0 ** -126)
        out[:, k0:k0 + 128] = _exact_e4m3(b * 448 / amax) * amax / 448
    return out


def _exact_hadamard(x, g, sign_in, sign_out):
    if not g:
        return x.double()
    i = torch.arange(g, device=x.device)
    bits = i.unsqueeze(0) & i.unsqueeze(1)
    parity = sum((bits >> b) & 1 for b in range(8)) % 2
    R = sign_in.double().unsqueeze(1) * (1.0 - 2.0 * parity.double()) * sign_out.double() / math.sqrt(g)
    return (x.double().reshape(-1, g) @ R).reshape(x.shape)


def _exact_code_values(codes):
    n = codes.view(torch.uint8).int()
    e, m = (n >> 3) & 15, (n & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(1 + m / 8, e - 7))
    return torch.where(n >= 128, -v, v)


def _exact_rows(codes, scales):
    kb = torch.arange(codes.shape[1], device=codes.device) // 128
    return _exact_code_values(codes) * scales.double()[kb].t()


def _exact_weights(codes, scales):
    n, k = (torch.arange(v, device=codes.device) // 128 for v in codes.shape)
    return _exact_code_values(codes) * scales.double()[n][:, k]


def _exact_route(logits, c, bias):
    """(expert ids, weights) of each token, groups and experts taken one at a time."""
    T, E = logits.shape
    G, l = c["groups"], logits.double()
    dead = ~(l > -math.inf)
    if c["scores"] == "sigmoid":
        s = torch.special.expit(l)
    else:
        s = torch.softmax(torch.where(dead, -math.inf, l), 1)
    s = torch.where(dead, 0.0, s)
    v = s + (0.0 if bias is None else bias.double())
    left = torch.where(dead, -math.inf, l if bias is None else v)
    if G > 1:
        of = torch.where(dead, -math.inf, v).reshape(T, G, E // G)
        first = of.max(2)
        worth = first.values
        if c["best"] == 2:
            second = of.scatter(2, first.indices.unsqueeze(2), -math.inf).amax(2)
            worth = worth + torch.where(second > -math.inf, second, 0.0)
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        for _ in range(c["top_groups"]):
            at = torch.where(keep, -math.inf, worth)
            at = torch.where(~keep & (at == at.amax(1, keepdim=True)), 1, 0).argmax(1, keepdim=True)
            keep.scatter_(1, at, True)
        left = torch.where(keep.unsqueeze(2), left.reshape(T, G, E // G), -math.inf).reshape(T, E)
    ids, ws = [], []
    for _ in range(c["k"]):
        top = left.amax(1, keepdim=True)
        first = (left == top).double().argmax(1, keepdim=True)
        none = top == -math.inf
        ids.append(torch.where(none, -1, first))
        ws.append(torch.where(none, 0.0, s.gather(1, first)))
        left = left.scatter(1, first, -math.inf)
    ids, ws = torch.cat(ids, 1), torch.cat(ws, 1)
    if c["renorm"]:
        total = ws.sum(1, keepdim=True)
        ws = torch.where(total > 0, ws / total, 0.0)
    return ids, ws * c["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return dict(weights=_exact_route(s["logits"], case, s["balance"])[1], experts=None, rows=None, pos=None,
                    offsets=None)
    if op in ("grouped", "gated"):
        a = _exact_rows(*s["a"])
        out = torch.zeros(case["T"] * case["k"], s["w"][0].shape[1], dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(case["E"]):
            at = slice(off[e], off[e + 1])
            out[at] = a[s["rows"][at].long()] @ _exact_weights(s["w"][0][e], s["w"][1][e]).t()
            if s["bias"] is not None:
                out[at] += s["bias"][e].double()
        if op == "grouped":
            return out
        gate, up = out[:, :case["F"]], out[:, case["F"]:]
        return _exact_blocks(gate * torch.sigmoid(gate) * up, 1)
    y = _exact_hadamard(s["x"], case["g"], s.get("sign_in"), s.get("sign_out"))
    if op == "weights":
        return _exact_blocks(y, 128)
    a = _exact_blocks(y, 1)
    if op == "quantize":
        return a
    if op == "linear":
        out = a @ _exact_weights(*s["w"]).t()
        return out if s["bias"] is None else out + s["bias"].double()
    ids, weights = _exact_route(s["logits"], case, s["balance"])
    F = case["F"]
    out = torch.zeros(case["T"], case["K"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        y = a[t] @ _exact_weights(s["w13"][0][e], s["w13"][1][e]).t()
        gate, up = y[:, :F], y[:, F:]
        y = _exact_blocks(gate * torch.sigmoid(gate) * up, 1) @ _exact_weights(s["w2"][0][e], s["w2"][1][e]).t()
        out.index_add_(0, t, y * weights[t, j].unsqueeze(1))
    return out
