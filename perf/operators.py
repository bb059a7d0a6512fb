"""Cases and plain forms of the microscaled 4-bit (MX4) operators: quantising activation
rows and reading them back, the linear layer on them, products grouped by expert,
routing, and the expert layer that runs all of them.

MX4: 32 consecutive k of a row share a power-of-two scale 2^X, X = floor(log2 absmax) - 2
(at least -127), and hold e2m1 elements rounded to nearest (ties to even).  Codes are
(rows, K/2) bytes, even k in the low nibble.  Scale bytes X + 127 are kept in slabs of
256 k: (ceil(K/256), rows, 8), unused bytes zero.  With a Hadamard rotation the rows are
first transformed per group of g values (signs, fast Walsh-Hadamard butterflies of
distance 1, 2, 4, ... in fp32, times 1/sqrt(g), signs).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # the activations of a decode batch, rotated in groups of 64
        dict(name="quantize decode", op="quantize", M=32, K=3840, g=64, dtype="bf16"),
        # the activations of a long prompt or a large image
        dict(name="quantize prefill", op="quantize", M=8192, K=3840, g=64, dtype="bf16"),
        # one token through a projection: latency
        dict(name="linear one token", op="linear", M=1, K=3840, N=3840, g=64, dtype="bf16", bias=True),
        # a ragged batch through a wide output projection, single-precision activations, no rotation
        dict(name="linear ragged f32", op="linear", M=333, K=5376, N=7168, g=0, dtype="f32", bias=False),
        # prefill
        dict(name="linear prefill", op="linear", M=8192, K=3840, N=3840, g=64, dtype="bf16", bias=False),
        # the down projection of a feed-forward layer: long K
        dict(name="linear wide K", op="linear", M=8192, K=10240, N=3840, g=256, dtype="f16", bias=True),
        # a decode batch's rows over the experts: one or two rows each, weights are the cost
        dict(name="grouped decode", op="grouped", T=32, k=4, E=32, K=3840, N=2560, skew=1.0, dtype="bf16", bias=True),
        # a prompt's rows over the experts: ragged groups, some of them empty
        dict(name="grouped prefill", op="grouped", T=4099, k=4, E=32, K=3840, N=2560, skew=1.5, dtype="f16", bias=False),
        # routing of a decode batch and of a prompt
        dict(name="route decode", op="route", T=32, E=32, k=4, skew=1.0, dtype="f32", renorm=True),
        dict(name="route prefill", op="route", T=8192, E=128, k=8, skew=1.0, dtype="bf16", renorm=False),
        # the whole expert layer: a small decode batch, and a prompt
        dict(name="experts decode", op="experts", T=16, k=4, E=32, K=3840, F=1280, skew=1.0, g=64, dtype="bf16"),
        dict(name="experts prefill", op="experts", T=8192, k=4, E=32, K=3840, F=1280, skew=1.0, g=64, dtype="bf16"),
    ]


def _size(rng, lo, hi, step=1):
    """A size of [lo, hi], a multiple of step, spread over the logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v not in (1536, 3072):
            return v


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "grouped", "grouped", "route", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    g = rng.choice([0, 16, 32, 64, 128, 256])
    step = max(32, g)
    if op == "quantize":
        return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, step, 10240, step), g=g, dtype=dtype)
    if op == "linear":
        return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, step, 10240, step), N=_size(rng, 16, 3840), g=g,
                    dtype=dtype, bias=rng.random() < 0.5)
    E = _size(rng, 4, 128)
    k = rng.randint(1, min(8, E))
    T = _size(rng, 1, 8192)
    skew = round(rng.uniform(0.0, 2.0), 2)
    if op == "route":
        return dict(op=op, T=T, E=E, k=k, skew=skew, dtype=dtype, renorm=rng.random() < 0.5)
    # rows, experts and widths together stay below the largest listed case
    E, T = min(E, 64), max(1, min(T, 32768 // k))
    k = min(k, E)
    if op == "grouped":
        return dict(op=op, T=T, k=k, E=E, K=_size(rng, 64, 3840, 32), N=_size(rng, 32, 2560), skew=skew, dtype=dtype,
                    bias=rng.random() < 0.5)
    K = _size(rng, max(64, step), 3840, step)
    return dict(op=op, T=T, k=k, E=E, K=K, F=_size(rng, 32, 1280, 32), skew=skew, g=g,
                dtype=rng.choice(["bf16", "f16"]))


def work(case):
    op, xb = case["op"], 4 if case["dtype"] == "f32" else 2
    mx = 17 / 32  # bytes of an MX4 value
    if op == "quantize":
        n = case["M"] * case["K"]
        # in, codes and scales out, in again, values out
        return dict(bytes=n * (2 * xb + 2 * mx), flops=n * (math.log2(case["g"]) if case["g"] else 1))
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return dict(bytes=M * K * xb + N * K * mx + M * N * xb, flops=2 * M * N * K)
    T, k, E = case["T"], case["k"], case["E"]
    if op == "route":
        return dict(bytes=T * E * xb + T * k * 16 + 4 * E, flops=T * E * 4)
    R, live = T * k, min(E, T * k)
    if op == "grouped":
        K, N = case["K"], case["N"]
        return dict(bytes=T * K * mx + live * N * K * mx + R * N * xb, flops=2 * R * N * K)
    K, F = case["K"], case["F"]
    return dict(bytes=2 * T * K * xb + T * E * 4 + live * 3 * F * K * mx, flops=6 * R * K * F)


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


def _pow2(n):
    """2^n in fp32 for integers n of [-127, 127], exactly."""
    return torch.where(n > -127, (n + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize(y):
    """fp32 rows -> (codes, scales in slabs); leading dimensions are kept."""
    K = y.shape[-1]
    b = y.reshape(*y.shape[:-1], K // 32, 32)
    amax = b.abs().amax(-1)
    X = ((amax.view(torch.int32) >> 23) - 129).clamp(min=-127)
    v = b.abs() * _pow2(-X).unsqueeze(-1)
    c = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    bad = ~(amax < math.inf)
    c = torch.where(bad.unsqueeze(-1), 0, c | (torch.signbit(b).to(torch.uint8) << 3)).reshape(*y.shape[:-1], K // 2, 2)
    s = torch.where(bad, 255, X + 127).to(torch.uint8)
    s = torch.nn.functional.pad(s, (0, -(K // 32) % 8))
    s = s.reshape(*s.shape[:-1], -1, 8).transpose(-3, -2).contiguous()
    return c[..., 0] | (c[..., 1] << 4), s


def _values(codes, scales):
    """(codes, scales in slabs) -> the fp32 values they stand for."""
    K = codes.shape[-1] * 2
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).int()].reshape(*codes.shape[:-1], K // 32, 32)
    s = scales.transpose(-3, -2).reshape(*codes.shape[:-1], -1)[..., :K // 32].int()
    f = torch.where(s == 255, math.nan, _pow2(s.clamp(max=254) - 127))
    return (v * f.unsqueeze(-1)).reshape(*codes.shape[:-1], K)


def _route(logits, k, renorm):
    l = logits.float()
    l = torch.where(l.isnan(), -math.inf, l)
    T, E = l.shape
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    live = val > -math.inf
    top = torch.where(live[:, :1], val[:, :1], 0)
    e = torch.where(live, torch.exp(val - top), 0)
    total = e.sum(1, keepdim=True) if renorm else torch.exp(l - top).sum(1, keepdim=True)
    w = torch.where(live, e / torch.where(live[:, :1], total, 1), 0)
    experts = torch.where(live, idx, -1).to(torch.int32)
    key = torch.where(live, idx, E).reshape(-1)
    counts = (key.unsqueeze(0) == torch.arange(E, device=l.device).unsqueeze(1)).sum(1)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0))).to(torch.int32)
    order = torch.sort(key, stable=True)[1]
    at = torch.arange(T * k, device=l.device)
    routed = at < offsets[E]
    rows = torch.where(routed, order // k, -1).to(torch.int32)
    pos = torch.empty_like(order)
    pos[order] = torch.where(routed, at, -1)
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
    return _quantize(torch.randn(*shape, device="cuda", generator=gen) * shape[-1] ** -0.5)


def _logits(case, gen, dtype):
    """Normal logits; experts differ in popularity by `skew`; one token in sixteen has masked
    experts, and every 61st token is padding, with nothing left."""
    T, E = case["T"], case["E"]
    l = torch.randn(T, E, device="cuda", generator=gen) + case["skew"] * torch.randn(E, device="cuda", generator=gen)
    t = torch.arange(T, device="cuda").unsqueeze(1)
    l = torch.where((t % 16 == 5) & (torch.rand(T, E, device="cuda", generator=gen) < 0.5), -math.inf, l)
    return torch.where(t % 61 == 60, -math.inf, l).to(DTYPES[dtype])


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
    s["logits"] = _logits(case, gen, dtype if op == "route" else "f32")
    if op == "route":
        return s
    E, K = case["E"], case["K"]
    r = _route(s["logits"], case["k"], True)
    # rows a batched plain product has to make room for, per expert
    s["cap"] = max(1, int((r["offsets"][1:] - r["offsets"][:-1]).max()))
    if op == "grouped":
        s["a"] = _quantize(_activations(case["T"], K, dtype, gen).float())
        s["w"] = _weights((E, case["N"], K), gen)
        s["bias"] = torch.randn(E, case["N"], device="cuda", generator=gen).to(DTYPES[dtype]) if case["bias"] else None
        s["offsets"], s["rows"] = r["offsets"], r["rows"]
    else:
        s["x"] = _activations(case["T"], K, dtype, gen)
        s["w13"] = _weights((E, 2 * case["F"], K), gen)
        s["w2"] = _weights((E, K, case["F"]), gen)
    return s


# ---- one pass ----------------------------------------------------------------

def _run_own(s):
    import bit_quantized_linear_rotate_amd as w4
    c = s["case"]
    op, dtype = c["op"], DTYPES[c["dtype"]]
    h = w4.Hadamard(c["g"], s["sign_in"], s["sign_out"]) if c.get("g") else None
    if op == "quantize":
        codes, scales = w4.w4a4_quantize_mx4(s["x"], h)
        return w4.w4a4_dequantize_mx4(codes, scales, dtype)
    if op == "linear":
        return w4.w4a4_linear_mx4(s["x"], *s["w"], h=h, bias=s["bias"])
    if op == "grouped":
        return w4.w4a4_grouped_gemm_mx4(*s["a"], *s["w"], s["offsets"], rows=s["rows"], bias=s["bias"], out_dtype=dtype)
    if op == "route":
        weights, experts, rows, pos, offsets = w4.w4a4_route_experts(s["logits"], c["k"], renormalize=c["renorm"])
        return dict(weights=weights, experts=experts, rows=rows, pos=pos, offsets=offsets)
    return w4.w4a4_experts_mx4(s["x"], s["logits"], c["k"], *s["w13"], *s["w2"], h=h)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, dtype = c["op"], DTYPES[c["dtype"]]
    if op == "route":
        return _route(s["logits"], c["k"], c["renorm"])
    if op == "grouped":
        y, e, live = _grouped(_values(*s["a"]), _values(*s["w"]), s["offsets"], s["rows"], s["cap"])
        if s["bias"] is not None:
            y = torch.where(live.unsqueeze(1), y + s["bias"].float()[e], 0)
        return y.to(dtype)
    a = _values(*_quantize(_rotate(s["x"].float(), c["g"], s.get("sign_in"), s.get("sign_out"))))
    if op == "quantize":
        return a.to(dtype)
    if op == "linear":
        y = a @ _values(*s["w"]).t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(dtype)
    r = _route(s["logits"], c["k"], True)
    F, K = c["F"], c["K"]
    y, _, _ = _grouped(a, _values(*s["w13"]), r["offsets"], r["rows"], s["cap"])
    gate, up = y[:, :F], y[:, F:]
    act = _values(*_quantize(gate / (1 + torch.exp(-gate)) * up))
    y, _, _ = _grouped(act, _values(*s["w2"]), r["offsets"], torch.arange(act.shape[0], device=act.device), s["cap"])
    picked = torch.where((r["pos"] >= 0).unsqueeze(2), y[r["pos"].clamp(min=0)], 0)
    return (picked * r["weights"].unsqueeze(2)).sum(1).to(dtype)


# ---- the definition in 64 bits -----------------------------------------------

def _exact_pow2(n):
    return ((n + 1023) << 52).view(torch.float64)


def _exact_grid(y):
    """The MX4 value of every element of y (float64), from the definition: the nearest of the
    block's sixteen values, the even code on a tie."""
    b = y.double().reshape(*y.shape[:-1], y.shape[-1] // 32, 32)
    amax = b.abs().max(-1, keepdim=True).values
    step = _exact_pow2(((amax.view(torch.int64) >> 52) - 1025).clamp(min=-127))
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=y.device)
    mag = b.abs() / step
    hi = torch.searchsorted(steps, mag.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dhi, dlo = steps[hi] - mag, mag - steps[lo]
    pick = torch.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(mag >= 6, 7, pick)
    return (torch.copysign(steps[pick], b) * step).reshape(y.shape)


def _exact_hadamard(x, g, sign_in, sign_out):
    if not g:
        return x.double()
    i = torch.arange(g, device=x.device)
    bits = i.unsqueeze(0) & i.unsqueeze(1)
    parity = sum((bits >> b) & 1 for b in range(8)) % 2
    R = sign_in.double().unsqueeze(1) * (1.0 - 2.0 * parity.double()) * sign_out.double() / math.sqrt(g)
    return (x.double().reshape(-1, g) @ R).reshape(x.shape)


def _exact_values(codes, scales):
    rows, K = codes.shape[0], codes.shape[1] * 2
    n = torch.empty(rows, K, dtype=torch.int64, device=codes.device)
    n[:, 0::2], n[:, 1::2] = codes.long() % 16, codes.long() // 16
    e, m = (n % 8) // 2, n % 2
    v = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * _exact_pow2(e - 1))
    kb = torch.arange(K, device=codes.device) // 32
    return v * (1.0 - 2.0 * (n // 8)) * _exact_pow2(scales[kb // 8, :, kb % 8].t().long() - 127)


def _exact_route(logits, k, renorm):
    """(expert ids, weights) of each token, the experts taken one at a time."""
    l = logits.double()
    left, ids, ws = l.clone(), [], []
    p = torch.exp(l - l.max(1, keepdim=True).values.clamp(min=-1e300))
    for _ in range(k):
        best = left.max(1, keepdim=True).values
        first = (left == best).double().argmax(1, keepdim=True)
        dead = best == -math.inf
        ids.append(torch.where(dead, -1, first))
        ws.append(torch.where(dead, 0.0, p.gather(1, first)))
        left = left.scatter(1, first, -math.inf)
    ids, ws = torch.cat(ids, 1), torch.cat(ws, 1)
    total = ws.sum(1, keepdim=True) if renorm else p.sum(1, keepdim=True)
    return ids, torch.where(total > 0, ws / total, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return dict(weights=_exact_route(s["logits"], case["k"], case["renorm"])[1], experts=None, rows=None, pos=None,
                    offsets=None)
    if op == "grouped":
        a, out = _exact_values(*s["a"]), torch.zeros(case["T"] * case["k"], case["N"], dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(case["E"]):
            at = slice(off[e], off[e + 1])
            out[at] = a[s["rows"][at].long()] @ _exact_values(s["w"][0][e], s["w"][1][e]).t()
            if s["bias"] is not None:
                out[at] += s["bias"][e].double()
        return out
    a = _exact_grid(_exact_hadamard(s["x"], case["g"], s.get("sign_in"), s.get("sign_out")))
    if op == "quantize":
        return a
    if op == "linear":
        out = a @ _exact_values(*s["w"]).t()
        return out if s["bias"] is None else out + s["bias"].double()
    ids, weights = _exact_route(s["logits"], case["k"], True)
    out = torch.zeros(case["T"], case["K"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        y = a[t] @ _exact_values(s["w13"][0][e], s["w13"][1][e]).t()
        gate, up = y[:, :case["F"]], y[:, case["F"]:]
        y = _exact_grid(gate * torch.sigmoid(gate) * up) @ _exact_values(s["w2"][0][e], s["w2"][1][e]).t()
        out.index_add_(0, t, y * weights[t, j].unsqueeze(1))
    return out
