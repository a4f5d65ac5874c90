"""Cases and plain forms of the feed-forward operators: routing, experts, 8-bit integers.

* route    scores of a router's logits [T, E] and the choice of k experts a token. An expert is available where its
           logit is neither NaN nor -inf. Scores s: softmax over the available experts, or sigmoid. The choice goes by
           c = s + bias, without a bias by the logit (which orders alike); with groups, only experts of the best
           `top_groups` groups of neighbours are chosen, a group's score being the sum of its two largest c (s without
           a bias). Weights: the chosen experts' s, renormalised to a sum of 1 if asked, times `scale`. Ties go to the
           lowest index. Outputs: weights float32 [T, k], experts int32 [T, k], best first.
* int8     a linear layer in 8-bit integers: s_x = max|x| / 127 a token, s_w = max|w| / 127 a channel,
           y = bf16(act(s_x s_w (x_q @ w_q^T) + bias) + residual). "swiglu" pairs the output columns in groups of 16
           gate and 16 up columns and gives silu(gate) * up.
* experts  the feed forward of the chosen experts: u = x_q @ Wu_e^T, h = silu(gate) * up in float32, d = h_q @ Wd_e^T,
           y = bf16(residual + sum_j w_j d_j). x and h are quantized as the linear layers of the weights' format
           quantize their input: per-tensor FP8, block FP8, MXFP8, MXFP4 or INT8.

Weights come as a checkpoint holds them: codes [N, K] (E2M1 two a byte, the even element in the low nibble) and scales
(FP8: one float32 an expert; block FP8: float32 [N/128, K/128]; MX: E8M0 [N, K/32]; INT8: float32 [N]), stacked over the
experts.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
FP8_SCALE_X = 0.08  # static scale of normed per-tensor FP8 activations: 448 * 0.08 = 36 covers their large channels
FP8_SCALE_H = 0.05  # of the experts' inner activations


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a chat: what counts is the launch
        {"name": "route 1x64", "op": "route", "T": 1, "E": 64, "k": 6, "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "renorm": True, "scale": 1.0, "f32": False},
        # a ragged mix of decode and prompt tokens
        {"name": "route 333x128", "op": "route", "T": 333, "E": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renorm": True, "scale": 1.0, "f32": False},
        # a full prompt batch, experts in groups with a bias that balances their load
        {"name": "route 8192x256 groups", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renorm": True, "scale": 2.5, "f32": True},
        # one token through the fused query, key and value projection, hidden size 4096
        {"name": "int8 M1", "op": "int8", "M": 1, "K": 4096, "N": 6144, "act": "none", "bias": False,
         "residual": False},
        # down projection onto the residual stream, an odd decode batch
        {"name": "int8 down M77", "op": "int8", "M": 77, "K": 14336, "N": 4096, "act": "none", "bias": False,
         "residual": True},
        # a prompt through the up projection with bias and SiLU
        {"name": "int8 up M4096", "op": "int8", "M": 4096, "K": 4096, "N": 14336, "act": "silu", "bias": True,
         "residual": False},
        # one token, eight of 64 small experts: latency and the chosen weights
        {"name": "experts block T1", "op": "experts", "fmt": "fp8_block", "T": 1, "E": 64, "k": 8, "H": 2048,
         "I": 1024},
        # a decode batch over few large experts: every weight is read
        {"name": "experts fp8 T48", "op": "experts", "fmt": "fp8", "T": 48, "E": 8, "k": 2, "H": 4096, "I": 14336},
        # a decode batch over many small experts, 4-bit weights
        {"name": "experts mxfp4 T128", "op": "experts", "fmt": "mxfp4", "T": 128, "E": 128, "k": 8, "H": 4096,
         "I": 1280},
        # an odd mix of decode and prompt tokens, integers
        {"name": "experts int8 T333", "op": "experts", "fmt": "int8", "T": 333, "E": 32, "k": 4, "H": 2048, "I": 1408},
        # a prompt batch over few large experts
        {"name": "experts block T2048", "op": "experts", "fmt": "fp8_block", "T": 2048, "E": 8, "k": 2, "H": 4096,
         "I": 7168},
        # a full prompt batch over many experts
        {"name": "experts mxfp8 T4096", "op": "experts", "fmt": "mxfp8", "T": 4096, "E": 64, "k": 8, "H": 4096,
         "I": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "int8", "experts", "experts"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        groups = rng.choice([1, 1, 4, 2]) if E % 8 == 0 else 1
        top = rng.randrange(1, groups + 1)
        k = min(rng.randrange(1, 11), top * E // groups)
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top, "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "f32": rng.random() < 0.5}
    if op == "int8":
        K = max(1, _log(rng, 256, 14336) // 32) * 32
        act = rng.choice(["none", "none", "relu", "gelu_tanh", "silu", "swiglu"])
        step = 32 if act == "swiglu" else 1
        N = max(1, _log(rng, 256, 28672) // step) * step
        M = min(_log(rng, 1, 4096), 4096 * 4096 * 14336 // (N * K))
        return {"op": op, "M": M, "K": K, "N": N, "act": act, "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5}
    fmt = rng.choice(["fp8", "fp8_block", "mxfp8", "mxfp4", "int8"])
    unit = 128 if fmt == "fp8_block" else 32
    H = max(4, _log(rng, 512, 6144) // unit) * unit
    E = rng.choice([4, 8, 16, 32, 60, 64, 128])
    I = max(4, _log(rng, 256, max(257, min(14336, 8 * 4096 * 14336 // (E * H)))) // unit) * unit
    k = rng.randrange(1, min(E, 8) + 1)
    T = max(1, min(_log(rng, 1, 4096), 4096 * 8 * 4096 * 1024 // (k * H * I)))
    return {"op": op, "fmt": fmt, "T": T, "E": E, "k": k, "H": H, "I": I}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _activations(g, M, K):
    """N(0, 1) with one channel in a hundred twenty times as large, as hidden states have."""
    x = _normal(g, M, K)
    big = torch.rand(K, generator=g, device=DEV) < 0.01
    return torch.where(big, 20 * x, x).to(torch.bfloat16)


def _encode_e2m1(v):
    """float32 values within +-6 -> E2M1 codes, to nearest, ties to the even code."""
    a = v.abs()
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    up = torch.bucketize(a, borders, right=True)  # a border counts as passed ...
    down = torch.bucketize(a, borders)  # ... or not
    code = torch.where(up % 2 == 0, up, down)
    return (code + torch.where(v < 0, 8, 0)).to(torch.uint8)


def _weight_codes(w, fmt):
    """float32 weights [E, N, K] as a checkpoint's codes and scales."""
    E, N, K = w.shape
    if fmt == "fp8":
        s = w.abs().amax((1, 2)) / 448
        return (w / s[:, None, None]).to(E4M3).view(torch.uint8), s
    if fmt == "fp8_block":
        t = w.view(E, N // 128, 128, K // 128, 128)
        s = t.abs().amax((2, 4)) / 448
        return (t / s[:, :, None, :, None]).to(E4M3).view(E, N, K).view(torch.uint8), s
    if fmt == "int8":
        s = w.abs().amax(2) / 127
        return torch.round(w / s[:, :, None]).clamp(-127, 127).to(torch.int8), s
    t = w.view(E, N, K // 32, 32)
    top = 9 if fmt == "mxfp8" else 3
    e = (torch.frexp(t.abs().amax(3))[1] - top).clamp(-127, 127)
    q = torch.ldexp(t, -e[..., None])
    if fmt == "mxfp8":
        codes = q.clamp(-448, 448).to(E4M3).view(E, N, K).view(torch.uint8)
    else:
        codes = _encode_e2m1(q.clamp(-6, 6)).view(E, N, K // 2, 2)
        codes = codes[..., 0] | (codes[..., 1] << 4)
    return codes, (e + 127).to(torch.uint8)


def _random_weights(g, E, N, K, fmt):
    """Expert by expert, so that the float32 weights never lie in memory all at once."""
    parts = [_weight_codes(_normal(g, 1, N, K, std=K ** -0.5), fmt) for _ in range(E)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    if c["op"] == "route":
        s["logits"] = _normal(g, c["T"], c["E"], std=1.5).to(torch.float32 if c["f32"] else torch.bfloat16)
        s["bias"] = _normal(g, c["E"], std=0.05) if c["bias"] else None
        return s
    if c["op"] == "int8":
        M, K, N = c["M"], c["K"], c["N"]
        s["x"] = _activations(g, M, K)
        s["wq"], s["ws"] = (t[0] for t in _weight_codes(_normal(g, 1, N, K, std=0.02), "int8"))
        s["b"] = _normal(g, N, std=0.01).to(torch.bfloat16) if c["bias"] else None
        s["res"] = _activations(g, M, N // 2 if c["act"] == "swiglu" else N) if c["residual"] else None
        if own:  # a user packs a layer's weight once, when it is loaded
            import fp8_quantized_linear_amd as fql

            s["W"] = fql.INT8Weight(fql.pack_weight_int8(s["wq"], s["ws"]), N, K)
        return s
    T, E, k, H, I, fmt = (c[n] for n in ("T", "E", "k", "H", "I", "fmt"))
    s["x"], s["res"] = _activations(g, T, H), _activations(g, T, H)
    # a router's choice: some experts are more popular than others, no token has one twice
    score = torch.sigmoid(_normal(g, T, E) + 0.5 * _normal(g, 1, E))
    w, e = torch.sort(score, 1, descending=True)
    s["w"] = w[:, :k] / w[:, :k].sum(1, keepdim=True)
    s["e"] = e[:, :k].to(torch.int32)
    s["uq"], s["us"] = _random_weights(g, E, 2 * I, H, fmt)
    s["dq"], s["ds"] = _random_weights(g, E, H, I, fmt)
    if own:  # packed once, when the layer is loaded
        import fp8_quantized_linear_amd as fql

        up, down = (FP8_SCALE_X, FP8_SCALE_H) if fmt == "fp8" else (None, None)
        s["U"] = fql.ExpertWeight.from_codes(fmt, s["uq"], s["us"], input_scale=up)
        s["D"] = fql.ExpertWeight.from_codes(fmt, s["dq"], s["ds"], input_scale=down)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _route(s):
    """In 64 bits: whether two experts change places hangs on the last bits of their scores."""
    c = s["c"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    logit = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(logit - logit.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logit))
    choice = logit if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        by = (p if s["bias"] is None else choice).view(T, G, E // G)
        best = torch.sort(by, 2, descending=True)[0][:, :, :2].sum(2)
        rank = torch.argsort(torch.sort(best, dim=1, descending=True, stable=True)[1], dim=1)
        out = (rank >= c["top_groups"])[:, :, None].expand(T, G, E // G).reshape(T, E)
        choice = choice.masked_fill(out, -math.inf)
    e = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(p, 1, e)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return (w * c["scale"]).float(), e.to(torch.int32)


def _scale(a, top):
    """A block's float32 scale and its reciprocal, rounded once each (codes next to a border go by them)."""
    s = (a.double() / top).float()
    return s, torch.where(s > 0, (1 / s.double()).clamp(max=3.4028234663852886e38).float(), 0.0)


def _fake(x, fmt, scale):
    """float32 x [..., K] through the 8-bit (or MXFP4) linear layers' input quantizer and back."""
    if fmt == "fp8":
        return (x * (1.0 / torch.tensor(scale))).clamp(-448, 448).to(E4M3).float() * scale
    if fmt == "int8":
        s, r = _scale(x.abs().amax(-1, keepdim=True), 127)
        return torch.round(x * r).clamp(-127, 127) * s
    if fmt == "fp8_block":
        t = x.unflatten(-1, (-1, 128))
        s, r = _scale(t.abs().amax(-1, keepdim=True), 448)
        return ((t * r).clamp(-448, 448).to(E4M3).float() * s).flatten(-2)
    t = x.unflatten(-1, (-1, 32))
    a = t.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a)[1] - (9 if fmt == "mxfp8" else 3), -127).clamp(-127, 127)
    q = torch.ldexp(t, -e)
    if fmt == "mxfp8":
        q = q.clamp(-448, 448).to(E4M3).float()
    else:
        q = _decode_e2m1(_encode_e2m1(q.clamp(-6, 6)))
    return torch.ldexp(q, e).flatten(-2)


def _decode_e2m1(code):
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.cat([values, -values])[code.int()]


def _weights(codes, scales, fmt):
    """A checkpoint's codes and scales [E, N, ...] -> float32 [E, N, K]."""
    if fmt == "int8":
        return codes.float() * scales[:, :, None]
    if fmt == "mxfp4":
        v = torch.stack([_decode_e2m1(codes & 15), _decode_e2m1(codes >> 4)], 3).flatten(2)
    else:
        v = codes.view(E4M3).float()
    E, N, K = v.shape
    if fmt == "fp8":
        return v * scales[:, None, None]
    if fmt == "fp8_block":
        return (v.view(E, N // 128, 128, K // 128, 128) * scales[:, :, None, :, None]).view(E, N, K)
    return torch.ldexp(v.view(E, N, K // 32, 32), scales.int()[..., None] - 127).view(E, N, K)


def _activation(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        t = z.unflatten(-1, (-1, 2, 16))
        gate, up = t[..., 0, :], t[..., 1, :]
        return (gate / (1 + torch.exp(-gate)) * up).flatten(-2)
    return z


def _int8(s):
    c = s["c"]
    x = s["x"].float()
    sx, r = _scale(x.abs().amax(1, keepdim=True), 127)
    q = torch.round(x * r).clamp(-127, 127)
    z = (q @ s["wq"].float().t()) * (sx * s["ws"])
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _activation(z, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(torch.bfloat16)


def _experts(s):
    """Pairs (token, place) sorted by expert, an expert's rows in blocks of B, one batched product over the blocks."""
    c = s["c"]
    T, E, k, fmt = c["T"], c["E"], c["k"], c["fmt"]
    P = T * k
    B = 128 if P >= 128 * E else 16 if P >= 4 * E else 1
    blocks = min(P, P // B + E)  # no more than this can be begun
    e, order = torch.sort(s["e"].view(-1).long(), stable=True)
    ids = torch.arange(E, device=DEV)
    first = torch.searchsorted(e, ids)
    need = (torch.searchsorted(e, ids, right=True) - first + B - 1) // B
    end = torch.cumsum(need, 0)
    i = torch.arange(P, device=DEV) - first[e]
    slot = (end - need)[e] * B + i  # a sorted pair's row among the blocks
    of_block = torch.searchsorted(end, torch.arange(blocks, device=DEV), right=True).clamp(max=E - 1)
    xq = _fake(s["x"].float(), fmt, FP8_SCALE_X)
    rows = torch.zeros((blocks * B, c["H"]), device=DEV)
    rows[slot] = xq[order // k]
    up = _weights(s["uq"], s["us"], fmt).transpose(1, 2).contiguous()
    u = torch.bmm(rows.view(blocks, B, -1), up[of_block])
    h = _fake(_activation(u, "swiglu"), fmt, FP8_SCALE_H)
    down = _weights(s["dq"], s["ds"], fmt).transpose(1, 2).contiguous()
    d = torch.bmm(h, down[of_block]).view(blocks * B, -1)
    back = torch.empty_like(slot)
    back[order] = slot
    y = (d[back].view(T, k, -1) * s["w"][:, :, None]).sum(1)
    return (y + s["res"].float()).to(torch.bfloat16)


def run(state):
    s, c = state, state["c"]
    if not own:
        return {"route": _route, "int8": _int8, "experts": _experts}[c["op"]](s)
    import fp8_quantized_linear_amd as fql

    if c["op"] == "route":
        return fql.route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "int8":
        return fql.linear_fused(s["x"], s["W"], activation=c["act"], bias=s["b"], residual=s["res"])
    return fql.experts_fused(s["x"], s["U"], s["D"], s["w"], s["e"], activation="swiglu", residual=s["res"])


# ---------------------------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * (4 if c["f32"] else 2) + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": 6 * c["T"] * c["E"]}
    if c["op"] == "int8":
        M, K, N = c["M"], c["K"], c["N"]
        No = N // 2 if c["act"] == "swiglu" else N
        return {"bytes": N * K + 4 * N + 2 * M * K + 2 * M * No * (2 if c["residual"] else 1)
                + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
    size = {"fp8": 1.0, "fp8_block": 1 + 4 / 128 ** 2, "mxfp8": 33 / 32, "mxfp4": 17 / 32, "int8": 1.0}[c["fmt"]]
    chosen = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, where all are as popular
    return {"bytes": chosen * 3 * H * I * size + 3 * 2 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _route64(s):
    c = s["c"]
    z = s["logits"].cpu().double()
    p = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
    by = p + s["bias"].cpu().double() if s["bias"] is not None else p
    choice = by if s["bias"] is not None else z
    T, E, G = c["T"], c["E"], c["groups"]
    if G > 1:
        two = by.view(T, G, -1).topk(min(2, E // G), 2)[0].sum(2)
        kept = torch.argsort(-two, dim=1, stable=True)[:, :c["top_groups"]]
        mask = torch.zeros((T, G), dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(mask.repeat_interleave(E // G, 1), choice, torch.full_like(choice, -math.inf))
    e = torch.argsort(-choice, dim=1, stable=True)[:, :c["k"]]
    w = p.gather(1, e)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return (w * c["scale"]).to(DEV), e.to(torch.int32).to(DEV)


def _round_e4m3(v):
    """float64 values rounded to the E4M3 grid: nearest, ties to even, saturating at 448."""
    quantum = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / quantum) * quantum).clamp(-448, 448)


def _round_e2m1(v):
    """float64 values rounded to the E2M1 grid, saturating at 6."""
    quantum = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=0).double() - 1)
    return (torch.round(v / quantum) * quantum).clamp(-6, 6)


def _f32(v):
    """float64 values rounded to float32."""
    return v.float().double()


def _fake64(x, fmt, scale):
    """The quantizers are defined with float32 scales and quotients (a value next to a border goes by them)."""
    if fmt == "fp8":
        s = _f32(torch.tensor(scale, dtype=torch.float64, device=DEV))
        return _round_e4m3(_f32(_f32(x) * _f32(1 / s))) * s
    n = {"int8": x.shape[-1], "fp8_block": 128, "mxfp8": 32, "mxfp4": 32}[fmt]
    t = _f32(x).reshape(x.shape[0], -1, n)
    a = t.abs().amax(2, keepdim=True)
    if fmt in ("int8", "fp8_block"):
        s = _f32(a / (127 if fmt == "int8" else 448))
        q = _f32(t * _f32(1 / torch.where(s > 0, s, 1.0)).clamp(max=torch.finfo(torch.float32).max))
        q = torch.round(q).clamp(-127, 127) if fmt == "int8" else _round_e4m3(q)
    else:
        s = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-119) - (8 if fmt == "mxfp8" else 2))
        q = (_round_e4m3 if fmt == "mxfp8" else _round_e2m1)(t / s)
    return (q * s).reshape(x.shape)


def _weight64(codes, scales, fmt):
    """One expert's codes and scales -> float64 [N, K]."""
    if fmt == "int8":
        return codes.double() * scales.double()[:, None]
    if fmt == "mxfp4":
        c = torch.stack([codes & 15, codes >> 4], 2).flatten(1).int()
        m, e = (c & 1).double(), (c >> 1) & 3
        v = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2) * torch.where(c >= 8, -1.0, 1.0)
    else:
        v = codes.view(E4M3).double()
    if fmt == "fp8":
        return v * scales.double()
    if fmt == "fp8_block":
        return v * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _act64(z, act):
    if act == "swiglu":
        t = z.view(z.shape[0], -1, 32)
        gate, up = t[..., :16], t[..., 16:]
        return (gate * torch.sigmoid(gate) * up).reshape(z.shape[0], -1)
    return {"none": lambda: z, "relu": lambda: torch.maximum(z, torch.zeros_like(z)),
            "silu": lambda: z * torch.sigmoid(z),
            "gelu_tanh": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[act]()


def _int8_64(s):
    z = _fake64(s["x"].double(), "int8", None) @ _weight64(s["wq"], s["ws"], "int8").t()
    if s["b"] is not None:
        z = z + s["b"].double()
    y = _act64(z, s["c"]["act"])
    return y + s["res"].double() if s["res"] is not None else y


def _experts64(s):
    c = s["c"]
    fmt = c["fmt"]
    x, y = _fake64(s["x"].double(), fmt, FP8_SCALE_X), s["res"].double()
    for e in range(c["E"]):
        t, j = torch.nonzero(s["e"] == e, as_tuple=True)
        if t.numel():
            h = _act64(x[t] @ _weight64(s["uq"][e], s["us"][e], fmt).t(), "swiglu")
            d = _fake64(h, fmt, FP8_SCALE_H) @ _weight64(s["dq"][e], s["ds"][e], fmt).t()
            y.index_add_(0, t, d * s["w"][t, j].double()[:, None])
    return y


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _route64, "int8": _int8_64, "experts": _experts64}[case["op"]](s)
