"""Timing cases of the operators around the routed layer.

Four operators, each with listed cases and a draw over the same ranges:

  quantize  bf16 / fp32 rows to MXFP4 (E2M1 codes, one E8M0 scale per 32
            elements) and back to the values they stand for
  linear    a dense MXFP4 x MXFP4 product from unquantised rows, with or
            without SwiGLU (the shared expert's projections)
  grouped   the same product over rows sorted by expert, ragged groups
  norm      the end of a block: norm of the block's output, its gate and
            residual scale, the residual sum, and the next block's norm

Where `own` is true `run` calls the package, else it computes the plain form
(elementary torch operations in 32 bits, rounded once at the end).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# the largest work of a drawn case, by operator (that of the largest listed one)
MOST_QUANTIZE = 65536 * 4096                    # elements
MOST_LINEAR = (8192 * 4096 * 8192, 8192 * 8192)  # multiply-adds; elements of either operand or the result
MOST_GROUPED = (256 * 4096 * 4096, 36864 * 2048 * 4096)  # weight elements; multiply-adds
MOST_PADDED = 6_000_000_000                     # elements of the plain form's padded rows and outputs
MOST_NORM = 16384 * 7168                        # elements


def listed():
    return [
        # the activations of one decode batch: latency
        dict(name="quantize decode rows", op="quantize", R=32, K=4096, xtype="bf16", strided=False),
        # columns of a wider fp32 buffer, odd row count, K not a multiple of 64
        dict(name="quantize odd strided fp32", op="quantize", R=1111, K=4128, xtype="fp32", strided=True),
        # one stack of weights, quantised when a checkpoint is converted: bandwidth
        dict(name="quantize weights", op="quantize", R=65536, K=4096, xtype="bf16", strided=False),
        # the shared expert's gate and up projection for a single token: latency and one read of the weights
        dict(name="linear one token", op="linear", M=1, K=4096, N=4096, swiglu=True, xtype="bf16", ytype="bf16"),
        # odd rows and features, K that ends inside a tile, fp32 result
        dict(name="linear odd", op="linear", M=333, K=1056, N=1000, swiglu=False, xtype="fp32", ytype="fp32"),
        # a prompt: tensor-core bound
        dict(name="linear prompt", op="linear", M=8192, K=4096, N=8192, swiglu=False, xtype="bf16", ytype="bf16"),
        # the experts' gate and up projections of a decode batch: the weights of every touched expert read once
        dict(name="grouped decode", op="grouped", T=32, k=8, E=256, K=4096, N=4096, swiglu=True, skew=0.0, empty=0,
             xtype="bf16", ytype="bf16"),
        # few experts, skewed load with an empty expert, odd feature count, fp32 result
        dict(name="grouped ragged", op="grouped", T=1000, k=2, E=9, K=1056, N=1001, swiglu=False, skew=1.5, empty=1,
             xtype="bf16", ytype="fp32"),
        # the experts' down projection of a prompt
        dict(name="grouped prompt", op="grouped", T=4608, k=8, E=256, K=2048, N=4096, swiglu=False, skew=0.0, empty=0,
             xtype="bf16", ytype="bf16"),
        # one decoded token at the end of its block: latency
        dict(name="norm one token", op="norm", T=1, d=4096, ytype="fp32", two=True, rtype="bf16", gate="token",
             sigmoid=True, post=True),
        # odd width (rows not 16-byte aligned), a gate for each element, no norm after the block
        dict(name="norm odd", op="norm", T=777, d=1001, ytype="bf16", two=False, rtype="fp32", gate="element",
             sigmoid=False, post=False),
        # a long prompt of the widest configuration: bandwidth
        dict(name="norm prompt", op="norm", T=16384, d=7168, ytype="fp32", two=True, rtype="bf16", gate="channel",
             sigmoid=False, post=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log32(rng, lo, hi):
    return max(32, 32 * int(round(math.exp(rng.uniform(math.log(lo / 32), math.log(hi / 32))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "grouped", "norm"])
    if op == "quantize":
        K = _log32(rng, 32, 16384)
        R = _log(rng, 1, max(1, min(131072, MOST_QUANTIZE // (K + 64))))
        return dict(op=op, R=R, K=K, xtype=rng.choice(["bf16", "fp32"]), strided=rng.random() < 0.3)
    if op == "linear":
        K = _log32(rng, 32, 8192)
        swiglu = rng.random() < 0.4
        N = _log(rng, 16, min(8192, MOST_LINEAR[1] // K))
        N += N % 2 if swiglu else 0
        M = _log(rng, 1, max(1, min(16384, MOST_LINEAR[0] // (K * N), MOST_LINEAR[1] // max(K, N))))
        return dict(op=op, M=M, K=K, N=N, swiglu=swiglu, xtype=rng.choice(["bf16", "bf16", "fp32"]),
                    ytype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "grouped":
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(8, E - 1))
        K = _log32(rng, 64, 4096)
        swiglu = rng.random() < 0.4
        N = _log(rng, 16, min(4096, MOST_GROUPED[0] // (E * K)))
        N += N % 2 if swiglu else 0
        most = min(4608, MOST_GROUPED[1] // (k * K * N), MOST_PADDED // (E * (K + N)))
        T = _log(rng, 1, max(1, most))
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, swiglu=swiglu, skew=rng.choice([0.0, 0.0, 1.0, 2.0]),
                    empty=rng.randint(0, max(0, min(3, E - k))), xtype="bf16", ytype=rng.choice(["bf16", "bf16", "fp32"]))
    d = _log(rng, 64, 16384)
    if rng.random() < 0.6:
        d = max(64, d // 64 * 64)
    T = _log(rng, 1, max(1, min(16384, MOST_NORM // d)))
    return dict(op=op, T=T, d=d, ytype=rng.choice(["bf16", "fp32"]), two=rng.random() < 0.5,
                rtype=rng.choice(["bf16", "fp32"]), gate=rng.choice(["none", "token", "channel", "element"]),
                sigmoid=rng.random() < 0.5, post=rng.random() < 0.7)


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _rows(g, R, K, dtype, strided=False):
    """Activation-like rows: normal, with a channel profile that has some large channels, and a few all-zero (padding) rows."""
    profile = torch.exp(0.8 * torch.randn(K, generator=g, device=DEV))
    x = torch.empty(R, K + (64 if strided else 0), dtype=dtype, device=DEV)
    step = max(1, (1 << 26) // K)
    for r in range(0, R, step):
        n = min(step, R - r)
        x[r:r + n, :K] = (torch.randn(n, K, generator=g, device=DEV) * profile).to(dtype)
    if R > 8:
        x[torch.randint(0, R, (max(1, R // 256),), generator=g, device=DEV)] = 0
    return x[:, :K]


def _weights(g, E, N, K):
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g, device=DEV)
    scales = torch.randint(120, 123, (E, N, K // 32), dtype=torch.uint8, generator=g, device=DEV)
    return codes, scales


def _tiled(s, swiglu):
    """Scales [E, N, K/32] in the product's layout: for SwiGLU gate and up rows in turn; tiles of 128 rows x 4 scales, in a
    tile the byte of row r and scale b at 16 (r % 32) + 4 (r / 32) + b; zeros past the ends."""
    E, N, KB = s.shape
    if swiglu:
        s = s.view(E, 2, N // 2, KB).transpose(1, 2).reshape(E, N, KB)
    rt, kt = -(-N // 128), -(-KB // 4)
    t = torch.zeros(E, rt * 128, kt * 4, dtype=torch.uint8, device=s.device)
    t[:, :N, :KB] = s
    return t.view(E, rt, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(E, rt, kt, 512)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        s["x"] = _rows(g, case["R"], case["K"], TYPES[case["xtype"]], case["strided"])
    elif op == "linear":
        s["x"] = _rows(g, case["M"], case["K"], TYPES[case["xtype"]])
        s["w"], s["w_scale"] = _weights(g, 1, case["N"], case["K"])
        s["w_tiled"] = _tiled(s["w_scale"], case["swiglu"])
    elif op == "grouped":
        T, k, E = case["T"], case["k"], case["E"]
        s["x"] = _rows(g, T, case["K"], TYPES[case["xtype"]])
        s["w"], s["w_scale"] = _weights(g, E, case["N"], case["K"])
        s["w_tiled"] = _tiled(s["w_scale"], case["swiglu"])
        # routing: the k experts of the largest logits of each token, slots sorted by expert
        bias = -case["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
        if case["empty"]:
            bias[:case["empty"]] = -1e4
        ids = (torch.randn(T, E, generator=g, device=DEV) + bias).topk(k, dim=1).indices.reshape(-1)
        s["sorted_slot"] = torch.sort(ids, stable=True).indices.to(torch.int32)
        counts = torch.bincount(ids, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most_rows"] = int(counts.max())
    else:
        T, d = case["T"], case["d"]
        rows = lambda t, scale: (scale * torch.randn(T, d, generator=g, device=DEV)).to(TYPES[t])  # noqa: E731
        s["residual"] = rows(case["rtype"], 4.0)
        s["y"] = rows(case["ytype"], 0.7)
        s["y2"] = rows("bf16", 0.5) if case["two"] else None
        shape = {"none": None, "token": (T,), "channel": (d,), "element": (T, d)}[case["gate"]]
        s["gate_values"] = None if shape is None else torch.randn(shape, generator=g, device=DEV).to(
            torch.float32 if case["gate"] == "token" else torch.bfloat16)
        s["scale"] = 0.5
        weight = lambda: (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)  # noqa: E731
        s["post_weight"], s["next_weight"] = weight(), weight()
    return s


# ---- the plain forms --------------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e in fp32, exact, for integers e in [-127, 127] (2^-127 is subnormal)"""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).to(torch.int32).view(torch.float32)


def _mxfp4(x):
    """The values (fp32) that the MXFP4 form of rows x stands for: per 32 elements the scale 2^(floor(log2 amax) - 2), elements to
    the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), saturated at 6"""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.clamp(torch.frexp(amax).exponent - 3, min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = b * _pow2(-e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.copysign(q, v) * _pow2(e)).reshape(x.shape)


def _dequantize(codes, scales):
    """The fp32 values of E2M1 codes [.., K/2] (low nibble first) with E8M0 scales [.., K/32]"""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([mag, -mag])
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([table[byte & 15], table[byte >> 4]], 1)
    v = pairs.index_select(0, codes.reshape(-1).to(torch.int32))
    return v.view(*scales.shape, 32).mul_(_pow2(scales.to(torch.int32) - 127)[..., None]).view(*codes.shape[:-1], -1)


def _swiglu(y):
    gate, up = y.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _mxfp4(s["x"]).to(torch.bfloat16)
    if op == "linear":
        y = _mxfp4(s["x"]) @ _dequantize(s["w"][0], s["w_scale"][0]).t()
        return (_swiglu(y) if s["swiglu"] else y).to(TYPES[s["ytype"]])
    if op == "grouped":
        rows = s["sorted_slot"].shape[0]
        first, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
        q = _mxfp4(s["x"])[s["sorted_slot"].long() // s["k"]]
        # every group's rows padded to the largest group's count, one batched product, and back
        at = first[:, None] + torch.arange(s["most_rows"], device=q.device)
        y = torch.bmm(q[at.clamp(max=rows - 1)], _dequantize(s["w"], s["w_scale"]).transpose(1, 2))
        r = torch.arange(rows, device=q.device)
        e = torch.searchsorted(end, r, right=True)
        y = y[e, r - first[e]]
        return (_swiglu(y) if s["swiglu"] else y).to(TYPES[s["ytype"]])
    y = s["y"].float()
    if s["y2"] is not None:
        y = y + s["y2"].float()
    if s["post"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    y = y * s["post_weight"].float()
    if s["gate_values"] is not None:
        gate = s["gate_values"].float()
        gate = 1 / (1 + torch.exp(-gate)) if s["sigmoid"] else gate
        y = y * (gate[:, None] if s["gate"] == "token" else gate)
    r = s["residual"].float() + s["scale"] * y
    n = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["next_weight"].float()
    return r.to(s["residual"].dtype), n.to(torch.bfloat16)


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import fp4_mixture_experts_gb300 as moe
    s = state
    op = s["op"]
    if op == "quantize":
        codes, scales = moe.mxfp4_quantize(s["x"])
        return moe.mxfp4_dequantize(codes, scales)
    if op == "linear":
        return moe.mxfp4_linear(s["x"], s["w"], s["w_tiled"], swiglu=s["swiglu"], dtype=TYPES[s["ytype"]])
    if op == "grouped":
        return moe.mxfp4_linear(s["x"], s["w"], s["w_tiled"], offsets=s["offsets"], row_index=s["sorted_slot"],
                                index_div=s["k"], swiglu=s["swiglu"], dtype=TYPES[s["ytype"]])
    return moe.block_residual(s["residual"], s["y"], y2=s["y2"], post_norm=s["post"], post_weight=s["post_weight"],
                              gate=s["gate_values"], gate_sigmoid=s["sigmoid"], scale=s["scale"],
                              next_weight=s["next_weight"], eps=EPS)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once (quantize: the codes and scales are
    written by the first call and read by the second)"""
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "quantize":
        n = case["R"] * case["K"]
        return {"bytes": n * (size[case["xtype"]] + 2 * 17 / 32 + 2), "flops": 4 * n}
    if op == "norm":
        n = case["T"] * case["d"]
        gate = {"none": 0, "token": 4 * case["T"], "channel": 2 * case["d"], "element": 2 * n}[case["gate"]]
        per = size[case["ytype"]] + (2 if case["two"] else 0) + 2 * size[case["rtype"]] + 2
        return {"bytes": n * per + gate + 4 * case["d"], "flops": 12 * n}
    K, N = case["K"], case["N"]
    out = N // 2 if case["swiglu"] else N
    if op == "linear":
        M = case["M"]
        return {"bytes": M * K * size[case["xtype"]] + N * K * 17 / 32 + M * out * size[case["ytype"]],
                "flops": 2 * M * N * K}
    rows = case["T"] * case["k"]
    # experts that get rows, at the mean of a uniform routing (the skewed ones touch fewer)
    E = case["E"] - case["empty"]
    touched = E * (1 - (1 - case["k"] / E) ** case["T"])
    return {"bytes": case["T"] * case["K"] * size[case["xtype"]] + touched * N * K * 17 / 32 + 4 * rows +
            rows * out * size[case["ytype"]], "flops": 2 * rows * N * K}


# ---- the definition in 64 bits ----------------------------------------------------------------------------------------

def _exact_mxfp4(x):
    """As _mxfp4, by counting the midpoints below a magnitude: a tie goes up where the upper code is even"""
    v = x.double().unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent.double() - 3, -127.0).clamp(min=-127.0)
    scale = torch.exp2(e).double()
    m = v.abs() / scale
    code = torch.zeros_like(m, dtype=torch.uint8)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (m > mid) | ((m == mid) & (i % 2 == 1))
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    return (value[code.int()] * v.sign() * scale).flatten(-2)


def _exact_weights(codes, scales):
    lo, hi = (codes & 15).int(), (codes >> 4).int()
    c = torch.stack([lo, hi], -1).flatten(-2)
    exponent, odd = (c & 7) >> 1, (c & 1).double()
    m = torch.where(exponent > 0, (2 + odd) * torch.exp2(exponent.double() - 2), 0.5 * odd)
    m = torch.where(c >= 8, -m, m)
    return m * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_swiglu(y):
    n = y.shape[-1] // 2
    return y[..., :n] * torch.sigmoid(y[..., :n]) * y[..., n:]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x, parts = s["x"], []
        step = max(1, (1 << 25) // case["K"])
        for r in range(0, case["R"], step):
            parts.append(_exact_mxfp4(x[r:r + step]))
        return torch.cat(parts)
    if op == "linear":
        y = _exact_mxfp4(s["x"]) @ _exact_weights(s["w"][0], s["w_scale"][0]).t()
        return _exact_swiglu(y) if case["swiglu"] else y
    if op == "grouped":
        q = _exact_mxfp4(s["x"])
        off = s["offsets"].tolist()
        token = torch.div(s["sorted_slot"].long(), case["k"], rounding_mode="floor")
        y = torch.zeros(token.shape[0], case["N"], dtype=torch.float64, device=q.device)
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                y[off[e]:off[e + 1]] = q[token[off[e]:off[e + 1]]] @ _exact_weights(s["w"][e], s["w_scale"][e]).t()
        return _exact_swiglu(y) if case["swiglu"] else y
    outs, norms = [], []
    step = max(1, (1 << 25) // case["d"])
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    for r in range(0, case["T"], step):
        at = slice(r, r + step)
        b = wide(s["y"][at])
        if case["two"]:
            b = b + wide(s["y2"][at])
        if case["post"]:
            b = b / torch.sqrt(b.pow(2).sum(-1, keepdim=True) / case["d"] + EPS)
        b = b * wide(s["post_weight"])
        if case["gate"] != "none":
            gv = wide(s["gate_values"])
            gv = {"token": lambda: gv[at, None], "channel": lambda: gv, "element": lambda: gv[at]}[case["gate"]]()
            b = b * (torch.sigmoid(gv) if case["sigmoid"] else gv)
        o = wide(s["residual"][at]) + s["scale"] * b
        outs.append(o)
        norms.append(o / torch.sqrt(o.pow(2).sum(-1, keepdim=True) / case["d"] + EPS) * wide(s["next_weight"]))
    return torch.cat(outs), torch.cat(norms)
