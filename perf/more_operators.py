"""Timing cases of the operators of a decoder layer's attention half.

Four operators, each with listed cases and a draw over the same ranges:

  linear   a product with weights in 8-bit floating point (E4M3), one
           power-of-two scale for each 128 x 128 of them, from rows that are
           quantised for each 128 elements; dense, with SwiGLU, or a matrix for
           each group of rows
  prompt   latent attention in its expanded form: keys and values of every head
           from the shared latent vectors, a ragged batch of new tokens behind
           cached ones
  decode   latent attention in its absorbed form: one new token a sequence over
           a paged cache of the latent vectors themselves
  pages    the block tables, slots and positions of a batch's new tokens, from
           the requests' lengths

Where `own` is true `run` calls the package, else it computes the plain form
(elementary torch operations in 32 bits, rounded once at the end).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NOPE, ROPE, VALUE, LATENT = 128, 64, 128, 512   # of a head: without and with positions, values; of a token: the latent vector
SCALE = (NOPE + ROPE) ** -0.5
# the largest work of a drawn case, by operator (that of the largest listed one)
MOST_LINEAR = (8192 * 4096 * 8192, 8192 * 8192)  # multiply-adds; elements of either operand or the result
MOST_PAIRS = 64 * 8192 * 8192 // 2               # heads x (query, key) pairs
MOST_TOKENS = 4 * 131072                         # cached tokens
MOST_DECODE = 4 * 131072 * 64                    # heads x cached tokens
MOST_SLOTS = 131072


def listed():
    return [
        # the down projection of one token: latency and one read of the weights
        dict(name="linear one token", op="linear", M=1, K=4096, N=2048, E=1, swiglu=False, xtype="bf16", ytype="bf16"),
        # a matrix for each group of rows (a head, an expert), uneven ones; odd features, K that ends inside a scale's block
        dict(name="linear grouped odd", op="linear", M=1999, K=1056, N=1001, E=9, swiglu=False, xtype="fp32", ytype="fp32"),
        # the shared expert's gate and up projection of a prompt
        dict(name="linear shared expert", op="linear", M=4608, K=4096, N=4096, E=1, swiglu=True, xtype="bf16", ytype="bf16"),
        # the output projection of a long prompt: tensor-core bound
        dict(name="linear prompt", op="linear", M=8192, K=8192, N=4096, E=1, swiglu=False, xtype="bf16", ytype="bf16"),
        # a short prompt on few heads (a layer that is split over GPUs): latency
        dict(name="prompt short", op="prompt", B=1, Q=200, C=0, H=16, spread=0.0, causal=True),
        # a ragged batch, some sequences behind a cached prefix, lengths down to one token
        dict(name="prompt ragged", op="prompt", B=13, Q=3001, C=5003, H=24, spread=1.0, causal=True),
        # a long prompt on all heads: tensor-core bound
        dict(name="prompt long", op="prompt", B=1, Q=8192, C=0, H=64, spread=0.0, causal=True),
        # one sequence: latency, and the split over its length
        dict(name="decode one sequence", op="decode", B=1, L=4608, H=64, page=64, spread=0.0),
        # a ragged batch on a number of heads that fills no tile, small pages
        dict(name="decode ragged", op="decode", B=33, L=33 * 1000, H=20, page=16, spread=1.0),
        # a few very long sequences: bandwidth
        dict(name="decode long", op="decode", B=4, L=4 * 131072, H=64, page=64, spread=0.2),
        # a decode step: one token each
        dict(name="pages step", op="pages", B=32, T=32, L=32 * 1000, page=64, spread=0.5),
        # a whole batch of prompts enters the cache
        dict(name="pages prompts", op="pages", B=256, T=131072, L=20000, page=64, spread=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _log32(rng, lo, hi):
    return max(32, 32 * int(round(math.exp(rng.uniform(math.log(lo / 32), math.log(max(lo, hi) / 32))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "prompt", "decode", "decode", "pages"])
    if op == "linear":
        E = rng.choice([1, 1, _log(rng, 2, 128)])
        K = _log32(rng, 32, 8192 if E == 1 else 1024)
        swiglu = rng.random() < 0.3
        N = _log(rng, 16, min(8192, MOST_LINEAR[1] // (K * E)))
        N += N % 2 if swiglu else 0
        M = _log(rng, 1, max(1, min(16384, MOST_LINEAR[0] // (K * N), MOST_LINEAR[1] // max(K, N))))
        return dict(op=op, M=M, K=K, N=N, E=E, swiglu=swiglu, xtype=rng.choice(["bf16", "bf16", "fp32"]),
                    ytype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "prompt":
        H = rng.choice([1, 8, 16, 24, 32, 64, 128])
        B = _log(rng, 1, 64)
        Q = _log(rng, B, min(16384, math.isqrt(2 * MOST_PAIRS // H)))
        C = rng.choice([0, _log(rng, 1, max(1, min(32768, MOST_PAIRS // (H * Q))))])
        case = dict(op=op, B=B, Q=Q, C=C, H=H, spread=rng.choice([0.0, 0.5, 1.0]), causal=rng.random() < 0.8)
        while H * sum(q * (q + c) for q, c in zip(*_prompt_lengths(case))) > 2 * MOST_PAIRS:
            case["Q"] = max(B, case["Q"] * 2 // 3)
            case["C"] = case["C"] // 2
        return case
    if op == "decode":
        H = rng.choice([1, 8, 16, 20, 32, 64, 128])
        B = _log(rng, 1, 256)
        L = _log(rng, B, min(MOST_TOKENS, MOST_DECODE // H))
        return dict(op=op, B=B, L=L, H=H, page=rng.choice([16, 32, 64, 64, 128]), spread=rng.choice([0.0, 0.5, 1.0]))
    B = _log(rng, 1, 1024)
    T = rng.choice([B, _log(rng, B, max(B, MOST_SLOTS))])
    return dict(op=op, B=B, T=T, L=_log(rng, B, 200 * B), page=rng.choice([16, 32, 64, 128]), spread=rng.choice([0.0, 0.5, 1.0]))


# ---- inputs -----------------------------------------------------------------------------------------------------------

def _split(total, n, spread, least, salt):
    """total in n parts of at least `least`, even (spread 0) to very uneven (1); the same for the same arguments"""
    rng = random.Random(f"{total} {n} {spread} {salt}")
    total = max(total, least * n)
    weights = [math.exp(3.0 * spread * rng.uniform(-1, 1)) for _ in range(n)]
    free = total - least * n
    parts = [least + int(free * w / sum(weights)) for w in weights]
    parts[0] += total - sum(parts)
    return parts


def _prompt_lengths(case):
    """new tokens and cached ones of each sequence"""
    q = _split(case["Q"], case["B"], case["spread"], 1, "new")
    c = _split(case["C"], case["B"], case["spread"], 0, "cached")
    return q, c


def _decode_lengths(case):
    return _split(case["L"], case["B"], case["spread"], 1, "cached")


def _pages_lengths(case):
    return _split(case["L"], case["B"], case["spread"], 0, "cached"), _split(case["T"], case["B"], case["spread"], 1, "new")


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _int32(values):
    return torch.tensor(values, dtype=torch.int32).to(DEV)


def _rows(g, R, K, dtype):
    """Activation-like rows: normal, with a channel profile that has some large channels, and a few all-zero (padding) rows."""
    profile = torch.exp(0.8 * torch.randn(K, generator=g, device=DEV))
    x = (torch.randn(R, K, generator=g, device=DEV) * profile).to(dtype)
    if R > 8:
        x[torch.randint(0, R, (max(1, R // 256),), generator=g, device=DEV)] = 0
    return x


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _tiled(s, N, swiglu):
    """Scales [E, ceil(N/128), ceil(K/128)] in the product's layout: for SwiGLU gate and up rows in turn; tiles of 128 rows by
    128 elements of K, four equal bytes a row, those of row r at 16 (r % 32) + 4 (r / 32); zeros past the end."""
    E, _, kt = s.shape
    rows = torch.arange(N, device=s.device)
    if swiglu:
        rows = rows.view(2, N // 2).t().reshape(-1)
    rt = -(-N // 128)
    t = torch.zeros(E, rt * 128, kt, dtype=torch.uint8, device=s.device)
    t[:, :N] = s[:, rows // 128]
    return t.view(E, rt, 4, 32, kt, 1).expand(-1, -1, -1, -1, -1, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, rt, kt, 512)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    order = random.Random(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "linear":
        M, K, N, E = (case[n] for n in "MKNE")
        s["x"] = _rows(g, M, K, TYPES[case["xtype"]])
        s["w"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
        for e in range(E):
            s["w"][e] = (120 * torch.randn(N, K, generator=g, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["w_scale"] = torch.randint(112, 115, (E, -(-N // 128), -(-K // 128)), dtype=torch.uint8, generator=g, device=DEV)
        s["w_tiled"] = _tiled(s["w_scale"], N, case["swiglu"])
        s["sizes"] = _split(M, E, 0.5, 0, "rows") if E > 1 else None
        s["offsets"] = _int32(_offsets(s["sizes"])) if E > 1 else None
    elif op == "prompt":
        H = case["H"]
        both = list(zip(*_prompt_lengths(case)))
        order.shuffle(both)
        s["q_lens"], s["k_lens"] = [q for q, _ in both], [q + c for q, c in both]
        s["q_offsets"], s["k_offsets"] = _int32(_offsets(s["q_lens"])), _int32(_offsets(s["k_lens"]))
        s["q"] = _normal(g, sum(s["q_lens"]), H, NOPE + ROPE)
        s["kv"] = _normal(g, sum(s["k_lens"]), H, NOPE + VALUE)     # as the up projection of the latent vectors writes it
        s["k_rope"] = _normal(g, sum(s["k_lens"]), ROPE)
    elif op == "decode":
        lens, page = _decode_lengths(case), case["page"]
        order.shuffle(lens)
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 8
        s["lens"], s["lengths"] = lens, _int32(lens)
        s["q"] = _normal(g, case["B"], case["H"], LATENT + ROPE)
        s["cache"] = _normal(g, pages, page, LATENT + ROPE)
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.zeros(case["B"], max(counts), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(counts):
            s["table"][b, :n] = ids[at:at + n]
            at += n
    else:
        both, page, B = list(zip(*_pages_lengths(case))), case["page"], case["B"]
        order.shuffle(both)
        owned = [-(-n // page) for n, _ in both]
        width = max(-(-(n + t) // page) for n, t in both) + 2
        total = sum(-(-(n + t) // page) for n, t in both) + 100
        ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        s["lengths"], s["new"] = _int32([n for n, _ in both]), _int32([t for _, t in both])
        s["tokens"] = sum(t for _, t in both)
        # the pages that requests own already, the rest of a row unset; the free ones
        col = torch.arange(width, device=DEV)[None]
        first = _int32(_offsets(owned))
        own_n = (first[1:] - first[:-1])[:, None]
        s["table"] = torch.where(col < own_n, ids[(first[:-1, None] + col).clamp(max=total - 1).long()], -1).to(torch.int32)
        s["free"] = ids[sum(owned):].clone()
    return s


# ---- the plain forms --------------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e in fp32, exact, for integers e in [-127, 127] (2^-127 is subnormal)"""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).to(torch.int32).view(torch.float32)


def _fp8(x):
    """The values (fp32) that the E4M3 form of rows x stands for: per 128 elements the least power of two that keeps them within
    448, elements to the nearest of 8 bits (ties to the even code)"""
    R, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(R, -1, 128)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(min=-127)
    return ((b * _pow2(-e)).to(torch.float8_e4m3fn).float() * _pow2(e)).view(R, -1)[:, :K]


def _dequantize(w, scale):
    """fp32 values of E4M3 [N, K] with E8M0 scales [ceil(N/128), ceil(K/128)]"""
    N, K = w.shape
    s = _pow2(scale.int() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return w.float() * s


def _swiglu(y):
    gate, up = y.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _attend(q, k, v, first):
    """softmax(SCALE q k^T) v of [H, Q, D], [H, L, D], [H, L, V], query i seeing the keys up to first + i (all: first None),
    some queries at a time; a query that sees none gets zeros"""
    out = torch.empty(q.shape[0], q.shape[1], v.shape[2], device=q.device)
    step = max(1, (1 << 30) // max(1, q.shape[0] * k.shape[1]))
    j = torch.arange(k.shape[1], device=q.device)
    for i in range(0, q.shape[1], step):
        p = torch.matmul(q[:, i:i + step], k.transpose(1, 2)) * SCALE
        if first is not None:
            rows = first + i + torch.arange(p.shape[1], device=q.device)
            p = torch.where(j[None, None] <= rows[None, :, None], p, -math.inf)
        p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
        out[:, i:i + step] = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out


def _plain(s):
    op = s["op"]
    if op == "linear":
        a = _fp8(s["x"])
        if s["offsets"] is None:
            y = a @ _dequantize(s["w"][0], s["w_scale"][0]).t()
        else:
            parts = a.split(s["sizes"])
            y = torch.cat([p @ _dequantize(s["w"][e], s["w_scale"][e]).t() for e, p in enumerate(parts)])
        return (_swiglu(y) if s["swiglu"] else y).to(TYPES[s["ytype"]])
    if op == "prompt":
        H, outs = s["H"], []
        q0 = k0 = 0
        for nq, nk in zip(s["q_lens"], s["k_lens"]):
            q = s["q"][q0:q0 + nq].float().transpose(0, 1)
            kv = s["kv"][k0:k0 + nk].float().transpose(0, 1)
            rope = s["k_rope"][k0:k0 + nk].float()[None].expand(H, -1, -1)
            k = torch.cat([kv[..., :NOPE], rope], -1)
            outs.append(_attend(q, k, kv[..., NOPE:], nk - nq if s["causal"] else None).transpose(0, 1))
            q0, k0 = q0 + nq, k0 + nk
        return torch.cat(outs).to(torch.bfloat16)
    if op == "decode":
        outs = []
        for b, n in enumerate(s["lens"]):
            pages = s["table"][b, :-(-n // s["page"])].long()
            c = s["cache"][pages].view(-1, LATENT + ROPE)[:n].float()
            outs.append(_attend(s["q"][b].float()[None], c[None], c[None, :, :LATENT], None)[0])
        return torch.stack(outs).to(torch.bfloat16)
    page, n, t = s["page"], s["lengths"].long(), s["new"].long()
    owned, after = (n + page - 1) // page, (n + t + page - 1) // page
    fresh = torch.cumsum(after - owned, 0) - (after - owned)
    table = s["table"]
    col = torch.arange(table.shape[1], device=table.device)[None]
    at = (fresh[:, None] + col - owned[:, None]).clamp(0, s["free"].shape[0] - 1)
    table = torch.where((col >= owned[:, None]) & (col < after[:, None]), s["free"][at], table)
    ends = torch.cumsum(t, 0)
    i = torch.arange(s["tokens"], device=table.device)
    b = torch.searchsorted(ends, i, right=True)
    position = n[b] + i - (ends - t)[b]
    slots = table[b, position // page].long() * page + position % page
    return table, slots, position.int(), (n + t).int(), (after - owned).sum().int()


# ---- one pass ---------------------------------------------------------------------------------------------------------

def run(state):
    if not own:
        return _plain(state)
    import fp4_mixture_experts_gb300 as moe
    s = state
    op = s["op"]
    if op == "linear":
        return moe.fp8_linear(s["x"], s["w"], s["w_tiled"], offsets=s["offsets"], swiglu=s["swiglu"],
                              dtype=TYPES[s["ytype"]])
    if op == "prompt":
        return moe.latent_attention(s["q"], s["kv"], s["k_rope"], s["q_offsets"], s["k_offsets"], scale=SCALE,
                                    causal=s["causal"])
    if op == "decode":
        return moe.latent_decode(s["q"], s["cache"], s["table"], s["lengths"], scale=SCALE)
    p = moe.page_slots(s["lengths"], s["new"], s["table"], s["free"], page_size=s["page"], tokens=s["tokens"])
    return s["table"], p.slots, p.positions, p.lengths, p.taken


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once"""
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "linear":
        M, K, N, E = (case[n] for n in "MKNE")
        out = N // 2 if case["swiglu"] else N
        return {"bytes": M * K * size[case["xtype"]] + min(E, M) * N * K * (1 + 1 / 16384) + M * out * size[case["ytype"]],
                "flops": 2 * M * N * K}
    if op == "prompt":
        H = case["H"]
        q, c = _prompt_lengths(case)
        pairs = sum(n * m + n * (n + 1) // 2 if case["causal"] else n * (n + m) for n, m in zip(q, c))
        keys = sum(q) + sum(c)
        return {"bytes": 2 * (sum(q) * H * (NOPE + ROPE + VALUE) + keys * (H * (NOPE + VALUE) + ROPE)),
                "flops": 2 * H * pairs * (NOPE + ROPE + VALUE)}
    if op == "decode":
        tokens, rows = sum(_decode_lengths(case)), case["B"] * case["H"]
        return {"bytes": 2 * (tokens * (LATENT + ROPE) + rows * (2 * LATENT + ROPE)),
                "flops": 2 * case["H"] * tokens * (2 * LATENT + ROPE)}
    n, t = _pages_lengths(case)
    page = case["page"]
    fresh = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(n, t))
    return {"bytes": 12 * sum(t) + 12 * case["B"] + 8 * fresh, "flops": 8 * sum(t)}


# ---- the definition in 64 bits ----------------------------------------------------------------------------------------

def _exact_fp8(x):
    """As _fp8: steps of 2^-3 of the leading power of two, 2^-9 at least"""
    R, K = x.shape
    out = torch.zeros(R, K, dtype=torch.float64, device=x.device)
    for k in range(0, K, 128):
        v = x[:, k:k + 128].double()
        amax = v.abs().max(1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0) / 448)) - 1
        for _ in range(3):
            e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
        scale = torch.exp2(torch.where(amax > 0, e, -127.0).clamp(min=-127.0))
        u = v / scale
        exponent = torch.frexp(u).exponent.double() - 1
        step = torch.exp2(exponent.clamp(min=-6.0) - 3)
        out[:, k:k + 128] = torch.round(u / step) * step * scale
    return out


def _exact_weights(w, scale):
    rows = torch.arange(w.shape[0], device=w.device) // 128
    cols = torch.arange(w.shape[1], device=w.device) // 128
    return w.to(torch.float32).double() * torch.exp2(scale.double() - 127)[rows][:, cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        a, parts = _exact_fp8(s["x"]), []
        off = [0, case["M"]] if case["E"] == 1 else s["offsets"].tolist()
        for e in range(case["E"]):
            parts.append(a[off[e]:off[e + 1]] @ _exact_weights(s["w"][e], s["w_scale"][e]).t())
        y = torch.cat(parts)
        if case["swiglu"]:
            gate, up = y[:, :case["N"] // 2], y[:, case["N"] // 2:]
            y = gate * torch.sigmoid(gate) * up
        return y
    if op == "prompt":
        qo, ko = s["q_offsets"].tolist(), s["k_offsets"].tolist()
        out = torch.zeros(qo[-1], case["H"], VALUE, dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
            seen = torch.arange(nq, device=DEV)[:, None] + (nk - nq) >= torch.arange(nk, device=DEV)[None]
            rope = s["k_rope"][ko[b]:ko[b + 1]].double()
            for h in range(case["H"]):
                q = s["q"][qo[b]:qo[b + 1], h].double()
                kv = s["kv"][ko[b]:ko[b + 1], h].double()
                z = (q[:, :NOPE] @ kv[:, :NOPE].t() + q[:, NOPE:] @ rope.t()) * SCALE
                if case["causal"]:
                    z = z.masked_fill(~seen, -math.inf)
                out[qo[b]:qo[b + 1], h] = torch.softmax(z, -1) @ kv[:, NOPE:]
        return out
    if op == "decode":
        out = torch.zeros(case["B"], case["H"], LATENT, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"]):
            t = torch.arange(n, device=DEV)
            c = s["cache"][s["table"][b, t // case["page"]].long(), t % case["page"]].double()
            out[b] = torch.softmax(s["q"][b].double() @ c.t() * SCALE, -1) @ c[:, :LATENT]
        return out
    table, free, page = s["table"].tolist(), s["free"].tolist(), case["page"]
    slots, positions, lengths, taken = [], [], [], 0
    for b, (n, t) in enumerate(zip(s["lengths"].tolist(), s["new"].tolist())):
        for i in range(n, n + t):
            if i % page == 0:
                table[b][i // page] = free[taken]
                taken += 1
            slots.append(table[b][i // page] * page + i % page)
            positions.append(i)
        lengths.append(n + t)
    return (_int32(table), torch.tensor(slots, device=DEV), _int32(positions), _int32(lengths), _int32(taken))
