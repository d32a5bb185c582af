"""The operators around a router and its experts' 8-bit products: cases, plain forms and 64-bit values.

Five operators (all sizes in elements; R: rows, T: tokens, K: chosen experts a token, E: experts):

  lists     the token lists of every expert from the router's choice: counts, offsets, rows, positions
  balance   the balance loss of a router with per-expert counts, and its gradient
  quantize  e4m3 codes with one power-of-two scale for each 1 x 128 block, along the rows and (for training)
            along the columns, of rows picked by an index
  matmul    y = x w^T of e4m3 codes with scales for each 1 x 128 (x) and 128 x 128 (w) block; plain or with one
            weight matrix for each expert's rows
  wgrad     each expert's dw = dy^T x of column-quantised dy and x
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 128


# ---------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch of 8 sequences: the lists of a layer of 256 experts, latency alone
        {"name": "lists_decode", "op": "lists", "tokens": 8, "top_k": 8, "experts": 256, "align": 1, "dropped": 0.0},
        # a training batch of 64 Ki tokens, segments padded to whole blocks of 128 rows
        {"name": "lists_train", "op": "lists", "tokens": 65536, "top_k": 8, "experts": 256, "align": 128, "dropped": 0.02},
        # sequences of one step of a sigmoid router, float32 logits as the router makes them
        {"name": "balance_sequences", "op": "balance", "tokens": 4099, "experts": 256, "top_k": 8, "score": 0, "dtype": "f32",
         "sequences": 9, "masked": 0.1},
        # one large batch of a softmax router with 64 experts
        {"name": "balance_batch", "op": "balance", "tokens": 131072, "experts": 64, "top_k": 8, "score": 1, "dtype": "bf16",
         "sequences": 1, "masked": 0.0},
        # a decode batch's activations before the gate and up products
        {"name": "quantize_decode", "op": "quantize", "tokens": 8, "rows": 8, "width": 6144, "dtype": "f32", "gather": False,
         "both": False},
        # a training step's tokens, gathered into their experts' segments, for the product and for the weights' gradient
        {"name": "quantize_train", "op": "quantize", "tokens": 8192, "rows": 73728, "width": 2048, "dtype": "bf16", "gather": True,
         "both": True},
        # one token through a shared expert's gate and up matrices
        {"name": "matmul_token", "op": "matmul", "rows": 1, "n": 4096, "k": 6144, "experts": 1, "dtype": "f32"},
        # a long prompt through the same matrices, an odd number of tokens
        {"name": "matmul_prompt", "op": "matmul", "rows": 16381, "n": 4096, "k": 6144, "experts": 1, "dtype": "bf16"},
        # 4 tokens of a decode batch through the gate and up matrices of their 8 experts each, of 256
        {"name": "matmul_experts_decode", "op": "matmul", "rows": 32, "n": 4096, "k": 6144, "experts": 256, "dtype": "bf16"},
        # 8 Ki tokens through 8 of 64 experts
        {"name": "matmul_experts_train", "op": "matmul", "rows": 65536, "n": 2048, "k": 2048, "experts": 64, "dtype": "bf16"},
        # the gradient of one layer's down matrices from a short step
        {"name": "wgrad_short", "op": "wgrad", "rows": 2048, "n": 2048, "k": 1024, "experts": 16, "dtype": "bf16"},
        # the gradient of 64 experts' gate and up matrices from 8 Ki tokens, in float32 as an optimiser takes it
        {"name": "wgrad_train", "op": "wgrad", "rows": 65536, "n": 2048, "k": 2048, "experts": 64, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["lists", "balance", "quantize", "matmul", "matmul", "wgrad"])
    if op == "lists":
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": _log(rng, 1, 65536), "top_k": rng.choice([k for k in (1, 2, 4, 6, 8) if k <= experts]),
                "experts": experts, "align": rng.choice([1, 16, 128]), "dropped": rng.choice([0.0, 0.05])}
    if op == "balance":
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": _log(rng, 16, 131072), "experts": experts, "top_k": rng.choice([1, 2, 4, 8]), "score": rng.choice([0, 1]),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "sequences": rng.choice([1, 2, 5, 16]), "masked": rng.choice([0.0, 0.2])}
    if op == "quantize":
        tokens, gather = _log(rng, 1, 16384), rng.random() < 0.5
        rows = min(65536, tokens * rng.choice([1, 2, 4])) if gather else tokens
        return {"op": op, "tokens": tokens, "rows": rows, "width": 16 * _log(rng, 8, 512), "dtype": rng.choice(["f32", "bf16", "f16"]),
                "gather": gather, "both": rng.random() < 0.5}
    if op == "matmul":
        return {"op": op, "rows": _log(rng, 1, 16384), "n": _log(rng, 128, 6144), "k": 16 * _log(rng, 8, 448),
                "experts": rng.choice([1, 1, 4, 16, 48]), "dtype": rng.choice(["f32", "bf16", "f16"])}
    return {"op": op, "rows": _log(rng, 64, 32768), "n": _log(rng, 128, 4096), "k": 16 * _log(rng, 8, 256), "experts": rng.choice([1, 4, 16, 40]),
            "dtype": rng.choice(["f32", "bf16"])}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = _drawn(rng)
        if _cost(case) <= most:
            return case


# --------------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _choice(g, tokens, experts, top_k, dropped):
    """A router's choice with uneven experts: [tokens, top_k] int32, distinct in a row; dropped rows hold -1."""
    liked = 0.5 * torch.randn(experts, generator=g, device="cuda")
    idx = (liked + 0.5 * torch.randn(tokens, experts, generator=g, device="cuda")).topk(top_k, dim=1).indices.to(torch.int32)
    if dropped:
        idx[torch.rand(tokens, generator=g, device="cuda") < dropped] = -1
    return idx


def _shares(g, rows, experts, align=1):
    """Offsets [experts + 1] of uneven segments, empty ones among them, of `rows` rows in all (a multiple of align)."""
    units = rows // align
    liked = torch.softmax(0.7 * torch.randn(experts, generator=g, device="cuda"), 0)
    at = torch.multinomial(liked, max(1, units), replacement=True, generator=g)
    counts = torch.bincount(at, minlength=experts)[:experts] * align
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    return off


def _codes(g, *shape):
    """e4m3 codes as quantising normal values with their blocks' largest at 448 leaves them."""
    out = torch.empty(shape, dtype=F8, device="cuda")
    flat = out.view(-1, shape[-1])
    for i in range(0, flat.shape[0], 1 << 15):
        part = flat[i:i + (1 << 15)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(110.0).clamp_(-448.0, 448.0))
    return out


def _pow2(g, *shape):
    return torch.exp2(torch.randint(-9, -5, shape, generator=g, device="cuda").float())


def _blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "lists":
        s["idx"] = _choice(g, case["tokens"], case["experts"], case["top_k"], case["dropped"])
    elif op == "balance":
        T, E, S = case["tokens"], case["experts"], case["sequences"]
        liked = 0.5 * torch.randn(E, generator=g, device="cuda")
        logits = liked + torch.randn(T, E, generator=g, device="cuda")
        s["idx"] = logits.topk(case["top_k"], dim=1).indices.to(torch.int32)
        s["logits"] = logits.to(FLOATS[case["dtype"]])
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        s["mask"] = (torch.rand(T, generator=g, device="cuda") >= case["masked"]) if case["masked"] else None
        s["grad"] = 0.5 + torch.rand(1, generator=g, device="cuda")
        s["coef"] = 0.01
    elif op == "quantize":
        x = torch.randn(case["tokens"], case["width"], generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(case["width"], generator=g, device="cuda"))  # some features are larger than others
        s["x"] = x.to(FLOATS[case["dtype"]])
        s["index"] = None
        if case["gather"]:
            index = torch.randint(0, case["tokens"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
            index[torch.rand(case["rows"], generator=g, device="cuda") < 0.1] = -1  # the padding behind each expert's rows
            s["index"] = index
    elif op == "matmul":
        R, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        s["x"], s["xs"] = _codes(g, R, K), _pow2(g, _blocks(K), R)
        s["w"] = _codes(g, E, N, K)
        s["ws"] = 2e-4 * (0.5 + torch.rand(E, _blocks(N), _blocks(K), generator=g, device="cuda"))
        s["offsets"] = _shares(g, R, E) if E > 1 else None
    else:
        N, K, E = case["n"], case["k"], case["experts"]
        R = _blocks(case["rows"]) * BLOCK
        s["offsets"] = _shares(g, R, E, BLOCK)
        pad = torch.rand(R, generator=g, device="cuda") < 0.05  # padded rows hold zeros
        s["xt"], s["dyt"] = _codes(g, K, R), _codes(g, N, R)
        for t in (s["xt"], s["dyt"]):
            t.view(torch.uint8).mul_((~pad).to(torch.uint8))
        s["xts"], s["dyts"] = _pow2(g, R // BLOCK, K), _pow2(g, R // BLOCK, N) * 2.0 ** -10
    return s


# ---------------------------------------------------------------------------------------------------- plain forms

def _plain_lists(s):
    idx, E, align = s["idx"], s["experts"], s["align"]
    T, K = idx.shape
    pairs = idx.reshape(-1).long()
    key = torch.where((pairs >= 0) & (pairs < E), pairs, E)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + align - 1) // align * align
    off = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    first = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = off[sorted_key] + torch.arange(T * K, device=idx.device) - first[sorted_key]
    used = sorted_key < E
    room = -(-(T * K + min(E, T * K) * (align - 1)) // align) * align
    rows = torch.full((room + 1,), -1, dtype=torch.int32, device=idx.device)
    rows[torch.where(used, place, room)] = (order // K).to(torch.int32)
    pos = torch.empty(T * K, dtype=torch.int32, device=idx.device)
    pos[order] = torch.where(used, place, -1).to(torch.int32)
    return counts.to(torch.int32), off.to(torch.int32), rows[:room], pos.view(T, K)


def _own_lists(s):
    import int4_moe_expert_gb300 as moe
    return moe.moe_expert_lists(s["idx"], s["experts"], align=s["align"])


def _segments(offsets, T):
    return torch.searchsorted(offsets[1:].long(), torch.arange(T, device=offsets.device), right=True)


def _plain_balance(s):
    x, E, K, S = s["logits"].float(), s["experts"], s["top_k"], s["sequences"]
    T = x.shape[0]
    keep = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=x.device)
    seg = _segments(s["offsets"], T)
    if s["score"] == 1:
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        sig = 1 / (1 + torch.exp(-x))
        z = sig.sum(1, keepdim=True) + 1e-20
        p = sig / z
    p = p * keep[:, None]
    sums = torch.zeros(S, E, dtype=torch.float64, device=x.device).index_add_(0, seg, p.double())
    tokens = torch.zeros(S, dtype=torch.int64, device=x.device).index_add_(0, seg, keep.long())
    counts = torch.zeros(S * E, dtype=torch.int64, device=x.device)
    counts.index_add_(0, (seg[:, None] * E + s["idx"].long()).reshape(-1), keep[:, None].expand(T, K).reshape(-1).long())
    counts = counts.view(S, E)
    n = tokens.clamp(min=1).double()
    each = s["coef"] * E / (K * S * n * n)
    loss = (each * (counts * sums).sum(1)).sum().float().reshape(1)
    up = (s["grad"].double() * each).float()[seg][:, None] * keep[:, None]
    c = counts.float()[seg]
    d = p * (c - (p * c).sum(1, keepdim=True)) * up
    if s["score"] == 0:
        d = d * (1 - sig)
    return loss, counts.to(torch.int32), sums.float(), d.to(s["logits"].dtype)


def _own_balance(s):
    import int4_moe_expert_gb300 as moe
    loss, counts, sums, tokens = moe.moe_balance_forward(s["logits"], s["idx"], s["coef"], s["score"], seq_offsets=s["offsets"], mask=s["mask"])
    d = moe.moe_balance_backward(s["logits"], s["top_k"], counts, tokens, s["coef"], s["score"], seq_offsets=s["offsets"], mask=s["mask"],
                                 grad_loss=s["grad"])
    return loss, counts, sums, d


def _plain_scale(largest):
    """The least power of two (from 2^-126) that brings `largest` to 448 or less; 1 for a block of zeros."""
    m, e = torch.frexp(largest)  # largest = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(largest > 0, torch.ldexp(torch.ones_like(largest), e), torch.ones_like(largest))


def _plain_rows(x):
    """Codes and scales of x [R, n] float32 in 1 x 128 blocks; the scales [blocks, R]."""
    R, n = x.shape
    wide = torch.zeros(R, _blocks(n) * BLOCK, device=x.device)
    wide[:, :n] = x
    wide = wide.view(R, -1, BLOCK)
    scale = _plain_scale(wide.abs().amax(2))
    return (wide / scale[:, :, None]).view(R, -1)[:, :n].to(F8), scale.t().contiguous()


def _plain_quantize(s):
    x = s["x"].float()
    if s["index"] is not None:
        x = x[s["index"].long().clamp(min=0)] * (s["index"] >= 0)[:, None]
    codes, scales = _plain_rows(x)
    if not s["both"]:
        return codes, scales
    tall = torch.zeros(_blocks(x.shape[0]) * BLOCK, x.shape[1], device=x.device)
    tall[:x.shape[0]] = x
    return (codes, scales) + _plain_rows(tall.t())


def _own_quantize(s):
    import int4_moe_expert_gb300 as moe
    return moe.moe_fp8_quantize(s["x"], rows=s["index"], transposed=s["both"])


def _spread(scale, n):
    return scale.repeat_interleave(BLOCK, dim=-1)[..., :n]


def _plain_matmul(s):
    R, N, K = s["rows"], s["n"], s["k"]
    x = s["x"].float() * _spread(s["xs"].t(), K)
    if s["offsets"] is None:
        w = s["w"][0].float() * _spread(s["ws"][0].repeat_interleave(BLOCK, dim=0)[:N], K)
        return (x @ w.t()).to(FLOATS[s["dtype"]])
    off = s["offsets"].long()
    counts = off[1:] - off[:-1]
    touched = counts.nonzero()[:, 0]
    w = s["w"].view(torch.uint8)[touched].view(F8).float() * _spread(s["ws"][touched].repeat_interleave(BLOCK, dim=1)[:, :N], K)
    most = torch.arange(int(counts.max()), device=x.device)
    at = off[touched][:, None] + most  # each touched expert's rows, the shorter ones filled up
    used = most < counts[touched][:, None]
    y = torch.bmm(x[torch.where(used, at, 0)], w.transpose(1, 2))
    out = torch.zeros(R, N, device=x.device)
    out[at[used]] = y[used]
    return out.to(FLOATS[s["dtype"]])


def _own_matmul(s):
    import int4_moe_expert_gb300 as moe
    return moe.moe_fp8_matmul(s["x"], s["xs"], s["w"] if s["offsets"] is not None else s["w"][0], s["ws"] if s["offsets"] is not None else s["ws"][0],
                              offsets=s["offsets"], out_dtype=FLOATS[s["dtype"]])


def _plain_wgrad(s):
    R = s["xt"].shape[1]
    x = torch.cat([(s["xt"].float() * _spread(s["xts"].t(), R)).t(), torch.zeros(1, s["k"], device="cuda")])
    dy = torch.cat([(s["dyt"].float() * _spread(s["dyts"].t(), R)).t(), torch.zeros(1, s["n"], device="cuda")])
    off = s["offsets"].long()
    counts = off[1:] - off[:-1]
    most = torch.arange(int(counts.max()), device=x.device)
    at = torch.where(most < counts[:, None], off[:-1, None] + most, R)  # each expert's rows, filled up with the row of zeros
    return torch.bmm(dy[at].transpose(1, 2), x[at]).to(FLOATS[s["dtype"]])


def _own_wgrad(s):
    import int4_moe_expert_gb300 as moe
    return moe.moe_fp8_wgrad(s["xt"], s["xts"], s["dyt"], s["dyts"], offsets=s["offsets"], out_dtype=FLOATS[s["dtype"]])


def run(state):
    if own:
        return {"lists": _own_lists, "balance": _own_balance, "quantize": _own_quantize, "matmul": _own_matmul, "wgrad": _own_wgrad}[state["op"]](state)
    return {"lists": _plain_lists, "balance": _plain_balance, "quantize": _plain_quantize, "matmul": _plain_matmul,
            "wgrad": _plain_wgrad}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------- exact values

def _exact_balance(s):
    logits = s["logits"].double()
    T, E = logits.shape
    K, S = s["top_k"], s["sequences"]
    keep = (s["mask"] if s["mask"] is not None else torch.ones(T, device="cuda")).double()
    off = s["offsets"].tolist()
    chosen = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    chosen.scatter_(1, s["idx"].long(), 1.0)
    chosen *= keep[:, None]
    grad = torch.zeros_like(logits)
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    sums = torch.zeros(S, E, dtype=torch.float64, device="cuda")
    for q in range(S):
        a, b = off[q], off[q + 1]
        part = logits[a:b].clone().requires_grad_(True)
        if s["score"] == 1:
            p = torch.softmax(part, dim=1)
        else:
            sig = torch.sigmoid(part)
            p = sig / (sig.sum(1, keepdim=True) + 1e-20)
        p = p * keep[a:b, None]
        n = max(1.0, float(keep[a:b].sum()))
        f = E / (K * n) * chosen[a:b].sum(0)
        one = s["coef"] / S * (f * (p.sum(0) / n)).sum()
        if b > a:
            grad[a:b] = torch.autograd.grad(one, part)[0] * s["grad"].double()
        loss += one.detach()
        sums[q] = p.detach().sum(0)
    return loss.reshape(1), None, sums, grad


def _exact_block(v):
    """Nearest e4m3 values (ties to even) of v over a block's scale, and the scale: v [..., 128] float64."""
    largest = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(largest > 0, largest, 448.0) / 448.0))
    e = torch.where(largest > 448.0 * torch.exp2(e), e + 1, e)  # log2 is rounded: settle it by comparison
    e = torch.where(largest <= 448.0 * torch.exp2(e - 1), e - 1, e)
    scale = torch.where(largest > 0, torch.exp2(e.clamp(min=-126)), torch.ones_like(e))
    u = v / scale
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step, scale[..., 0]


def _exact_rows(x):
    R, n = x.shape
    wide = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(R, -1, BLOCK)
    codes, scale = _exact_block(wide)
    return codes.view(R, -1)[:, :n], scale.t()


def _exact_quantize(s):
    x = s["x"].double()
    if s["index"] is not None:
        x = torch.cat([x, x.new_zeros(1, x.shape[1])])[torch.where(s["index"] < 0, x.shape[0], s["index"]).long()]
    codes, scales = _exact_rows(x)
    if not s["both"]:
        return codes, scales
    codes_t, scales_t = _exact_rows(torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % BLOCK)).t())
    return codes, scales, codes_t, scales_t


def _exact_matmul(s):
    R, N, K = s["rows"], s["n"], s["k"]
    out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    off = [0, R] if s["offsets"] is None else s["offsets"].tolist()
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        for i in range(_blocks(K)):  # block by block of the inner axis, its scales on the sums
            k = slice(i * BLOCK, min(K, (i + 1) * BLOCK))
            part = s["x"][a:b, k].double() @ s["w"][e][:, k].double().t()
            out[a:b] += part * s["xs"][i, a:b, None].double() * s["ws"][e, :, i].double().repeat_interleave(BLOCK)[:N]
    return out


def _exact_wgrad(s):
    off = s["offsets"].tolist()
    E, N, K = len(off) - 1, s["n"], s["k"]
    out = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            each = torch.arange(a // BLOCK, b // BLOCK, device="cuda").repeat_interleave(BLOCK)
            dy = s["dyt"][:, a:b].double() * s["dyts"][each].t().double()
            out[e] = dy @ (s["xt"][:, a:b].double() * s["xts"][each].t().double()).t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lists":
        return None  # whole numbers alone
    return {"balance": _exact_balance, "quantize": _exact_quantize, "matmul": _exact_matmul, "wgrad": _exact_wgrad}[case["op"]](s)


# ------------------------------------------------------------------------------------------------------------ work

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2, "f16": 2}
    if op == "lists":
        pairs, E, align = case["tokens"] * case["top_k"], case["experts"], case["align"]
        room = -(-(pairs + min(E, pairs) * (align - 1)) // align) * align
        return {"bytes": 4 * (2 * pairs + room + 2 * E + 1), "flops": 0}
    if op == "balance":  # the logits for the sums, again for the gradient (which needs all counts), and the gradient
        T, E, S = case["tokens"], case["experts"], case["sequences"]
        return {"bytes": 3 * T * E * size[case["dtype"]] + 4 * T * case["top_k"] + 8 * S * E, "flops": 16 * T * E}
    if op == "quantize":
        R, n, picked = case["rows"], case["width"], min(case["rows"], case["tokens"])
        out = R * n + 4 * _blocks(n) * R
        if case["both"]:
            out += n * _blocks(R) * BLOCK + 4 * n * _blocks(R)
        return {"bytes": picked * n * size[case["dtype"]] + out + (4 * R if case["gather"] else 0), "flops": 2 * R * n}
    R, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
    if op == "matmul":
        touched = min(E, R)
        return {"bytes": R * K + 4 * R * _blocks(K) + touched * (N * K + 4 * _blocks(N) * _blocks(K)) + R * N * size[case["dtype"]],
                "flops": 2 * R * N * K}
    R = _blocks(R) * BLOCK
    return {"bytes": R * (N + K) + 4 * (R // BLOCK) * (N + K) + E * N * K * size[case["dtype"]], "flops": 2 * R * N * K}
