"""The operators before and behind a layer's experts, for serving and for training: cases, plain forms and 64-bit values.

Four operators (all sizes in elements; T: tokens, E: experts, K: chosen experts a token):

  route    the choice of a router from its logits: scores, a bias for balance, groups, the K best experts, their weights;
           with `grad` also the gradient of the logits from that of the weights
  norm     root-mean-square norm of a residual stream after an addition to it, in the inputs' type, in e4m3 with one
           power-of-two scale for each 1 x 128 block, or both; with `grad` also the gradients of the stream and of the weight
  combine  the weighted sum of a token's rows in the experts' lists; with `grad` also the gradients of the rows and weights
  clip     the norm of all gradients together, and the gradients scaled to a largest norm
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128


# ---------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch of 8 sequences: latency alone
        {"name": "route_decode", "op": "route", "tokens": 8, "experts": 256, "top_k": 8, "score": 0, "bias": True, "groups": 1, "kept": 1,
         "dtype": "f32", "masked": 0.0, "renorm": True, "grad": False},
        # a long prompt through a group-limited router (4 of 8 groups), logits in 16 bits, an odd number of tokens
        {"name": "route_groups", "op": "route", "tokens": 16381, "experts": 256, "top_k": 8, "score": 0, "bias": True, "groups": 8, "kept": 4,
         "dtype": "bf16", "masked": 0.0, "renorm": True, "grad": False},
        # a training step of a softmax router without renormalised weights (its gradient reaches every logit)
        {"name": "route_softmax", "op": "route", "tokens": 32768, "experts": 64, "top_k": 8, "score": 1, "bias": False, "groups": 1, "kept": 1,
         "dtype": "bf16", "masked": 0.1, "renorm": False, "grad": True},
        # a training step of a sigmoid router with a bias for balance, padding tokens masked
        {"name": "route_train", "op": "route", "tokens": 65536, "experts": 256, "top_k": 8, "score": 0, "bias": True, "groups": 1, "kept": 1,
         "dtype": "f32", "masked": 0.1, "renorm": True, "grad": True},
        # a decode batch before a layer: float32 stream, values for the router and codes for the 8-bit experts
        {"name": "norm_decode", "op": "norm", "tokens": 4, "width": 6144, "dtype": "f32", "stream": "f32", "values": True, "codes": True,
         "grad": False},
        # a long prompt: 16-bit stream, values and codes
        {"name": "norm_prompt", "op": "norm", "tokens": 16381, "width": 6144, "dtype": "bf16", "stream": "bf16", "values": True, "codes": True,
         "grad": False},
        # a training step: 16-bit activations on a float32 stream, and the way back
        {"name": "norm_train", "op": "norm", "tokens": 32768, "width": 2048, "dtype": "bf16", "stream": "f32", "values": True, "codes": False,
         "grad": True},
        # a decode batch of 4 sequences behind its experts, the shared expert's output added
        {"name": "combine_decode", "op": "combine", "tokens": 4, "experts": 256, "top_k": 8, "width": 6144, "align": 1, "dtype": "bf16", "add": True,
         "grad": False},
        # a training step: segments of whole blocks of rows, a few dropped pairs, and the way back
        {"name": "combine_train", "op": "combine", "tokens": 16384, "experts": 64, "top_k": 8, "width": 2048, "align": 128, "dtype": "bf16",
         "add": False, "grad": True},
        # the gradients of one small layer: norms, router, a shared expert
        {"name": "clip_layer", "op": "clip", "tensors": 9, "values": 1500000, "dtype": "f32"},
        # the gradients of the layers that one card trains: few large tensors of experts, many small ones, of both types
        {"name": "clip_model", "op": "clip", "tensors": 56, "values": 700000000, "dtype": "mixed"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["route", "route", "norm", "norm", "combine", "clip"])
    if op == "route":
        score = rng.choice([0, 0, 1])
        groups = rng.choice([1, 1, 4, 8]) if score == 0 else 1
        kept = rng.randint(1, groups)
        experts = groups * max(1, _log(rng, 8, 512) // groups)
        top_k = rng.choice([k for k in (1, 2, 4, 6, 8, 12) if k <= kept * (experts // groups)])
        return {"op": op, "tokens": _log(rng, 1, 65536), "experts": experts, "top_k": top_k, "score": score,
                "bias": score == 0 and rng.random() < 0.7, "groups": groups, "kept": kept, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "masked": rng.choice([0.0, 0.2]), "renorm": top_k > 1 and rng.random() < 0.7,  # one renormalised weight is a constant
                "grad": rng.random() < 0.5}
    if op == "norm":
        dtype = rng.choice(["f32", "bf16", "f16"])
        codes = rng.random() < 0.6
        return {"op": op, "tokens": _log(rng, 1, 32768), "width": 16 * _log(rng, 4, 512) if codes or rng.random() < 0.6 else _log(rng, 64, 8192),
                "dtype": dtype, "stream": rng.choice([dtype, "f32", "none"]), "values": not codes or rng.random() < 0.5, "codes": codes,
                "grad": rng.random() < 0.5}
    if op == "combine":
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "top_k": rng.choice([1, 2, 4, 6, 8]), "width": _log(rng, 64, 8192),
                "align": rng.choice([1, 16, 128]), "dtype": rng.choice(["f32", "bf16", "f16"]), "add": rng.random() < 0.5,
                "grad": rng.random() < 0.5}
    return {"op": op, "tensors": rng.randint(1, 60), "values": _log(rng, 1000, 500000000), "dtype": rng.choice(["f32", "bf16", "mixed"])}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        case = _drawn(rng)
        if _cost(case) <= most[case["op"]]:
            return case


# --------------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _blocks(n):
    return -(-n // BLOCK)


def _room(case):
    """Rows that the lists of any choice of this size need."""
    pairs, align = case["tokens"] * case["top_k"], case["align"]
    return -(-(pairs + min(case["experts"], pairs) * (align - 1)) // align) * align


def _lists(idx, E, align, room):
    """Rows (token of each, -1 without one) and pos (row of each pair, -1 for dropped ones) of a choice."""
    T, K = idx.shape
    pairs = idx.reshape(-1).long()
    key = torch.where(pairs >= 0, pairs, E)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + align - 1) // align * align
    order = torch.argsort(key, stable=True)
    at = key[order]
    start = torch.cat([padded.cumsum(0) - padded, padded.new_zeros(1)])
    first = torch.cat([counts.cumsum(0) - counts, counts.new_zeros(1)])
    place = start[at] + torch.arange(T * K, device=idx.device) - first[at]
    rows = torch.full((room + 1,), -1, dtype=torch.int32, device=idx.device)
    rows[torch.where(at < E, place, room)] = (order // K).to(torch.int32)
    pos = torch.empty(T * K, dtype=torch.int32, device=idx.device)
    pos[order] = torch.where(at < E, place, -1).to(torch.int32)
    rows[room] = -1
    return rows[:room].contiguous(), pos.view(T, K)


def _parts(case):
    """Sizes of the tensors: three large ones in four hold most values, the others fall off; and their types."""
    n, left, sizes = case["tensors"], case["values"], []
    for i in range(n):
        size = left if i == n - 1 else max(1, left // (3 if i < 8 else 2 + n // 8) + 7 * i)
        size = max(1, min(size, left - (n - 1 - i)))
        sizes.append(size)
        left -= size
    kinds = ["bf16" if case["dtype"] == "bf16" or (case["dtype"] == "mixed" and i % 3 == 1) else "f32" for i in range(n)]
    return list(zip([max(1, s) for s in sizes], kinds))


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "route":
        T, E = case["tokens"], case["experts"]
        liked = 0.5 * torch.randn(E, generator=g, device="cuda")
        s["logits"] = (liked + torch.randn(T, E, generator=g, device="cuda")).to(FLOATS[case["dtype"]])
        s["b"] = 0.1 * torch.randn(E, generator=g, device="cuda") - 0.3 * liked if case["bias"] else None
        s["mask"] = (torch.rand(T, generator=g, device="cuda") >= case["masked"]) if case["masked"] else None
        s["dw"] = torch.randn(T, case["top_k"], generator=g, device="cuda")
        s["scale"] = 2.5
    elif op == "norm":
        T, H, dt = case["tokens"], case["width"], FLOATS[case["dtype"]]
        s["x"] = torch.randn(T, H, generator=g, device="cuda").to(dt)
        s["res"] = None
        if case["stream"] != "none":
            res = torch.randn(T, H, generator=g, device="cuda")
            res *= 2 * torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))  # some features of the stream are larger than others
            s["res"] = res.to(FLOATS[case["stream"]])
        s["w"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
        s["eps"] = 1e-5
        if case["grad"]:
            s["dy"] = torch.randn(T, H, generator=g, device="cuda").to(dt)
            s["dh"] = torch.randn(T, H, generator=g, device="cuda").to(FLOATS[case["stream"]] if s["res"] is not None else dt)
    elif op == "combine":
        T, E, K, N, dt = case["tokens"], case["experts"], case["top_k"], case["width"], FLOATS[case["dtype"]]
        liked = 0.5 * torch.randn(E, generator=g, device="cuda")
        idx = (liked + 0.5 * torch.randn(T, E, generator=g, device="cuda")).topk(K, dim=1).indices.to(torch.int32)
        idx[torch.rand(T, K, generator=g, device="cuda") < 0.02] = -1
        R = _room(case)
        s["tokens_of"], s["pos"] = _lists(idx, E, case["align"], R)
        s["rows"] = torch.randn(R, N, generator=g, device="cuda").to(dt)
        s["w"] = 2.5 * torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
        s["more"] = torch.randn(T, N, generator=g, device="cuda").to(dt) if case["add"] else None
        s["dy"] = torch.randn(T, N, generator=g, device="cuda").to(dt) if case["grad"] else None
    else:
        s["grads"], s["out"] = [], []
        for n, kind in _parts(case):
            x = torch.empty(n, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g).mul_(10.0 ** (-2 - n % 3))
            s["grads"].append(x.to(FLOATS[kind]))
            s["out"].append(torch.empty_like(s["grads"][-1]))
        s["most"] = 1.0
    return s


# ---------------------------------------------------------------------------------------------------- plain forms

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _plain_choice(s):
    """The K best experts of every token; scores compared in 64 bits, since neighbours can be nearer than 32 bits tell."""
    x = s["logits"].double()
    T, E = x.shape
    key = x if s["score"] == 1 or s["b"] is None else _sigmoid(x) + s["b"].double()
    if s["groups"] > 1:
        score = _sigmoid(x) if s["b"] is None else key
        best = score.view(T, s["groups"], -1).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        on = torch.zeros(T, s["groups"], dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(on.repeat_interleave(E // s["groups"], dim=1), key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, -1)
    return idx.to(torch.int32)


def _plain_route(s):
    idx = _plain_choice(s)
    at, used, scale = idx.clamp(min=0).long(), (idx >= 0).float(), s["scale"]
    x = s["logits"].float()
    if s["score"] == 1:
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = _sigmoid(x)
    chosen = p.gather(1, at) * used
    total = chosen.sum(1, keepdim=True) + 1e-20
    w = scale * chosen / total if s["renorm"] else scale * chosen
    if not s["grad"]:
        return idx, w
    d = s["dw"] * used * scale
    if s["renorm"]:
        d = (d - (d * chosen).sum(1, keepdim=True) / total) / total * used
    dp = torch.zeros_like(x).scatter_add_(1, at, d)
    dx = p * (dp - (dp * p).sum(1, keepdim=True)) if s["score"] == 1 else dp * p * (1 - p)
    return idx, w, dx.to(s["logits"].dtype)


def _own_route(s):
    import int4_moe_expert_gb300 as moe
    idx, w = moe.moe_route_forward(s["logits"], s["top_k"], bias=s["b"], score_func=s["score"], n_group=s["groups"], topk_group=s["kept"],
                                   norm_topk=s["renorm"], routed_scale=s["scale"], mask=s["mask"])
    if not s["grad"]:
        return idx, w
    return idx, w, moe.moe_route_backward(s["logits"], idx, s["dw"], score_func=s["score"], norm_topk=s["renorm"], routed_scale=s["scale"])


def _plain_scale(largest):
    """The least power of two (from 2^-126) that brings `largest` to 448 or less; 1 for a block of zeros."""
    m, e = torch.frexp(largest)  # largest = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(largest > 0, torch.ldexp(torch.ones_like(largest), e), torch.ones_like(largest))


def _plain_norm(s):
    x, T, H = s["x"], s["tokens"], s["width"]
    h = x if s["res"] is None else (s["res"].float() + x.float()).to(s["res"].dtype)
    v = h.float()
    r64 = torch.rsqrt(v.double().square().mean(1) + s["eps"])  # 64 bits: the codes' scales step at a border
    rstd = r64.float()
    w = s["w"].float()
    y = v * rstd[:, None] * w
    out = {"rstd": rstd}
    if s["res"] is not None:
        out["h"] = h
    if s["values"]:
        out["y"] = y.to(x.dtype)
    if s["codes"]:
        wide = torch.zeros(T, _blocks(H) * BLOCK, dtype=torch.float64, device=x.device)
        wide[:, :H] = (v.double() * w.double()).abs()
        scale = _plain_scale(wide.view(T, -1, BLOCK).amax(2) * r64[:, None]).float()
        out["codes"] = (y / scale.repeat_interleave(BLOCK, dim=1)[:, :H]).to(F8)
        out["scales"] = scale.t().contiguous()
    if s["grad"]:
        dy = s["dy"].float()
        n = v * rstd[:, None]
        d = dy * w
        out["dw"] = (dy * n).sum(0)
        out["dh"] = ((d - n * (d * n).mean(1, keepdim=True)) * rstd[:, None] + s["dh"].float()).to(h.dtype)
    return out


def _own_norm(s):
    import int4_moe_expert_gb300 as moe
    got = moe.moe_norm_forward(s["x"], residual=s["res"], weight=s["w"], eps=s["eps"], values=s["values"], quantize=s["codes"])
    y, h, rstd = got[:3]
    out = {"rstd": rstd}
    if s["res"] is not None:
        out["h"] = h
    if s["values"]:
        out["y"] = y
    if s["codes"]:
        out["codes"], out["scales"] = got[3:]
    if s["grad"]:
        out["dh"], out["dw"] = moe.moe_norm_backward(s["dy"], h, rstd, weight=s["w"], grad_h=s["dh"])
    return out


def _plain_combine(s):
    rows, pos, w = s["rows"].float(), s["pos"], s["w"]
    used = (pos >= 0).float()
    each = rows[pos.clamp(min=0).long()]  # [T, K, N]
    y = (each * (w * used)[:, :, None]).sum(1)
    if s["more"] is not None:
        y = y + s["more"].float()
    y = y.to(s["rows"].dtype)
    if not s["grad"]:
        return y
    dy = s["dy"].float()
    dw = (each * dy[:, None, :]).sum(2) * used
    at = torch.where(pos >= 0, pos.long(), rows.shape[0])
    d = torch.zeros(rows.shape[0] + 1, rows.shape[1], dtype=s["rows"].dtype, device=rows.device)
    d[at.reshape(-1)] = (w[:, :, None] * dy[:, None, :]).to(d.dtype).view(-1, rows.shape[1])
    d[rows.shape[0]] = 0
    return y, d[:-1], dw


def _own_combine(s):
    import int4_moe_expert_gb300 as moe
    y = moe.moe_combine_forward(s["rows"], s["pos"], s["w"], add=s["more"])
    if not s["grad"]:
        return y
    d, dw = moe.moe_combine_backward(s["dy"], s["rows"], s["pos"], s["tokens_of"], s["w"])
    return y, d, dw


def _plain_clip(s):
    total = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["grads"]]).sum()  # long sums
    norm = total.sqrt().float().reshape(1)
    c = torch.clamp(s["most"] / (norm + 1e-6), max=1.0)
    for x, y in zip(s["grads"], s["out"]):
        y.copy_(x.float() * c)
    return norm, s["out"]


def _own_clip(s):
    import int4_moe_expert_gb300 as moe
    norm = moe.moe_grad_norm(s["grads"])
    moe.moe_grad_clip(s["grads"], norm, s["most"], out=s["out"])
    return norm, s["out"]


def run(state):
    if own:
        return {"route": _own_route, "norm": _own_norm, "combine": _own_combine, "clip": _own_clip}[state["op"]](state)
    return {"route": _plain_route, "norm": _plain_norm, "combine": _plain_combine, "clip": _plain_clip}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------- exact values

def _exact_best(key, k):
    """The k largest of every row one by one, the lowest index first among equals."""
    key, E = key.clone(), key.shape[1]
    number = torch.arange(E, device=key.device).expand_as(key)
    got = []
    for _ in range(k):
        best = torch.where(key == key.amax(1, keepdim=True), number, E).amin(1)
        got.append(best)
        key.scatter_(1, best[:, None], -math.inf)
    return torch.stack(got, 1)


def _exact_route(s):
    x = s["logits"].double()
    T, E = x.shape
    score = torch.sigmoid(x) + (s["b"].double() if s["b"] is not None else 0.0) if s["score"] == 0 else x
    if s["groups"] > 1:
        two = score.view(T, s["groups"], -1).topk(min(2, E // s["groups"]), dim=2).values.sum(2)
        out = torch.ones(T, s["groups"], dtype=torch.bool, device=x.device).scatter_(1, _exact_best(two, s["kept"]), False)
        score = score.masked_fill(out.repeat_interleave(E // s["groups"], 1), -math.inf)
    idx = _exact_best(score, s["top_k"])
    x.requires_grad_(True)
    p = torch.softmax(x, 1) if s["score"] == 1 else torch.sigmoid(x)
    w = p.gather(1, idx)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = s["scale"] * w
    if s["mask"] is not None:
        w = w * s["mask"][:, None]
    if not s["grad"]:
        return None, w.detach()
    return None, w.detach(), torch.autograd.grad((w * s["dw"].double()).sum(), x)[0]


def _exact_codes(v):
    """Nearest e4m3 values (ties to even) of v over its 1 x 128 blocks' scales, and the scales: v [T, H] float64."""
    T, H = v.shape
    v = torch.nn.functional.pad(v, (0, -H % BLOCK)).view(T, -1, BLOCK)
    largest = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(largest > 0, largest, 448.0) / 448.0))
    e = torch.where(largest > 448.0 * torch.exp2(e), e + 1, e)  # log2 is rounded: settle it by comparison
    e = torch.where(largest <= 448.0 * torch.exp2(e - 1), e - 1, e)
    scale = torch.where(largest > 0, torch.exp2(e.clamp(min=-126)), torch.ones_like(e))
    u = v / scale
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(u / step) * step).view(T, -1)[:, :H], scale[..., 0].t()


def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:  # the stream is what its type holds: the sum in 32 bits, then rounded to it
        h = (s["x"].float() + s["res"].float()).to(s["res"].dtype).double()
    h.requires_grad_(True)
    w = s["w"].double().requires_grad_(True)
    rstd = 1 / torch.sqrt((h * h).mean(1) + s["eps"])
    y = h * rstd[:, None] * w
    out = {"rstd": rstd.detach()}
    if s["res"] is not None:
        out["h"] = h.detach()
    if s["values"]:
        out["y"] = y.detach()
    if s["codes"]:
        out["codes"], out["scales"] = _exact_codes(y.detach())
    if s["grad"]:
        dh, out["dw"] = torch.autograd.grad(y, (h, w), s["dy"].double())
        out["dh"] = dh + s["dh"].double()
    return out


def _exact_combine(s):
    rows, w = s["rows"].double(), s["w"].double()
    R, N = rows.shape
    y = torch.zeros(s["tokens"], N, dtype=torch.float64, device="cuda") if s["more"] is None else s["more"].double()
    d, dw = torch.zeros(R + 1, N, dtype=torch.float64, device="cuda"), torch.zeros_like(w)
    for k in range(s["top_k"]):
        on, at = s["pos"][:, k] >= 0, s["pos"][:, k].long()
        one = torch.where(on[:, None], rows[at.clamp(min=0)], 0.0)
        y = y + w[:, k, None] * one
        if s["grad"]:
            dy = s["dy"].double()
            dw[:, k] = torch.einsum("tn,tn->t", one, dy)
            d[torch.where(on, at, R)] = w[:, k, None] * dy
    return (y, d[:R], dw) if s["grad"] else y


def _exact_clip(s):
    squares = [float(torch.linalg.vector_norm(x.double())) ** 2 for x in s["grads"]]
    norm = math.sqrt(math.fsum(squares))
    c = min(1.0, s["most"] / (norm + 1e-6))
    return torch.tensor([norm], dtype=torch.float64, device="cuda"), [x.double() * c for x in s["grads"]]


def exact(case, seed):
    return {"route": _exact_route, "norm": _exact_norm, "combine": _exact_combine, "clip": _exact_clip}[case["op"]](prepare(case, seed))


# ------------------------------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "route":  # the logits once, the choice; the gradient: chosen logits again (all of them without renormalised softmax weights), written whole
        T, E, K, el = case["tokens"], case["experts"], case["top_k"], SIZE[case["dtype"]]
        bytes_ = T * E * el + 8 * T * K + (4 * E if case["bias"] else 0) + (T if case["masked"] else 0)
        flops = 8 * T * E
        if case["grad"]:
            dense = case["score"] == 1 and not case["renorm"]
            bytes_ += T * E * el + 8 * T * K + (T * E * el if dense else T * K * el)
            flops += (8 * T * E if dense else 12 * T * K)
        return {"bytes": bytes_, "flops": flops}
    if op == "norm":
        T, H, el = case["tokens"], case["width"], SIZE[case["dtype"]]
        st = 0 if case["stream"] == "none" else SIZE[case["stream"]]
        one = T * H
        bytes_ = one * (el + 2 * st + (el if case["values"] else 0) + (1 if case["codes"] else 0)) + 4 * T + el * H
        bytes_ += 4 * T * _blocks(H) if case["codes"] else 0
        flops = 6 * one
        if case["grad"]:  # the stream, dy and the stream's own gradient read, the gradient written
            bytes_ += one * (el + 3 * (st or el)) + 4 * T + 4 * H
            flops += 12 * one
        return {"bytes": bytes_, "flops": flops}
    if op == "combine":
        T, K, N, el = case["tokens"], case["top_k"], case["width"], SIZE[case["dtype"]]
        bytes_ = T * K * N * el + T * N * el * (2 if case["add"] else 1) + 8 * T * K
        flops = 2 * T * K * N
        if case["grad"]:
            bytes_ += T * N * el + T * K * N * el + _room(case) * (N * el + 4) + 12 * T * K
            flops += 3 * T * K * N
        return {"bytes": bytes_, "flops": flops}
    return {"bytes": sum(2 * n * SIZE[kind] for n, kind in _parts(case)), "flops": 3 * case["values"]}
