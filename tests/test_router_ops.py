"""Token lists and the balance loss (moe_expert_lists, moe_balance_*): refusals on the host, values,
gradients and edge cases on the GPU against plain 64-bit implementations."""
import ctypes as C

import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import int4_moe_expert_gb300 as m
    return m


@pytest.fixture(scope="module")
def gpu(moe):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return moe


NEW = ["moe_expert_lists_rows", "moe_expert_lists_workspace", "moe_expert_lists", "moe_balance_workspace", "moe_balance_forward",
       "moe_balance_backward", "moe_fp8_quantize", "moe_fp8_quantize_weights", "moe_fp8_matmul", "moe_fp8_wgrad", "moe_fp8_device_error"]


def test_entry_points_are_declared_and_exported(moe):
    from pathlib import Path
    text = (Path(__file__).resolve().parents[1] / "include" / "moe.h").read_text()
    L = C.CDLL(str(moe.library_path()))
    for name in NEW:
        assert f"{name}(" in text and hasattr(L, name), name
        if not name.endswith(("_rows", "_workspace")):
            assert name in moe.__all__ and callable(getattr(moe, name)), name


# ------------------------------------------------------------------ refusals (no GPU: nothing is launched)

P = 4096          # an aligned address that no call below reaches


def test_lists_refusals(moe):
    L = moe.lib()
    call = lambda T=4, K=2, E=8, align=1, idx=P, cnt=P, off=P, rows=P, pos=P, ws=None, n=0: L.moe_expert_lists(   # noqa: E731
        idx, T, K, E, align, cnt, off, rows, pos, ws, n, None)
    assert call(T=-1) == moe.MOE_ERR_INVALID and "T=-1" in moe.moe_last_error()
    assert call(E=0) == call(E=1025) == moe.MOE_ERR_UNSUPPORTED
    assert call(K=0) == call(K=1025) == moe.MOE_ERR_UNSUPPORTED
    assert call(align=0) == call(align=4097) == moe.MOE_ERR_UNSUPPORTED
    assert call(T=1 << 30, K=8) == moe.MOE_ERR_UNSUPPORTED and "2^31" in moe.moe_last_error()
    for k in ("idx", "cnt", "off", "rows", "pos"):
        assert call(**{k: None}) == moe.MOE_ERR_INVALID
        assert call(**{k: P + 2}) == moe.MOE_ERR_INVALID
    assert call(T=100000, K=8) == moe.MOE_ERR_INVALID and "workspace" in moe.moe_last_error()
    assert call(T=100000, K=8, ws=P, n=16) == moe.MOE_ERR_INVALID
    assert L.moe_expert_lists_rows(3, 2, 8, 128) == 6 * 128 and L.moe_expert_lists_rows(1000, 8, 4, 128) == 8576
    assert L.moe_expert_lists_rows(0, 2, 8, 16) == 0 and L.moe_expert_lists_rows(-1, 2, 8, 16) == -1


def test_balance_refusals(moe):
    L = moe.lib()
    base = dict(x=P, dt=0, ld=8, T=4, E=8, idx=P, K=2, score=0, coef=0.1, seq=None, S=1, mask=None, loss=P, cnt=P, sums=P, tok=P, ws=P,
                n=1 << 20)

    def fwd(**kw):
        a = {**base, **kw}
        return L.moe_balance_forward(a["x"], a["dt"], a["ld"], a["T"], a["E"], a["idx"], a["K"], a["score"], a["coef"], a["seq"], a["S"],
                                     a["mask"], a["loss"], a["cnt"], a["sums"], a["tok"], a["ws"], a["n"], None)

    def bwd(d=P, ldd=8, g=None, **kw):
        a = {**base, **kw}
        return L.moe_balance_backward(a["x"], a["dt"], a["ld"], a["T"], a["E"], a["K"], a["score"], a["coef"], a["cnt"], a["tok"], a["seq"],
                                      a["S"], a["mask"], g, d, ldd, 0, None)
    for call in (fwd, bwd):
        for kw in (dict(x=None), dict(dt=3), dict(dt=-1), dict(ld=7), dict(T=-1), dict(K=0), dict(K=9), dict(score=2), dict(S=2),
                   dict(coef=float("nan")), dict(x=P + 1), dict(cnt=None), dict(tok=None), dict(seq=P + 1, S=2)):
            assert call(**kw) == moe.MOE_ERR_INVALID, kw
        for kw in (dict(E=0, ld=8), dict(E=1025, ld=1025), dict(S=0), dict(S=65536, seq=P)):
            assert call(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(idx=None), dict(loss=None), dict(sums=None), dict(ws=None), dict(n=8), dict(ws=P + 8)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(d=None), dict(ldd=7), dict(d=P + 2), dict(g=P + 2)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw
    assert bwd(T=0) == moe.MOE_OK


def test_balance_refuses_token_numbers_beyond_32_bits(moe):
    """The kernels step up to a block of 128 tokens past T in 32-bit token numbers, so the last 127
    values of T are refused."""
    L = moe.lib()
    most = 2**31 - 128
    fwd = lambda T, K=1: L.moe_balance_forward(P, 2, 4, T, 4, P, K, 0, 0.1, None, 1, None, P, P, P, P, P, 1 << 40, None)   # noqa: E731
    bwd = lambda T, K=1: L.moe_balance_backward(P, 2, 4, T, 4, K, 0, 0.1, P, P, None, 1, None, None, P, 4, 0, None)        # noqa: E731
    for T in (2**31 - 1, 2**31 - 8, 2**31 - 63, most + 1):
        for call in (fwd, bwd):
            assert call(T) == moe.MOE_ERR_UNSUPPORTED and f"T={T}" in moe.moe_last_error()
        assert L.moe_balance_workspace(T, 4, 1) == 0
    assert fwd(most, 0) == bwd(most, 0) == moe.MOE_ERR_INVALID           # refused for top_k, not for T
    assert L.moe_balance_workspace(most, 4, 1) >= most // 128 * 4 * 8


def test_binding_refuses_what_is_not_on_the_device(moe):
    with pytest.raises(moe.MoeError):
        moe.moe_expert_lists(torch.zeros(2, 2, dtype=torch.int32), 4)
    with pytest.raises(moe.MoeError):
        moe.moe_balance_forward(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), 0.1)


# ------------------------------------------------------------------------------------------ token lists

def lists_ref(idx, E, align):
    """Plain loops over the pairs."""
    idx = idx.tolist()
    K = len(idx[0]) if idx else 1
    pairs = [[] for _ in range(E)]
    for t, row in enumerate(idx):
        for k, e in enumerate(row):
            if 0 <= e < E:
                pairs[e].append((t, k))
    off, rows, pos = [0], [], [[-1] * K for _ in idx]
    for e in range(E):
        for i, (t, k) in enumerate(pairs[e]):
            pos[t][k] = off[e] + i
            rows.append(t)
        rows += [-1] * (-len(pairs[e]) % align)
        off.append(len(rows))
    return [len(p) for p in pairs], off, rows, pos


def check_lists(moe, idx, E, align):
    counts, off, rows, pos = moe.moe_expert_lists(idx.cuda(), E, align)
    c, o, r, p = lists_ref(idx, E, align)
    assert counts.tolist() == c and off.tolist() == o and pos.cpu().tolist() == p
    assert rows[:len(r)].tolist() == r
    assert bool((rows[len(r):] == -1).all()) and rows.numel() % align == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,E,align", [(1, 1, 1, 1), (1, 8, 256, 1), (3, 2, 5, 16), (33, 4, 7, 128), (100, 6, 300, 1), (64, 1, 1024, 2),
                                         (1024, 8, 64, 128), (1025, 8, 64, 128), (2000, 5, 1000, 4096), (30011, 8, 40, 128),
                                         (20000, 3, 1024, 1), (400000, 1, 3, 1)])
def test_lists(gpu, T, K, E, align):
    g = torch.Generator().manual_seed(T + K + E)
    idx = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32)
    check_lists(gpu, idx, E, align)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 3000])
def test_lists_extremes(gpu, T):
    check_lists(gpu, torch.full((T, 4), 2, dtype=torch.int32), 6, 128)                   # one expert has all
    check_lists(gpu, torch.full((T, 4), -1, dtype=torch.int32), 6, 16)                   # nothing routed
    far = torch.tensor([[-2**31, 6, 2**31 - 1, 5]] * T, dtype=torch.int32)               # values that are no expert
    check_lists(gpu, far, 6, 1)
    counts, off, rows, pos = gpu.moe_expert_lists(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 6, 128)
    assert counts.tolist() == [0] * 6 and off.tolist() == [0] * 7 and rows.numel() == 0 and pos.shape == (0, 4)


@pytest.mark.gpu
def test_lists_up_to_the_last_row_number(gpu):
    """Segments that end next to row 2^31: a warp's lanes behind them have numbers beyond it."""
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GB")
    T, K = 2**28 - 1, 8
    for E, align, dropped in ((3, 1, 0), (3, 2, 5), (1, 2, 1)):
        t = torch.arange(T, dtype=torch.int32, device="cuda")
        idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
        for k in range(K):
            idx[:, k] = (t + k) % E
        idx.view(-1)[T * K - dropped:] = -1
        counts, off, rows, pos = gpu.moe_expert_lists(idx, E, align)
        want = torch.zeros(E, dtype=torch.int64, device="cuda")
        for k in range(K):
            for e in range(E):
                want[e] += (idx[:, k] == e).sum()
        assert counts.tolist() == want.tolist() and rows.numel() < 2**31
        seg = [0]
        for c in counts.tolist():
            seg.append(seg[-1] + -(-c // align) * align)
        assert off.tolist() == seg and seg[-1] >= 2**31 - 16
        for k in range(K):      # every pair's row holds its token, in its expert's segment
            p, e = pos[:, k].long(), idx[:, k]
            on = e >= 0
            assert bool((p[~on] == -1).all())
            p, e = p[on], e[on].long()
            assert torch.equal(rows[p], t[on])
            assert bool((p >= off[:-1].long()[e]).all()) and bool((p < off[1:].long()[e]).all())
            del p, e, on
        assert int((rows == -1).sum()) == rows.numel() - int(counts.sum())
        del t, idx, counts, off, rows, pos
        torch.cuda.empty_cache()


@pytest.mark.gpu
def test_lists_refuses_in_the_binding(gpu):
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in (idx.long(), idx[:, ::2], idx[0], idx.cpu()):
        with pytest.raises(gpu.MoeError):
            gpu.moe_expert_lists(bad, 4)
    for kw in (dict(n_experts=0), dict(n_experts=2000), dict(n_experts=4, align=0), dict(n_experts=4, align=5000), dict(n_experts=2.5)):
        with pytest.raises(gpu.MoeError):
            gpu.moe_expert_lists(idx, **kw)


# ------------------------------------------------------------------------------------------ balance loss

def balance_ref(logits, idx, coef, score, seq, mask):
    """Loss, counts, sums, tokens and the gradient for grad_loss = 1, segment by segment in float64."""
    x = logits.double().cpu()
    T, E = x.shape
    K = idx.shape[1]
    S = len(seq) - 1
    grad = torch.zeros(T, E, dtype=torch.float64)
    size = torch.zeros(T, E, dtype=torch.float64)       # what the gradient's rounding errors are relative to
    loss, counts, sums, tokens = 0.0, [], [], []
    for s in range(S):
        rows = [t for t in range(seq[s], seq[s + 1]) if mask is None or mask[t]]
        n = max(1, len(rows))
        c = torch.zeros(E, dtype=torch.float64)
        for t in rows:
            for e in idx[t].tolist():
                if 0 <= e < E:
                    c[e] += 1
        if score == 1:
            m = x[rows].amax(1, keepdim=True) if rows else x[rows].sum(1, keepdim=True)
            ex = torch.exp(x[rows] - torch.where(torch.isinf(m), torch.zeros_like(m), m))
            z = ex.sum(1, keepdim=True)
            p = ex / torch.where(z == 0, torch.ones_like(z), z)
            f = torch.ones_like(p)
        else:
            sig = torch.sigmoid(x[rows])
            p = sig / (sig.sum(1, keepdim=True) + 1e-20)
            f = torch.sigmoid(-x[rows])
        k = coef * E / (K * S * n * n)
        loss += k * float((c * p.sum(0)).sum())
        dot = (p * c).sum(1, keepdim=True)
        grad[rows] = k * p * (c - dot) * f
        size[rows] = k * p * (c + dot) * f
        counts.append(c.int())
        sums.append(p.sum(0))
        tokens.append(len(rows))
    return loss, torch.stack(counts), torch.stack(sums), torch.tensor(tokens, dtype=torch.int32), grad, size


def check_balance(moe, logits, idx, coef, score, seq=None, mask=None, g=None):
    """Tolerances: a score is a few roundings of 2^-24 (exp within 2 of them, the sum over E in a tree),
    so 2^-19 of the value covers it; a sum over tokens adds one rounding a level and chunk; a gradient
    adds the same relative to p (c + dot), then the rounding to its type."""
    dev = "cuda"
    T = logits.shape[0]
    lo, hi = (seq[0], seq[-1]) if seq else (0, T)
    x = logits.to(dev) if not logits.is_cuda else logits
    sq = torch.tensor(seq, dtype=torch.int32, device=dev) if seq else None
    mk = mask.to(dev) if mask is not None else None
    ref = balance_ref(x, idx, coef, score, seq or [0, T], mask)
    loss, counts, sums, tokens = moe.moe_balance_forward(x, idx.to(dev), coef, score, seq_offsets=sq, mask=mk)
    assert torch.equal(counts.cpu(), ref[1]) and torch.equal(tokens.cpu(), ref[3])
    assert abs(loss.item() - ref[0]) <= 2.0 ** -18 * abs(ref[0])
    assert bool(((sums.cpu().double() - ref[2]).abs() <= 2.0 ** -18 * ref[2]).all())
    out = torch.full((T, logits.shape[1]), 7.0, dtype=logits.dtype, device=dev)
    up = None if g is None else torch.tensor([g], device=dev)
    d = moe.moe_balance_backward(x, idx.shape[1], counts, tokens, coef, score, seq_offsets=sq, mask=mk, grad_loss=up, out=out)
    assert d is out
    d = d.cpu().double()
    scale = 1.0 if g is None else g
    err = (d[lo:hi] - scale * ref[4][lo:hi]).abs()
    fin = torch.finfo(logits.dtype)
    least = fin.smallest_normal * fin.eps           # half a step of subnormal results, rounded up
    assert bool((err <= 2.0 ** -18 * scale * ref[5][lo:hi] + fin.eps / 2 * (scale * ref[4][lo:hi]).abs() + least).all())
    assert bool((d[:lo] == 7.0).all()) and bool((d[hi:] == 7.0).all())        # rows outside every segment
    fill = torch.full_like(out, 7.0)                # a new tensor, likely in this one's memory
    del fill
    n = moe.moe_balance_backward(x, idx.shape[1], counts, tokens, coef, score, seq_offsets=sq, mask=mk, grad_loss=up).cpu().double()
    assert torch.equal(n[lo:hi], d[lo:hi]) and bool((n[:lo] == 0).all()) and bool((n[hi:] == 0).all())
    return loss, counts, sums, tokens


def router(T, E, K, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = (1.5 * torch.randn(T, E, generator=g)).to(dtype)
    return x, x.float().topk(K, dim=1).indices.int()


@pytest.mark.gpu
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,K,dtype", [(1, 1, 1, torch.float32), (1, 8, 2, torch.bfloat16), (7, 13, 3, torch.float16),
                                         (65, 32, 4, torch.float32), (130, 64, 8, torch.bfloat16), (100, 100, 2, torch.float32),
                                         (70, 129, 5, torch.float32), (333, 256, 8, torch.float32), (50, 257, 8, torch.bfloat16),
                                         (40, 512, 6, torch.float32), (30, 1000, 8, torch.float16), (20, 1023, 1, torch.float32)])
def test_balance_values_and_gradient(gpu, score, T, E, K, dtype):
    x, idx = router(T, E, K, 3 * T + E, dtype)
    check_balance(gpu, x, idx, 300.0, score, g=1.25)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("seq", [[0, 200], [0, 0, 200], [0, 1, 1, 77, 200, 200], [13, 50, 51, 180]])
def test_balance_segments_and_masks(gpu, score, seq):
    x, idx = router(200, 48, 4, 5)
    g = torch.Generator().manual_seed(6)
    mask = torch.rand(200, generator=g) < 0.7
    check_balance(gpu, x, idx, 1.0, score, seq, None)
    check_balance(gpu, x, idx, 1.0, score, seq, mask)
    check_balance(gpu, x, idx, 1.0, score, seq, torch.zeros(200, dtype=torch.bool))      # no token is left
    idx[::5] = -1                                                                        # dropped choices
    idx[3] = 48
    check_balance(gpu, x, idx, 1.0, score, seq, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [0, 1])
def test_balance_small_scores_and_gradients(gpu, score):
    """Logits whose sigmoids are near the smallest numbers, and an upstream gradient that makes the scaled
    counts small too: no product of the two may underflow where the result does not."""
    x, idx = router(300, 64, 4, 11)
    for low in (-42.0, -60.0, -85.0):
        check_balance(gpu, x + low, idx, 1.0, score, g=1e-22)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 8, 40, 300, 1024])
@pytest.mark.parametrize("S", [1, 5, 30, 130, 600])
def test_balance_numbers_of_segments(gpu, S, E):
    x, idx = router(2500, E, min(E, 3), S + E)
    cut = sorted(torch.randint(0, 2501, (S - 1,), generator=torch.Generator().manual_seed(S)).tolist())
    mask = torch.rand(2500, generator=torch.Generator().manual_seed(E)) < 0.9
    check_balance(gpu, x, idx, 1.0, 1, [0] + cut + [2500], mask)


@pytest.mark.gpu
def test_balance_many_segments_and_long_ones(gpu):
    x, idx = router(3000, 16, 2, 7)
    check_balance(gpu, x, idx, 1.0, 0, sorted([0, 3000] + torch.randint(0, 3001, (700,), generator=torch.Generator().manual_seed(8)).tolist()))
    x, idx = router(20000, 16, 2, 9, torch.bfloat16)
    check_balance(gpu, x, idx, 1e4, 1, [0, 19999, 20000])


@pytest.mark.gpu
@pytest.mark.parametrize("score", [0, 1])
def test_balance_infinities_and_masked_nans(gpu, score):
    x, idx = router(64, 20, 2, 10)
    x[:, 3] = -float("inf")                      # an expert that no token may take
    x[5] = -float("inf")                         # no expert left
    x[6] = torch.finfo(torch.float32).min
    mask = torch.ones(64, dtype=torch.bool)
    mask[10:14] = False
    x[10], x[11], x[12] = float("nan"), float("inf"), -float("inf")
    check_balance(gpu, x, idx, 1.0, score, mask=mask)
    x[0, 0] = float("nan")                       # an unmasked one shows
    loss, *_ = gpu.moe_balance_forward(x.cuda(), idx.cuda(), 1.0, score)
    assert bool(loss.isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,dtype", [(8, torch.float32), (13, torch.bfloat16), (64, torch.bfloat16), (300, torch.float16), (1024, torch.float32)])
@pytest.mark.parametrize("g", [float("inf"), -float("inf"), float("nan"), 3e38])
def test_balance_masked_rows_are_zeros_for_any_upstream_gradient(gpu, score, E, dtype, g):
    """An upstream gradient that overflowed: zeros in masked rows (and outside the segments), the formula's
    infinities and NaN in the others."""
    T, K = 77, 4
    x, idx = router(T, E, K, 5, dtype)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(6)) < 0.6
    mask[60:70] = False                                       # a segment without a token left
    x[~mask] = float("nan")
    seq = torch.tensor([3, 20, 60, 70, 75], dtype=torch.int32, device="cuda")
    x, idx, m = x.cuda(), idx.cuda(), mask.cuda()
    _, counts, _, tokens = gpu.moe_balance_forward(x, idx, 0.5, score, seq_offsets=seq, mask=m)
    up = torch.tensor([g], device="cuda")
    d = gpu.moe_balance_backward(x, K, counts, tokens, 0.5, score, seq_offsets=seq, mask=m, grad_loss=up)
    inside = torch.zeros(T, dtype=torch.bool)
    inside[3:75] = True
    assert bool((d.cpu()[~mask | ~inside] == 0).all())
    if g != 3e38:
        assert not bool(d.cpu()[mask & inside].float().isfinite().all(1).any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (4, 4), (8, 0)])
def test_balance_strided_rows(gpu, dtype, pad, shift):
    """Logits as columns of a wider buffer, at aligned and unaligned places."""
    x, idx = router(77, 64, 4, 11, dtype)
    wide = torch.full((77, 64 + pad + shift), float("nan"), dtype=dtype, device="cuda")
    view = wide[:, shift:shift + 64]
    view.copy_(x)
    check_balance(gpu, view, idx, 1.0, 0)
    loss, counts, sums, tokens = gpu.moe_balance_forward(view, idx.cuda(), 1.0)
    want = gpu.moe_balance_backward(view, 4, counts, tokens, 1.0)
    out = torch.zeros(77, 64 + pad + shift, dtype=dtype, device="cuda")
    gpu.moe_balance_backward(view, 4, counts, tokens, 1.0, out=out[:, shift:shift + 64])
    assert torch.equal(out[:, shift:shift + 64], want)
    assert int(out[:, :shift].abs().sum()) == 0 and int(out[:, shift + 64:].abs().sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("score", [0, 1])
def test_balance_gradient_against_differences(gpu, score):
    """Central differences of the float64 loss, the counts held: the formula, not the kernel's rounding."""
    x, idx = router(12, 6, 2, 12)
    seq, coef, h = [0, 5, 12], 3.0, 1e-5
    loss, counts, sums, tokens = check_balance(gpu, x, idx, coef, score, seq)
    d = gpu.moe_balance_backward(x.cuda(), 2, counts, tokens, coef, score, seq_offsets=torch.tensor(seq, dtype=torch.int32, device="cuda")).cpu()
    for t, e in [(0, 0), (4, 5), (5, 1), (11, 3)]:
        up, down = x.double().clone(), x.double().clone()
        up[t, e] += h
        down[t, e] -= h
        diff = (balance_ref(up, idx, coef, score, seq, None)[0] - balance_ref(down, idx, coef, score, seq, None)[0]) / (2 * h)
        # the difference is off by h^2 / 6 of the third derivative and 2^-52 / h of the loss
        assert abs(d[t, e].item() - diff) <= 1e-6 * max(1.0, abs(diff))


@pytest.mark.gpu
def test_balance_no_tokens(gpu):
    z = torch.zeros(0, 8, device="cuda")
    loss, counts, sums, tokens = gpu.moe_balance_forward(z, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 1.0)
    assert loss.item() == 0 and int(counts.sum()) == 0 and float(sums.sum()) == 0 and tokens.tolist() == [0]
    assert gpu.moe_balance_backward(z, 2, counts, tokens, 1.0).shape == (0, 8)


@pytest.mark.gpu
def test_balance_more_than_two_to_the_31_elements(gpu):
    """The last sequence of a call whose logits pass 2^31 elements: as in a call of its own."""
    T, E, last = 2_200_000, 1024, 300
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    tail, idx = router(last, E, 2, 13, torch.bfloat16)
    x[-last:] = tail.cuda()
    full = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    full[-last:] = idx.cuda()
    seq = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    _, counts, sums, tokens = gpu.moe_balance_forward(x, full, 2.0, seq_offsets=seq)
    _, c1, s1, t1 = gpu.moe_balance_forward(tail.cuda(), idx.cuda(), 1.0)
    assert torch.equal(counts[1], c1[0]) and tokens.tolist() == [T - last, last] and counts[0, 0] == 2 * (T - last)
    assert bool(((sums[1] - s1[0]).abs() <= 2.0 ** -18 * s1[0]).all())
    d = gpu.moe_balance_backward(x, 2, counts, tokens, 2.0, seq_offsets=seq)
    want = gpu.moe_balance_backward(tail.cuda(), 2, c1, t1, 1.0)
    assert torch.equal(d[-last:], want)


@pytest.mark.gpu
def test_balance_refuses_in_the_binding(gpu):
    x, idx = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    f = gpu.moe_balance_forward
    for bad in (lambda: f(x.double(), idx, 1.0), lambda: f(x.t(), idx, 1.0), lambda: f(x, idx[:3], 1.0), lambda: f(x, idx.long(), 1.0),
                lambda: f(x, idx, 1.0, 2), lambda: f(x, idx, 1.0, seq_offsets=seq.long()), lambda: f(x, idx, 1.0, seq_offsets=seq[:1]),
                lambda: f(x, idx, 1.0, mask=torch.ones(3, dtype=torch.bool, device="cuda")), lambda: f(x, idx, float("inf")),
                lambda: f(x, torch.zeros(4, 9, dtype=torch.int32, device="cuda"), 1.0)):
        with pytest.raises(gpu.MoeError):
            bad()
    loss, counts, sums, tokens = f(x, idx, 1.0)
    b = gpu.moe_balance_backward
    for bad in (lambda: b(x, 0, counts, tokens, 1.0), lambda: b(x, 2, counts[:, :4], tokens, 1.0), lambda: b(x, 2, counts, tokens.float(), 1.0),
                lambda: b(x, 2, counts, tokens, 1.0, out=torch.zeros(4, 8, dtype=torch.float16, device="cuda")),
                lambda: b(x, 2, counts, tokens, 1.0, grad_loss=torch.ones(2, device="cuda"))):
        with pytest.raises(gpu.MoeError):
            bad()


@pytest.mark.gpu
def test_router_ops_capture_and_side_stream(gpu):
    """Captured calls replay on the buffers' new contents; a side stream gets its own allocations; two
    graphs replay at once; repeated calls give the same bits."""
    xs, idxs = zip(*(router(3000, 64, 4, 20 + i) for i in range(3)))
    x, idx = xs[0].cuda(), idxs[0].cuda()

    def step(stream=None):
        r = gpu.moe_expert_lists(idx, 64, 128, stream=stream)
        f = gpu.moe_balance_forward(x, idx, 1.0, stream=stream)
        return [*r, *f, gpu.moe_balance_backward(x, 4, f[1], f[3], 1.0, stream=stream)]
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        idx.copy_(idxs[i])
        want = [t.clone() for t in step()]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o))
