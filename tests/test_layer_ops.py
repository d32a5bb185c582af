"""The operators before and behind a layer's experts (moe_route_*, moe_norm_*, moe_combine_*, moe_grad_*):
refusals on the host, values, gradients and edge cases on the GPU against plain 64-bit implementations,
and a training step that runs them together with the lists, quantisers and products."""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
inf, nan = math.inf, math.nan


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


def half_step(t):
    return torch.finfo(t).eps / 2


def gen(*seed):
    return torch.Generator().manual_seed(sum(int(s) * (2 * i + 1) for i, s in enumerate(seed)))


def strided(x, pad, shift):
    """x [T, n] in rows pad elements longer, the first one shift elements behind the allocation's start."""
    T, n = x.shape
    buf = torch.zeros(T * (n + pad) + shift, dtype=x.dtype, device="cuda")
    v = buf[shift:shift + T * (n + pad)].view(T, n + pad)[:, :n]
    v.copy_(x)
    return v


NEW = ["moe_route_forward", "moe_route_backward", "moe_norm_forward", "moe_norm_workspace", "moe_norm_backward", "moe_combine_forward",
       "moe_combine_backward", "moe_grad_norm_workspace", "moe_grad_norm", "moe_grad_clip"]


def test_entry_points_are_declared_and_exported(moe):
    from pathlib import Path
    text = (Path(__file__).resolve().parents[1] / "include" / "moe.h").read_text()
    L = C.CDLL(str(moe.library_path()))
    for name in NEW:
        assert f"{name}(" in text and hasattr(L, name), name
        if not name.endswith("_workspace"):
            assert name in moe.__all__ and callable(getattr(moe, name)), name


# ------------------------------------------------------------------ refusals (no GPU: nothing is launched)

P = 4096          # an aligned address that no call below reaches


def test_route_refusals(moe):
    L = moe.lib()
    base = dict(x=P, dt=0, ld=8, T=4, E=8, b=None, K=2, score=0, G=1, kept=1, norm=1, scale=1.0, mask=None, idx=P, w=P, dw=P, d=P, ldd=8)

    def fwd(**kw):
        a = {**base, **kw}
        return L.moe_route_forward(a["x"], a["dt"], a["ld"], a["T"], a["E"], a["b"], a["K"], a["score"], a["G"], a["kept"], a["norm"],
                                   a["scale"], a["mask"], a["idx"], a["w"], None)

    def bwd(**kw):
        a = {**base, **kw}
        return L.moe_route_backward(a["x"], a["dt"], a["ld"], a["T"], a["E"], a["idx"], a["K"], a["score"], a["norm"], a["scale"], a["dw"],
                                    a["d"], a["ldd"], 0, None)
    for call in (fwd, bwd):
        for kw in (dict(x=None), dict(dt=3), dict(ld=7), dict(T=-1), dict(K=0), dict(K=9), dict(E=64, ld=64, ldd=64, K=33), dict(score=2),
                   dict(norm=2), dict(scale=nan), dict(scale=inf), dict(x=P + 1), dict(idx=None), dict(idx=P + 2)):
            assert call(**kw) == moe.MOE_ERR_INVALID, kw
        for kw in (dict(E=0, ld=8), dict(E=1025, ld=1025, ldd=1025)):
            assert call(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
        assert call(T=0, x=None, idx=None, w=None, dw=None, d=None) == moe.MOE_OK
    for kw in (dict(w=None), dict(w=P + 2), dict(b=P + 2), dict(G=0), dict(G=3), dict(E=66, ld=66, G=33), dict(G=4, kept=0), dict(G=4, kept=5),
               dict(G=4, kept=1, K=3), dict(score=1, G=2, kept=2), dict(score=1, b=P)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(dw=None), dict(d=None), dict(ldd=7), dict(d=P + 2), dict(dw=P + 1)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw


def test_norm_refusals(moe):
    L = moe.lib()
    base = dict(x=P, dt=2, ldx=64, r=P, sd=0, ldr=64, w=P, wd=2, T=4, H=64, eps=1e-5, h=P, ldh=64, y=P, ldy=64, rs=P, q=P, s=P)

    def fwd(**kw):
        a = {**base, **kw}
        return L.moe_norm_forward(a["x"], a["dt"], a["ldx"], a["r"], a["sd"], a["ldr"], a["w"], a["wd"], a["T"], a["H"], a["eps"], a["h"], a["ldh"],
                                  a["y"], a["ldy"], a["rs"], a["q"], a["s"], None)
    for kw in (dict(x=None), dict(h=None), dict(dt=3), dict(sd=1), dict(wd=1), dict(T=-1), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(q=None),
               dict(s=None), dict(ldx=63), dict(ldr=63), dict(ldh=63), dict(ldy=63), dict(x=P + 1), dict(x=P + 8), dict(r=P + 8), dict(w=P + 8),
               dict(y=P + 2), dict(ldx=68), dict(ldr=65), dict(q=P + 8), dict(rs=P + 2), dict(s=P + 2), dict(h=P + 2)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(H=0), dict(H=16385, ldx=16385, ldr=16385, ldh=16385, ldy=16385), dict(H=40), dict(H=63)):
        assert fwd(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    assert fwd(T=0, x=None, r=None, w=None) == moe.MOE_OK
    back = dict(dy=P, dt=2, lddy=64, h=P, sd=0, ldh=64, rs=P, w=P, wd=2, g=P, ldg=64, T=4, H=64, o=P, ldo=64, dw=P, ws=P, n=1 << 20)

    def bwd(**kw):
        a = {**back, **kw}
        return L.moe_norm_backward(a["dy"], a["dt"], a["lddy"], a["h"], a["sd"], a["ldh"], a["rs"], a["w"], a["wd"], a["g"], a["ldg"], a["T"], a["H"],
                                   a["o"], a["ldo"], a["dw"], a["ws"], a["n"], None)
    for kw in (dict(dy=None), dict(h=None), dict(rs=None), dict(o=None), dict(dt=-1), dict(sd=1), dict(wd=1), dict(T=-1), dict(lddy=63), dict(ldh=63),
               dict(ldg=63), dict(ldo=63), dict(ws=None), dict(ws=P + 8), dict(n=64), dict(dw=P + 2), dict(dy=P + 1), dict(g=P + 2), dict(rs=P + 1)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw
    assert bwd(H=0) == bwd(H=20000, lddy=20000, ldh=20000, ldg=20000, ldo=20000) == moe.MOE_ERR_UNSUPPORTED
    assert bwd(T=0, dw=None, dy=None) == moe.MOE_OK
    assert L.moe_norm_workspace(0, 64) == L.moe_norm_workspace(-1, 64) == L.moe_norm_workspace(4, 20000) == 0 < L.moe_norm_workspace(1, 1)


def test_combine_refusals(moe):
    L = moe.lib()
    base = dict(r=P, dt=2, ld=8, R=16, N=8, pos=P, T=4, K=2, w=P, add=P, lda=8, y=P, yd=2, ldy=8)

    def fwd(**kw):
        a = {**base, **kw}
        return L.moe_combine_forward(a["r"], a["dt"], a["ld"], a["R"], a["N"], a["pos"], a["T"], a["K"], a["w"], a["add"], a["lda"], a["y"], a["yd"],
                                     a["ldy"], None)
    for kw in (dict(r=None), dict(pos=None), dict(y=None), dict(dt=3), dict(yd=-1), dict(T=-1), dict(R=-1), dict(ld=7), dict(lda=7), dict(ldy=7),
               dict(r=P + 1), dict(y=P + 1), dict(add=P + 1), dict(pos=P + 2), dict(w=P + 2)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(N=0), dict(N=131073, ld=131073, lda=131073, ldy=131073), dict(K=0), dict(K=33), dict(T=2**31 - 1, N=131072, ld=131072, lda=131072, ldy=131072)):
        assert fwd(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    assert fwd(T=0, r=None, pos=None, y=None) == moe.MOE_OK
    back = dict(dy=P, dt=2, lddy=8, r=P, ld=8, R=16, N=8, pos=P, T=4, K=2, tok=P, w=P, d=P, ldd=8, dw=P)

    def bwd(**kw):
        a = {**back, **kw}
        return L.moe_combine_backward(a["dy"], a["dt"], a["lddy"], a["r"], a["ld"], a["R"], a["N"], a["pos"], a["T"], a["K"], a["tok"], a["w"], a["d"],
                                      a["ldd"], a["dw"], None)
    for kw in (dict(dy=None), dict(r=None), dict(pos=None), dict(tok=None), dict(dt=3), dict(T=-1), dict(R=-1), dict(ld=7), dict(lddy=7), dict(ldd=7),
               dict(dy=P + 1), dict(d=P + 1), dict(tok=P + 2), dict(pos=P + 1), dict(w=P + 2), dict(dw=P + 2)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(N=0), dict(K=0), dict(K=33), dict(T=2**30 + 1)):
        assert bwd(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    assert bwd(T=0, R=0, dy=None, pos=None, tok=None, r=None) == moe.MOE_OK
    assert bwd(d=None, dw=None) == moe.MOE_OK


def test_grad_refusals(moe):
    L = moe.lib()

    def lists(*ts):       # (address, dtype, size)
        return ((C.c_void_p * len(ts))(*[t[0] for t in ts]), (C.c_int32 * len(ts))(*[t[1] for t in ts]), (C.c_int64 * len(ts))(*[t[2] for t in ts]))

    def norm(*ts, n=None, ws=P, size=1 << 20, to=P):
        p, d, s = lists(*ts)
        return L.moe_grad_norm(len(ts) if n is None else n, p, d, s, to, ws, size, None)

    def clip(*ts, most=1.0, out=None, norm=P):
        p, d, s = lists(*ts)
        o = None if out is None else (C.c_void_p * len(out))(*out)
        return L.moe_grad_clip(len(ts), p, d, s, norm, most, o, None)
    good = (P, 0, 16)
    for call in (norm, clip):
        for bad in ((P, 3, 16), (P, 0, -1), (None, 0, 1), (P + 2, 0, 4), (P + 1, 2, 4)):
            assert call(good, bad) == moe.MOE_ERR_INVALID, bad
        assert call((P, 0, 1 << 45), good) == moe.MOE_ERR_UNSUPPORTED
    assert norm(good, to=None) == norm(good, to=P + 2) == norm(good, ws=None) == norm(good, ws=P + 8) == norm(good, size=8) == moe.MOE_ERR_INVALID
    assert norm(good, n=-1) == moe.MOE_ERR_INVALID and norm(good, n=65537) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_grad_norm(2, None, None, None, P, P, 1 << 20, None) == moe.MOE_ERR_INVALID
    for most in (-1.0, nan, inf):
        assert clip(good, most=most) == moe.MOE_ERR_INVALID
    assert clip(good, norm=None) == moe.MOE_ERR_INVALID
    # outputs on top of other tensors
    for ts, out in ([(good, good), None], [(good, (P + 60, 0, 4)), None], [(good, (P + 4, 2, 1)), None], [(good,), [P + 4]],
                    [(good, (2 * P, 0, 16)), [4 * P, 4 * P + 32]], [(good, (2 * P, 0, 16)), [2 * P, 4 * P]], [(good,), [None]], [(good,), [P + 2]],
                    [((P, 0, 1000), (2 * P, 0, 1), (P + 2000, 0, 1)), None]):
        assert clip(*ts, out=out) == moe.MOE_ERR_INVALID, (ts, out)
    assert clip((P, 0, 0), (P, 0, 0)) == moe.MOE_OK == clip()                 # nothing to scale: nothing is launched
    assert L.moe_grad_norm_workspace(-1) == L.moe_grad_norm_workspace(65537) == 0 < L.moe_grad_norm_workspace(0) < L.moe_grad_norm_workspace(600)


def test_outputs_on_top_of_what_others_read_are_refused(moe):
    L, Q = moe.lib(), P + 4096
    assert L.moe_route_backward(P, 0, 8, 4, 8, Q, 2, 0, 1, 1.0, Q, P, 8, 0, None) == moe.MOE_ERR_INVALID
    assert L.moe_combine_forward(P, 0, 8, 4, 8, Q, 4, 2, Q, None, 0, P, 0, 8, None) == moe.MOE_ERR_INVALID
    assert L.moe_combine_backward(Q, 0, 8, P, 8, 4, 8, Q, 4, 2, Q, Q, P, 8, Q, None) == moe.MOE_ERR_INVALID
    assert L.moe_combine_backward(P, 0, 8, Q, 8, 4, 8, Q, 4, 2, Q, Q, P, 8, Q, None) == moe.MOE_ERR_INVALID


def test_norm_refuses_outputs_on_top_of_other_tensors(moe):
    L, T, H = moe.lib(), 4, 64
    far = {n: P + 65536 * (i + 1) for i, n in enumerate("xrwhyscb")}

    def fwd(dt=2, sd=0, ld=64, quant=True, **kw):
        a = {**far, **kw}
        return L.moe_norm_forward(a["x"], dt, ld, a["r"], sd, ld, a["w"], dt, T, H, 1e-5, a["h"], ld, a["y"], ld, a["s"],
                                  a["c"] if quant else None, a["b"] if quant else None, None)
    x, r, w, h, y, s, c, b = (far[n] for n in "xrwhyscb")
    for kw in (dict(y=x, r=None), dict(y=x + 128, r=None), dict(y=x - 128, r=None), dict(y=h, sd=2), dict(y=h + 16), dict(y=x + 16), dict(y=r), dict(y=r + 256, sd=2),
               dict(h=r + 256), dict(h=r - 16), dict(h=x), dict(h=x + 128, sd=2), dict(h=r + 4, quant=False), dict(y=x + 2, quant=False), dict(y=w), dict(w=h),
               dict(s=x), dict(s=y + 4), dict(s=h + 1020), dict(c=x), dict(c=y + 16), dict(c=w), dict(b=r), dict(b=c + 252), dict(b=s + 12), dict(s=c)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw
    # columns that run into the next one's, in rows of one buffer; single rows inside another tensor's rows
    assert fwd(ld=128, r=None, y=x + 112) == fwd(ld=128, r=None, y=x + 144) == fwd(ld=128, h=r + 240) == moe.MOE_ERR_INVALID


def test_norm_gradient_refuses_outputs_on_top_of_other_tensors(moe):
    L, T, H = moe.lib(), 4, 64
    far = {n: P + 1048576 * (i + 1) for i, n in enumerate("dhsgwozk")}

    def bwd(dt=2, sd=0, ld=64, **kw):
        a = {**far, **kw}
        return L.moe_norm_backward(a["d"], dt, ld, a["h"], sd, ld, a["s"], a["w"], dt, a["g"], ld, T, H, a["o"], ld, a["z"], a["k"], 1 << 19, None)
    d, h, s, g, w, o, z, k = (far[n] for n in "dhsgwozk")
    for kw in (dict(o=h + 256), dict(o=h - 256), dict(o=g + 4), dict(o=d), dict(o=d + 128, sd=2), dict(o=s), dict(o=s - 1020), dict(o=w), dict(z=o), dict(z=o + 1020),
               dict(k=d), dict(k=h), dict(k=g), dict(k=o), dict(k=z), dict(k=w), dict(k=s), dict(ld=128, o=h + 144), dict(ld=128, o=g - 144)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw


def test_route_refuses_outputs_on_top_of_other_tensors(moe):
    L, T, E, K = moe.lib(), 4, 64, 2
    x, b, m, i, w, d = (P + 65536 * (k + 1) for k in range(6))

    def fwd(i=i, w=w, b=b, ld=E, dt=0):
        return L.moe_route_forward(x, dt, ld, T, E, b, K, 0, 1, 1, 1, 1.0, m, i, w, None)
    for kw in (dict(i=x), dict(w=x + 1020), dict(i=x - 28), dict(i=b), dict(w=b + 252), dict(i=m), dict(w=m - 28), dict(i=w), dict(w=i + 28), dict(i=x + 228, ld=128, dt=2)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw

    def bwd(d=d, ld=E, ldd=E, i=i, w=w, dt=0, add=0):
        return L.moe_route_backward(x, dt, ld, T, E, i, K, 0, 1, 1.0, w, d, ldd, add, None)
    for kw in (dict(d=x), dict(d=x + 256), dict(d=x - 256), dict(d=x + 4), dict(d=x + 256, ld=192), dict(d=x + 256, ldd=192), dict(d=x + 252, ld=128, ldd=128),
               dict(d=x - 252, ld=128, ldd=128), dict(d=i), dict(d=w + 16), dict(d=w - 1020), dict(d=x + 128, dt=2, add=1)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw


def test_combine_refuses_outputs_on_top_of_other_tensors(moe):
    L, T, R, N, K = moe.lib(), 4, 16, 64, 2
    r, y, a, q, w, t, d, z = (P + 65536 * (k + 1) for k in range(8))

    def fwd(y=y, a=a, ld=N, ldy=N, dt=0, yt=0):
        return L.moe_combine_forward(r, dt, ld, R, N, q, T, K, w, a, N, y, yt, ldy, None)
    for kw in (dict(y=r), dict(y=r + 256), dict(y=r + 4), dict(y=r - 1020), dict(y=r + 15 * 256), dict(y=r + 256, ld=192), dict(y=r + 252, ld=128, ldy=128),
               dict(y=a + 256), dict(y=a - 4), dict(y=a, ldy=128), dict(y=q), dict(y=w - 1020), dict(y=r + 128, yt=2)):
        assert fwd(**kw) == moe.MOE_ERR_INVALID, kw

    def bwd(d=d, z=z, dy=y, ld=N, ldd=N):
        return L.moe_combine_backward(dy, 0, N, r, ld, R, N, q, T, K, t, w, d, ldd, z, None)
    for kw in (dict(d=r), dict(d=r + 256), dict(d=r - 4), dict(d=y), dict(d=y - 15 * 256), dict(d=r + 256, ld=192), dict(d=q), dict(d=t - 4092), dict(d=w), dict(d=z),
               dict(z=d + 16), dict(z=r), dict(z=y + 1020), dict(z=q + 28), dict(z=t), dict(z=w + 4), dict(d=r + 252, ld=128, ldd=128)):
        assert bwd(**kw) == moe.MOE_ERR_INVALID, kw


def test_grad_norm_on_top_of_gradients_is_refused(moe):
    """The clipping's blocks read the norm while others write; the norm's blocks write their sums while others read."""
    L, n = moe.lib(), 1000
    g, h, ws, far = P, P + 65536, P + 131072, P + 262144
    ptr = lambda *a: (C.c_void_p * len(a))(*a)   # noqa: E731
    kinds, sizes = (C.c_int32 * 2)(0, 2), (C.c_int64 * 2)(n, n)
    for norm in (g, g + 4 * n - 4, h, h + 2 * n - 4):
        assert L.moe_grad_clip(2, ptr(g, h), kinds, sizes, norm, 1.0, None, None) == moe.MOE_ERR_INVALID
        assert L.moe_grad_clip(2, ptr(far, far + 65536), kinds, sizes, norm, 1.0, ptr(g, h), None) == moe.MOE_ERR_INVALID
        assert L.moe_grad_norm(2, ptr(g, h), kinds, sizes, norm, ws, 1 << 16, None) == moe.MOE_ERR_INVALID
    for w in (g, g + 4 * n - 16, h):
        assert L.moe_grad_norm(2, ptr(g, h), kinds, sizes, far, w, 1 << 16, None) == moe.MOE_ERR_INVALID
    assert L.moe_grad_norm(2, ptr(g, h), kinds, sizes, ws + 16, ws, 1 << 16, None) == moe.MOE_ERR_INVALID


def test_combine_refuses_more_blocks_than_a_grid_has(moe):
    """Rows off the boundaries have fewer columns a warp than the others: the limit is theirs, and a refusal, not a failed launch."""
    L, T, far = moe.lib(), 2**31 - 1, 1 << 50
    for N, dt in ((1023, 0), (1021, 2), (997, 1)):
        assert L.moe_combine_forward(P, dt, N, 16, N, far, T, 2, None, None, N, 2 * far, dt, N, None) == moe.MOE_ERR_UNSUPPORTED, N


def test_binding_refuses_what_is_not_on_the_device(moe):
    x, i = torch.zeros(2, 16), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: moe.moe_route_forward(x, 1), lambda: moe.moe_norm_forward(x), lambda: moe.moe_combine_forward(x, i),
                 lambda: moe.moe_route_backward(x, i, torch.zeros(2, 1)), lambda: moe.moe_grad_norm([x])):
        with pytest.raises(moe.MoeError):
            call()


# ------------------------------------------------------------------------------------------ routing

def route_ref(x, K, bias=None, score=0, G=1, kept=1, renorm=True, scale=1.0, mask=None):
    """Choice and weights in float64; NaN ranks with -infinity, the lower index wins a tie."""
    v = x.detach().double().cpu()
    T, E = v.shape
    b = 0.0 if bias is None else bias.double().cpu()
    sig = torch.sigmoid(v)
    key = v if score == 1 or bias is None else sig + b
    if G > 1:
        each = torch.nan_to_num(sig + b, nan=-inf, posinf=inf, neginf=-inf).view(T, G, E // G).sort(2, descending=True).values[:, :, :2].sum(2)
        order = torch.nan_to_num(each, nan=-inf, posinf=inf, neginf=-inf).sort(dim=1, descending=True, stable=True).indices[:, :kept]
        on = torch.zeros(T, G, dtype=torch.bool).scatter_(1, order, True).repeat_interleave(E // G, 1)
        key = torch.where(on, key, -inf)
    key = torch.where(torch.isnan(key), -inf, key)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = route_weights(v, idx, score, renorm, scale)
    if mask is not None:
        off = ~mask.cpu()
        idx[off], w[off] = -1, 0
    return idx, w


def route_weights(v, idx, score, renorm, scale):
    p = torch.softmax(v, 1) if score == 1 else torch.sigmoid(v)
    w = p.gather(1, idx.clamp(min=0)) * (idx >= 0)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return scale * w


def check_route(moe, x, K, dw_seed=0, **kw):
    """A score is within 2^-21 of its value (exp 2 units, a sum, a quotient; the softmax's sum a tree), a
    weight within 2^-20, the sum over K and the quotient included.  The gradient: 2^-18 of the sizes of
    its terms, then the rounding to its type."""
    bias, mask = kw.get("bias"), kw.get("mask")
    T, E = x.shape
    args = {**kw, "bias": None if bias is None else bias.cuda(), "mask": None if mask is None else mask.cuda()}
    xd = x if x.is_cuda else x.cuda()
    idx, w = moe.moe_route_forward(xd, K, bias=args["bias"], score_func=kw.get("score", 0), n_group=kw.get("G", 1), topk_group=kw.get("kept", 1),
                                   norm_topk=kw.get("renorm", True), routed_scale=kw.get("scale", 1.0), mask=args["mask"])
    ref, want = route_ref(x, K, **kw)
    assert torch.equal(idx.cpu().long(), ref)
    assert bool(((w.cpu().double() - want).abs() <= 2.0 ** -20 * want.abs() + 1e-30).all())
    dw = torch.randn(T, K, generator=gen(dw_seed, T, E))
    score, renorm, scale = kw.get("score", 0), kw.get("renorm", True), kw.get("scale", 1.0)
    d = moe.moe_route_backward(xd, idx, dw.cuda(), score_func=score, norm_topk=renorm, routed_scale=scale)
    grad, size = route_grad_ref(x.detach().double().cpu(), ref, dw.double(), score, renorm, scale)
    tol = 2.0 ** -18 * size + half_step(x.dtype) * grad.abs() + torch.finfo(x.dtype).tiny
    assert bool(((d.cpu().double() - grad).abs() <= tol).all())
    return idx, w


def route_grad_ref(v, idx, dw, score, renorm, scale):
    """The formulas' gradient and the size that its roundings are relative to."""
    T, E = v.shape
    used, at = idx >= 0, idx.clamp(min=0)
    p = torch.softmax(v, 1) if score == 1 else torch.sigmoid(v)
    ch, d = p.gather(1, at) * used, dw * used
    f = (1 - p) if score == 0 else torch.ones_like(p)
    z = ch.sum(1, keepdim=True) + (1e-20 if renorm else 0)
    q = ch / z if renorm else ch
    if renorm or score == 0:
        dot = (q * d).sum(1, keepdim=True) if renorm else torch.zeros(T, 1, dtype=torch.float64)
        top = (q * d).abs().sum(1, keepdim=True) if renorm else torch.zeros(T, 1, dtype=torch.float64)
        g = scale * q * (d - dot) * f.gather(1, at)
        s = abs(scale) * q * (d.abs() + top) * f.gather(1, at)
        return torch.zeros_like(v).scatter_add_(1, at, g * used), torch.zeros_like(v).scatter_add_(1, at, s * used)
    de = torch.zeros_like(v).scatter_add_(1, at, d)
    dot, top = (q * d).sum(1, keepdim=True), (q * d).abs().sum(1, keepdim=True)
    any_ = used.any(1, keepdim=True)
    return torch.where(any_, scale * p * (de - dot), 0.0), torch.where(any_, abs(scale) * p * (de.abs() + top), 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,dtype,kw", [
    (1, 1, 1, F32, {}), (1, 256, 8, F32, dict(b=1)), (3, 8, 8, BF16, dict(score=1)), (7, 13, 3, F16, dict(renorm=False)),
    (33, 22, 8, F16, dict(score=1)), (500, 22, 8, F32, {}), (65, 16, 16, F32, dict(score=1, renorm=False)), (130, 40, 6, BF16, dict(b=1)),
    (129, 64, 8, BF16, dict(score=1, renorm=False)), (257, 64, 6, F32, dict(b=1, masked=0.3)), (100, 100, 5, F32, dict(score=1, masked=0.5)),
    (77, 128, 8, F16, dict(b=1, G=8, kept=3)), (300, 256, 8, F32, dict(b=1, G=8, kept=4, masked=0.1)), (64, 256, 8, BF16, dict(G=16, kept=2)),
    (50, 256, 12, F32, dict(b=1)), (41, 300, 8, F32, dict(b=1, scale=2.5)), (20, 512, 8, BF16, dict(score=1, scale=-1.5)),
    (19, 60, 32, F32, dict(b=1)), (9, 1000, 32, F16, dict(score=1, renorm=False)), (9, 1024, 32, F32, dict(b=1, G=32, kept=5)),
    (12, 96, 4, F32, dict(G=32, kept=2)), (30, 7, 2, BF16, dict(G=7, kept=3)), (4000, 256, 8, F32, dict(b=1, masked=0.1))])
def test_route_values_and_gradient(gpu, T, E, K, dtype, kw):
    g = gen(T, E, K)
    kw = dict(kw)
    x = torch.randn(T, E, generator=g).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g) if kw.pop("b", 0) else None
    p = kw.pop("masked", 0)
    mask = torch.rand(T, generator=g) >= p if p else None
    check_route(gpu, x, K, bias=bias, mask=mask, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("E,K", [(5, 3), (32, 8), (64, 8), (256, 8), (256, 32), (1024, 32)])
def test_route_ties_go_to_the_lowest_index(gpu, E, K):
    g = gen(E, K)
    for x in (torch.zeros(3, E), torch.full((3, E), -0.0), torch.randint(0, 3, (9, E), generator=g).float(), torch.randint(0, 2, (9, E), generator=g) * -0.0,
              (torch.randn(9, E, generator=g) * 2).round() / 2):
        for kw in (dict(), dict(bias=torch.zeros(E)), dict(score=1), dict(bias=(torch.arange(E) % 2).float())):
            check_route(gpu, x, K, **kw)
    if E % 8 == 0 and K <= 4 * (E // 8):
        for x in (torch.zeros(3, E), torch.randint(0, 2, (9, E), generator=g).float()):
            check_route(gpu, x, K, G=8, kept=4)
            check_route(gpu, x, K, G=8, kept=4, bias=torch.zeros(E))


@pytest.mark.gpu
@pytest.mark.parametrize("E,G,dtype,shift", [(64, 4, F32, 0), (64, 4, BF16, 1), (128, 8, F16, 0), (160, 4, F32, 0), (160, 8, BF16, 0), (200, 8, F32, 0), (250, 5, F16, 0),
                                             (255, 15, F32, 0), (256, 8, BF16, 0), (256, 8, F32, 1), (256, 16, F16, 0), (512, 8, F32, 0), (1000, 4, BF16, 0), (256, 32, F32, 0)])
def test_route_groups_of_every_layout(gpu, E, G, dtype, shift):
    """Groups that lanes hold in runs of one, two and four logits; ties, keys near one another, rows of one value, NaN and infinities."""
    T = 67
    g = gen(E, G, shift)
    K = min(8, E // G)
    x = torch.randn(T, E, generator=g)
    x[:9] = (x[:9] * 2).round() / 2
    x[9:18] = torch.randint(0, 2, (9, E), generator=g).float()
    x[18] = 0.0
    x[19, ::3] = nan
    x[20, 1::2] = -inf
    x[21] = -inf
    x = x.to(dtype)
    bias = 0.2 * torch.randn(E, generator=g)
    near = (0.7 + 1e-8 * torch.randperm(E, generator=g).double() - torch.sigmoid(x[40].double())).float()      # row 40: all keys next to 0.7
    for b in (None, torch.zeros(E), bias, near):
        for kept in sorted({1, (G + 1) // 2, G}):
            v = strided(x, shift, shift)
            idx, w = gpu.moe_route_forward(v, K, bias=None if b is None else b.cuda(), n_group=G, topk_group=kept)
            ref, want = route_ref(x, K, bias=b, G=G, kept=kept)
            assert torch.equal(idx.cpu().long(), ref), (kept, (idx.cpu() != ref).nonzero()[:4])
            ok = ~torch.isnan(want)
            assert bool(((w.cpu().double() - want)[ok].abs() <= 2.0 ** -20 * want[ok] + 1e-30).all()) and torch.equal(torch.isnan(w.cpu()), ~ok)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [64, 128, 256, 512, 1024])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,G", [(1, 8, 1), (37, 6, 1), (70, 12, 1), (41, 8, 4)])
def test_route_experts_that_fill_the_lanes(gpu, E, dtype, T, K, G):
    """Rows without an end inside a run, on their boundary and off it; the last expert is among the choices."""
    g = gen(E, T)
    x = torch.randn(T, E, generator=g)
    x[:, E - 1] = 4.0
    x = x.to(dtype)
    bias = 0.2 * torch.randn(E, generator=g)
    for b in (None, bias):
        for v in (x.cuda(), strided(x, 1, 1), strided(x, 8, 0)):
            check_route(gpu, v, K, bias=b, G=G, kept=max(1, G // 2))


@pytest.mark.gpu
@pytest.mark.parametrize("E,K,G,dtype", [(64, 6, 1, F32), (256, 8, 1, BF16), (256, 8, 8, F32), (1000, 32, 1, F32), (96, 4, 4, F16), (40, 8, 1, F32), (33, 33 - 1, 1, F32)])
def test_route_many_equal_keys(gpu, E, K, G, dtype):
    """Rows with more equal keys than a warp has lanes: of one logit, of few, with infinities, NaN, and neighbours that float32 does not tell apart."""
    T = 24
    g = gen(E, K, G)
    x = torch.zeros(T, E)
    x[1] = -3.5
    x[2] = torch.randint(0, 2, (E,), generator=g).float()
    x[3] = torch.randint(0, 3, (E,), generator=g).float() - 40.0
    x[4, E // 2:] = -inf
    x[5, ::3] = nan
    x[6, 3] = inf
    x[7] = nan
    x[8] = -inf
    x[9, 1::2] = -0.0
    x[10, E - K // 2:] = 2.0
    x[11] = torch.randn(E, generator=g)
    x[12] = 90.0                                       # a sigmoid of 1
    x[13] = (torch.arange(E) % 2) * 1e-6
    x[14, :5] = inf
    x = x.to(dtype)
    off = torch.zeros(E)
    off[torch.randperm(E, generator=g)[K // 2:]] = -inf          # fewer experts than choices
    lone = torch.zeros(E)
    lone[E - 1] = inf
    step = (0.25 + 2.0 ** -26 * torch.randint(0, 3, (E,), generator=g).double()).float()
    for score, bias in ((0, None), (1, None), (0, torch.zeros(E)), (0, off), (0, lone), (0, step), (0, torch.full((E,), nan))):
        for kept in sorted({1, G}) if score == 0 else (1,):
            if K > kept * (E // G) or (score == 1 and G > 1):
                continue
            idx, _ = gpu.moe_route_forward(x.cuda(), K, bias=None if bias is None else bias.cuda(), score_func=score, n_group=G, topk_group=kept)
            ref, _ = route_ref(x, K, bias=bias, score=score, G=G, kept=kept)
            assert torch.equal(idx.cpu().long(), ref), (score, kept, (idx.cpu() != ref).nonzero()[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("gap", [0.0, 1e-12, 1e-9, 3e-8, 1e-7, 1e-6])
def test_route_keys_nearer_than_float32_tells(gpu, gap):
    """Keys sigmoid(l) + bias that are `gap` apart: the order is that of their float64 values."""
    E, T = 64, 40
    g = gen(7)
    x = torch.randn(T, E, generator=g)
    sig = torch.sigmoid(x.double())
    bias = (0.7 + gap * torch.randperm(E, generator=g).double() - sig[0]).float()          # row 0: all keys next to 0.7
    check_route(gpu, x, 8, bias=bias)
    check_route(gpu, x, 8, bias=bias, G=8, kept=3)
    check_route(gpu, x - 40.0, 4, bias=torch.full((E,), 0.25))                             # sigmoids of 1e-17
    check_route(gpu, x + 20.0, 4, bias=torch.full((E,), 0.25))                             # next to 1


@pytest.mark.gpu
def test_route_infinities_and_nan(gpu):
    E, K = 24, 4
    x = torch.randn(8, E, generator=gen(3))
    x[0] = nan
    x[1] = -inf
    x[2, 3] = nan
    x[3, 5] = inf
    x[4, :E - 2] = -inf
    x[5, 1::2] = nan
    x[6, 0], x[6, 1] = inf, inf
    for score, bias in ((0, None), (0, torch.linspace(-1, 1, E)), (1, None)):
        for renorm in (True, False):
            idx, w = gpu.moe_route_forward(x.cuda(), K, bias=None if bias is None else bias.cuda(), score_func=score, norm_topk=renorm)
            ref, want = route_ref(x, K, bias=bias, score=score, renorm=renorm)
            assert torch.equal(idx.cpu().long(), ref), (score, renorm)
            if score == 0:
                ok = ~torch.isnan(want)
                assert bool(((w.cpu().double() - want)[ok].abs() <= 2.0 ** -20 * want[ok]).all()) and torch.equal(torch.isnan(w.cpu()), ~ok)
            assert bool((w[1] == 0).all()) or score == 0 and not renorm
            assert bool((w[7].cpu() - want[7]).abs().max() <= 2.0 ** -20)
    big = torch.full((2, E), torch.finfo(F32).min)          # masks of the type's lowest value
    big[0, 7:9] = 0.0
    check_route(gpu, big, K, score=1)
    check_route(gpu, big, K)


@pytest.mark.gpu
@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
@pytest.mark.parametrize("E,dtype", [(8, F32), (13, BF16), (64, BF16), (300, F16), (1024, F32)])
def test_route_masked_tokens(gpu, score, renorm, E, dtype):
    """Masked tokens have no choice and a gradient of zeros, whatever their logits and the gradient hold."""
    T, K = 37, 4
    x = torch.randn(T, E, generator=gen(E)).to(dtype)
    mask = torch.arange(T) % 3 != 1
    x[1] = nan
    x[4] = inf
    idx, w = gpu.moe_route_forward(x.cuda(), K, score_func=score, norm_topk=renorm, mask=mask.cuda())
    ref, want = route_ref(x, K, score=score, renorm=renorm, mask=mask)
    assert torch.equal(idx.cpu().long(), ref) and bool((w.cpu()[~mask] == 0).all())
    dw = torch.randn(T, K, generator=gen(1))
    dw[~mask] = nan
    d = gpu.moe_route_backward(x.cuda(), idx, dw.cuda(), score_func=score, norm_topk=renorm)
    assert bool((d.cpu()[~mask] == 0).all()) and bool(torch.isfinite(d.float()).all())
    none = gpu.moe_route_forward(x.cuda(), K, score_func=score, mask=torch.zeros(T, dtype=torch.bool, device="cuda"))
    assert bool((none[0] == -1).all()) and bool((none[1] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (4, 4), (8, 0)])
@pytest.mark.parametrize("E", [64, 256])
def test_route_strided_rows(gpu, dtype, pad, shift, E):
    T, K = 45, 8
    x = torch.randn(T, E, generator=gen(pad, shift, E)).to(dtype)
    v = strided(x, pad, shift)
    for score, renorm in ((0, True), (1, False)):
        idx, w = check_route(gpu, v, K, score=score, renorm=renorm)
        dw = torch.randn(T, K, generator=gen(2))
        buf = torch.full((T * (E + pad) + shift,), 7.0, dtype=dtype, device="cuda")
        out = buf[shift:shift + T * (E + pad)].view(T, E + pad)
        gpu.moe_route_backward(v, idx, dw.cuda(), score_func=score, norm_topk=renorm, out=out[:, :E])
        grad, size = route_grad_ref(x.double(), idx.cpu().long(), dw.double(), score, renorm, 1.0)
        assert bool(((out[:, :E].cpu().double() - grad).abs() <= 2.0 ** -18 * size + half_step(dtype) * grad.abs() + torch.finfo(dtype).tiny).all())
        assert bool((out[:, E:] == 7).all()) and bool((buf[:shift] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
@pytest.mark.parametrize("E,K", [(6, 3), (64, 12), (300, 32)])
def test_route_gradient_of_repeated_and_foreign_experts(gpu, score, renorm, E, K):
    """An expert twice in a row gets the sum of its gradients; entries outside [0, E) have no weight."""
    T = 21
    g = gen(E, K)
    x = torch.randn(T, E, generator=g)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    idx[0] = 2
    idx[1, 0] = idx[1, K - 1] = E - 1
    idx[2] = -1
    for i, v in enumerate((E, -2**31, 2**31 - 1)):
        idx[3 + i, 1] = v
    dw = torch.randn(T, K, generator=g)
    known = torch.where((idx >= 0) & (idx < E), idx, -1).long()
    grad, size = route_grad_ref(x.double(), known, dw.double(), score, renorm, 1.5)
    d = gpu.moe_route_backward(x.cuda(), idx.cuda(), dw.cuda(), score_func=score, norm_topk=renorm, routed_scale=1.5)
    # K equal terms at most meet in one expert: K roundings more
    assert bool(((d.cpu().double() - grad).abs() <= (2.0 ** -18 + K * 2.0 ** -24) * size + 1e-37).all())
    # on top of what is there
    for dtype in (F32, BF16):
        base = torch.randn(T, E, generator=g).to(dtype)
        out = base.cuda()
        gpu.moe_route_backward(x.to(dtype).cuda(), idx.cuda(), dw.cuda(), score_func=score, norm_topk=renorm, routed_scale=1.5, out=out, accumulate=True)
        grad, size = route_grad_ref(x.to(dtype).double(), known, dw.double(), score, renorm, 1.5)
        want = base.double() + grad
        tol = (2.0 ** -18 + K * 2.0 ** -24) * size + 2.0 ** -23 * want.abs() + (half_step(dtype) if dtype != F32 else 0) * want.abs() + 1e-37
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
        assert torch.equal(out[2].cpu(), base[2])


@pytest.mark.gpu
@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
def test_route_gradient_against_differences(gpu, score, renorm):
    T, E, K, e = 5, 12, 4, 1e-5
    x = torch.randn(T, E, generator=gen(9), dtype=torch.float64)
    idx, _ = route_ref(x, K, score=score)
    dw = torch.randn(T, K, generator=gen(10))
    d = gpu.moe_route_backward(x.float().cuda(), idx.int().cuda(), dw.cuda(), score_func=score, norm_topk=renorm).cpu().double()
    f = lambda v: (route_weights(v, idx, score, renorm, 1.0) * dw.double()).sum()   # noqa: E731
    for t in range(T):
        for j in range(E):
            a, b = x.clone(), x.clone()
            a[t, j] += e
            b[t, j] -= e
            # central differences: e^2 times a third derivative of order 1, and 2^-53 / e; logits rounded to float32
            assert abs(float((f(a) - f(b)) / (2 * e)) - float(d[t, j])) <= 1e-6 + 2.0 ** -18


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_gradient_beside_its_logits(gpu, dtype):
    """Logits and their gradient in columns of one buffer, or in every other of its rows; rows in common are refused."""
    T, E, K = 33, 64, 4
    x = torch.randn(T, E, generator=gen(E)).to(dtype).cuda()
    dw = torch.randn(T, K, generator=gen(2)).cuda()
    idx, _ = gpu.moe_route_forward(x, K)
    want = gpu.moe_route_backward(x, idx, dw)
    for both in (torch.zeros(T, 2, E, dtype=dtype, device="cuda"), torch.zeros(T, 5, E, dtype=dtype, device="cuda")):
        both[:, 0] = x
        gpu.moe_route_backward(both[:, 0], idx, dw, out=both[:, 1])
        assert torch.equal(both[:, 0], x) and torch.equal(both[:, 1], want) and bool((both[:, 2:] == 0).all())
    flat = torch.zeros(T + 1, E, dtype=dtype, device="cuda")
    for a, b in ((flat[:-1], flat[1:]), (flat[1:], flat[:-1]), (flat.view(-1)[:T * E].view(T, E), flat.view(-1)[1:T * E + 1].view(T, E))):
        with pytest.raises(gpu.MoeError):
            gpu.moe_route_backward(a, idx, dw, out=b)


@pytest.mark.gpu
def test_route_agrees_with_the_layer_router(gpu):
    """The same choice as moe_route_noalloc's where its float32 logits leave no doubt."""
    H, E, K, T = 256, 64, 6, 8
    g = gen(21)
    w, b, x = torch.randn(E, H, generator=g) / 16, 0.1 * torch.randn(E, generator=g), torch.randn(T, H, generator=g)
    for kw in (dict(), dict(n_group=8, topk_group=3), dict(score_func=1), dict(norm_topk=0)):
        cfg = gpu.make_config(H, E, K, 32, routed_scale=2.5, **kw)
        idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
        wt = torch.empty(T, K, device="cuda")
        gpu.moe_route_noalloc(cfg, w.cuda(), b.cuda(), x.cuda(), T, idx, wt)
        logits = x.double() @ w.double().t()
        soft = kw.get("score_func", 0) == 1
        i2, w2 = gpu.moe_route_forward(logits.float().cuda(), K, bias=None if soft else b.cuda(), score_func=int(soft), n_group=kw.get("n_group", 1),
                                       topk_group=kw.get("topk_group", 1), norm_topk=bool(kw.get("norm_topk", 1)), routed_scale=2.5)
        key = logits if soft else torch.sigmoid(logits) + b.double()
        if kw.get("n_group"):
            two = key.view(T, 8, 8).topk(2).values.sum(2).sort(1, descending=True).values
            clear = two[:, 2] - two[:, 3] > 1e-4
        else:
            clear = torch.ones(T, dtype=torch.bool)
        top = key.sort(1, descending=True).values
        clear &= (top[:, :-1] - top[:, 1:]).amin(1) > 1e-5
        assert int(clear.sum()) >= 2
        assert torch.equal(idx.cpu()[clear], i2.cpu()[clear])
        assert bool(((wt - w2).cpu()[clear].abs() <= 1e-4).all())      # logits to 256 roundings of float32


@pytest.mark.gpu
def test_route_no_tokens(gpu):
    idx, w = gpu.moe_route_forward(torch.zeros(0, 16, device="cuda"), 4)
    assert idx.shape == w.shape == (0, 4)
    assert gpu.moe_route_backward(torch.zeros(0, 16, device="cuda"), idx, w).shape == (0, 16)


@pytest.mark.gpu
def test_route_more_than_two_to_the_31_elements(gpu):
    if torch.cuda.mem_get_info()[0] < 40 * 2**30:
        pytest.skip("needs 40 GB")
    T, E, K = 2**25 + 77, 65, 4
    x = torch.randn(T, E, device="cuda", dtype=BF16)
    idx, w = gpu.moe_route_forward(x, K)
    dw = torch.randn(T, K, device="cuda")
    d = gpu.moe_route_backward(x, idx, dw, norm_topk=True)
    for at in (0, T // 2, T - 40):
        i2, w2 = gpu.moe_route_forward(x[at:at + 40].contiguous(), K)
        assert torch.equal(idx[at:at + 40], i2) and torch.equal(w[at:at + 40], w2)
        assert torch.equal(d[at:at + 40], gpu.moe_route_backward(x[at:at + 40].contiguous(), i2, dw[at:at + 40].contiguous()))


@pytest.mark.gpu
def test_route_refuses_in_the_binding(gpu):
    x = torch.zeros(4, 16, device="cuda")
    i, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    for bad in (x.double(), x[0], x.t(), x.cpu()):
        with pytest.raises(gpu.MoeError):
            gpu.moe_route_forward(bad, 2)
    for kw in (dict(top_k=0), dict(top_k=17), dict(top_k=2.5), dict(top_k=2, bias=w), dict(top_k=2, bias=torch.zeros(16, device="cuda").half()),
               dict(top_k=2, mask=torch.ones(3, dtype=torch.bool, device="cuda")), dict(top_k=2, score_func=1, bias=torch.zeros(16, device="cuda")),
               dict(top_k=2, n_group=3), dict(top_k=5, n_group=4, topk_group=1), dict(top_k=2, routed_scale=inf), dict(top_k=2, score_func=5)):
        with pytest.raises(gpu.MoeError):
            gpu.moe_route_forward(x, **kw)
    for kw in (dict(topk_idx=i.long()), dict(grad_w=w.half()), dict(grad_w=w[:3]), dict(out=x.half()), dict(out=x[:, :8]), dict(accumulate=True)):
        with pytest.raises(gpu.MoeError):
            gpu.moe_route_backward(**{**dict(logits=x, topk_idx=i, grad_w=w), **kw})


# ------------------------------------------------------------------------------------------ norm

def norm_ref(x, res, w, eps):
    h = x if res is None else (x.float() + res.float()).to(res.dtype)
    v = h.double()
    r = 1 / torch.sqrt((v * v).mean(1) + eps)
    return h, r, v * r[:, None] * (1.0 if w is None else w.double())


def scales_ref(y):
    """Scales [blocks, T] of y [T, H] float64 (finite)."""
    T, H = y.shape
    m = torch.nn.functional.pad(y, (0, -H % 128)).view(T, -1, 128).abs().amax(2)
    f, e = torch.frexp(m)
    s = torch.ldexp(torch.ones_like(m), (e - 9 + (f > 0.875).int()).clamp(min=-126))
    return torch.where(m > 0, s, 1.0).t()


def check_codes(codes, scales, y):
    """Scales equal; a code is the nearest e4m3 value, but float32's y is within 2^-18 of y."""
    T, H = y.shape
    s = scales_ref(y)
    assert torch.equal(scales.cpu().double(), s)
    u = y / s.t().repeat_interleave(128, 1)[:, :H]
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    assert bool(((codes.cpu().float().double() - u).abs() <= step / 2 + 2.0 ** -18 * u.abs()).all())


def check_norm(moe, x, res=None, w=None, eps=1e-5, quantize=False, values=True, out=None, inputs=None):
    """y: the sum of squares of at most 32 elements a thread and 10 levels, half of it in the root, and
    three more roundings: 2^-18 of the value, then the rounding to its type."""
    xd, rd = inputs or (x.cuda(), None if res is None else res.cuda())
    wd = None if w is None else w.cuda()
    got = moe.moe_norm_forward(xd, residual=rd, weight=wd, eps=eps, values=values, quantize=quantize, out=out)
    h, r, y = norm_ref(x, res, w, eps)
    assert torch.equal(got[1].cpu(), h) and (res is not None or got[1] is xd or got[1].data_ptr() == xd.data_ptr())
    assert bool(((got[2].cpu().double() - r).abs() <= 2.0 ** -18 * r).all())
    if values:
        assert got[0].dtype == x.dtype
        assert bool(((got[0].cpu().double() - y).abs() <= (2.0 ** -18 + half_step(x.dtype)) * y.abs() + torch.finfo(x.dtype).tiny).all())
    else:
        assert got[0] is None
    if quantize:
        check_codes(got[3], got[4], y)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,dtype,stream,wt,quantize", [
    (1, 1, F32, F32, F32, False), (1, 6144, F32, F32, F32, True), (4, 6144, BF16, BF16, BF16, True), (3, 16, F16, None, F16, True),
    (5, 144, BF16, F32, F32, True), (300, 256, F16, F16, None, True), (9, 272, F32, None, F32, True), (1000, 1024, BF16, F32, BF16, True),
    (700, 1040, F32, F32, F32, True), (310, 2048, BF16, F32, BF16, True), (7, 2047, F16, F16, F16, False), (311, 2047, BF16, F32, F32, False),
    (33, 1001, F32, F32, None, False), (2, 8192, F16, F32, F32, True), (400, 8192, F16, F16, F16, True), (3, 16384, BF16, BF16, F32, True),
    (330, 16384, F32, F32, F32, True), (3, 16383, F16, F16, F16, False), (8, 66, BF16, None, None, False), (2500, 48, F32, F32, F32, True)])
def test_norm_values_and_codes(gpu, T, H, dtype, stream, wt, quantize):
    g = gen(T, H)
    x = torch.randn(T, H, generator=g).to(dtype)
    res = None if stream is None else (2 * torch.randn(T, H, generator=g)).to(stream)
    w = None if wt is None else (1 + 0.3 * torch.randn(H, generator=g)).to(wt)
    got = check_norm(gpu, x, res, w, quantize=quantize)
    if quantize:      # codes alone are the same codes
        more = check_norm(gpu, x, res, w, quantize=True, values=False)
        assert torch.equal(got[3].view(torch.uint8), more[3].view(torch.uint8)) and torch.equal(got[4], more[4])


@pytest.mark.gpu
@pytest.mark.parametrize("H", [128, 1008, 2048, 6144])
@pytest.mark.parametrize("T", [2, 400])
def test_norm_scales_at_their_step(gpu, T, H):
    """Blocks whose largest value is within float32's error of 448 times a power of two: the scale is the
    one that float64 gives, on either side."""
    g = gen(T, H)
    x = torch.randn(T, H, generator=g)
    x[:, 5] = 0.5
    _, r, _ = norm_ref(x, None, None, 1e-5)
    wanted = 3.5 * 2.0 ** -3 * torch.exp2(torch.randint(0, 6, (T,), generator=g).double())     # 448 is 3.5 x 2^7
    x[:, 5:6] *= 1.0          # a column that meets the step through the weight of one row at a time
    sides = set()
    for t in range(0, T, max(1, T // 12)):
        for ulps in (-3, -1, 0, 1, 2, 7):
            w = 0.001 * torch.ones(H)
            w[5] = float(wanted[t] / (0.5 * r[t])) * (1 + ulps * 2.0 ** -24)
            y = norm_ref(x, None, w, 1e-5)[2]
            got = gpu.moe_norm_forward(x.cuda(), weight=w.cuda(), quantize=True)
            s = scales_ref(y)
            assert torch.equal(got[4].cpu().double(), s)
            sides.add(float(s[0, t] * 448 / wanted[t]))
    assert sides == {1.0, 2.0}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,stream", [(F32, F32), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 0), (16, 8)])
@pytest.mark.parametrize("H", [200, 2048])
def test_norm_strided_rows(gpu, dtype, stream, pad, shift, H):
    T = 19
    g = gen(pad, shift, H)
    x, res = torch.randn(T, H, generator=g).to(dtype), torch.randn(T, H, generator=g).to(stream)
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype)
    xs, rs = strided(x, pad, shift), strided(res, pad, shift)
    buf = torch.full((T, H + 24), 7.0, dtype=stream, device="cuda")
    got = check_norm(gpu, x, res, w, inputs=(xs, rs), out=buf[:, :H])
    assert bool((buf[:, H:] == 7).all()) and got[1].data_ptr() == buf.data_ptr()
    dy, gh = torch.randn(T, H, generator=g).to(dtype), torch.randn(T, H, generator=g).to(stream)
    want = gpu.moe_norm_backward(dy.cuda(), got[1].contiguous(), got[2], weight=w.cuda(), grad_h=gh.cuda())
    ghs = strided(gh, pad, shift)
    d, dw = gpu.moe_norm_backward(strided(dy, pad, shift), got[1], got[2], weight=w.cuda(), grad_h=ghs, out=ghs)      # in place
    tol = 2.0 ** -18 + half_step(stream)
    assert d.data_ptr() == ghs.data_ptr() and bool(((d - want[0]).double().abs() <= tol * (2 + 2 * want[0].double().abs())).all())
    assert bool(((dw - want[1]).abs() <= 2.0 ** -17 * (dy.double().abs() * 6).sum(0).cuda()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("H", [256, 1024, 4096])
def test_norm_in_place_and_repeatable(gpu, H):
    x, res = torch.randn(500, H, generator=gen(H)).to(BF16), torch.randn(500, H, generator=gen(H + 1))
    w = torch.ones(H, dtype=BF16)
    a = gpu.moe_norm_forward(x.cuda(), residual=res.cuda(), weight=w.cuda(), quantize=True)
    r = res.cuda()
    b = gpu.moe_norm_forward(x.cuda(), residual=r, weight=w.cuda(), quantize=True, out=r)
    assert b[1].data_ptr() == r.data_ptr()
    for u, v in zip(a, b):
        assert torch.equal(u.view(torch.uint8) if u.dtype == torch.float8_e4m3fn else u, v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v)
    dy = torch.randn(500, H, generator=gen(2)).to(BF16).cuda()
    p, q = (gpu.moe_norm_backward(dy, a[1], a[2], weight=w.cuda()) for _ in range(2))
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@pytest.mark.gpu
def test_norm_in_place_and_beside_its_inputs(gpu):
    """y on top of x or residual, outputs in other columns of the inputs' buffer: what separate tensors give."""
    T, H = 40, 512
    L, st = gpu.lib(), torch.cuda.current_stream().cuda_stream
    x, res, w = torch.randn(T, H, generator=gen(1)).to(BF16).cuda(), torch.randn(T, H, generator=gen(2)).to(BF16).cuda(), torch.ones(H, dtype=BF16, device="cuda")
    y, h, r, q, s = gpu.moe_norm_forward(x, residual=res, weight=w, quantize=True)
    alone = gpu.moe_norm_forward(x, weight=w)[0]
    wide = torch.full((T, 3 * H), 7.0, dtype=BF16, device="cuda")
    wide[:, :H], wide[:, H:2 * H] = x, res
    got = gpu.moe_norm_forward(wide[:, :H], residual=wide[:, H:2 * H], weight=w, quantize=True, out=wide[:, 2 * H:])
    for a, b in zip(got, (y, h, r, q, s)):
        assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a, b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
    assert torch.equal(wide[:, :H], x) and torch.equal(wide[:, H:2 * H], res)

    def call(x, res, h, y, codes):
        c, b = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(H // 128, T, device="cuda")
        assert gpu.MOE_OK == L.moe_norm_forward(x.data_ptr(), 2, H, res.data_ptr() if res is not None else None, 2, H, w.data_ptr(), 2, T, H, 1e-5,
                                                h.data_ptr() if h is not None else None, H, y.data_ptr(), H, None, c.data_ptr() if codes else None,
                                                b.data_ptr() if codes else None, st)
        return (c, b) if codes else None
    z = x.clone()
    call(z, None, None, z, False)
    assert torch.equal(z, alone)
    z, hh = x.clone(), torch.empty_like(x)
    c, b = call(z, res, hh, z, True)
    assert torch.equal(z, y) and torch.equal(hh, h) and torch.equal(c, q.view(torch.uint8)) and torch.equal(b, s)
    z, hh = res.clone(), torch.empty_like(x)
    c, b = call(x, z, hh, z, True)
    assert torch.equal(z, y) and torch.equal(hh, h) and torch.equal(c, q.view(torch.uint8)) and torch.equal(b, s)
    z = torch.empty_like(x)
    call(x, res, z, z, False)
    assert torch.equal(z, y)


@pytest.mark.gpu
def test_norm_zeros_nan_and_extremes(gpu):
    T, H = 8, 384
    x = torch.randn(T, H, generator=gen(1))
    x[0] = 0
    x[1, 7] = nan
    x[2, 300] = inf
    x[3] = 1e-30
    x[4] *= 1e15
    x[5, :128] = 0
    y, h, r, q, s = gpu.moe_norm_forward(x.cuda(), weight=torch.ones(H, device="cuda"), quantize=True)
    y, q, s = y.cpu(), q.cpu().float(), s.cpu()
    assert bool((y[0] == 0).all()) and bool((q[0] == 0).all()) and s[:, 0].tolist() == [1.0] * 3
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(s[:, 1]).all())
    assert bool((y[2, :300] == 0).all()) and bool(torch.isnan(y[2, 300])) and bool(torch.isnan(s[2, 2])) and s[:2, 2].tolist() == [1.0, 1.0]
    keep = [3, 4, 5, 6, 7]
    _, _, want = norm_ref(x[keep], None, None, 1e-5)
    assert bool(((y[keep].double() - want).abs() <= 2.0 ** -17 * want.abs()).all())
    check_codes(q[keep].to(torch.float8_e4m3fn), s[:, keep], want)
    assert bool(torch.isnan(gpu.moe_norm_forward(torch.zeros(1, 16, device="cuda"), eps=0.0)[0]).all())      # 0 times 1 / sqrt(0)
    z = gpu.moe_norm_forward(torch.full((1, 16), 4.0, device="cuda", dtype=F16), weight=torch.full((16,), 7e4, device="cuda"))
    assert bool(torch.isinf(z[0]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 324])
@pytest.mark.parametrize("H", [1, 200, 255, 1001, 2046, 2048, 6144, 8192])
@pytest.mark.parametrize("dtype,stream", [(F32, None), (BF16, None), (BF16, BF16), (BF16, F32)])
def test_norm_rows_whose_squares_leave_float32(gpu, T, H, dtype, stream):
    """Rows from 1e-37 to 1e38, without an epsilon and with one: values, codes and gradients are the formula's."""
    g = gen(T, H, 9)
    size = torch.tensor([1e-37, 1e-30, 1e-24, 1e-21, 1.0, 1e17, 1e20, 1e30, 1e38], dtype=torch.float64).repeat(T // 9)[:, None]
    x = (torch.randn(T, H, generator=g).clamp(-3, 3).double() * size)
    x[4, 0] = 2e19                                     # one value alone
    x = x.to(dtype)
    x[x == 0] = 1e-37
    res = None if stream is None else (0.1 * torch.randn(T, H, generator=g).clamp(-3, 3).double() * size).to(stream)
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dtype)
    dy = torch.randn(T, H, generator=g).to(dtype)
    for eps in (0.0, 1e-5):
        y, h, r, *codes = gpu.moe_norm_forward(x.cuda(), residual=None if res is None else res.cuda(), weight=w.cuda(), eps=eps, quantize=H % 16 == 0)
        h64, r64, y64 = norm_ref(x, res, w, eps)
        # 1 / rms beyond float32's largest value (one value below 2^-128 and no epsilon) is rounded to infinity; y is the formula's
        held = r64 <= torch.finfo(F32).max
        assert torch.equal(h.cpu(), h64) and bool((r.cpu()[~held] == inf).all())
        assert bool(((r.cpu().double() - r64)[held].abs() <= 2.0 ** -18 * r64[held]).all())
        assert bool(((y.cpu().double() - y64).abs() <= (2.0 ** -18 + half_step(dtype)) * y64.abs() + torch.finfo(dtype).tiny).all())
        if codes:
            check_codes(codes[0], codes[1], y64)
        check_norm_grad(gpu, x[held], None if res is None else res[held], w, dy[held], None, eps=eps)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [128, 2048, 6144])
def test_norm_scales_at_their_step_of_large_and_small_rows(gpu, H):
    """A power of two times a row is the same row behind the norm (eps = 0): the same codes and scales, next to a scale's step too."""
    x = torch.randn(6, H, generator=gen(H, 2))
    _, r, _ = norm_ref(x, None, None, 0.0)
    for t in range(6):
        for ulps in (-2, 0, 2):
            w = 0.001 * torch.ones(H)
            w[5] = float(1.75 / (x[t, 5].double().abs() * r[t])) * (1 + ulps * 2.0 ** -24)
            want = gpu.moe_norm_forward(x.cuda(), weight=w.cuda(), quantize=True, eps=0.0)
            assert torch.equal(want[4].cpu().double(), scales_ref(norm_ref(x, None, w, 0.0)[2]))
            for by in (2.0 ** -80, 2.0 ** 60, 2.0 ** 120):
                got = gpu.moe_norm_forward((x * by).cuda(), weight=w.cuda(), quantize=True, eps=0.0)
                assert torch.equal(got[4], want[4])
                check_codes(got[3], got[4], norm_ref(x, None, w, 0.0)[2])


def check_norm_grad(moe, x, res, w, dy, gh, eps=1e-5):
    """dh: 2^-17 of the sizes of its terms (the row's sum has 16 or 32 additions a thread and 10 levels),
    then the rounding; dw: the tokens of a block one after another (34 at most here) and 32 + 5 more: 2^-17."""
    wd = None if w is None else w.cuda()
    _, h, r = moe.moe_norm_forward(x.cuda(), residual=None if res is None else res.cuda(), weight=wd, eps=eps)
    d, dw = moe.moe_norm_backward(dy.cuda(), h, r, weight=wd, grad_h=None if gh is None else gh.cuda())
    v = h.cpu().double().requires_grad_(True)
    w64 = (torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()).requires_grad_(True)
    y = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * w64
    gv, gw = torch.autograd.grad(y, (v, w64), dy.double())
    g = 0.0 if gh is None else gh.double()
    v, rr = v.detach(), 1 / torch.sqrt((v.detach() ** 2).mean(1, keepdim=True) + eps)
    n, dd = (v * rr).abs(), (dy.double() * w64.detach()).abs()
    size = (dd + n * (dd * n).mean(1, keepdim=True)) * rr + (0.0 if gh is None else gh.double().abs())
    want = gv + g
    assert d.dtype == h.dtype
    assert bool(((d.cpu().double() - want).abs() <= 2.0 ** -17 * size + half_step(h.dtype) * want.abs() + torch.finfo(h.dtype).tiny).all())
    if w is None:
        assert dw is None
    else:
        assert dw.dtype == F32 and bool(((dw.cpu().double() - gw).abs() <= 2.0 ** -17 * (dy.double().abs() * n).sum(0)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,dtype,stream,wt,through", [
    (1, 1, F32, F32, F32, True), (1, 6144, F32, F32, F32, False), (5, 16, F16, None, F16, True), (700, 144, BF16, F32, F32, True),
    (3000, 64, F32, F32, F32, True), (300, 1024, F16, F16, None, True), (333, 1032, BF16, BF16, BF16, False), (1000, 2048, BF16, F32, BF16, True),
    (200, 2047, F16, F16, F16, True), (90, 1001, F32, None, F32, True), (77, 8192, BF16, F32, F32, True), (160, 8200, F32, F32, F32, True),
    (155, 16384, F16, F16, F16, True), (5, 16383, BF16, F32, F32, False)])
def test_norm_gradient(gpu, T, H, dtype, stream, wt, through):
    g = gen(T, H, 5)
    x = torch.randn(T, H, generator=g).to(dtype)
    res = None if stream is None else torch.randn(T, H, generator=g).to(stream)
    w = None if wt is None else (1 + 0.3 * torch.randn(H, generator=g)).to(wt)
    dy = torch.randn(T, H, generator=g).to(dtype)
    gh = torch.randn(T, H, generator=g).to(stream or dtype) if through else None
    check_norm_grad(gpu, x, res, w, dy, gh)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [200, 1001, 2048])
@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_norm_gradient_in_place(gpu, H, dtype, stream):
    """dh on top of dy, h or grad_h, or in other columns of their buffer."""
    T = 700
    g = gen(H)
    dy, res, gh = torch.randn(T, H, generator=g).to(dtype).cuda(), torch.randn(T, H, generator=g).to(stream).cuda(), torch.randn(T, H, generator=g).to(stream).cuda()
    w = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    _, h, r = gpu.moe_norm_forward(dy, residual=res, weight=w)
    d, dw = gpu.moe_norm_backward(dy, h, r, weight=w, grad_h=gh)
    for name in ("dy", "h", "gh")[0 if dtype == stream else 1:]:
        t = dict(dy=dy.clone(), h=h.clone(), gh=gh.clone())
        a, b = gpu.moe_norm_backward(t["dy"], t["h"], r, weight=w, grad_h=t["gh"], out=t[name])
        assert a.data_ptr() == t[name].data_ptr() and torch.equal(a, d) and torch.equal(b, dw)
    n = (H + 7) // 8 * 8
    wide = torch.zeros(T, 3 * n, dtype=stream, device="cuda")
    wide[:, :H], wide[:, n:n + H] = h, gh
    a, b = gpu.moe_norm_backward(dy, wide[:, :H], r, weight=w, grad_h=wide[:, n:n + H], out=wide[:, 2 * n:2 * n + H])
    tol = 2.0 ** -18 + half_step(stream)       # rows of another boundary may be added in another order
    assert bool(((a - d).double().abs() <= tol * (2 + 2 * d.double().abs())).all()) and torch.equal(wide[:, :H], h)


@pytest.mark.gpu
def test_norm_gradient_against_differences(gpu):
    H, e = 24, 1e-5
    x, w, dy = torch.randn(2, H, generator=gen(4)).double(), (1 + 0.2 * torch.randn(H, generator=gen(5))), torch.randn(2, H, generator=gen(6))
    _, h, r = gpu.moe_norm_forward(x.float().cuda(), weight=w.cuda())
    d = gpu.moe_norm_backward(dy.cuda(), h, r, weight=w.cuda())[0].cpu()
    f = lambda v: (norm_ref(v, None, w, 1e-5)[2] * dy.double()).sum()   # noqa: E731
    for t in range(2):
        for j in range(H):
            a, b = x.clone(), x.clone()
            a[t, j] += e
            b[t, j] -= e
            assert abs(float((f(a) - f(b)) / (2 * e)) - float(d[t, j])) <= 1e-6 + 2.0 ** -16


@pytest.mark.gpu
def test_norm_no_tokens(gpu):
    x, w = torch.zeros(0, 48, device="cuda"), torch.ones(48, device="cuda")
    y, h, r, q, s = gpu.moe_norm_forward(x, residual=x, weight=w, quantize=True)
    assert y.shape == h.shape == q.shape == (0, 48) and r.shape == (0,) and s.shape == (1, 0)
    d, dw = gpu.moe_norm_backward(x, h, r, weight=w)
    assert d.shape == (0, 48) and dw.tolist() == [0.0] * 48


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1024, 16384])
def test_norm_more_than_two_to_the_31_elements(gpu, H):
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GB")
    T = 2**31 // H + 1029
    x = torch.randn(T, H, device="cuda", dtype=BF16)
    w = torch.randn(H, device="cuda")
    y, h, r, q, s = gpu.moe_norm_forward(x, residual=x, weight=w, quantize=True)
    d, dw = gpu.moe_norm_backward(y, h, r, weight=w, grad_h=x)
    for at in (0, T - 40):
        i = slice(at, at + 40)
        a = gpu.moe_norm_forward(x[i], residual=x[i], weight=w, quantize=True)
        # another number of elements a thread: another order of the sum of squares
        assert torch.equal(h[i], a[1]) and bool(((r[i] - a[2]).abs() <= 2.0 ** -18 * r[i]).all())
        assert torch.equal(s[:, i], a[4]) and bool(((y[i] - a[0]).float().abs() <= 2.0 ** -7 * a[0].float().abs()).all())
        b = gpu.moe_norm_backward(y[i], h[i], r[i], weight=w, grad_h=x[i])
        assert torch.equal(d[i], b[0])
    del y, h, d, q
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_norm_of_almost_two_to_the_31_rows(gpu):
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GB")
    T = 2**31 - 1
    x = torch.randn(T, 1, device="cuda", dtype=BF16)
    y, h, r = gpu.moe_norm_forward(x)
    d = gpu.moe_norm_backward(y, h, r, grad_h=x)[0]
    for at in (0, T // 2, T - 40):
        i = slice(at, at + 40)
        a = gpu.moe_norm_forward(x[i])
        assert torch.equal(y[i], a[0]) and torch.equal(r[i], a[2])
        assert torch.equal(d[i], gpu.moe_norm_backward(y[i], h[i], r[i], grad_h=x[i])[0])
    del x, y, h, r, d
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_norm_refuses_in_the_binding(gpu):
    x, w = torch.zeros(4, 32, device="cuda", dtype=BF16), torch.ones(32, device="cuda", dtype=BF16)
    for kw in (dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(residual=x.half()), dict(residual=x[:3]), dict(weight=w.half()), dict(weight=w[:16]),
               dict(eps=-1.0), dict(eps="a"), dict(out=x), dict(residual=x, out=x.float()), dict(residual=x.float(), out=x), dict(residual=x, out=x[:, :16])):
        with pytest.raises(gpu.MoeError):
            gpu.moe_norm_forward(**{**dict(x=x, weight=w), **kw})
    for bad in (torch.zeros(4, 24, device="cuda"), strided(torch.zeros(4, 32), 1, 0), strided(torch.zeros(4, 32), 0, 1)):
        with pytest.raises(gpu.MoeError):
            gpu.moe_norm_forward(bad, quantize=True)
    r = torch.ones(4, device="cuda")
    for kw in (dict(dy=x.float()), dict(h=x.half()), dict(rstd=r[:3]), dict(rstd=r.half()), dict(grad_h=x.float()), dict(out=x.float()), dict(weight=w[:3])):
        with pytest.raises(gpu.MoeError):
            gpu.moe_norm_backward(**{**dict(dy=x, h=x, rstd=r, weight=w), **kw})


# ------------------------------------------------------------------------------------------ combine

def lists_of(moe, T, E, K, align, seed, dropped=0.1):
    g = gen(T, E, K, seed)
    idx = torch.rand(T, E, generator=g).topk(K, 1).indices.int()
    idx[torch.rand(T, K, generator=g) < dropped] = -1
    _, _, rows, pos = moe.moe_expert_lists(idx.cuda(), E, align)
    return rows, pos


def check_combine(moe, rows, pos, w, add, out_dtype=None, out=None):
    """K + 1 roundings of float32 of the terms' sizes, then one to the type."""
    y = moe.moe_combine_forward(rows, pos, w, add=add, out=out, out_dtype=out_dtype)
    R, N = rows.shape
    T, K = pos.shape
    on = ((pos >= 0) & (pos < R)).cpu()
    each = rows.cpu().double()[pos.cpu().clamp(0, max(R - 1, 0)).long()] if R else torch.zeros(T, K, N, dtype=torch.float64)
    each = torch.where(on[:, :, None], each, 0.0)
    ww = (torch.ones(T, K) if w is None else w.cpu()).double()[:, :, None]
    more = torch.zeros(T, N, dtype=torch.float64) if add is None else add.cpu().double()
    want, size = (ww * each).sum(1) + more, (ww * each).abs().sum(1) + more.abs()
    assert y.dtype == (out_dtype or (rows.dtype if add is None else add.dtype))
    assert bool(((y.cpu().double() - want).abs() <= (K + 1) * 2.0 ** -24 * size + half_step(y.dtype) * want.abs() + torch.finfo(y.dtype).tiny).all())
    return y


def check_combine_grad(moe, dy, rows, pos, tokens, w, out=None):
    """drows: one product (and K sums), rounded; dw: N / 128 additions a thread of 8, then 7 levels."""
    d, dw = moe.moe_combine_backward(dy, rows, pos, tokens, w, out=out)
    R, N = rows.shape
    T, K = pos.shape
    p, tok, g = pos.cpu(), tokens.cpu(), dy.cpu().double()
    ww = (torch.ones(T, K) if w is None else w.cpu()).double()
    want, s, size = torch.zeros(R, N, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            r = int(p[t, k])
            if 0 <= r < R:
                s[t, k] = (rows[r].cpu().double() * g[t]).sum()
                size[t, k] = (rows[r].cpu().double() * g[t]).abs().sum()
                if tok[r] == t:
                    want[r] += ww[t, k] * g[t]
    assert d.dtype == rows.dtype and dw.dtype == F32
    assert bool(((d.cpu().double() - want).abs() <= (half_step(d.dtype) + (K + 1) * 2.0 ** -24) * want.abs() + torch.finfo(d.dtype).tiny).all())
    assert bool(((dw.cpu().double() - s).abs() <= (N / 128 + 16) * 2.0 ** -24 * size).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,N,align,dtype,add", [
    (1, 1, 1, 1, 1, F32, False), (1, 256, 8, 6144, 1, BF16, True), (4, 256, 8, 2048, 1, F16, True), (37, 8, 2, 40, 16, BF16, False),
    (130, 6, 3, 1000, 128, F32, True), (65, 40, 32, 130, 1, F16, False), (50, 300, 12, 257, 128, BF16, True), (20, 16, 9, 4100, 8, F32, False),
    (3, 5, 5, 33, 1, BF16, True)])
def test_combine_values_and_gradients(gpu, T, E, K, N, align, dtype, add):
    g = gen(T, E, K, N)
    tokens, pos = lists_of(gpu, T, E, K, align, N)
    R = tokens.numel()
    rows = torch.randn(R, N, generator=g).to(dtype)
    rows[tokens.cpu() < 0] = nan                       # rows without a token are never read
    rows = rows.cuda()
    w = torch.randn(T, K, generator=g).cuda()
    more = torch.randn(T, N, generator=g).to(dtype).cuda() if add else None
    check_combine(gpu, rows, pos, w, more)
    check_combine(gpu, rows, pos, None, None, out_dtype=F32)
    dy = torch.randn(T, N, generator=g).to(dtype).cuda()
    check_combine_grad(gpu, dy, rows, pos, tokens, w, out=torch.full((R, N), 7.0, dtype=dtype, device="cuda"))
    check_combine_grad(gpu, dy, rows, pos, tokens, None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_combine_rows_named_twice_or_by_others(gpu, dtype):
    """A row takes the gradient of its own token alone, with the sum of the weights where that names it
    more than once; rows that no pair of their token names get zeros; positions outside [0, R) none."""
    T, K, R, N = 6, 4, 20, 72
    g = gen(8)
    pos = torch.randint(0, R, (T, K), generator=g, dtype=torch.int32)
    pos[0] = 3
    pos[1, 1] = pos[1, 3] = 5
    pos[2] = torch.tensor([-1, R, -2**31, 2**31 - 1], dtype=torch.int32)
    tokens = torch.randint(-1, T, (R,), generator=g, dtype=torch.int32)
    tokens[3], tokens[5], tokens[6], tokens[7] = 0, 1, T, 2**31 - 1
    rows, dy = torch.randn(R, N, generator=g).to(dtype).cuda(), torch.randn(T, N, generator=g).to(dtype).cuda()
    w = torch.randn(T, K, generator=g).cuda()
    check_combine(gpu, rows, pos.cuda(), w, None)
    check_combine_grad(gpu, dy, rows, pos.cuda(), tokens.cuda(), w, out=torch.full((R, N), 7.0, dtype=dtype, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [1, 7, 17, 248, 257, 1030])
def test_combine_rows_on_every_boundary(gpu, dtype, N):
    """Rows, sums and gradients that start on different boundaries, the first and last rows of a tensor among the chosen ones."""
    T, K = 9, 3
    for shift in range(16 // rows_el(dtype)):
        g = gen(N, shift)
        tokens, pos = lists_of(gpu, T, 4, K, 1, shift, dropped=0.0)
        R = tokens.numel()
        rows = strided(torch.randn(R, N, generator=g).to(dtype), 0, shift)
        dy = strided(torch.randn(T, N, generator=g).to(dtype), 1, 1)
        w = torch.randn(T, K, generator=g).cuda()
        for out_dtype in (F32, BF16):
            more = strided(torch.randn(T, N, generator=g).to(out_dtype), 1, shift)
            out = torch.full((T + 1, N + 3), 7.0, dtype=out_dtype, device="cuda")
            check_combine(gpu, rows, pos, w, more, out_dtype=out_dtype, out=out[:T, 2:N + 2])
            assert bool((out[:, :2] == 7).all()) and bool((out[:, N + 2:] == 7).all()) and bool((out[T] == 7).all())
        same = torch.full((R * N + shift + 9,), 7.0, dtype=dtype, device="cuda")
        check_combine_grad(gpu, dy, rows, pos, tokens, w, out=same[shift:shift + R * N].view(R, N))
        assert bool((same[:shift] == 7).all()) and bool((same[shift + R * N:] == 7).all())
        other = torch.full((R + 1, N + 2), 7.0, dtype=dtype, device="cuda")
        check_combine_grad(gpu, dy, rows, pos, tokens, w, out=other[:R, 1:N + 1])
        assert bool((other[:, :1] == 7).all()) and bool((other[:, N + 1:] == 7).all()) and bool((other[R] == 7).all())


def rows_el(dtype):
    return torch.finfo(dtype).bits // 8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (2, 2), (8, 8)])
def test_combine_strided_rows(gpu, dtype, pad, shift):
    T, K, N = 23, 3, 136
    g = gen(pad, shift)
    tokens, pos = lists_of(gpu, T, 8, K, 16, 1)
    R = tokens.numel()
    rows, more, dy = (strided(torch.randn(n, N, generator=g).to(dtype), pad, shift) for n in (R, T, T))
    w = torch.randn(T, K, generator=g).cuda()
    y = check_combine(gpu, rows, pos, w, more)
    assert torch.equal(y, gpu.moe_combine_forward(rows.contiguous(), pos, w, add=more.contiguous()))
    got = gpu.moe_combine_forward(rows, pos, w, add=more, out=more)                     # on top of add
    assert got.data_ptr() == more.data_ptr() and torch.equal(got, y)
    out = torch.full((R, N + pad + 1), 7.0, dtype=dtype, device="cuda")
    check_combine_grad(gpu, dy, rows, pos, tokens, w, out=out[:, :N])
    assert bool((out[:, N:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("N", [64, 67])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_combine_beside_its_inputs(gpu, dtype, N):
    """Rows and their gradient, or add and the sum, in columns of one buffer; the weights' gradient on top of the weights; rows in common are refused."""
    T, E, K = 33, 6, 3
    g = gen(N)
    tokens, pos = lists_of(gpu, T, E, K, 4, N)
    R = tokens.numel()
    rows, dy, w = torch.randn(R, N, generator=g).to(dtype).cuda(), torch.randn(T, N, generator=g).to(dtype).cuda(), torch.randn(T, K, generator=g).cuda()
    d, dw = gpu.moe_combine_backward(dy, rows, pos, tokens, w)
    both = torch.zeros(R, 2, N, dtype=dtype, device="cuda")
    both[:, 0] = rows
    a, b = gpu.moe_combine_backward(dy, both[:, 0], pos, tokens, w, out=both[:, 1])
    check_combine_grad(gpu, dy, both[:, 0], pos, tokens, w, out=both[:, 1])
    assert torch.equal(both[:, 0], rows) and bool(((b - dw).abs() <= 2.0 ** -17 * N).all()) and torch.equal(a, d)
    ww = w.clone()
    code = {F32: 0, BF16: 2}[dtype]
    out = torch.empty_like(rows)
    assert gpu.MOE_OK == gpu.lib().moe_combine_backward(dy.data_ptr(), code, N, rows.data_ptr(), N, R, N, pos.data_ptr(), T, K, tokens.data_ptr(), ww.data_ptr(),
                                                        out.data_ptr(), N, ww.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert torch.equal(ww, dw) and torch.equal(out, d)
    y = gpu.moe_combine_forward(rows, pos, w, add=dy)
    both = torch.zeros(T, 2, N, dtype=dtype, device="cuda")
    both[:, 0] = dy
    gpu.moe_combine_forward(rows, pos, w, add=both[:, 0], out=both[:, 1])
    assert torch.equal(both[:, 0], dy)
    check_combine(gpu, rows, pos, w, both[:, 0], out=both[:, 1])
    check_combine(gpu, rows, pos, w, dy.clone())
    assert y.shape == (T, N)
    flat = torch.zeros(R + 1, N, dtype=dtype, device="cuda")
    for call in (lambda: gpu.moe_combine_forward(flat[:-1], pos, w, out=flat[1:T + 1]), lambda: gpu.moe_combine_forward(rows, pos, w, add=flat[:T], out=flat[1:T + 1]),
                 lambda: gpu.moe_combine_backward(dy, flat[:-1], pos, tokens, w, out=flat[1:]), lambda: gpu.moe_combine_backward(flat[:T], rows, pos, tokens, w, out=flat[1:])):
        with pytest.raises(gpu.MoeError):
            call()


@pytest.mark.gpu
def test_combine_nothing(gpu):
    z = torch.zeros(0, 16, device="cuda")
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    assert gpu.moe_combine_forward(z, none[:0]).shape == (0, 16)
    assert bool((gpu.moe_combine_forward(z, none) == 0).all())                          # no rows at all
    rows = torch.full((5, 16), nan, device="cuda")
    tokens = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    assert bool((gpu.moe_combine_forward(rows, none) == 0).all())
    d, dw = gpu.moe_combine_backward(torch.ones(3, 16, device="cuda"), rows, none, tokens, out=rows.clone())
    assert bool((d == 0).all()) and bool((dw == 0).all())
    d, dw = gpu.moe_combine_backward(z, rows, none[:0], tokens, out=rows.clone())       # no tokens
    assert bool((d == 0).all()) and dw.shape == (0, 2)
    d, dw = gpu.moe_combine_backward(torch.ones(3, 16, device="cuda"), z, none, tokens[:0])
    assert d.shape == (0, 16) and bool((dw == 0).all())


@pytest.mark.gpu
def test_combine_more_than_two_to_the_31_elements(gpu):
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GB")
    T, K, N = 150000, 8, 2048
    tokens, pos = torch.arange(T * K, device="cuda", dtype=torch.int32) // K, torch.arange(T * K, device="cuda", dtype=torch.int32).view(T, K)
    rows = torch.randn(T * K, N, device="cuda", dtype=BF16)
    w, dy = torch.randn(T, K, device="cuda"), torch.randn(T, N, device="cuda", dtype=BF16)
    y = gpu.moe_combine_forward(rows, pos, w)
    d, dw = gpu.moe_combine_backward(dy, rows, pos, tokens, w)
    for at in (0, T - 20):
        i, r = slice(at, at + 20), slice(at * K, (at + 20) * K)
        first = pos[:20].contiguous()
        assert torch.equal(y[i], gpu.moe_combine_forward(rows[r], first, w[i].contiguous()))
        a = gpu.moe_combine_backward(dy[i], rows[r], first, tokens[:20 * K], w[i].contiguous())
        assert torch.equal(d[r], a[0]) and torch.equal(dw[i], a[1])
    del rows, d
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_combine_refuses_in_the_binding(gpu):
    rows, pos, w = torch.zeros(6, 16, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    tok, dy = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(3, 16, device="cuda")
    for kw in (dict(rows=rows.double()), dict(rows=rows.t()), dict(pos=pos.long()), dict(pos=pos[0]), dict(topk_w=w.half()), dict(topk_w=w[:2]), dict(add=rows),
               dict(add=dy.half(), out_dtype=F32), dict(out=rows), dict(out=dy.half(), out_dtype=F32), dict(out_dtype=torch.float64),
               dict(pos=torch.zeros(3, 33, dtype=torch.int32, device="cuda"), topk_w=None)):
        with pytest.raises(gpu.MoeError):
            gpu.moe_combine_forward(**{**dict(rows=rows, pos=pos, topk_w=w), **kw})
    for kw in (dict(dy=dy.half()), dict(dy=dy[:2]), dict(tokens=tok[:5]), dict(tokens=tok.long()), dict(out=rows.half()), dict(topk_w=w[:2])):
        with pytest.raises(gpu.MoeError):
            gpu.moe_combine_backward(**{**dict(dy=dy, rows=rows, pos=pos, tokens=tok, topk_w=w), **kw})


# ------------------------------------------------------------------------------------------ gradients' norm and clipping

def check_clip(moe, grads, most, place):
    """The squares' float32 sums of 32 at most, then float64 and a root: 2^-20; the factor three more
    roundings, a gradient one more and that to its type."""
    was = [g.clone() for g in grads]
    n = moe.moe_grad_norm(grads)
    want = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in was))
    assert n.shape == (1,) and abs(float(n) - want) <= 2.0 ** -20 * want
    out = None if place else [torch.full_like(g, 7.0) for g in grads]
    assert moe.moe_grad_clip(grads, n, most, out=out) is None
    c = min(1.0, most / (want + 1e-6))
    for g, o, w in zip(grads, grads if place else out, was):
        ref = w.double() * c
        assert bool(((o.double() - ref).abs() <= (2.0 ** -19 + half_step(w.dtype)) * ref.abs() + torch.finfo(w.dtype).smallest_normal).all())
        assert place or torch.equal(g, w)
        if most > 1.001 * want:
            assert torch.equal(o, w)


@pytest.mark.gpu
@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("sizes", [[1], [0], [0, 5, 0], [1, 2, 3, 4, 5, 6, 7, 8, 9], [32768, 32767, 32769, 100001], [10**6, 3, 65536],
                                   list(range(1, 70)), [7] * 65, [i % 50 for i in range(600)]])
def test_clip(gpu, sizes, place):
    g = gen(len(sizes), sum(sizes))
    kinds = (F32, BF16, F16)
    mk = lambda: [torch.randn(n, generator=g).to(kinds[i % 3]).cuda() for i, n in enumerate(sizes)]   # noqa: E731
    for most in (0.5, 1e9, 0.0):
        check_clip(gpu, mk(), most, place)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_clip_unaligned_and_permuted(gpu, shift):
    buf, more = torch.randn(200000, device="cuda"), torch.randn(200000, device="cuda").to(BF16)
    w = torch.randn(40, 30, 20, device="cuda")
    grads = [buf[shift:shift + 70001], buf[100000 + shift:100000 + shift + 9], more[shift:shift + 66000], w.permute(2, 0, 1), torch.randn(300, 200, device="cuda").t()]
    check_clip(gpu, grads, 1.0, True)
    check_clip(gpu, grads, 0.3, False)
    n = gpu.moe_grad_norm(grads)
    out = [torch.empty(70004, device="cuda")[2:70003], torch.empty(9, device="cuda")]             # other boundaries than their gradients'
    gpu.moe_grad_clip(grads[:2], n, 0.25, out=out)
    for a, b in zip(grads, out):
        assert bool(((b.double() - a.double() * 0.25 / (float(n) + 1e-6)).abs() <= 2.0 ** -19 * a.double().abs()).all())
    assert bool((buf[:shift] != 0).all())


@pytest.mark.gpu
def test_clip_norm_beside_the_gradients(gpu):
    """One buffer holds a gradient, the norm and a gradient; the norm inside one of them is refused."""
    flat = torch.randn(2049, device="cuda")
    a, norm, b = flat[:1024], flat[1024:1025], flat[1025:]
    was = [a.clone(), b.clone()]
    norm.copy_(gpu.moe_grad_norm([a, b]))
    n = float(norm)
    gpu.moe_grad_clip([a, b], norm, 0.5)
    for x, y in zip((a, b), was):
        assert bool(((x.double() - y.double() * 0.5 / (n + 1e-6)).abs() <= 2.0 ** -19 * y.double().abs()).all())
    assert float(norm) == n
    with pytest.raises(gpu.MoeError):
        gpu.moe_grad_clip([flat], norm, 0.5)
    other = [torch.zeros_like(a), torch.zeros_like(b)]
    gpu.moe_grad_clip([a, b], a[5:6], 0.5, out=other)          # read alone: one of the inputs may hold it
    with pytest.raises(gpu.MoeError):
        gpu.moe_grad_clip([a, b], other[1][5:6], 0.5, out=other)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-12, 1e12, 1e18, 1e30, 2e37])
def test_clip_magnitudes(gpu, scale):
    """Squares that float32 cannot hold."""
    grads = [torch.randn(50001, generator=gen(1)).clamp(-5, 5).mul(scale).cuda(), torch.randn(33, generator=gen(2)).clamp(-5, 5).mul(scale).to(BF16).cuda()]
    n = gpu.moe_grad_norm(grads)
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    assert float(n) == inf if want > torch.finfo(F32).max else abs(float(n) - want) <= 2.0 ** -20 * want + 2.0 ** -149
    gpu.moe_grad_clip(grads, n, 1.0)
    assert all(bool(torch.isfinite(g).all()) for g in grads)


@pytest.mark.gpu
def test_clip_nan_and_infinity(gpu):
    a, b = torch.randn(1000, device="cuda"), torch.randn(70000, device="cuda").to(BF16)
    b[69999] = nan
    n = gpu.moe_grad_norm([a, b])
    assert math.isnan(float(n))
    gpu.moe_grad_clip([a, b], n, 1.0)
    assert bool(torch.isnan(a).all()) and bool(torch.isnan(b).all())
    a, b = torch.randn(1000, device="cuda"), torch.randn(70000, device="cuda").to(F16)
    a[3] = -inf
    n = gpu.moe_grad_norm([a, b])
    assert float(n) == inf
    gpu.moe_grad_clip([a, b], n, 1.0)
    assert bool(torch.isnan(a[3])) and bool((a[:3] == 0).all()) and bool((b == 0).all())
    assert float(gpu.moe_grad_norm([])) == 0.0 and gpu.moe_grad_clip([], n, 1.0) is None


@pytest.mark.gpu
def test_clip_more_than_two_to_the_31_elements(gpu):
    if torch.cuda.mem_get_info()[0] < 40 * 2**30:
        pytest.skip("needs 40 GB")
    x = torch.full((2**31 + 70001,), 0.5, dtype=BF16, device="cuda")
    x[-1] = 3.0
    n = gpu.moe_grad_norm([x])
    want = math.sqrt((x.numel() - 1) * 0.25 + 9.0)
    assert abs(float(n) - want) <= 2.0 ** -20 * want
    gpu.moe_grad_clip([x], n, float(n) / 2)
    assert float(x[-1]) == 1.5 and float(x[2**31 + 5]) == 0.25 and float(x[0]) == 0.25 and bool((x[:-1] == 0.25).all())
    a, b = gpu.moe_grad_norm([x]), gpu.moe_grad_norm([x])
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_clip_refuses_in_the_binding(gpu):
    x, n = torch.zeros(8, 8, device="cuda"), torch.ones(1, device="cuda")
    for grads in ([x.double()], [x[:, :4]], [x, x.cpu()], [x, 3], [torch.zeros(1, 8, device="cuda").expand(8, 8)]):
        with pytest.raises(gpu.MoeError):
            gpu.moe_grad_norm(grads)
        with pytest.raises(gpu.MoeError):
            gpu.moe_grad_clip(grads, n, 1.0)
    for kw in (dict(norm=n.half()), dict(norm=torch.ones(2, device="cuda")), dict(norm=n.cpu()), dict(max_norm=-1.0), dict(max_norm=nan), dict(max_norm="a"),
               dict(grads=[x, x]), dict(grads=[x, x[2:4]]), dict(out=[]), dict(out=[x.half()]), dict(out=[x.t()]), dict(out=[x.view(64)])):
        with pytest.raises(gpu.MoeError):
            gpu.moe_grad_clip(**{**dict(grads=[x], norm=n, max_norm=1.0), **kw})
    assert bool((x == 0).all())


# ------------------------------------------------------------------------------------------ streams, graphs, together

@pytest.mark.gpu
def test_capture_and_side_stream(gpu):
    """Captured calls, replayed on other contents of the same inputs, and calls on a side stream give what
    plain calls give; two graphs that run at once share nothing."""
    T, E, K, H = 300, 64, 6, 512
    g = gen(31)

    def inputs():
        return [torch.randn(T, E, generator=g), torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)]

    def step(logits, x, res, s=None):
        idx, w = gpu.moe_route_forward(logits, K, stream=s)
        counts, off, rows, pos = gpu.moe_expert_lists(idx, E, 16, stream=s)
        y, h, r, q, sc = gpu.moe_norm_forward(x, residual=res, quantize=True, weight=torch_w, stream=s)
        each = y.index_select(0, rows.clamp(min=0).long()) if s is None else y[:1].expand(rows.numel(), H).contiguous()
        z = gpu.moe_combine_forward(each, pos, w, add=y, stream=s)
        d, dw = gpu.moe_combine_backward(z, each, pos, rows, w, stream=s)
        dl = gpu.moe_route_backward(logits, idx, dw, stream=s)
        dh, dn = gpu.moe_norm_backward(z, h, r, weight=torch_w, grad_h=z, stream=s)
        n = gpu.moe_grad_norm([dl, dn, d], stream=s)
        gpu.moe_grad_clip([dl, dn, d], n, 1.0, stream=s)
        return [idx, w, y, h, r, q.view(torch.uint8), sc, z, d, dl, dh, dn, n]
    torch_w = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    graphs = []
    for _ in range(2):
        held = [t.cuda() for t in inputs()]
        step(*held)                                   # first calls outside
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*held)
        graphs.append((graph, held, out))
    for _ in range(3):
        fresh = [inputs(), inputs()]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for (graph, held, _), new, s in zip(graphs, fresh, streams):
            with torch.cuda.stream(s):
                for a, b in zip(held, new):
                    a.copy_(b)
                graph.replay()
        torch.cuda.synchronize()
        for (_, held, out), new in zip(graphs, fresh):
            want = step(*[t.cuda() for t in new])
            for a, b in zip(out, want):
                assert torch.equal(a, b)
    s = torch.cuda.Stream()
    held = [t.cuda() for t in inputs()]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a = step(*held)
    torch.cuda.synchronize()
    for u, v in zip(a, step(*held)):
        assert torch.equal(u, v)
    # stream given as an argument
    idx, w = gpu.moe_route_forward(held[0], K, stream=s)
    y = gpu.moe_norm_forward(held[1], residual=held[2], weight=torch_w, stream=s.cuda_stream)[0]
    s.synchronize()
    assert torch.equal(idx, a[0]) and torch.equal(w, a[1]) and torch.equal(y, a[2])


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_stream_argument_of_every_operator(gpu, handle):
    """stream= (an object or its handle) while another stream is the current one: each call waits for what that stream makes before it."""
    T, E, K, H = 300, 64, 6, 512
    g = gen(77)
    inputs = [torch.randn(T, E, generator=g).cuda(), torch.randn(T, H, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()]
    weight = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    other = torch.cuda.Stream()

    def step(held, at=None):
        s = at if at is None or not handle else at.cuda_stream

        def call(f, *a, **kw):
            if at is not None:                       # the stream is behind by a millisecond or so before every call
                with torch.cuda.stream(at):
                    torch.cuda._sleep(1000000)
            return f(*a, stream=s, **kw)
        if at is not None:
            with torch.cuda.stream(at):
                torch.cuda._sleep(1000000)
                for a, b in zip(held, inputs):
                    a.copy_(b)
        logits, x, res = held
        idx, w = call(gpu.moe_route_forward, logits, K)
        _, _, rows, pos = call(gpu.moe_expert_lists, idx, E, 16)
        y, h, r, q, sc = call(gpu.moe_norm_forward, x, residual=res, weight=weight, quantize=True)
        with torch.cuda.stream(at or torch.cuda.current_stream()):
            each = y.index_select(0, rows.clamp(min=0).long())
        z = call(gpu.moe_combine_forward, each, pos, w, add=y)
        d, dw = call(gpu.moe_combine_backward, z, each, pos, rows, w)
        dl = call(gpu.moe_route_backward, logits, idx, dw)
        dh, dn = call(gpu.moe_norm_backward, z, h, r, weight=weight, grad_h=z)
        n = call(gpu.moe_grad_norm, [dl, dn, d])
        call(gpu.moe_grad_clip, [dl, dn, d], n, 1.0)
        return [idx, w, pos, y, h, r, q.view(torch.uint8), sc, z, d, dw, dl, dh, dn, n]
    want = step(inputs)
    held = [torch.zeros_like(t) for t in inputs]
    torch.cuda.synchronize()
    got = step(held, other)
    other.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_training_step_of_a_layer(gpu):
    """Norm, routing, lists, quantised products, combine and back, as a trainer runs them: gradients against
    autograd in float64 on the dequantised operands of the same step."""
    T, H, I, E, K = 200, 256, 128, 8, 3
    g = gen(55)
    dev = "cuda"
    x, res = torch.randn(T, H, generator=g).to(BF16).cuda(), torch.randn(T, H, generator=g).cuda()
    nw = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    rw, bias = (torch.randn(E, H, generator=g) / 16).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()
    w = (torch.randn(E, I, H, generator=g) / 16).cuda()
    wq, ws, wt, wts = gpu.moe_fp8_quantize_weights(w, transposed=True)

    def deq(codes, scales):       # rows: 1 x 128 blocks
        return codes.double() * scales.double().t().repeat_interleave(128, 1)[:, :codes.shape[1]]
    w64 = wq.double() * ws.double().repeat_interleave(128, 1)[:, :I].repeat_interleave(128, 2)[:, :, :H]

    # forward
    y, h, rstd = gpu.moe_norm_forward(x, residual=res, weight=nw)
    logits = y.float() @ rw.t()
    idx, tw = gpu.moe_route_forward(logits, K, bias=bias, routed_scale=2.5)
    counts, off, rows, pos = gpu.moe_expert_lists(idx, E, 128)
    yq, ys, yt, yts = gpu.moe_fp8_quantize(y, rows=rows, transposed=True)
    e = gpu.moe_fp8_matmul(yq, ys, wq, ws, offsets=off)
    z = gpu.moe_combine_forward(e, pos, tw)
    # backward
    dz = torch.randn(T, I, generator=g).to(BF16).cuda()
    de, dtw = gpu.moe_combine_backward(dz, e, pos, rows, tw)
    dq, ds, dt, dts = gpu.moe_fp8_quantize(de, transposed=True)
    dyr = gpu.moe_fp8_matmul(dq, ds, wt, wts, offsets=off)
    dw = gpu.moe_fp8_wgrad(yt, yts, dt, dts, offsets=off)
    dl = gpu.moe_route_backward(logits, idx, dtw, routed_scale=2.5)
    drw = dl.t() @ y.float()
    dy = gpu.moe_combine_forward(dyr, pos, add=(dl @ rw).to(BF16))
    dh, dnw = gpu.moe_norm_backward(dy, h, rstd, weight=nw, grad_h=res)
    norm = gpu.moe_grad_norm([dw, drw, dnw])

    # the same step in float64: the rounded activations that the products read, and the gradients through them
    nw64, h64 = nw.double().requires_grad_(True), h.double().requires_grad_(True)
    rw64, w_ = rw.double().requires_grad_(True), w64.clone().requires_grad_(True)
    y64 = h64 / torch.sqrt((h64 ** 2).mean(1, keepdim=True) + 1e-5) * nw64
    p = torch.sigmoid(y64 @ rw64.t()).gather(1, idx.long())
    tw64 = 2.5 * p / (p.sum(1, keepdim=True) + 1e-20)
    z64 = torch.zeros(T, I, dtype=torch.float64, device=dev)
    for k in range(K):
        z64 = z64 + tw64[:, k, None] * torch.einsum("th,tih->ti", y64, w_[idx[:, k].long()])
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())   # noqa: E731
    # activations in e4m3: relative roundings of at most 2^-4 with random signs, 2^-5 on average, in the
    # 2-norm of a sum no more than that of its terms; bf16's 2^-8 beside it
    assert rel(z, z64.detach()) <= 2.0 ** -4
    assert rel(tw, tw64.detach()) <= 2.0 ** -6      # logits from y in bf16
    gh, gnw, grw, gw = torch.autograd.grad(z64, (h64, nw64, rw64, w_), dz.double())
    assert rel(dw, gw) <= 2.0 ** -3                 # both factors of the product in e4m3
    assert rel(drw, grw) <= 2.0 ** -3
    assert rel(dh - res, gh) <= 2.0 ** -3 and rel(dnw, gnw) <= 2.0 ** -3
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in (dw, drw, dnw)))
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    grads = [dw, drw, dnw]
    gpu.moe_grad_clip(grads, norm, want / 4)
    assert abs(float(gpu.moe_grad_norm(grads)) - want / 4) <= 1e-5 * want
    # the row gradients behind the products: rows without a token are zeros, so the weights' gradient has nothing of them
    assert bool((de[rows < 0] == 0).all())
