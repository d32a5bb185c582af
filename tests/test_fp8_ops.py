"""Block-scaled e4m3 quantisers and products (moe_fp8_*): refusals on the host; on the GPU, codes bit
for bit against a plain 64-bit quantiser and products against 64-bit sums of the codes' values."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

F8 = getattr(torch, "float8_e4m3fn", None)
B = 128
P = 4096          # an aligned address that no refused call reaches


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
    yield moe
    assert moe.moe_fp8_device_error() == 0           # no pipeline wait of any call ran out


# ------------------------------------------------------------------------------------ refusals on the host

def test_quantize_refusals(moe):
    L = moe.lib()

    def call(x=P, dt=0, ld=64, T=4, width=64, rows=None, R=4, c=P, s=P, ct=None, st=None):
        return L.moe_fp8_quantize(x, dt, ld, T, width, rows, R, c, s, ct, st, None)
    for kw in (dict(dt=5), dict(T=-1, R=-1), dict(R=5), dict(ld=48), dict(x=None), dict(c=None), dict(s=None), dict(x=P + 8), dict(ld=66),
               dict(c=P + 8), dict(s=P + 2), dict(rows=P + 2), dict(ct=P), dict(st=P), dict(ct=P + 8, st=P), dict(dt=1, ld=68)):
        assert call(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(width=8), dict(width=24), dict(width=131088, ld=131088), dict(rows=P, R=65535 * 128 + 1)):
        assert call(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    assert call(T=0, R=0) == moe.MOE_OK

    def weights(w=P, dt=0, E=2, N=64, K=64, c=P, s=P, ct=None, st=None):
        return L.moe_fp8_quantize_weights(w, dt, E, N, K, c, s, ct, st, None)
    for kw in (dict(dt=3), dict(w=None), dict(w=P + 4), dict(c=None), dict(s=None), dict(ct=P), dict(st=P), dict(c=P + 1), dict(s=P + 1)):
        assert weights(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(E=0), dict(E=65536), dict(N=0), dict(N=131073), dict(K=0), dict(K=40)):
        assert weights(**kw) == moe.MOE_ERR_UNSUPPORTED, kw


def test_product_refusals(moe):
    L = moe.lib()

    def mm(x=P, xs=P, R=4, w=P, ws=P, E=1, N=64, K=64, off=None, y=P, dt=0, ldy=64):
        return L.moe_fp8_matmul(x, xs, R, w, ws, E, N, K, off, y, dt, ldy, None)
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=P + 8), dict(w=P + 8), dict(xs=P + 2),
               dict(ws=P + 1), dict(off=P + 2), dict(y=P + 2), dict(dt=7), dict(ldy=63), dict(R=-1), dict(E=2)):
        assert mm(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(E=0), dict(E=1025, off=P), dict(N=0), dict(N=131073, ldy=131073), dict(K=0), dict(K=72), dict(K=131088), dict(R=65535 * 128 + 1)):
        assert mm(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    assert mm(R=0) == moe.MOE_OK

    def wg(xt=P, xs=P, dyt=P, ds=P, R=128, N=64, K=64, E=1, off=None, dw=P, dt=0):
        return L.moe_fp8_wgrad(xt, xs, dyt, ds, R, N, K, E, off, dw, dt, None)
    for kw in (dict(xt=None), dict(xs=None), dict(dyt=None), dict(ds=None), dict(dw=None), dict(R=64), dict(R=-128), dict(E=2), dict(dt=-1),
               dict(xt=P + 8), dict(dyt=P + 4), dict(ds=P + 2), dict(dw=P + 2), dict(off=P + 1)):
        assert wg(**kw) == moe.MOE_ERR_INVALID, kw
    for kw in (dict(E=0), dict(E=1025, off=P), dict(N=0), dict(K=0), dict(N=131073), dict(R=65536 * 128)):
        assert wg(**kw) == moe.MOE_ERR_UNSUPPORTED, kw
    assert "need" in moe.moe_last_error()
    assert L.moe_fp8_device_error(None) == moe.MOE_ERR_INVALID


def test_stall_refusals(moe):
    f = moe.lib().moe_fp8_debug_stall_next_call
    for a in ((-1, 0), (0, -1), (0, 8)):
        assert f(*a) == moe.MOE_ERR_INVALID, a


# ------------------------------------------------------------------------------------------------ quantisers

def quant_ref(v):
    """Blocks along the last axis of v (float64, any number of blocks of 128): the codes' values and the
    scales, from the definition: all finite e4m3 values in a table, the nearest by comparison."""
    table = sorted({(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)} |
                   {m / 8 * 2.0 ** -6 for m in range(8)})
    table = torch.tensor(table, dtype=torch.float64)
    mid = (table[:-1] + table[1:]) / 2
    n = v.shape[-1]
    pad = torch.zeros(*v.shape[:-1], -(-n // B) * B, dtype=torch.float64)
    pad[..., :n] = v
    blocks = pad.view(*v.shape[:-1], -1, B)
    big = blocks.abs().amax(-1)
    scale = torch.ones_like(big)
    for i in np.ndindex(*big.shape):
        b = big[i].item()
        if not np.isfinite(b):
            scale[i] = float("nan")
        elif b > 0:
            s = 2.0 ** -126
            while b / s > 448:
                s *= 2
            scale[i] = s
    u = blocks / scale[..., None]
    a = u.abs()
    at = torch.searchsorted(mid, a.contiguous(), right=False)               # ties go below here ...
    tie = (at < len(mid)) & (a == mid[at.clamp(max=len(mid) - 1)]) & (at % 2 == 1)
    val = table[(at + tie.long()).clamp(max=len(table) - 1)] * torch.sign(u)  # ... and to the even code
    val = torch.where(scale.isnan()[..., None].expand_as(val), torch.full_like(val, float("nan")), val)
    return val.reshape(*v.shape[:-1], -1)[..., :n], scale


def same(got, want):
    got = got.double().cpu()
    return torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0))


def hard_values(rows, width, seed, dtype):
    """Rows of different sizes, ties, zeros, subnormals, values at the range's ends."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g)
    big = torch.finfo(dtype).max
    x *= torch.exp2(torch.randint(-14, 12, (rows, 1), generator=g).float())
    if rows > 6 and width >= 16:
        x[1] = 0.0
        x[2] = torch.round(torch.rand(width, generator=g) * 256) / 256 * 448       # many ties between codes
        x[3] = big
        x[4, ::3] = torch.finfo(dtype).smallest_normal
        x[4, 1::3] = 0.0
        x[5] = torch.linspace(-1, 1, width) * torch.finfo(dtype).smallest_normal / 4
        x[6, 0] = 448.0
    return x.clamp(-big, big).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,width", [(1, 16), (1, 128), (9, 144), (130, 256), (257, 400), (33, 2048)])
def test_quantize(gpu, T, width, dtype):
    x = hard_values(T, width, T + width, dtype)
    val, scale = quant_ref(x.double())
    codes, scales = gpu.moe_fp8_quantize(x.cuda())
    assert codes.dtype == F8 and codes.shape == (T, width) and scales.shape == (-(-width // B), T)
    assert same(codes.float(), val) and same(scales, scale.t())
    c2, s2, ct, st = gpu.moe_fp8_quantize(x.cuda(), transposed=True)
    assert same(c2.float(), val) and same(s2, scale.t())
    tall = torch.zeros(-(-T // B) * B, width, dtype=torch.float64)
    tall[:T] = x.double()
    val_t, scale_t = quant_ref(tall.t().contiguous())
    assert ct.shape == val_t.shape and same(ct.float(), val_t) and same(st, scale_t.t())


@pytest.mark.gpu
def test_quantize_many_rows(gpu):
    """The variant for many rows gives the same codes as the one for few and the one for both ways."""
    for width, dtype in ((528, torch.bfloat16), (640, torch.float32), (400, torch.float16)):
        x = hard_values(20011, width, 1, dtype).cuda()
        codes, scales = gpu.moe_fp8_quantize(x)
        c2, s2, _, _ = gpu.moe_fp8_quantize(x, transposed=True)
        assert torch.equal(codes.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(scales, s2)
        val, scale = quant_ref(x[-50:].double().cpu())
        assert same(codes[-50:].float(), val) and same(scales[:, -50:], scale.t())


@pytest.mark.gpu
@pytest.mark.parametrize("both", [False, True])
def test_quantize_picked_rows(gpu, both):
    """Rows by index: repeated, negative, behind the last token; rows of a wider buffer."""
    wide = hard_values(20, 336, 2, torch.bfloat16).cuda()
    x = wide[:, 16:288]                                 # 16-byte aligned rows, a stride of their own
    idx = torch.tensor([3, 3, -1, 19, 0, 20, -2**31, 2**31 - 1] + list(range(20)) * 9, dtype=torch.int32)
    out = gpu.moe_fp8_quantize(x, rows=idx.cuda(), transposed=both)
    rows = [x[i].double().cpu() if 0 <= i < 20 else torch.zeros(272, dtype=torch.float64) for i in idx.tolist()]
    full = torch.stack(rows)
    val, scale = quant_ref(full)
    assert same(out[0].float(), val) and same(out[1], scale.t())
    if both:
        tall = torch.zeros(-(-len(rows) // B) * B, 272, dtype=torch.float64)
        tall[:len(rows)] = full
        val, scale = quant_ref(tall.t().contiguous())
        assert same(out[2].float(), val) and same(out[3], scale.t())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_not_finite(gpu, bad, dtype):
    """A block with a NaN or an infinity has the scale NaN, in each orientation its own block alone."""
    x = torch.ones(140, 272, dtype=dtype)
    x[5, 130] = bad
    c, s, ct, st = gpu.moe_fp8_quantize(x.cuda(), transposed=True)
    c1, s1 = gpu.moe_fp8_quantize(x.cuda())
    for q in (s, s1):
        assert bool(q[1, 5].isnan()) and int(q.isnan().sum()) == 1
    assert bool(st[0, 130].isnan()) and int(st.isnan().sum()) == 1
    assert torch.equal(c.view(torch.uint8), c1.view(torch.uint8)) and bool((c[4].float() * s[:, 4].repeat_interleave(B)[:272] == 1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 200, 272), (2, 137, 400), (1, 16, 2048)])
def test_quantize_weights(gpu, E, N, K, dtype):
    w = (0.05 * torch.randn(E, N, K, generator=torch.Generator().manual_seed(N + K))).to(dtype)
    nb, kb = -(-N // B), -(-K // B)
    pad = torch.zeros(E, nb * B, kb * B, dtype=torch.float64)
    pad[:, :N, :K] = w.double()
    blocks = pad.view(E, nb, B, kb, B).permute(0, 1, 3, 2, 4).reshape(E, nb, kb, B * B)
    # one scale for the block: quantise its values against the block's own largest
    big = blocks.abs().amax(-1)
    scale = torch.where(big > 0, torch.exp2(torch.ceil(torch.log2(torch.where(big > 0, big, 1.0) / 448.0))), torch.ones_like(big))
    scale = torch.where(big > 448 * scale, 2 * scale, torch.where(big <= 224 * scale, scale / 2, scale))
    scale = torch.where(big > 0, scale, torch.ones_like(scale))
    spread = scale.repeat_interleave(B, 1)[:, :N].repeat_interleave(B, 2)[:, :, :K]
    codes, s, ct, st = gpu.moe_fp8_quantize_weights(w.cuda(), transposed=True)
    assert same(s, scale) and same(st, scale.transpose(1, 2))
    # rounding: within half a step of the value (2^-4 of it, or half the step of subnormal codes)
    u = w.double() / spread
    err = (codes.double().cpu() - u).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * u.abs(), torch.full_like(u, 2.0 ** -10))).all())
    assert torch.equal(ct.view(torch.uint8), codes.view(torch.uint8).transpose(1, 2).contiguous())
    c2, s2 = gpu.moe_fp8_quantize_weights(w[0].contiguous().cuda())
    assert c2.shape == (N, K) and torch.equal(c2.view(torch.uint8), codes[0].view(torch.uint8)) and torch.equal(s2, s[0])


# -------------------------------------------------------------------------------------------------- products

def codes_of(g, *shape):
    return (100 * torch.randn(*shape, generator=g)).clamp(-448, 448).to(F8)


def spread(s, n):
    return s.double().repeat_interleave(B, dim=-1)[..., :n]


def close(got, ref, size, terms, dtype):
    """got is ref rounded to dtype, off by the float32 sums: the products of two codes are exact, every
    one of `terms` additions and the scales' products round or truncate by at most 2^-23 of the running
    sum, which `size` (the sum of the magnitudes) bounds.  Rounding to nearest takes what lies half a step
    beyond the largest finite value or farther, here max + 16 = 65520 for float16 (its last step is 32), to
    the infinity of its sign."""
    fin = torch.finfo(dtype)
    got = got.double().cpu()
    sums = (terms + 8) * 2.0 ** -23 * size
    edge = fin.max * (1 + fin.eps / (4 - 2 * fin.eps))
    over = ref.abs() + sums >= edge
    assert bool((got.isinf() == over)[(ref.abs() - sums >= edge) | ~over].all()) and bool((got.sign() == ref.sign())[got.isinf()].all())
    tol = sums + fin.eps / 2 * ref.abs() + fin.smallest_normal * fin.eps
    err = torch.where(got.isinf(), torch.zeros_like(ref), (got - ref).abs())
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the tolerance"


def matmul_case(R, N, K, E, seed, offsets=None):
    g = torch.Generator().manual_seed(seed)
    kb, nb = -(-K // B), -(-N // B)
    x, w = codes_of(g, R, K), codes_of(g, E, N, K)
    xs = torch.exp2(torch.randint(-8, 3, (kb, R), generator=g).float()) * (1 + torch.rand(kb, R, generator=g))
    ws = 0.001 * (0.5 + torch.rand(E, nb, kb, generator=g)) * torch.where(torch.rand(E, nb, kb, generator=g) < 0.1, -1.0, 1.0)
    return x, xs, w, ws


def matmul_ref(x, xs, w, ws, off):
    R, K = x.shape
    E, N, _ = w.shape
    xd = x.double() * spread(xs.t(), K)
    ref, size = torch.full((R, N), 7.0, dtype=torch.float64), torch.zeros(R, N, dtype=torch.float64)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            wd = w[e].double() * spread(ws[e].repeat_interleave(B, 0)[:N], K)
            ref[a:b] = xd[a:b] @ wd.t()
            size[a:b] = xd[a:b].abs() @ wd.abs().t()
    return ref, size


def check_matmul(moe, R, N, K, E=1, dtype=torch.float32, off=None, pad=0, shift=0):
    x, xs, w, ws = matmul_case(R, N, K, E, R + N + K + E)
    grouped = off is not None
    ref, size = matmul_ref(x, xs, w, ws, off or [0, R])
    out = torch.full((R, N + pad + shift), 7.0, dtype=dtype, device="cuda")
    view = out[:, shift:shift + N]
    o = torch.tensor(off, dtype=torch.int32, device="cuda") if grouped else None
    y = moe.moe_fp8_matmul(x.cuda(), xs.cuda(), w.cuda() if grouped else w[0].cuda(), ws.cuda() if grouped else ws[0].cuda(), offsets=o, out=view)
    assert y is view
    assert y.dtype == dtype
    close(y, ref, size, K, dtype)
    assert bool((out[:, :shift] == 7).all()) and bool((out[:, shift + N:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,N,K", [(1, 1, 16), (1, 128, 128), (2, 300, 1040), (16, 256, 4096), (17, 129, 272), (64, 512, 640), (65, 257, 144),
                                   (128, 256, 128), (200, 1000, 400), (256, 130, 2048), (257, 256, 128), (400, 640, 1168), (1000, 333, 512)])
def test_matmul(gpu, R, N, K, dtype):
    check_matmul(gpu, R, N, K, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("R,off", [(1, [0, 0, 1, 1]), (5, [0, 2, 2, 5]), (40, [0, 17, 18, 40]), (40, [3, 20, 20, 33]), (200, [0, 0, 199, 200]),
                                   (300, [1, 130, 131, 299]), (900, [0, 900, 900, 900]), (1500, [7, 500, 777, 1400]), (20, [4, 4, 4, 4])])
def test_matmul_experts(gpu, R, off):
    """Rows of three experts: empty ones, uneven ones, rows outside every segment (left as they were)."""
    check_matmul(gpu, R, 264, 400, E=3, off=off)
    check_matmul(gpu, R, 129, 144, E=3, dtype=torch.bfloat16, off=off)


@pytest.mark.gpu
@pytest.mark.parametrize("R,E", [(8, 300), (64, 1024), (700, 48), (3000, 5)])
def test_matmul_many_experts(gpu, R, E):
    cut = sorted(torch.randint(0, R + 1, (E - 1,), generator=torch.Generator().manual_seed(E)).tolist())
    check_matmul(gpu, R, 136, 272, E=E, off=[0] + cut + [R], dtype=torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [3, 50, 150, 600])
@pytest.mark.parametrize("dtype,pad,shift", [(torch.bfloat16, 8, 0), (torch.bfloat16, 1, 1), (torch.float32, 3, 0), (torch.float16, 0, 2)])
def test_matmul_into_strided_rows(gpu, R, dtype, pad, shift):
    check_matmul(gpu, R, 320, 256, dtype=dtype, pad=pad, shift=shift)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N,pad,shift", [(torch.bfloat16, 2000, 0, 0), (torch.float32, 1924, 4, 0), (torch.float16, 2047, 1, 0),
                                               (torch.float16, 1928, 16, 8), (torch.float32, 2000, 1, 0)])
@pytest.mark.parametrize("off", [None, [0, 1303, 3990], [5, 2100, 3900]])
def test_matmul_large_tiles(gpu, dtype, N, pad, shift, off):
    """Sizes whose tiles two blocks share: full and ragged tiles, rows on 16-byte boundaries or not, columns
    beside the output and rows outside every segment left as they were."""
    check_matmul(gpu, 3990, N, 2560, E=len(off) - 1 if off else 1, dtype=dtype, off=off, pad=pad, shift=shift)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [4, 60, 200, 600])
def test_matmul_keeps_rows_apart(gpu, R):
    """A NaN in one row's codes or scale, or in a row that no expert has, stays in that row."""
    x, xs, w, ws = matmul_case(R, 200, 384, 2, R)
    off = [1, R // 2, R - 1]
    ref, size = matmul_ref(x, xs, w, ws, off)
    x[0] = float("nan")
    xs[:, R - 1] = float("nan")
    xs[1, R // 2] = float("nan")
    y = torch.full((R, 200), 7.0, device="cuda")
    gpu.moe_fp8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out=y)
    assert bool(y[R // 2].isnan().all())
    keep = [r for r in range(R) if r != R // 2]
    close(y[keep], ref[keep], size[keep], 384, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K,E", [(3, 300, 400, 1), (40, 200, 272, 5), (60, 640, 1168, 1), (200, 640, 2048, 1), (700, 1300, 1024, 1),
                                     (2300, 1300, 1280, 1), (2300, 2048, 2048, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matmul_scales_whose_product_leaves_float32(gpu, R, N, K, E, dtype):
    """Scales as small and as large as float32 has them: their product alone may be subnormal, zero or
    infinite where the scaled sum is an ordinary number (or 0)."""
    g = torch.Generator().manual_seed(R + N)
    kb, nb = -(-K // B), -(-N // B)
    small = (2.0 ** -6 * torch.randn(E, N, K, generator=g)).clamp(-0.0625, 0.0625)
    x, w = codes_of(g, R, K).float(), small.to(F8)
    xe, we = torch.randint(-4, 3, (kb, R), generator=g).float(), torch.randint(-8, 0, (E, nb, kb), generator=g).float()
    far = torch.arange(R) % 5
    x[far == 1] = 2.0 ** -9 * torch.randint(-1, 2, (int((far == 1).sum()), K), generator=g).float()       # tiny sums, some of them 0
    x[far == 2] = 0.0
    xe[:, far == 1] = 100.0 + torch.randint(0, 4, (kb, int((far == 1).sum())), generator=g)
    xe[:, far == 2] = 120.0
    xe[:, far == 3] = -126.0
    xe[:, far == 4] = -149.0 + 24
    we[:, :, ::2] = 30.0                                    # every other block: 2^130 with the rows of sums of 2^-9 2^-6 n
    we[:, :, 1::4] = -20.0
    xs, ws = torch.exp2(xe) * (1 + torch.rand(kb, R, generator=g)), torch.exp2(we) * (1 + torch.rand(E, nb, kb, generator=g))
    xs[:, far == 4] = torch.where(torch.rand(kb, int((far == 4).sum()), generator=g) < 0.5, xs[:, far == 4] * 2.0 ** -20, xs[:, far == 4])    # subnormal
    x = x.to(F8)
    off = [R * e // E for e in range(E + 1)]
    ref, size = matmul_ref(x, xs, w, ws, off)
    assert float(ref.abs().max()) < torch.finfo(dtype).max / 4 and bool((ref[far == 2] == 0).all())
    y = gpu.moe_fp8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=dtype)
    close(y, ref, size, K, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K", [(1, 512, 6144), (16, 4096, 6144), (128, 1024, 6144), (512, 2000, 6144), (1500, 4096, 4096), (2300, 2048, 6144)])
def test_matmul_error_in_the_2_norm(gpu, R, N, K):
    """Random signs: a block's 4 truncated steps are off by 4 x 2^-23 of its sum at most, and the nb float32
    additions of the blocks by 2^-24 of running sums, whose roots of the sums of squares make
    sqrt(nb / 2) of the last one's: with 48 blocks 13 x 2^-24 in all."""
    x, xs, w, ws = (t.cuda() for t in matmul_case(R, N, K, 1, 4))
    xs.fill_(0.75), ws.fill_(0.0013)
    y = gpu.moe_fp8_matmul(x, xs, w[0], ws[0], out_dtype=torch.float32)
    ref = (x.double() @ w[0].double().t()) * (xs[0, 0].double() * ws[0, 0, 0].double())
    assert float((y.double() - ref).norm() / ref.norm()) <= 16 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("R,E,most", [(4000, 300, 4000), (16384, 1024, 15000), (9000, 8, 8993), (20000, 64, 12345)])
def test_matmul_skewed_routing(gpu, R, E, most):
    """One expert has nearly all rows, so that the rows of an expert on average say little."""
    N, K = 200, 272
    x, xs, w, ws = (t.cuda() for t in matmul_case(R, N, K, E, 3))
    g = torch.Generator().manual_seed(R)
    counts = torch.bincount(torch.randint(0, E, (R - most,), generator=g), minlength=E)
    counts[E // 2] += most
    off = [0] + counts.cumsum(0).tolist()
    y = gpu.moe_fp8_matmul(x, xs, w, ws, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    ref, size = matmul_ref(x.cpu(), xs.cpu(), w.cpu(), ws.cpu(), off)
    close(y, ref, size, K, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K", [(5, 200, 272), (300, 640, 400), (2300, 2048, 2048)])
def test_matmul_of_the_smallest_quantised_rows(gpu, R, N, K):
    """Rows whose scale is the quantiser's least, 2^-126, with weights' scales below 1: the products are
    subnormal powers of two.  Others with a scale that is none (NaN rows), which stay NaN."""
    g = torch.Generator().manual_seed(R)
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-127, -116, (R, 1), generator=g).float())
    x[1] = float("inf")
    w = 0.02 * torch.randn(N, K, generator=g)
    q, s = gpu.moe_fp8_quantize(x.cuda())
    wq, wscale = gpu.moe_fp8_quantize_weights(w.cuda())
    y = gpu.moe_fp8_matmul(q, s, wq, wscale, out_dtype=torch.float32)
    keep = torch.arange(R) != 1
    assert bool(y[1].isnan().all())
    ref, size = matmul_ref(q.float().cpu()[keep], s.cpu()[:, keep], wq.float().cpu()[None], wscale.cpu()[None], [0, R - 1])
    assert float(s[:, 0].min()) >= 2.0 ** -126 and bool((s == 2.0 ** -126).any())
    close(y[keep.cuda()], ref, size, K, torch.float32)


@pytest.mark.gpu
def test_matmul_bad_offsets_stay_in_bounds(gpu):
    """Offsets outside the rows or falling are cut to the rows: nothing else is read or written."""
    x, xs, w, ws = matmul_case(100, 136, 144, 3, 1)
    for off in ([-5, 40, 60, 400], [0, 2**31 - 1, -2**31, 100]):
        pool = torch.full((300, 136), 7.0, device="cuda")
        gpu.moe_fp8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out=pool[100:200])
        assert bool((pool[:100] == 7).all()) and bool((pool[200:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K,E", [(20, 256, 384, 1), (700, 272, 400, 1), (900, 256, 128, 3)])
def test_activation_gradient_is_the_product_with_the_transposed_weights(gpu, R, N, K, E):
    g = torch.Generator().manual_seed(R)
    w, dy = 0.05 * torch.randn(E, N, K, generator=g), torch.randn(R, N, generator=g)
    codes, s, ct, st = gpu.moe_fp8_quantize_weights(w.cuda(), transposed=True)
    q, qs = gpu.moe_fp8_quantize(dy.cuda())
    off = [0, R] if E == 1 else [0, R // 4, R // 4, R]
    o = None if E == 1 else torch.tensor(off, dtype=torch.int32, device="cuda")
    dx = gpu.moe_fp8_matmul(q, qs, ct if E > 1 else ct[0], st if E > 1 else st[0], offsets=o, out_dtype=torch.float32)
    wd = codes.double().cpu() * spread(s.cpu().repeat_interleave(B, 1)[:, :N], K)
    dd = q.double().cpu() * spread(qs.cpu().t(), N)
    for e in range(E):
        a, b = off[e], off[e + 1]
        close(dx[a:b], dd[a:b] @ wd[e], dd[a:b].abs() @ wd[e].abs(), N, torch.float32)


def wgrad_case(R, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    p2 = lambda *s: torch.exp2(torch.randint(-20, 4, s, generator=g).float())   # noqa: E731
    return codes_of(g, K, R), p2(R // B, K), codes_of(g, N, R), p2(R // B, N)


def check_wgrad(moe, R, N, K, off=None, dtype=torch.float32):
    xt, xs, dyt, ds = wgrad_case(R, N, K, R + N + K)
    dw = moe.moe_fp8_wgrad(xt.cuda(), xs.cuda(), dyt.cuda(), ds.cuda(), out_dtype=dtype,
                           offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda"))
    x, d = xt.double() * spread(xs.t(), R), dyt.double() * spread(ds.t(), R)
    segs = off or [0, R]
    got = dw if off is not None else dw[None]
    assert got.shape == (len(segs) - 1, N, K) and got.dtype == dtype
    for e in range(len(segs) - 1):
        a, b = segs[e], segs[e + 1]
        ref = d[:, a:b] @ x[:, a:b].t()
        if a == b:
            assert bool((got[e] == 0).all())
        close(got[e], ref, d[:, a:b].abs() @ x[:, a:b].abs().t(), max(1, b - a), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,N,K", [(128, 1, 1), (128, 128, 16), (256, 300, 272), (640, 129, 257), (1280, 256, 512), (384, 1000, 136)])
def test_wgrad(gpu, R, N, K, dtype):
    check_wgrad(gpu, R, N, K, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("off", [[0, 128, 128, 1024], [0, 0, 0, 0], [128, 256, 896, 896], [0, 1024, 1024, 1024],
                                 [0, 128, 256, 256, 512, 512, 640, 1024]])
def test_wgrad_experts(gpu, off):
    check_wgrad(gpu, 1024, 200, 272, off)
    check_wgrad(gpu, 1024, 520, 144, off, torch.bfloat16)


@pytest.mark.gpu
def test_wgrad_many_tiles_with_and_without_rows(gpu):
    """More tiles than blocks, experts without rows between the others: both accumulators, many times."""
    cut = sorted(torch.randint(0, 17, (15,), generator=torch.Generator().manual_seed(1)).tolist())
    check_wgrad(gpu, 2048, 1000, 1000, [0] + [128 * c for c in cut] + [2048])


@pytest.mark.gpu
@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 6, 7, 10, 13, 30])
def test_wgrad_pairs_with_scales_of_every_stage(gpu, blocks):
    """Tiles of two blocks, whose scales are staged in batches of row blocks by either block and copied to
    the tensor cores by the first: sums of fewer, as many and more row blocks than a batch or the ring of
    batches holds, each with scales of its own; the same bits every time."""
    R, N, K = 128 * blocks, 2048, 1152
    check_wgrad(gpu, R, N, K)
    xt, xs, dyt, ds = (t.cuda() for t in wgrad_case(R, N, K, blocks))
    off = torch.tensor([0, 0, 128 * (blocks // 2), 128 * (blocks // 2), R], dtype=torch.int32, device="cuda")
    first = [gpu.moe_fp8_wgrad(xt, xs, dyt, ds), gpu.moe_fp8_wgrad(xt, xs, dyt, ds, offsets=off)]
    for _ in range(10):
        assert torch.equal(gpu.moe_fp8_wgrad(xt, xs, dyt, ds), first[0])
        assert torch.equal(gpu.moe_fp8_wgrad(xt, xs, dyt, ds, offsets=off), first[1])


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,off", [(256, 256, None), (130, 300, None), (200, 136, [0, 2048, 2048, 4096]), (512, 500, [0, 128, 4096])])
def test_wgrad_few_outputs_from_many_rows(gpu, N, K, off):
    """Blocks that share a tile's rows, experts with fewer row blocks than sharers and with none."""
    check_wgrad(gpu, 4096, N, K, off)
    check_wgrad(gpu, 4096, N, K, off, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(256, 256), (2000, 2560)])
def test_wgrad_long_sums_keep_float32(gpu, N, K):
    """32768 rows: the 2-norm of the error against 64 bits stays within a few float32 roundings a level,
    16 x 2^-24 (sums of 2048 rows by the tensor core, which truncates, then float32 additions); sums in
    one go would be off by 6e-6."""
    R = 32768
    xt, xs, dyt, ds = (t.cuda() for t in wgrad_case(R, N, K, 7))
    xs.fill_(1.0), ds.fill_(1.0)
    dw = gpu.moe_fp8_wgrad(xt, xs, dyt, ds)
    ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for r in range(0, R, 4096):
        ref += dyt[:, r:r + 4096].double() @ xt[:, r:r + 4096].double().t()
    assert float((dw.double() - ref).norm() / ref.norm()) <= 16 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K", [(256, 256, 256), (2048, 2048, 1152), (32768, 256, 256), (32768, 2000, 2560)])
def test_wgrad_sums_of_one_sign(gpu, R, N, K):
    """Codes of one sign, where truncated additions all err the same way.  The tensor core adds the 128 rows
    of a block in 4 steps, 16 blocks in a row: at most 64 truncations of 2^-23 of the running sum, which is
    half of the last one on average; then a float32 addition of 2^-24 for each 16 blocks, of a running
    sum again."""
    xt, _, dyt, _ = (t.cuda() for t in wgrad_case(R, N, K, 9))
    xt, dyt = xt.float().abs().to(F8), dyt.float().abs().to(F8)
    dw = gpu.moe_fp8_wgrad(xt, torch.ones(R // B, K, device="cuda"), dyt, torch.ones(R // B, N, device="cuda"))
    ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for r in range(0, R, 4096):
        ref += dyt[:, r:r + 4096].double() @ xt[:, r:r + 4096].double().t()
    steps, flushes = 4 * min(16, R // B), -(-R // (16 * B))
    assert float((dw.double() - ref).norm() / ref.norm()) <= (steps + 1) / 2 * 2.0 ** -23 + (flushes + 1) / 2 * 2.0 ** -24


@pytest.mark.gpu
def test_pairs_one_after_another(gpu):
    """Short calls of both products in tiles of two blocks, each starting as the one before ends: the
    arrivals on a block's barriers belong to its own call."""
    xt, xs, dyt, ds = (t.cuda() for t in wgrad_case(256, 2048, 1152, 8))
    x, xsc, w, ws = (t.cuda() for t in matmul_case(2300, 2048, 2048, 1, 8))
    first = None
    for _ in range(60):
        got = [gpu.moe_fp8_wgrad(xt, xs, dyt, ds), gpu.moe_fp8_wgrad(xt[:, :128].contiguous(), xs[:1], dyt[:, :128].contiguous(), ds[:1]),
               gpu.moe_fp8_matmul(x, xsc, w[0], ws[0]), gpu.moe_fp8_matmul(x, xsc, w[0], ws[0])]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.gpu
def test_wgrad_no_rows_and_nan(gpu):
    z = lambda *s: torch.zeros(*s, device="cuda")    # noqa: E731
    dw = gpu.moe_fp8_wgrad(z(16, 0).to(F8), z(0, 16), z(24, 0).to(F8), z(0, 24), offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert dw.shape == (3, 24, 16) and bool((dw == 0).all())
    xt, xs, dyt, ds = wgrad_case(256, 40, 48, 3)
    xs[1, 5], ds[0, 7] = float("nan"), float("nan")
    dw = gpu.moe_fp8_wgrad(xt.cuda(), xs.cuda(), dyt.cuda(), ds.cuda()).cpu()
    want = torch.zeros(40, 48, dtype=torch.bool)
    want[:, 5] = want[7] = True
    assert torch.equal(dw.isnan(), want)


@pytest.mark.gpu
def test_wgrad_bad_offsets_stay_in_bounds(gpu):
    xt, xs, dyt, ds = wgrad_case(512, 40, 48, 4)
    pool = torch.full((5, 40, 48), 7.0, device="cuda")
    for off in ([-128, 130, 2**31 - 1, 100], [512, 0, -2**31, 2**31 - 1]):
        gpu.moe_fp8_wgrad(xt.cuda(), xs.cuda(), dyt.cuda(), ds.cuda(), offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out=pool[1:4])
        assert bool((pool[0] == 7).all()) and bool((pool[4] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("op,R,N,K,E,blocks,stalls", [
    ("matmul", 700, 640, 1152, 48, (0,), (0, 4, 7)),          # 16-row tiles
    ("matmul", 1, 640, 4096, 1, (0, 3), (0, 3)),              # shared by a cluster
    ("matmul", 200, 640, 2048, 1, (0, 3), (0, 2)),            # 128 x 128, shared
    ("matmul", 700, 1300, 1024, 1, (0,), (0, 6)),             # 128 x 128
    ("matmul", 2300, 1300, 1280, 1, (0,), (0, 2, 8)),         # 128 x 256
    ("matmul", 2300, 2048, 2048, 1, (0, 1), (0, 3, 9)),       # a pair's 256 x 256
    ("wgrad", 1664, 2048, 1152, 1, (0, 1), (0, 3, 9)),        # a pair's
    ("wgrad", 4096, 256, 256, 1, (0, 5), (0, 3))])            # 128 x 128, shared
def test_waits_that_run_out_end_the_call(gpu, op, R, N, K, E, blocks, stalls):
    """A block that stops copying its operands: the waits for them give up after half a second (no fault, no
    hang), the call returns and reports the flag, and the next calls are right again."""
    if op == "matmul":
        x, xs, w, ws = (t.cuda() for t in matmul_case(R, N, K, E, 1))
        off = torch.arange(E + 1, device="cuda").mul_(R).div_(E, rounding_mode="floor").int()
        call = lambda: gpu.moe_fp8_matmul(x, xs, w, ws, offsets=off)        # noqa: E731
    else:
        xt, xs, dyt, ds = (t.cuda() for t in wgrad_case(R, N, K, 1))
        call = lambda: gpu.moe_fp8_wgrad(xt, xs, dyt, ds)                    # noqa: E731
    want = call()
    assert gpu.moe_fp8_device_error() == 0
    for block in blocks:
        for stages in stalls:
            gpu.moe_fp8_debug_stall_next_call(stages, block)
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            waited = time.perf_counter() - t0
            assert gpu.moe_fp8_device_error(check=False) == gpu.MOE_DEVICE_ERR_TC, (block, stages)
            assert waited < 10.0, waited
            assert gpu.moe_fp8_device_error() == 0               # cleared by the read
            for _ in range(2):
                assert torch.equal(call(), want), (block, stages)
            assert gpu.moe_fp8_device_error() == 0
    gpu.moe_fp8_debug_stall_next_call(1000, 0)               # more stages than a block has: the usual call
    assert torch.equal(call(), want) and gpu.moe_fp8_device_error() == 0


@pytest.mark.gpu
def test_binding_refusals(gpu):
    x, xs, w, ws = (t.cuda() for t in matmul_case(8, 64, 256, 2, 5))
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    f = gpu.moe_fp8_matmul
    bad = [lambda: f(x.float(), xs, w[0], ws[0]), lambda: f(x, xs, w, ws), lambda: f(x, xs, w[0], ws[0], offsets=off), lambda: f(x, xs.t(), w[0], ws[0]),
           lambda: f(x, xs, w[0], ws), lambda: f(x[:, :128], xs[:1], w[0], ws[0]), lambda: f(x, xs, w, ws, offsets=off[:2]),
           lambda: f(x, xs, w, ws, offsets=off.long()), lambda: f(x, xs, w[0], ws[0], out=torch.zeros(8, 63, device="cuda")),
           lambda: f(x, xs, w[0], ws[0], out_dtype=torch.float64), lambda: f(x.cpu(), xs, w[0], ws[0]), lambda: f(x, xs.cpu(), w[0], ws[0]),
           lambda: f(x, xs, w[0], ws[0], out=torch.zeros(8, 64, device="cuda"), out_dtype=torch.float16)]
    q = gpu.moe_fp8_quantize
    y = torch.zeros(8, 256, device="cuda")
    bad += [lambda: q(y.double()), lambda: q(y.t()), lambda: q(y[0]), lambda: q(y, rows=off.float()), lambda: q(y[:, :24]), lambda: q(y[:, 1:17]),
            lambda: q(torch.zeros(8, 258, device="cuda")[:, :256]), lambda: gpu.moe_fp8_quantize_weights(y[:, ::2]),
            lambda: gpu.moe_fp8_quantize_weights(y[None, None])]
    xt, txs, dyt, tds = (t.cuda() for t in wgrad_case(256, 32, 48, 6))
    g = gpu.moe_fp8_wgrad
    bad += [lambda: g(xt[:, :128], txs, dyt, tds), lambda: g(xt, txs[:1], dyt, tds), lambda: g(xt, txs, dyt, tds.double()),
            lambda: g(xt, txs, dyt, tds, offsets=off[:1]), lambda: g(xt, txs, dyt, tds, out=torch.zeros(48, 32, device="cuda")),
            lambda: g(xt[:, :64].contiguous(), txs[:0], dyt[:, :64].contiguous(), tds[:0])]
    for i, b in enumerate(bad):
        with pytest.raises(gpu.MoeError):
            b()
            pytest.fail(f"call {i} was taken")


# ------------------------------------------------------------------- together: one training step of the experts

def expert_step(moe, x, idx, tw, wq, wd_q, dy, E):
    """Forward and gradients of sum_k tw[t, k] down_e(silu(gate_e x) * up_e x), the way a program runs it."""
    T, K = idx.shape
    I = wq[0].shape[1] // 2
    counts, off, rows, pos = moe.moe_expert_lists(idx, E, align=B)
    xq, xs, xt, xts = moe.moe_fp8_quantize(x, rows=rows, transposed=True)
    gu = moe.moe_fp8_matmul(xq, xs, wq[0], wq[1], offsets=off, out=torch.zeros(rows.numel(), 2 * I, device=x.device))
    gate, up = gu[:, :I], gu[:, I:]
    sig = torch.sigmoid(gate)
    h = gate * sig * up
    hq, hs, ht, hts = moe.moe_fp8_quantize(h, transposed=True)
    d = moe.moe_fp8_matmul(hq, hs, wd_q[0], wd_q[1], offsets=off, out=torch.zeros(rows.numel(), x.shape[1], device=x.device))
    y = (d[pos.reshape(-1).long()].view(T, K, -1) * tw[:, :, None]).sum(1)
    # backward
    dd = torch.zeros_like(d)
    dd[pos.reshape(-1).long()] = (tw[:, :, None] * dy[:, None]).reshape(T * K, -1)
    dq, ds, dt, dts = moe.moe_fp8_quantize(dd, transposed=True)
    dh = moe.moe_fp8_matmul(dq, ds, wd_q[2], wd_q[3], offsets=off, out=torch.zeros_like(h))
    dwd = moe.moe_fp8_wgrad(ht, hts, dt, dts, offsets=off)
    dgu = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], 1)
    gq, gs, gt, gts = moe.moe_fp8_quantize(dgu, transposed=True)
    dxr = moe.moe_fp8_matmul(gq, gs, wq[2], wq[3], offsets=off, out=torch.zeros(rows.numel(), x.shape[1], device=x.device))
    dwgu = moe.moe_fp8_wgrad(xt, xts, gt, gts, offsets=off)
    dx = dxr[pos.reshape(-1).long()].view(T, K, -1).sum(1)
    return y, dx, dwgu, dwd, counts


def step_inputs(T, E, K, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    x, dy = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    idx = torch.rand(T, E, generator=g).topk(K, 1).indices.int()
    tw = torch.rand(T, K, generator=g) + 0.5
    wgu, wdn = torch.randn(E, 2 * I, H, generator=g) / H ** 0.5, torch.randn(E, H, I, generator=g) / I ** 0.5
    return x, dy, idx, tw, wgu, wdn


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,H,I", [(1, 4, 2, 128, 64), (50, 6, 2, 256, 128), (700, 4, 3, 272, 144)])
def test_training_step_of_the_experts(gpu, T, E, K, H, I):
    """Against autograd of the exact layer in float64.  Each of the values that are quantised on the way
    is off by at most 2^-4 of itself, the weights too, so a product of n random terms is off by about
    2^-4 sqrt(2) / sqrt(3) of its root mean square; four such products follow one another at most, hence
    the 2-norm within 4 x 0.051 < 0.25 of the result's.  A wrong row, expert or scale is off by 1."""
    x, dy, idx, tw, wgu, wdn = (t.cuda() for t in step_inputs(T, E, K, H, I, T))
    wq, wd_q = gpu.moe_fp8_quantize_weights(wgu, transposed=True), gpu.moe_fp8_quantize_weights(wdn, transposed=True)
    y, dx, dwgu, dwd, counts = expert_step(gpu, x, idx, tw, wq, wd_q, dy, E)
    xr, wgr, wdr = (t.double().cpu().requires_grad_(True) for t in (x, wgu, wdn))
    out = []
    for t in range(T):
        acc = 0
        for k in range(K):
            e = int(idx[t, k])
            gu = wgr[e] @ xr[t]
            acc = acc + tw[t, k].double().cpu() * (wdr[e] @ (torch.nn.functional.silu(gu[:I]) * gu[I:]))
        out.append(acc)
    ref = torch.stack(out)
    ref.backward(dy.double().cpu())
    assert counts.tolist() == torch.bincount(idx.cpu().reshape(-1).long(), minlength=E).tolist()
    for got, want in ((y, ref.detach()), (dx, xr.grad), (dwgu, wgr.grad), (dwd, wdr.grad)):
        assert float((got.double().cpu() - want).norm() / want.norm()) < 0.25
    idle = (counts == 0).nonzero()[:, 0]
    assert bool((dwgu[idle] == 0).all()) and bool((dwd[idle] == 0).all())


@pytest.mark.gpu
def test_step_is_the_same_captured_replayed_and_on_another_stream(gpu):
    T, E, K, H, I = 300, 6, 2, 256, 128
    first = [t.cuda() for t in step_inputs(T, E, K, H, I, 1)]
    second = [t.cuda() for t in step_inputs(T, E, K, H, I, 2)]
    x, dy, idx, tw = (t.clone() for t in first[:4])
    wq, wd_q = gpu.moe_fp8_quantize_weights(first[4], transposed=True), gpu.moe_fp8_quantize_weights(first[5], transposed=True)
    run = lambda: expert_step(gpu, x, idx, tw, wq, wd_q, dy, E)   # noqa: E731
    want = [t.clone() for t in run()]
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for src in (second, first):
        for a, b in zip((x, dy, idx, tw), src):
            a.copy_(b)
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        for g, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o))


@pytest.mark.gpu
def test_explicit_stream_argument(gpu):
    """stream= runs and allocates on that stream, given as a torch stream or as a raw handle."""
    x, xs, w, ws = (t.cuda() for t in matmul_case(70, 200, 256, 1, 9))
    want = gpu.moe_fp8_matmul(x, xs, w[0], ws[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for h in (s, s.cuda_stream, 0):
        y = gpu.moe_fp8_matmul(x, xs, w[0], ws[0], stream=h)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_more_than_two_to_the_31_elements(gpu):
    """Rows whose elements lie beyond 2^31 of x, of the codes, of the transposed codes and of y: the last
    rows of a long call are those of a short one."""
    R, width, N = 1_100_032, 2048, 2048
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(R, width, dtype=torch.bfloat16, device="cuda")
    x[:-512] = 1.0
    x[-512:] = torch.randn(512, width, generator=g, device="cuda").bfloat16()
    w = gpu.moe_fp8_quantize_weights(0.02 * torch.randn(N, width, generator=g, device="cuda"))
    c, s, ct, st = gpu.moe_fp8_quantize(x, transposed=True)
    c1, s1 = gpu.moe_fp8_quantize(x)
    c2, s2, ct2, st2 = gpu.moe_fp8_quantize(x[-512:].contiguous(), transposed=True)
    for a, b in ((c[-512:], c2), (c1[-512:], c2), (ct[:, -512:], ct2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(s[:, -512:], s2) and torch.equal(s1[:, -512:], s2) and torch.equal(st[-4:], st2)
    del x, c1, ct
    y = gpu.moe_fp8_matmul(c, s, *w)
    # against 64 bits (a short call may add the blocks up in another order)
    ref, size = matmul_ref(c2.cpu(), s2.cpu(), w[0].cpu()[None], w[1].cpu()[None], [0, 512])
    close(y[-512:], ref, size, width, torch.bfloat16)
    assert bool((y[1000] == y[R - 600]).all())


@pytest.mark.gpu
def test_first_calls_of_a_process_may_be_captured(gpu):
    """Nothing that a first call sets up (kernels' shared memory, the error word, the encoder of tensor
    maps) breaks a capture: a fresh process whose first calls are captured gets the same results."""
    import subprocess
    import sys
    from pathlib import Path
    code = """
import torch, int4_moe_expert_gb300 as moe
torch.manual_seed(0)
x = torch.randn(300, 256, device="cuda"); w = torch.randn(3, 264, 256, device="cuda")
idx = torch.randint(0, 3, (300, 2), dtype=torch.int32, device="cuda"); logits = torch.randn(300, 3, device="cuda")
torch.cuda.synchronize()
def step():
    c, off, rows, pos = moe.moe_expert_lists(idx, 3, 128)
    loss, n, s, t = moe.moe_balance_forward(logits, idx, 1.0)
    q, qs, qt, qts = moe.moe_fp8_quantize(x, rows=rows, transposed=True)
    few = moe.moe_fp8_quantize(x[:4])
    wq, ws, wt, wts = moe.moe_fp8_quantize_weights(w, transposed=True)
    y = moe.moe_fp8_matmul(q, qs, wq, ws, offsets=off, out=torch.zeros(rows.numel(), 264, device="cuda"))
    z = moe.moe_fp8_matmul(few[0], few[1], wq[0], ws[0])
    return [c, off, rows, pos, loss, moe.moe_balance_backward(logits, 2, n, t, 1.0), y, z, moe.moe_fp8_wgrad(qt, qts, qt, qts, offsets=off)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay(); torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parents[1], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
