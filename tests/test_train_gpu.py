"""The training operators against their formulas in 64 bits, and each gradient against
differences of its forward formula.

Tolerances.  u = 2^-24 is half a unit in the last place of fp32.  A sum of n terms whose
every partial sum is rounded at most r times is within r * u * (sum of the terms'
magnitudes); the kernels' sums round at most n / 64 + 64 times (a thread's or a step's share
in sequence, then a tree).  A tensor-core step of 16 products rounds the running sum once,
towards zero (2u).  A result rounded to bf16 is off by 2^-9 of itself more (2^-8 here, for
the rounding of a value that is itself off), and no result is nearer to a value than its type's
smallest subnormal (2^-133 in bf16, 2^-149 in fp32) lets it be.
"""
import numpy as np
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * scale).to(dtype)


def nan(shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def check(got, ref, mag, rounds, name=""):
    """|got - ref| <= rounds u mag (+ bf16's own rounding), everywhere; NaN where ref is NaN."""
    torch.cuda.synchronize()
    g = got.double()
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{name}: NaN at other places"
    bound = rounds * U * mag + (2.0 ** -8 * ref.abs() + 2.0 ** -133 if got.dtype == BF16 else 2.0 ** -149)
    bad = ((g - ref).abs() > bound) & ~torch.isnan(ref)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {g[i].item()} "
                             f"wanted {ref[i].item()} within {torch.as_tensor(bound)[i].item()}")


def rounds(n):
    return n / 64 + 64


# ---------------------------------------------------------------- layer norm

def ln_ref(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    y = xh if gamma is None else xh * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd


def ln_run(x, gamma, beta, eps=1e-5):
    T, d = x.shape
    plan = binding.moe_plan(T, d, 1, 1, 256)
    y, mean, rstd = nan((T, d), BF16), nan((T,)), nan((T,))
    binding.moe_layernorm(plan, x, gamma, beta, eps, y, mean, rstd)
    return plan, y, mean, rstd


LN_SHAPES = [(1, 16), (3, 48), (333, 272), (5, 1024), (65, 2064), (1000, 4096), (7, 7168), (2, 16400), (9, 32784),
             (2, 65536)]


@pytest.mark.parametrize("T,d", LN_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layernorm(T, d, dtype):
    x = (randn((T, d), 1) * 3 + randn((T, 1), 2)).to(dtype)
    gamma, beta = 1 + randn((d,), 3, scale=0.1), randn((d,), 4, scale=0.1)
    _, y, mean, rstd = ln_run(x, gamma, beta)
    ry, rmean, rrstd = ln_ref(x, gamma, beta, 1e-5)
    xa = x.double().abs().mean(1)
    check(mean, rmean[:, 0], xa, rounds(d), "mean")
    check(rstd, rrstd[:, 0], rrstd[:, 0] * (1 + xa * rrstd[:, 0]), rounds(d), "rstd")
    mag = (x.double().abs() + xa[:, None]) * rrstd * (1 + xa[:, None] * rrstd) * gamma.abs().double() + beta.abs().double()
    check(y, ry, mag, rounds(d), "y")


def test_layernorm_without_weights_or_statistics():
    x = randn((37, 528), 5, BF16)
    plan, y, _, _ = ln_run(x, None, None)
    y2 = nan((37, 528), BF16)
    binding.moe_layernorm(plan, x, None, None, 1e-5, y2)
    ry, _, _ = ln_ref(x, None, None, 1e-5)
    check(y, ry, ry.abs() + 1, rounds(528))
    assert torch.equal(y, y2)


def test_layernorm_of_constant_and_far_rows():
    """A row of equal values has variance 0 (y = beta); a row far from zero keeps its spread
    (the variance is summed about the mean)."""
    d = 4096
    x = torch.full((3, d), 1000.0, device=DEV)
    x[1] += randn((d,), 6, scale=0.5)
    x[2] = 0.0
    beta = randn((d,), 7)
    _, y, mean, rstd = ln_run(x, None, beta)
    ry, rm, rr = ln_ref(x, None, beta, 1e-5)
    assert torch.equal(y[0], beta.to(BF16)) and torch.equal(y[2], beta.to(BF16))
    # the mean is off by up to rounds(d) u |x| = 1e3 * 128 u = 7.6e-3, and y by that times rstd
    check(y[1], ry[1], 1000.0 * rr[1] + ry[1].abs(), rounds(d))
    check(rstd, rr[:, 0], rr[:, 0] * (1 + 1000.0 * 1000.0 * U * rounds(d) * rr[:, 0]), rounds(d))


def test_layernorm_passes_nan_and_infinity_on_within_their_row():
    x = randn((4, 272), 8)
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    _, y, mean, rstd = ln_run(x, None, None)
    ry, _, _ = ln_ref(x, None, None, 1e-5)
    assert torch.isnan(y[1:3]).all()
    check(y[[0, 3]], ry[[0, 3]], ry[[0, 3]].abs() + 1, rounds(272))


def ln_back_ref(dy, x, gamma, mean, rstd, dres):
    dy, x = dy.double(), x.double()
    g = 1.0 if gamma is None else gamma.double()
    r = rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * r
    v = dy * g
    m1, m2 = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    dx = r * (v - m1 - xh * m2)
    mag = r * (v.abs() + v.abs().mean(1, keepdim=True) + xh.abs() * (v * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    # xh's own error: x - mean is rounded relative to |x| + |mean|
    big = (x.abs() + mean.double().abs()[:, None]) * r + xh.abs()
    mag = mag + r * big * m2.abs() + r * xh.abs() * (v.abs() * big).mean(1, keepdim=True)
    return dx, mag, (dy * xh).sum(0), (dy.abs() * big).sum(0), dy.sum(0), dy.abs().sum(0)


def ln_back_run(dy, x, gamma, dres, in_place=False):
    T, d = x.shape
    plan = binding.moe_plan(T, d, 1, 1, 256)
    _, mean, rstd = ln_ref(x, None, None, 1e-5)
    mean, rstd = mean[:, 0].float().contiguous(), rstd[:, 0].float().contiguous()
    scratch = binding.backward_scratch(plan)
    dx = dres.clone() if in_place else nan((T, d), x.dtype)
    dg, db = nan((d,)), nan((d,))
    binding.moe_layernorm_backward(plan, dy, x, gamma, mean, rstd, dx if in_place else dres, dx, dg, db, scratch)
    return plan, scratch, mean, rstd, dx, dg, db


@pytest.mark.parametrize("T,d", LN_SHAPES + [(20000, 48), (5000, 2064), (1500, 4112), (1501, 8192), (600, 12304), (300, 32768)])
@pytest.mark.parametrize("x_dtype,dy_dtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
def test_layernorm_backward(T, d, x_dtype, dy_dtype):
    x = (randn((T, d), 11) + randn((T, 1), 12)).to(x_dtype)
    dy, dres = randn((T, d), 13, dy_dtype), randn((T, d), 14, x_dtype)
    gamma = 1 + randn((d,), 15, scale=0.1)
    _, _, mean, rstd, dx, dg, db = ln_back_run(dy, x, gamma, dres)
    rdx, mdx, rdg, mdg, rdb, mdb = ln_back_ref(dy, x, gamma, mean, rstd, dres)
    check(dx, rdx, mdx, rounds(d), "dx")
    check(dg, rdg, mdg, rounds(T), "dgamma")
    check(db, rdb, mdb, rounds(T), "dbeta")


def test_layernorm_backward_optional_arguments_and_repeats():
    T, d = 700, 1040
    x, dy, dres = randn((T, d), 16, BF16), randn((T, d), 17), randn((T, d), 18, BF16)
    plan, scratch, mean, rstd, dx, dg, db = ln_back_run(dy, x, None, dres)
    rdx, mdx, rdg, mdg, rdb, mdb = ln_back_ref(dy, x, None, mean, rstd, dres)
    check(dx, rdx, mdx, rounds(d))
    in_place = ln_back_run(dy, x, None, dres, in_place=True)
    for a, b in zip((dx, dg, db), in_place[4:]):
        assert torch.equal(a, b)
    for want_g, want_b in ((True, False), (False, True), (False, False)):
        dx2, dg2, db2 = nan((T, d), BF16), nan((d,)), nan((d,))
        binding.moe_layernorm_backward(plan, dy, x, None, mean, rstd, None, dx2, dg2 if want_g else None,
                                       db2 if want_b else None, scratch if want_g or want_b else None)
        check(dx2, rdx - dres.double(), mdx, rounds(d))
        assert torch.equal(dg2, dg) if want_g else torch.isnan(dg2).all()
        assert torch.equal(db2, db) if want_b else torch.isnan(db2).all()


@pytest.mark.parametrize("T,d", [(1, 16), (3, 272), (16, 64), (1, 2064), (1, 9008), (2, 9008), (1, 16400)])
@pytest.mark.parametrize("want_g,want_b", [(True, True), (True, False), (False, True), (False, False)])
def test_layernorm_backward_of_few_rows(T, d, want_g, want_b):
    """One CTA writes the weights' gradients itself, those that are wanted."""
    x, dy, dres = randn((T, d), 26, BF16), randn((T, d), 27), randn((T, d), 28, BF16)
    plan, scratch, mean, rstd, dx, dg, db = ln_back_run(dy, x, None, dres)
    _, _, rdg, mdg, rdb, mdb = ln_back_ref(dy, x, None, mean, rstd, dres)
    check(dg, rdg, mdg, rounds(T))
    check(db, rdb, mdb, rounds(T))
    dx2, dg2, db2 = nan((T, d), BF16), nan((d,)), nan((d,))
    binding.moe_layernorm_backward(plan, dy, x, None, mean, rstd, dres, dx2, dg2 if want_g else None,
                                   db2 if want_b else None, scratch if want_g or want_b else None)
    assert torch.equal(dx2, dx)
    assert torch.equal(dg2, dg) if want_g else torch.isnan(dg2).all()
    assert torch.equal(db2, db) if want_b else torch.isnan(db2).all()


def test_layernorm_gradient_against_differences():
    T, d = 9, 272
    x, gamma, beta, r = (randn(s, 20 + i) for i, s in enumerate(((T, d), (d,), (d,), (T, d))))
    _, _, _, _, dx, dg, db = ln_back_run(r, x, gamma, torch.zeros_like(x))
    f = lambda x, g, b: float((ln_ref(x, g, b, 1e-5)[0] * r.double()).sum())  # noqa: E731
    x64, g64, b64 = x.double(), gamma.double(), beta.double()
    h = 1e-4
    for i, (got, at) in enumerate(((dx, x64), (dg, g64), (db, b64))):
        v = randn(at.shape, 30 + i).double()
        args = lambda s: [a + s * h * v if j == i else a for j, a in enumerate((x64, g64, b64))]  # noqa: E731
        want = (f(*args(1)) - f(*args(-1))) / (2 * h)
        # differences: h^2 f''' / 6 is below 1e-6 here; the gradient: 4096 u of the sum of magnitudes
        assert abs(float((got.double() * v).sum()) - want) <= 1e-5 * float((got.double() * v).abs().sum())


# ---------------------------------------------------------------- SwiGLU and its 8-bit checkpoint

def ckpt_ref(GU):
    """codes, scales (the definition's fp32 steps in numpy) of GU [S][2F]."""
    S, F2 = GU.shape
    F = F2 // 2
    nb = binding.checkpoint_blocks(F)
    v = np.zeros((S, 2, nb * 128), np.float32)
    v[:, :, :F] = GU.float().cpu().numpy().reshape(S, 2, F)
    v = v.reshape(S, 2, nb, 128)
    bad = ~np.isfinite(v).all(-1)
    amax = np.abs(np.where(np.isfinite(v), v, 0)).max(-1).astype(np.float32)
    small = amax < np.float32(2.0 ** -121)
    safe = np.where(small | bad, np.float32(1), amax)
    inv = (np.float32(127) / safe).astype(np.float32)
    with np.errstate(invalid="ignore"):
        codes = np.rint((v * inv[..., None]).astype(np.float32))
    codes = np.where((small | bad)[..., None], 0, codes).astype(np.int8)
    scales = np.where(small, np.float32(0), (safe / np.float32(127)).astype(np.float32))
    scales = np.where(bad, np.float32("nan"), scales)
    codes = codes.reshape(S, 2, nb * 128)[:, :, :F].reshape(S, F2)
    return torch.from_numpy(np.ascontiguousarray(codes)), torch.from_numpy(scales.reshape(S, 2 * nb))


def restored(codes, scales):
    S, F2 = codes.shape
    F, nb = F2 // 2, scales.shape[1] // 2
    col = torch.arange(F, device=codes.device) // 128
    sc = scales.double()
    return codes[:, :F].double() * sc[:, :nb][:, col], codes[:, F:].double() * sc[:, nb:][:, col]


def ckpt_plan(S, F, dtype):
    return binding.moe_plan(S, 256, 8, 1, 2 * F, out_dtype=binding.MOE_OUT_BF16 if dtype == BF16 else binding.MOE_OUT_F32)


def ckpt_run(GU, with_h=True):
    S, F = GU.shape[0], GU.shape[1] // 2
    plan = ckpt_plan(S, F, GU.dtype)
    H = nan((S, F), BF16) if with_h else None
    codes = torch.full((S, 2 * F), 77, dtype=torch.int8, device=DEV)
    scales = nan((S, 2 * binding.checkpoint_blocks(F)))
    binding.moe_swiglu_checkpoint(plan, GU, H, codes, scales)
    torch.cuda.synchronize()
    return plan, H, codes, scales


CKPT_SHAPES = [(1, 8), (3, 24), (50, 120), (7, 128), (33, 136), (257, 1408), (5, 1000), (2, 14336)]


@pytest.mark.parametrize("S,F", CKPT_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu_checkpoint(S, F, dtype):
    GU = randn((S, 2 * F), 40)
    GU[:, :: 7] *= 20
    GU = GU.to(dtype)
    plan, H, codes, scales = ckpt_run(GU)
    rc, rs = ckpt_ref(GU)
    assert torch.equal(codes.cpu(), rc) and torch.equal(scales.cpu(), rs)
    g, u = GU[:, :F].double(), GU[:, F:].double()
    # sigmoid: expf within 2 ulp, an addition, a division, two products
    check(H, g * torch.sigmoid(g) * u, (g * torch.sigmoid(g) * u).abs() * (1 + g.abs()), 16, "H")
    _, _, codes2, scales2 = ckpt_run(GU, with_h=False)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


def test_swiglu_checkpoint_of_zero_tiny_huge_and_invalid_blocks():
    S, F = 8, 264
    GU = randn((S, 2 * F), 41)
    GU[0, :128] = 0
    GU[1, 128:256] *= 1e-38
    GU[2, F:F + 128] *= 3e38 / GU[2, F:F + 128].abs().max()
    GU[3, 5], GU[4, F + 130], GU[5, 256] = float("nan"), float("inf"), float("-inf")
    GU[6, :128] = 2.0 ** -121
    GU[7, :128] = 2.0 ** -122
    _, H, codes, scales = ckpt_run(GU)
    rc, rs = ckpt_ref(GU)
    assert torch.equal(codes.cpu(), rc)
    assert torch.equal(torch.isnan(scales.cpu()), torch.isnan(rs))
    assert torch.equal(torch.nan_to_num(scales.cpu(), nan=-1.0), torch.nan_to_num(rs, nan=-1.0))
    assert scales[7, 0] == 0 and scales[6, 0] > 0
    dH = randn((S, F), 42)
    H2, dGU = nan((S, F), BF16), torch.zeros((S, 2 * F), dtype=BF16, device=DEV)
    binding.moe_swiglu_checkpoint_backward(ckpt_plan(S, F, F32), dH, codes, scales, H2, dGU)
    # the block that held a NaN or an infinity gives NaN gradients, its neighbours do not
    assert torch.isnan(dGU[3, :128]).all() and not torch.isnan(dGU[3, 128:F]).any()
    assert torch.isnan(dGU[4, 128:256]).all() and not torch.isnan(dGU[4, :128]).any()
    assert torch.isnan(dGU[5, 256:F]).all()


def swiglu_back_ref(g, u, dH):
    s, dH = torch.sigmoid(g), dH.double()
    return torch.cat([dH * u * (s + g * s * (1 - s)), dH * g * s], 1), g * s * u


@pytest.mark.parametrize("S,F", CKPT_SHAPES)
@pytest.mark.parametrize("dh_dtype", [F32, BF16])
def test_swiglu_checkpoint_backward(S, F, dh_dtype):
    GU = randn((S, 2 * F), 43, scale=3.0)
    plan, _, codes, scales = ckpt_run(GU)
    dH = randn((S, F), 44, dh_dtype)
    H, dGU = nan((S, F), BF16), nan((S, 2 * F), BF16)
    binding.moe_swiglu_checkpoint_backward(plan, dH, codes, scales, H, dGU)
    g, u = restored(codes, scales)
    rd, rh = swiglu_back_ref(g, u, dH)
    s = torch.sigmoid(g)
    d64 = dH.double().abs()
    mag = torch.cat([d64 * u.abs() * s * (1 + g.abs()) ** 2, d64 * (g * s).abs() * (1 + g.abs())], 1)
    check(dGU, rd, mag, 32, "dGU")
    check(H, rh, rh.abs() * (1 + g.abs()), 16, "H")
    dGU2 = nan((S, 2 * F), BF16)
    binding.moe_swiglu_checkpoint_backward(plan, dH, codes, scales, None, dGU2)
    assert torch.equal(dGU, dGU2)


def test_swiglu_gradient_against_differences():
    """The stored values are what the backward pass differentiates at."""
    S, F = 6, 136
    plan, _, codes, scales = ckpt_run(randn((S, 2 * F), 45))
    dH = randn((S, F), 46)
    dGU = nan((S, 2 * F), BF16)
    binding.moe_swiglu_checkpoint_backward(plan, dH, codes, scales, None, dGU)
    v64 = torch.cat(restored(codes, scales), 1)
    f = lambda v: ((v[:, :F] * torch.sigmoid(v[:, :F]) * v[:, F:]) * dH.double()).sum(1)  # noqa: E731
    h = 1e-4
    for c in (0, 7, F - 1, F, 2 * F - 1):
        step = torch.zeros_like(v64)
        step[:, c] = h
        want = (f(v64 + step) - f(v64 - step)) / (2 * h)
        assert ((dGU[:, c].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()


# ---------------------------------------------------------------- combine backward

def cb_run(T, k, N, y_dtype, dout_dtype, seed=50, dest=None):
    S = T * k
    plan = binding.moe_plan(T, 256, max(32, k), k, N,
                            out_dtype=binding.MOE_OUT_BF16 if y_dtype == BF16 else binding.MOE_OUT_F32)
    dout, Y = randn((T, N), seed, dout_dtype), randn((S, N), seed + 1, y_dtype)
    w = torch.softmax(randn((T, k), seed + 2), 1)
    if dest is None:
        dest = torch.randperm(S, generator=_gen(seed + 3), device=DEV).to(torch.int32)
    dY, dw = nan((S, N), BF16), nan((T, k))
    binding.moe_combine_backward(plan, dout, Y, w, dest, dY, dw)
    torch.cuda.synchronize()
    return dout, Y, w, dest, dY, dw


def cb_ref(dout, Y, w, dest):
    T, k = w.shape
    d = dest.long()
    dY = torch.zeros(T * k, dout.shape[1], dtype=torch.float64, device=DEV)
    dY[d] = (w.double()[:, :, None] * dout.double()[:, None]).reshape(T * k, -1)
    terms = Y.double()[d].reshape(T, k, -1) * dout.double()[:, None]
    return dY, terms.sum(-1), terms.abs().sum(-1)


@pytest.mark.parametrize("T,k,N", [(1, 1, 16), (5, 2, 48), (333, 4, 1408), (64, 8, 4096), (17, 3, 272), (9, 32, 528),
                                   (40, 12, 2064), (2, 5, 65536)])
@pytest.mark.parametrize("y_dtype,dout_dtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
def test_combine_backward(T, k, N, y_dtype, dout_dtype):
    dout, Y, w, dest, dY, dw = cb_run(T, k, N, y_dtype, dout_dtype)
    rY, rw, mw = cb_ref(dout, Y, w, dest)
    check(dY, rY, rY.abs(), 2, "dY")
    check(dw, rw, mw, rounds(N), "dw")


@pytest.mark.parametrize("k,N", [(3, 1408), (8, 1040), (11, 528), (1, 2032)])
@pytest.mark.parametrize("y_dtype,dout_dtype", [(F32, BF16), (BF16, F32)])
def test_combine_backward_many_tokens(k, N, y_dtype, dout_dtype):
    """A warp a token, with rows of several passes and more tokens than warps at once."""
    T = 10 * torch.cuda.get_device_properties(0).multi_processor_count * 8 // 3 + 5
    dout, Y, w, dest, dY, dw = cb_run(T, k, N, y_dtype, dout_dtype)
    rY, rw, mw = cb_ref(dout, Y, w, dest)
    check(dY, rY, rY.abs(), 2, "dY")
    check(dw, rw, mw, rounds(N), "dw")


def test_combine_backward_skips_slots_outside_the_rows():
    T, k, N = 6, 2, 272
    dest = torch.randperm(T * k, generator=_gen(1), device=DEV).to(torch.int32)
    lost = dest.clone()
    lost[3], lost[8] = -1, T * k
    dout, Y, w, _, dY, dw = cb_run(T, k, N, BF16, F32, dest=lost)
    rY, rw, mw = cb_ref(dout, Y, w, dest)
    gone = dest[[3, 8]].long()
    keep = torch.ones(T * k, dtype=torch.bool, device=DEV)
    keep[gone] = False
    assert torch.isnan(dY[gone]).all() and (dw.reshape(-1)[[3, 8]] == 0).all()
    check(dY[keep], rY[keep], rY[keep].abs(), 2)
    slots = torch.ones(T * k, dtype=torch.bool, device=DEV)
    slots[[3, 8]] = False
    check(dw.reshape(-1)[slots], rw.reshape(-1)[slots], mw.reshape(-1)[slots], rounds(N))


def test_combine_gradient_against_differences():
    T, k, N = 7, 3, 48
    dout, Y, w, dest, dY, dw = cb_run(T, k, N, F32, F32, seed=60)
    f = lambda Y, w: float(((Y[dest.long()].reshape(T, k, N) * w[:, :, None]).sum(1) * dout.double()).sum())  # noqa: E731
    vy, vw, h = randn(Y.shape, 61).double(), randn(w.shape, 62).double(), 1e-3
    Y64, w64 = Y.double(), w.double()
    # the function is linear in each argument: differences are exact but for rounding
    for got, v, want in ((dY, vy, (f(Y64 + h * vy, w64) - f(Y64 - h * vy, w64)) / (2 * h)),
                         (dw, vw, (f(Y64, w64 + h * vw) - f(Y64, w64 - h * vw)) / (2 * h))):
        tol = 2.0 ** -8 if got.dtype == BF16 else 1e-5
        assert abs(float((got.double() * v).sum()) - want) <= tol * float((got.double() * v).abs().sum())


# ---------------------------------------------------------------- gradients of the grouped product

def grad_setup(counts, d, N, seed=70, plan_kw=None):
    S, E = sum(counts), len(counts)
    plan = binding.moe_plan(S, d, E, 1, N, **(plan_kw or {}))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    off = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device=DEV)
    A, dY = randn((S, d), seed, BF16), randn((S, N), seed + 1, BF16)
    W = randn((E, d, N), seed + 2, BF16)
    return plan, ws, st, off, A, dY, W


def segments(counts):
    ends = np.cumsum(counts).tolist()
    return [(e, b - c, b) for e, (c, b) in enumerate(zip(counts, ends))]


def dgrad_ref(counts, dY, W):
    out = [dY[a:b].double() @ W[e].double().T for e, a, b in segments(counts)]
    mag = [dY[a:b].double().abs() @ W[e].double().abs().T for e, a, b in segments(counts)]
    return torch.cat(out), torch.cat(mag)


def wgrad_ref(counts, A, dY):
    out = [A[a:b].double().T @ dY[a:b].double() for _, a, b in segments(counts)]
    mag = [A[a:b].double().abs().T @ dY[a:b].double().abs() for _, a, b in segments(counts)]
    return torch.stack(out), torch.stack(mag)


def mma_rounds(K):
    """one rounding of 2u per step of 16, twice over for what happens inside a step, and the joins"""
    return 4 * (K / 16 + 16)


GRAD_CASES = [
    ([1], 16, 16),
    ([3], 272, 48),
    ([0, 1, 0, 2, 0], 64, 528),
    ([15, 16, 17, 0, 31, 33], 48, 272),
    ([63, 64, 65, 1], 272, 1040),
    ([127, 128, 129], 528, 64),
    ([255, 0, 257, 256], 512, 144),
    ([700], 1040, 528),
    ([2000, 5, 0, 300], 80, 592),
    ([701, 1003, 77, 1], 272, 336),   # long odd reductions before another expert's rows
    ([513] * 5 + [449], 528, 512),
    # few tiles and a long reduction, which is split: over the rows, over N, with other experts beside it
    ([5000], 64, 80),
    ([4501, 70, 0, 6213], 80, 144),
    ([5], 272, 2608),
    ([130, 0, 3], 528, 4624),
    ([2] * 64, 256, 512),
    ([0] * 31 + [100], 128, 256),
    # experts whose offsets just fit beside seven stages of loads, and more
    ([66] * 255 + [400], 48, 80),
    ([66] * 299 + [700], 272, 80),
    ([65] * 1023 + [90], 16, 32),
]


@pytest.mark.parametrize("counts,d,N", GRAD_CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_dgrad(counts, d, N, dtype):
    plan, ws, st, off, _, dY, W = grad_setup(counts, d, N)
    dA = nan((sum(counts), d), dtype)
    binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
    assert binding.moe_read_status(st)[0] == 0
    ref, mag = dgrad_ref(counts, dY, W)
    check(dA, ref, mag, mma_rounds(N), "dA")


@pytest.mark.parametrize("counts,d,N", GRAD_CASES)
@pytest.mark.parametrize("dtype,accumulate", [(F32, False), (BF16, False), (F32, True)])
def test_grouped_wgrad(counts, d, N, dtype, accumulate):
    plan, ws, st, off, A, dY, _ = grad_setup(counts, d, N)
    before = randn((len(counts), d, N), 77) if accumulate else nan((len(counts), d, N), dtype)
    dW = before.clone()
    binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st, accumulate=accumulate)
    assert binding.moe_read_status(st)[0] == 0
    ref, mag = wgrad_ref(counts, A, dY)
    if accumulate:
        ref, mag = ref + before.double(), mag + before.double().abs()
    check(dW, ref, mag, mma_rounds(max(counts)), "dW")
    if not accumulate:
        for e, c in enumerate(counts):
            assert c or (dW[e] == 0).all()


def test_grouped_gradients_keep_other_experts_values_out():
    """Rows of one expert that hold NaN or infinities reach no other expert's results."""
    counts, d, N = [37, 5, 70, 129, 9], 272, 336
    plan, ws, st, off, A, dY, W = grad_setup(counts, d, N)
    ref_a, _ = dgrad_ref(counts, dY, W)
    ref_w, mag_w = wgrad_ref(counts, A, dY)
    for e, a, b in segments(counts):
        if e % 2 == 1:
            A[a:b], dY[a:b], W[e] = float("nan"), float("inf"), float("nan")
    dA, dW = nan((sum(counts), d)), nan((len(counts), d, N))
    binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
    binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
    assert binding.moe_read_status(st)[0] == 0
    for e, a, b in segments(counts):
        if e % 2 == 0:
            assert torch.isfinite(dA[a:b]).all() and torch.isfinite(dW[e]).all()
            check(dW[e], ref_w[e], mag_w[e], mma_rounds(counts[e]))
            assert float((dA[a:b].double() - ref_a[a:b]).norm()) <= 1e-5 * float(ref_a[a:b].norm())
        else:
            assert torch.isnan(dA[a:b]).all() and torch.isnan(dW[e]).all()


@pytest.mark.parametrize("K", [1024, 16384])
def test_grouped_gradients_keep_32_bit_sums_over_long_reductions(K):
    """fp32 results of a long reduction stay within 1e-6 (norm): 512 products at a time in the
    tensor cores' sum (about 5e-7 by its rounding towards zero), the sums of those in fp32."""
    plan, ws, st, off, A, dY, _ = grad_setup([K], 128, 256, seed=80)
    dW = nan((1, 128, 256))
    binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
    ref, _ = wgrad_ref([K], A, dY)
    assert binding.moe_read_status(st)[0] == 0
    assert float((dW.double() - ref).norm()) <= 1e-6 * float(ref.norm())
    plan, ws, st, off, _, dY, W = grad_setup([130], 256, K, seed=81)
    dA = nan((130, 256))
    binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
    ref, _ = dgrad_ref([130], dY, W)
    assert binding.moe_read_status(st)[0] == 0
    assert float((dA.double() - ref).norm()) <= 1e-6 * float(ref.norm())


def test_grouped_gradients_against_differences():
    """Y is linear in A and in W: (Y(A + hV) - Y(A - hV)) / 2h is exact but for rounding."""
    counts, d, N = [5, 0, 40, 17], 64, 80
    plan, ws, st, off, A, dY, W = grad_setup(counts, d, N, seed=85)
    dA, dW = nan((sum(counts), d)), nan((4, d, N))
    binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
    binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
    assert binding.moe_read_status(st)[0] == 0

    def f(A, W):
        return sum(float(((A[a:b] @ W[e]) * dY[a:b].double()).sum()) for e, a, b in segments(counts))
    A64, W64, h = A.double(), W.double(), 1e-3
    va, vw = randn(A.shape, 86).double(), randn(W.shape, 87).double()
    for got, v, want in ((dA, va, (f(A64 + h * va, W64) - f(A64 - h * va, W64)) / (2 * h)),
                         (dW, vw, (f(A64, W64 + h * vw) - f(A64, W64 - h * vw)) / (2 * h))):
        assert abs(float((got.double() * v).sum()) - want) <= 1e-5 * float((got.double() * v).abs().sum())


def test_grouped_gradients_report_offsets_that_are_no_segments():
    counts, d, N = [40, 60], 64, 64
    for bad in ([0, 40, 99], [1, 40, 100], [0, 120, 100], [0, -5, 100]):
        plan, ws, st, _, A, dY, W = grad_setup(counts, d, N)
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        dA, dW = nan((100, d)), nan((2, d, N))
        binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
        assert binding.moe_read_status(st)[0] == binding.MOE_ERR_DEVICE
        st.zero_()
        binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
        assert binding.moe_read_status(st)[0] == binding.MOE_ERR_DEVICE
        assert torch.isnan(dA).all() and torch.isnan(dW).all()


def test_grouped_gradients_repeat_share_a_workspace_and_run_in_a_graph():
    """The same bits every time, on another stream, between forward calls on the same
    workspace, and replayed from a CUDA graph."""
    counts, d, N = [300, 0, 41, 513, 90], 272, 400
    plan, ws, st, off, A, dY, W = grad_setup(counts, d, N)
    S = sum(counts)
    first = []
    side = torch.cuda.Stream()
    Y = nan((S, N))
    for i in range(3):
        dA, dW = nan((S, d)), nan((len(counts), d, N), BF16)
        s = side if i == 1 else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        binding.moe_grouped_gemm(plan, A, off, W, Y, ws, st, s)
        binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st, s)
        binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st, stream=s)
        binding.moe_grouped_gemm(plan, A, off, W, Y, ws, st, s)
        torch.cuda.synchronize()
        first.append((dA, dW, Y.clone()))
    for other in first[1:]:
        for a, b in zip(first[0], other):
            assert torch.equal(a, b)
    dA, dW = nan((S, d)), nan((len(counts), d, N), BF16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
        binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
    for _ in range(2):
        dA.fill_(float("nan"))
        dW.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dA, first[0][0]) and torch.equal(dW, first[0][1])
    assert binding.moe_read_status(st)[0] == 0


def test_grouped_wgrad_adds_up_exactly_over_many_calls():
    """Few rows an expert: the epilogue's loads and stores of the accumulated sums are the whole work, and every
    role runs as far ahead of it as the rings let it.  Whole numbers: each sum is exact, a tile that is missed, done
    twice or done with another's rows shows."""
    counts, d, N, calls = [64, 0, 17, 64] * 12, 2048, 1536, 150
    plan, ws, st, off, A, dY, _ = grad_setup(counts, d, N)
    dY.fill_(1)
    A.copy_((torch.arange(sum(counts), device=DEV) % 3 + 1)[:, None])
    want = torch.stack([A[r0:r1, 0].double().sum() for _, r0, r1 in segments(counts)])
    dW = torch.zeros(len(counts), d, N, device=DEV)
    for i in range(calls):
        binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st, accumulate=True)
    assert binding.moe_read_status(st)[0] == 0
    for e in range(len(counts)):
        assert (dW[e] == float(want[e]) * calls).all(), e


def test_split_reductions_repeat_and_share_a_workspace():
    """Pieces of a reduction are added in their order whichever is done first, and offsets that split nothing
    leave nothing of an earlier call behind."""
    counts, d, N = [9001, 9, 130], 272, 4624
    S = sum(counts)
    plan, ws, st, off, A, dY, W = grad_setup(counts, d, N)
    even = torch.tensor([0, 3050, 6100, S], dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(3):
        dA, dW = nan((S, d), BF16), nan((3, d, N))
        binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
        binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
        dW2 = nan((3, d, N))
        binding.moe_grouped_gemm_wgrad(plan, A, dY, even, dW2, ws, st)
        torch.cuda.synchronize()
        outs.append((dA, dW, dW2))
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)
    ref, mag = wgrad_ref(counts, A, dY)
    check(outs[0][1], ref, mag, mma_rounds(max(counts)))
    ref, mag = wgrad_ref([3050, 3050, S - 6100], A, dY)
    check(outs[0][2], ref, mag, mma_rounds(3050))
    assert binding.moe_read_status(st)[0] == 0


def test_calls_wait_for_their_stream_and_for_events_of_others():
    """Launched while the kernel before them ends, the calls still see all that their stream has been told to wait
    for: a kernel, a copy and a fill before them, and another stream's work through an event."""
    T, d, k, N = 512, 1040, 2, 528
    plan = binding.moe_plan(T, d, 1, 1, 256)
    cplan = binding.moe_plan(T, 256, 8, k, N, out_dtype=1)
    x, other = randn((T, d), 90, BF16), randn((T, d), 91, BF16)
    dout, w = randn((T, N), 92), randn((T, k), 93)
    Y = randn((T * k, N), 94, BF16)
    dest = torch.randperm(T * k, generator=_gen(95), device=DEV).to(torch.int32)

    def results(x, dout, stream):
        y, mean, rstd = nan((T, d), BF16), nan((T,)), nan((T,))
        dx, dg, db = nan((T, d), BF16), nan((d,)), nan((d,))
        dY, dw = nan((T * k, N), BF16), nan((T, k))
        scratch = binding.backward_scratch(plan)
        torch.cuda.synchronize()

        def run():
            binding.moe_layernorm(plan, x, None, None, 1e-5, y, mean, rstd, stream)
            binding.moe_layernorm_backward(plan, y, x, None, mean, rstd, None, dx, dg, db, scratch, stream)
            binding.moe_combine_backward(cplan, dout, Y, w, dest, dY, dw, stream)
            return y, mean, rstd, dx, dg, db, dY, dw
        return run

    want = [t.clone() for t in results(x, dout, None)()]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for how in ("copy", "fill and add", "event"):
        late_x, late_dout = other.clone(), torch.zeros_like(dout)
        run = results(late_x, late_dout, b)
        with torch.cuda.stream(a if how == "event" else b):
            torch.cuda._sleep(10_000_000)
            if how == "fill and add":
                late_x.zero_()
                late_x.add_(x)
            else:
                late_x.copy_(x)
            late_dout.copy_(dout)
        if how == "event":
            binding.moe_layernorm(plan, other, None, None, 1e-5, nan((T, d), BF16), None, None, b)
            b.wait_stream(a)
        got = run()
        torch.cuda.synchronize()
        for g, r in zip(got, want):
            assert torch.equal(g, r), how


def test_no_rows():
    """T = 0: nothing is read; sums over rows are zero."""
    plan = binding.moe_plan(0, 64, 4, 2, 64)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    dW, dg, db = nan((4, 64, 64)), nan((64,)), nan((64,))
    binding.moe_grouped_gemm_wgrad(plan, e(0, 64), e(0, 64), off, dW, ws, st)
    kept = randn((4, 64, 64), 1)
    want = kept.clone()
    binding.moe_grouped_gemm_wgrad(plan, e(0, 64), e(0, 64), off, kept, ws, st, accumulate=True)
    binding.moe_grouped_gemm_dgrad(plan, e(0, 64), off, e(4, 64, 64), e(0, 64), ws, st)
    binding.moe_layernorm(plan, e(0, 64), None, None, 1e-5, e(0, 64))
    binding.moe_layernorm_backward(plan, e(0, 64), e(0, 64), None, e(0, dt=F32), e(0, dt=F32), None, e(0, 64), dg, db,
                                   binding.backward_scratch(plan))
    binding.moe_swiglu_checkpoint(plan, e(0, 64, dt=F32), None, e(0, 64, dt=torch.int8), e(0, 2, dt=F32))
    binding.moe_swiglu_checkpoint_backward(plan, e(0, 32), e(0, 64, dt=torch.int8), e(0, 2, dt=F32), None, e(0, 64))
    binding.moe_combine_backward(plan, e(0, 64), e(0, 64, dt=F32), e(0, 2, dt=F32), e(0, 2, dt=torch.int32), e(0, 64),
                                 e(0, 2, dt=F32))
    assert binding.moe_read_status(st)[0] == 0
    assert (dW == 0).all() and (dg == 0).all() and (db == 0).all() and torch.equal(kept, want)


# ---------------------------------------------------------------- refusals

def test_refusals_of_the_binding():
    plan = binding.moe_plan(8, 64, 4, 2, 64)
    x = randn((8, 64), 1, BF16)
    y = torch.empty_like(x)
    for bad, word in ((x[:4], "elements"), (randn((64, 8), 1, BF16).T, "strided"), (x.half(), "float16"),
                      (x.cpu(), "cpu"), (None, "missing")):
        with pytest.raises(ValueError, match=word):
            binding.moe_layernorm(plan, bad, None, None, 1e-5, y)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    dY, W = randn((16, 64), 2, BF16), randn((4, 64, 64), 3, BF16)
    with pytest.raises(ValueError, match="offsets"):
        binding.moe_grouped_gemm_dgrad(plan, dY, off.long(), W, randn((16, 64), 4), ws, st)
    with pytest.raises(ValueError, match="W"):
        binding.moe_grouped_gemm_dgrad(plan, dY, off, W[:3], randn((16, 64), 4), ws, st)


def test_refusals_of_the_library():
    plan = binding.moe_plan(8, 64, 4, 2, 64)
    lib = binding.load_library()
    h = plan.handle
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    p = buf.data_ptr()
    bad, ws_err, unsup = binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_WORKSPACE, binding.MOE_ERR_UNSUPPORTED
    assert lib.moe_layernorm(h, p, 2, p, p, 1e-5, p, p, p, None) == bad        # dtype
    assert lib.moe_layernorm(h, p, 1, p, p, 0.0, p, p, p, None) == bad         # eps
    assert lib.moe_layernorm(h, p, 1, p, p, float("nan"), p, p, p, None) == bad
    assert lib.moe_layernorm(h, p, 1, p, p, float("inf"), p, p, p, None) == bad
    assert lib.moe_layernorm(h, p + 2, 1, p, p, 1e-5, p, p, p, None) == bad    # alignment
    assert lib.moe_layernorm(h, None, 1, p, p, 1e-5, p, p, p, None) == bad
    assert lib.moe_layernorm(h, p, 1, p + 4, p, 1e-5, p, p, p, None) == bad
    assert lib.moe_layernorm_backward(h, p, 0, p, 1, p, p, p, p, p, p, p, None, None) == ws_err
    assert lib.moe_layernorm_backward(h, p, 0, p, 1, p, p, p, p, p, p, p, p + 16, None) == ws_err
    assert lib.moe_layernorm_backward(h, p, 0, p, 1, p, None, p, p, p, p, p, p, None) == bad
    assert lib.moe_layernorm_backward(h, p, 0, p, 5, p, p, p, p, p, p, p, p, None) == bad
    assert lib.moe_swiglu_checkpoint(h, p, p, p + 8, p, None) == bad
    assert lib.moe_swiglu_checkpoint(h, p, p, None, p, None) == bad
    assert lib.moe_swiglu_checkpoint_backward(h, p, 7, p, p, p, p, None) == bad
    assert lib.moe_swiglu_checkpoint_backward(h, p, 1, p, p, p, None, None) == bad
    assert lib.moe_combine_backward(h, p, 1, p, p, p + 1, p, p, None) == bad
    assert lib.moe_combine_backward(h, p, 3, p, p, p, p, p, None) == bad
    assert lib.moe_grouped_gemm_dgrad(h, p, p, p, p, 9, p, p, None) == bad
    assert lib.moe_grouped_gemm_dgrad(h, p, p, p, p, 0, None, p, None) == ws_err
    assert lib.moe_grouped_gemm_dgrad(h, p, p, p, p, 0, p, None, None) == bad
    assert lib.moe_grouped_gemm_dgrad(h, p, p, p + 8, p, 0, p, p, None) == bad
    assert lib.moe_grouped_gemm_wgrad(h, p, p, p, p, 1, 1, p, p, None) == unsup  # bf16 sums
    assert lib.moe_grouped_gemm_wgrad(h, p, p, p, p, 0, 2, p, p, None) == bad
    assert lib.moe_grouped_gemm_wgrad(h, p, p, p, p, 0, 0, p + 64, p, None) == ws_err
    assert lib.moe_grouped_gemm_wgrad(h, p, p, p, None, 0, 0, p, p, None) == bad
    assert (buf == 0).all()
