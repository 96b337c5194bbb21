"""The 8-bit forward operators against their formulas in 64 bits.

Tolerances.  u = 2^-24 is half a unit in the last place of fp32.  An fp32 sum whose partial sums are rounded at most r
times is within r u (sum of the terms' magnitudes).  A row's sum of squares is rounded at most d / 64 + 64 times (a
thread's share in sequence, then a tree).  A block of 128 products takes four tensor-core steps, each rounding the running
sum once, towards zero (2u); the blocks' sums are added in sequence, the product of two scales and the multiplication by
it are a rounding each.  A result rounded to bf16 is off by 2^-8 of itself at most, an e4m3 code by 2^-4 of itself or (below
2^-6) by 2^-10.
"""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
F32, BF16, E4M3, I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale).to(dtype)


def nan(shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=F32, device=DEV).to(dtype)


def blocks(n):
    return (n + 127) // 128


def within(got, ref, bound, name=""):
    torch.cuda.synchronize()
    g = got.double()
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{name}: NaN at other places"
    bad = ((g - ref).abs() > bound) & ~torch.isnan(ref)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {g[i].item()} wanted "
                             f"{ref[i].item()} within {torch.as_tensor(bound)[i].item()}")


def spread(scales, n):
    """[rows, blocks] as [rows, n]."""
    return scales.double().repeat_interleave(128, 1)[:, :n]


def block_amax(v):
    n = v.shape[1]
    return torch.nn.functional.pad(v.abs(), (0, blocks(n) * 128 - n)).reshape(v.shape[0], -1, 128).amax(-1)


def check_8bit(codes, scales, ref, err, name=""):
    """codes, scales: ref (64 bits, known to `err`) in 8 bits."""
    n = ref.shape[1]
    amax, e = block_amax(ref), block_amax(err)
    within(scales, amax / 448, e / 448 + 2 * U * amax / 448, name + " scales")
    s = spread(scales, n)
    got = codes.double() * s
    half = torch.maximum(2.0 ** -4 * (ref.abs() + err), 2.0 ** -10 * s)
    within(got, ref, half * (1 + 4 * U) + err + 4 * U * ref.abs(), name + " values")


# ---------------------------------------------------------------- RMS norm

def rms_run(x, res, gamma, h_dtype, eps=1e-5, y=True, codes=True, in_place=False):
    T, d = x.shape
    plan = binding.moe_plan(T, d, 1, 1, 256)
    h = None if res is None else res.clone() if in_place else nan((T, d), h_dtype)
    out = dict(h=h, y=nan((T, d), BF16) if y else None, codes=nan((T, d), E4M3) if codes else None,
               scales=nan((T, blocks(d))) if codes else None, rstd=nan((T,)))
    binding.moe_rmsnorm(plan, x, h if in_place else res, gamma, eps, h, out["y"], out["codes"], out["scales"], out["rstd"])
    return plan, out


def rms_ref(x, res, gamma, h_dtype, eps=1e-5):
    h = x if res is None else (x.float() + res.float()).to(h_dtype)
    hd = h.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1) + eps)
    y = hd * rstd[:, None]
    return h, rstd, y if gamma is None else y * gamma.double()


def rms_check(out, ref, d, name=""):
    h, rstd, y = ref
    r = (d / 64 + 64) / 2 + 8  # half of the sum's relative error, and the roundings after it
    if out["h"] is not None:
        assert torch.equal(out["h"], h)
    within(out["rstd"], rstd, r * U * rstd, name + " rstd")
    err = r * U * y.abs()
    if out["y"] is not None:
        within(out["y"], y, err + 2.0 ** -8 * y.abs() + 2.0 ** -133, name + " y")
    if out["codes"] is not None:
        check_8bit(out["codes"], out["scales"], y, err, name)


RMS_SHAPES = [(1, 16), (3, 48), (333, 272), (5, 1024), (65, 2064), (1000, 4096), (7, 7168), (2, 16400), (3, 32768),
              (2, 32784), (2, 65536)]


@pytest.mark.parametrize("T,d", RMS_SHAPES)
@pytest.mark.parametrize("x_dtype,h_dtype", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_rmsnorm_with_residual(T, d, x_dtype, h_dtype):
    x, res, gamma = randn((T, d), 1, x_dtype), randn((T, d), 2, h_dtype, 3.0), 1 + randn((d,), 3, scale=0.1)
    _, out = rms_run(x, res, gamma, h_dtype)
    rms_check(out, rms_ref(x, res, gamma, h_dtype), d)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,d", [(37, 528), (2, 40016)])
def test_rmsnorm_alone_and_in_place(T, d, dtype):
    x, res = randn((T, d), 4, dtype), randn((T, d), 5, dtype)
    _, out = rms_run(x, None, None, dtype)
    rms_check(out, rms_ref(x, None, None, dtype), d, "no residual")
    _, only_y = rms_run(x, None, None, dtype, codes=False)
    _, only_8 = rms_run(x, None, None, dtype, y=False)
    assert torch.equal(out["y"], only_y["y"])
    assert torch.equal(out["codes"].view(torch.uint8), only_8["codes"].view(torch.uint8))
    assert torch.equal(out["scales"], only_8["scales"])
    _, placed = rms_run(x, res, None, dtype, in_place=True)
    rms_check(placed, rms_ref(x, res, None, dtype), d, "in place")


def test_rmsnorm_of_rows_that_are_zero_tiny_huge_or_not_numbers():
    d = 400
    x = randn((8, d), 6)
    x[1] = 0.0
    x[2] *= 2.0 ** -100       # sum of squares is 0 in fp32: rstd = 1 / sqrt(eps)
    x[3, 130:256] = 0.0       # a block of almost nothing else
    x[4] *= 1e15
    x[5, 3], x[6, 7], x[7, 399] = float("nan"), float("inf"), float("-inf")
    _, out = rms_run(x, None, None, F32)
    ref = rms_ref(x, None, None, F32)
    good = slice(0, 5)
    rms_check({k: None if v is None else v[good] for k, v in out.items()}, tuple(v[good] for v in ref), d)
    assert (out["codes"][1].float() == 0).all() and (out["scales"][1] == 0).all()
    # tiny values: the scale of y = x / sqrt(eps) is far above the smallest that is stored, and in range
    assert (out["scales"][2] > 0).all()
    assert torch.isnan(out["y"][5]).all() and torch.isnan(out["scales"][5]).all()
    for r, c in ((6, 7), (7, 399)):  # infinity times 1 / infinity; the others are 0
        assert torch.isnan(out["y"][r, c]) and torch.isnan(out["scales"][r, c // 128])
    assert (out["codes"][5].float() == 0).all()


@pytest.mark.parametrize("d", [16, 48, 400, 1024, 2064, 4096, 7168, 16400, 32768, 40016])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rmsnorm_of_rows_whose_squares_pass_the_range(d, dtype):
    """Finite rows up to the type's largest values, beside ordinary ones: their sum of squares is beyond fp32."""
    scale = torch.tensor([1.0, 1e18, 1e19, 1e20, 1e30, 1e36, 6e37], device=DEV)[:, None]
    x = (randn((7, d), 15).clamp(-5, 5) * scale).to(dtype)
    x[6, 0] = torch.finfo(dtype).max
    gamma = 1 + randn((d,), 16, scale=0.1)
    _, out = rms_run(x, None, gamma, dtype)
    rms_check(out, rms_ref(x, None, gamma, dtype), d)
    res = (randn((7, d), 17).clamp(-5, 5) * scale * 0.25).to(dtype)
    x[6, 0] = 0
    _, placed = rms_run(x * 0.25, res, gamma, dtype, in_place=True)
    rms_check(placed, rms_ref(x * 0.25, res, gamma, dtype), d, "in place")


@pytest.mark.parametrize("T,d", [(20000, 16), (9000, 272), (5000, 1040), (3001, 4096), (700, 16400), (400, 40016)])
def test_rmsnorm_of_a_few_such_rows_among_many(T, d):
    """Rows are worked on several to a CTA, and more than one after the other: the others stay to the bit as without them."""
    x, res = randn((T, d), 18, BF16), randn((T, d), 19, BF16)
    at = torch.tensor([0, 5, T // 2, T - 1], device=DEV)
    big, big_res = x.clone(), res.clone()
    big[at] *= 1e30
    big_res[at] *= 1e30
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[at] = False
    for r, br in ((None, None), (res, big_res)):
        _, plain = rms_run(x, r, None, BF16, in_place=r is not None)
        _, out = rms_run(big, br, None, BF16, in_place=r is not None)
        ref = rms_ref(big[at], None if br is None else br[at], None, BF16)
        rms_check({n: None if v is None else v[at] for n, v in out.items()}, ref, d)
        for n, v in out.items():
            if v is not None:
                assert torch.equal(v[rest].float(), plain[n][rest].float()), n


def test_rmsnorm_with_an_eps_near_the_range():
    """h^2 / d and eps are in range, their sum is not."""
    d = 64
    x = torch.full((3, d), 1.5e19, device=DEV)
    x[0] = 1.0
    _, out = rms_run(x, None, None, F32, eps=3e38)
    rms_check(out, rms_ref(x, None, None, F32, eps=3e38), d)


@pytest.mark.parametrize("d", [16, 400, 4096, 40016])
def test_rmsnorm_of_a_row_with_infinities(d):
    """NaN where they are (in 8 bits their block) and 0 elsewhere; its neighbours are not touched."""
    x = randn((3, d), 14)
    _, plain = rms_run(x, None, None, F32)
    x[1, 3], x[1, d - 1] = float("inf"), float("-inf")
    _, out = rms_run(x, None, None, F32)
    torch.cuda.synchronize()
    there = torch.zeros(d, dtype=torch.bool, device=DEV)
    there[3] = there[d - 1] = True
    block = torch.nn.functional.pad(there, (0, blocks(d) * 128 - d)).reshape(-1, 128).any(1)
    assert out["rstd"][1] == 0
    assert torch.equal(torch.isnan(out["y"][1]), there) and (out["y"][1][~there] == 0).all()
    assert torch.equal(torch.isnan(out["scales"][1]), block) and (out["scales"][1][~block] == 0).all()
    assert (out["codes"][1].float() == 0).all()
    for n in ("y", "codes", "scales", "rstd"):
        assert torch.equal(out[n][::2].float(), plain[n][::2].float()), n


def test_blocks_below_the_smallest_scale_are_stored_as_zeros():
    d = 256
    x = torch.full((2, d), 1.0, device=DEV)
    gamma = torch.ones(d, device=DEV)
    gamma[:128] = 2.0 ** -118
    gamma[128:] = 2.0 ** -116
    _, out = rms_run(x, None, gamma, F32)
    assert (out["scales"][:, 0] == 0).all() and (out["codes"][:, :128].float() == 0).all()
    assert (out["scales"][:, 1] > 0).all() and (out["codes"][:, 128:].float() == 448).all()


@pytest.mark.parametrize("T,d", [(1, 16), (1, 512), (333, 272), (65, 992), (129, 2064), (700, 4096), (5, 16384), (3, 16400)])
@pytest.mark.parametrize("dy_dtype,h_dtype", [(F32, F32), (BF16, BF16), (F32, BF16)])
def test_rmsnorm_backward(T, d, dy_dtype, h_dtype):
    h, dy, dres = randn((T, d), 7, h_dtype), randn((T, d), 8, dy_dtype), randn((T, d), 9, h_dtype)
    gamma = 1 + randn((d,), 10, scale=0.1)
    plan = binding.moe_plan(T, d, 1, 1, 256)
    rstd = rms_ref(h, None, None, h_dtype)[1].float()
    scratch = binding.backward_scratch(plan)
    for res in (dres, None):
        dx, dgamma = nan((T, d), h_dtype), nan((d,))
        binding.moe_rmsnorm_backward(plan, dy, h, gamma, rstd, res, dx, dgamma, scratch)
        hd, r, v = h.double(), rstd.double()[:, None], dy.double() * gamma.double()
        hh = hd * r
        ref = r * (v - hh * (v * hh).mean(1, keepdim=True))
        mag = r * (v.abs() + hh.abs() * (v * hh).abs().mean(1, keepdim=True))
        if res is not None:
            ref, mag = ref + res.double(), mag + res.double().abs()
        n = d / 64 + 64
        within(dx, ref, n * U * mag + (2.0 ** -8 * ref.abs() + 2.0 ** -133 if h_dtype == BF16 else 2.0 ** -149), "dx")
        within(dgamma, (dy.double() * hh).sum(0), (T / 64 + 64) * U * (dy.double() * hh).abs().sum(0), "dgamma")
    placed = dres.clone()  # dres may be dx, and dgamma may be left out
    dx2 = nan((T, d), h_dtype)
    binding.moe_rmsnorm_backward(plan, dy, h, gamma, rstd, dres, dx2, dgamma, scratch)
    binding.moe_rmsnorm_backward(plan, dy, h, gamma, rstd, placed, placed, None, None)
    assert torch.equal(placed, dx2)


@pytest.mark.parametrize("d", [272, 2064])
def test_rmsnorm_backward_takes_scratch_that_holds_anything(d):
    """Also where the weights' columns end within a CTA of the kernel that joins them (d an odd multiple of 16)."""
    T = 333
    h, dy, rstd = randn((T, d), 7), randn((T, d), 8), 1 + randn((T,), 9, scale=0.1)
    plan = binding.moe_plan(T, d, 1, 1, 256)
    results = []
    for fill in (0, 0xFF):  # zeros, NaN
        dx, dgamma = nan((T, d)), nan((d,))
        binding.moe_rmsnorm_backward(plan, dy, h, None, rstd, None, dx, dgamma, torch.full_like(binding.backward_scratch(plan), fill))
        results.append((dx, dgamma))
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(*results))


def test_rmsnorm_backward_is_the_derivative_of_the_forward_formula():
    T, d = 4, 48
    h, dy, gamma = randn((T, d), 11), randn((T, d), 12), 1 + randn((d,), 13, scale=0.1)
    x = h.double().requires_grad_(True)
    g = gamma.double().requires_grad_(True)
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5) * g
    (y * dy.double()).sum().backward()
    # a difference quotient of the formula agrees with the automatic derivative used below
    step = randn((T, d), 14).double()
    f = lambda a: float(((a / torch.sqrt((a * a).mean(1, keepdim=True) + 1e-5) * gamma.double()) * dy.double()).sum())  # noqa: E731
    slope = (f(h.double() + 1e-6 * step) - f(h.double() - 1e-6 * step)) / 2e-6
    assert abs(slope - float((x.grad * step).sum())) < 1e-6 * float((x.grad * step).abs().sum())
    plan = binding.moe_plan(T, d, 1, 1, 256)
    rstd = rms_ref(h, None, None, F32)[1].float()
    dx, dgamma = nan((T, d)), nan((d,))
    binding.moe_rmsnorm_backward(plan, dy, h, gamma, rstd, None, dx, dgamma, binding.backward_scratch(plan))
    within(dx, x.grad, 128 * U * (x.grad.abs() + 4 * dy.double().abs().mean()), "dx")
    within(dgamma, g.grad, 128 * U * (g.grad.abs() + dy.double().abs().sum(0) * 4), "dgamma")


def test_rmsnorm_of_no_tokens():
    plan = binding.moe_plan(0, 64, 1, 1, 256)
    empty = torch.empty(0, 64, device=DEV)
    binding.moe_rmsnorm(plan, empty, None, None, 1e-5, None, empty.to(BF16))
    dgamma = nan((64,))
    binding.moe_rmsnorm_backward(plan, empty, empty, None, torch.empty(0, device=DEV), None, empty, dgamma,
                                 binding.backward_scratch(plan))
    torch.cuda.synchronize()
    assert (dgamma == 0).all()


# ---------------------------------------------------------------- weights in 8 bits

def quantize(W, halves):
    E, d, N = W.shape
    plan = binding.moe_plan(1, d, E, 1, N)
    codes, scales = nan((E, N, d), E4M3), nan((E, halves * blocks(N // halves), blocks(d)))
    binding.moe_quantize_weights(plan, W, codes, scales, halves)
    return codes, scales


def weight_scale(scales, N, d, halves):
    """Scales of [E][N][d] weights, one a weight."""
    n = N // halves
    row = torch.arange(N, device=DEV)
    row = row // n * blocks(n) + row % n // 128
    return scales.double()[:, row][:, :, torch.arange(d, device=DEV) // 128]


@pytest.mark.parametrize("E,d,N,halves", [(1, 16, 16, 1), (3, 144, 272, 1), (2, 1040, 528, 1), (2, 400, 32, 2), (5, 256, 2816, 2),
                                          (3, 128, 288, 2), (16, 512, 1024, 1)])
def test_quantize_weights(E, d, N, halves):
    W = randn((E, d, N), 20, BF16)
    W[:, : d // 2] *= 8.0
    codes, scales = quantize(W, halves)
    t = W.double().transpose(1, 2)
    n = N // halves
    tiles = torch.nn.functional.pad(t.reshape(E, halves, n, d), (0, blocks(d) * 128 - d, 0, blocks(n) * 128 - n))
    amax = tiles.reshape(E, halves * blocks(n), 128, blocks(d), 128).abs().amax((2, 4))
    within(scales, amax / 448, 2 * U * amax / 448, "scales")
    s = weight_scale(scales, N, d, halves)
    within(codes.double() * s, t, torch.maximum(2.0 ** -4 * t.abs(), 2.0 ** -10 * s) * (1 + 8 * U), "values")


def test_quantize_weights_with_infinities_and_zeros():
    W = randn((2, 256, 256), 21, BF16)
    W[0, 130, 5] = float("inf")
    W[1, 3, 200] = float("nan")
    W[1, 128:, :128] = 0.0
    W[0, :128, 128:] = 2.0 ** -120
    codes, scales = quantize(W, 1)
    torch.cuda.synchronize()
    bad = torch.zeros(2, 2, 2, dtype=torch.bool, device=DEV)
    bad[0, 0, 1] = bad[1, 1, 0] = True
    assert torch.equal(torch.isnan(scales), bad)
    assert scales[1, 0, 1] == 0 and scales[0, 1, 0] == 0
    assert (codes[0, :128, 128:].float() == 0).all() and (codes[1, 128:, :128].float() == 0).all()
    assert (codes[0, 128:, :128].float() == 0).all()


# ---------------------------------------------------------------- per-expert product

def routing(T, E, k, load, seed):
    """Experts of the slots ("even", "skew": most on expert 0 and none on the last half), offsets and perm."""
    logits = torch.randn(T, E, generator=gen(seed), device=DEV)
    if load == "skew":
        logits[:, 0] += 8.0
        logits[:, max(k, E - E // 2):] -= 50.0
    idx = torch.topk(logits, k, 1).indices.reshape(-1)
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(I32)
    return offsets, torch.argsort(idx, stable=True).to(I32)


def codes_of(shape, seed):
    return randn(shape, seed, scale=120.0).clamp(-448, 448).to(E4M3)


def scales_of(shape, seed, typical):
    return torch.exp(randn(shape, seed, scale=0.5)) * typical


def operands(T, d, E, k, N, halves, gather, load, seed=30):
    offsets, perm = routing(T, E, k, load, seed)
    rows = T if gather else T * k
    A, As = codes_of((rows, d), seed + 1), scales_of((rows, blocks(d)), seed + 2, 0.01)
    W, Ws = codes_of((E, N, d), seed + 3), scales_of((E, halves * blocks(N // halves), blocks(d)), seed + 4, 0.01 / d ** 0.5)
    return offsets, perm if gather else None, A, As, W, Ws


def product(ops, k, halves):
    """(result, sum of the magnitudes) in 64 bits."""
    offsets, perm, A, As, W, Ws = ops
    E, N, d = W.shape
    a = A.double() * spread(As, d)
    if perm is not None:
        a = a[(perm // k).long()]
    w = W.double() * weight_scale(Ws, N, d, halves)
    off = offsets.tolist()
    Y = torch.cat([a[off[e]:off[e + 1]] @ w[e].T for e in range(E)])
    mag = torch.cat([a[off[e]:off[e + 1]].abs() @ w[e].abs().T for e in range(E)])
    return Y, mag


def product_rounds(d):
    return 8 + blocks(d) + 4


def buffers(plan):
    return torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV), torch.zeros(4, dtype=I32, device=DEV)


def fp8_run(T, d, E, k, N, ops, dtype):
    plan = binding.moe_plan(T, d, E, k, N, out_dtype=binding.MOE_OUT_BF16 if dtype == BF16 else binding.MOE_OUT_F32)
    offsets, perm, A, As, W, Ws = ops
    Y = torch.full((T * k + 3, N), 7.0, dtype=dtype, device=DEV)  # rows behind the last are left as they were
    Y[:T * k] = float("nan")
    ws, st = buffers(plan)
    binding.moe_grouped_gemm_fp8(plan, A, As, perm, offsets, W, Ws, Y[:T * k], ws, st)
    rc, status = binding.moe_read_status(st)
    assert rc == 0, status
    assert (Y[T * k:] == 7.0).all()
    return Y[:T * k]


FP8_SHAPES = [(1, 16, 1, 1, 16, "even"), (1, 64, 4, 2, 48, "even"), (5, 128, 3, 1, 272, "even"), (37, 144, 8, 2, 528, "skew"),
              (64, 1040, 16, 8, 512, "even"), (200, 1040, 5, 3, 1296, "skew"), (600, 2064, 2, 2, 784, "even"),
              (129, 4096, 1, 1, 256, "even"), (3000, 512, 8, 2, 1024, "skew"), (4096, 256, 64, 2, 1408, "even"),
              (500, 384, 256, 2, 512, "even"), (20, 14336, 8, 2, 272, "even"), (3300, 400, 2, 1, 784, "even"),
              (5000, 1040, 2, 2, 288, "skew")]


@pytest.mark.parametrize("T,d,E,k,N,load", FP8_SHAPES)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_gemm_fp8(T, d, E, k, N, load, gather, dtype):
    ops = operands(T, d, E, k, N, 1, gather, load)
    Y = fp8_run(T, d, E, k, N, ops, dtype)
    ref, mag = product(ops, k, 1)
    within(Y, ref, product_rounds(d) * U * mag + (2.0 ** -8 * ref.abs() if dtype == BF16 else 0.0) + 2.0 ** -126, "Y")


@pytest.mark.parametrize("T,d,E,k,F,load", [(1, 16, 1, 1, 16, "even"), (5, 128, 3, 1, 144, "even"), (37, 144, 8, 2, 272, "skew"),
                                            (64, 1040, 16, 8, 256, "even"), (600, 2064, 2, 2, 400, "even"),
                                            (4096, 256, 64, 2, 704, "skew"), (500, 384, 256, 2, 128, "even"),
                                            (3300, 400, 2, 1, 272, "even"), (5000, 1040, 2, 2, 144, "skew")])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_gemm_fp8_swiglu(T, d, E, k, F, load, gather):
    ops = operands(T, d, E, k, 2 * F, 2, gather, load)
    offsets, perm, A, As, W, Ws = ops
    plan = binding.moe_plan(T, d, E, k, 2 * F)
    S = T * k
    H, Hs = torch.full((S + 3, F), 7.0, device=DEV).to(E4M3), torch.full((S + 3, blocks(F)), 7.0, device=DEV)
    Hs[:S] = float("nan")
    ws, st = buffers(plan)
    binding.moe_grouped_gemm_fp8_swiglu(plan, A, As, perm, offsets, W, Ws, H[:S], Hs[:S], ws, st)
    rc, status = binding.moe_read_status(st)
    assert rc == 0, status
    assert (H[S:].float() == 7.0).all() and (Hs[S:] == 7.0).all()
    gu, mag = product(ops, k, 2)
    g, u = gu[:, :F], gu[:, F:]
    e = product_rounds(d) * U * mag
    s = torch.sigmoid(g)
    ref = g * s * u
    # silu's slope is at most 1.1; its own roundings are 8 + 1.2 |g| units
    err = 1.1 * u.abs() * e[:, :F] + (g * s).abs() * e[:, F:] + e[:, :F] * e[:, F:] + (8 + 1.2 * g.abs()) * 2 * U * ref.abs()
    check_8bit(H[:S], Hs[:S], ref, err, "H")


@pytest.mark.parametrize("T,E", [(40, 4), (1200, 4), (3300, 4)])
@pytest.mark.parametrize("gather", [False, True])
def test_fp8_rows_and_columns_that_are_not_numbers_stay_alone(T, E, gather):
    """A NaN code or scale of a row of A is that row's alone, one of W's rows its expert's column's."""
    d, k, N = 400, 2, 528
    offsets, perm, A, As, W, Ws = operands(T, d, E, k, N, 1, gather, "even", seed=40)
    A.view(torch.uint8)[3, 17] = 0x7F
    As[5, 2] = float("nan")
    As[7, 0] = float("inf")
    W.view(torch.uint8)[1, 300, 9] = 0xFF
    Ws[2, 4, 3] = float("nan")   # columns 512 .. 527 of expert 2
    Y = fp8_run(T, d, E, k, N, (offsets, perm, A, As, W, Ws), F32)
    off = offsets.tolist()
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), torch.tensor([off[e + 1] - off[e] for e in range(E)], device=DEV))
    src = (perm // k).long() if gather else torch.arange(T * k, device=DEV)
    bad = torch.zeros(T * k, N, dtype=torch.bool, device=DEV)
    bad |= ((src == 3) | (src == 5))[:, None]
    bad[expert == 1, 300] = True
    bad[expert == 2, 512:] = True
    loose = src == 7  # infinite (or NaN, where a block's sum is 0)
    assert torch.equal(torch.isnan(Y)[~loose], bad[~loose])
    assert not torch.isfinite(Y[loose]).any()
    ok = (offsets, perm, torch.where(torch.isnan(A.float()), 0.0, A.float()).to(E4M3), torch.nan_to_num(As, 0.01, 0.01),
          torch.where(torch.isnan(W.float()), 0.0, W.float()).to(E4M3), torch.nan_to_num(Ws, 0.01))
    ref, mag = product(ok, k, 1)
    good = ~bad & ~loose[:, None]
    assert ((Y.double() - ref).abs()[good] <= (product_rounds(d) * U * mag + 2.0 ** -126)[good]).all()


def test_fp8_offsets_that_do_not_ascend_are_reported_and_write_nothing():
    T, d, E, k, N = 40, 128, 4, 2, 256
    offsets, perm, A, As, W, Ws = operands(T, d, E, k, N, 1, False, "even")
    plan = binding.moe_plan(T, d, E, k, N)
    for bad in ([0, 30, 20, 60, 80], [0, 20, 40, 60, 81], [1, 20, 40, 60, 80], [0, 20, 40, 60, 79], [0, -5, 40, 60, 80]):
        ws, st = buffers(plan)
        Y = torch.full((T * k, N), 7.0, device=DEV)
        binding.moe_grouped_gemm_fp8(plan, A, As, perm, torch.tensor(bad, dtype=I32, device=DEV), W, Ws, Y, ws, st)
        rc, _ = binding.moe_read_status(st)
        assert rc == binding.MOE_ERR_DEVICE and (Y == 7.0).all()


def test_fp8_perm_outside_the_slots_reads_no_other_memory():
    T, d, E, k, N = 40, 128, 4, 2, 256
    offsets, perm, A, As, W, Ws = operands(T, d, E, k, N, 1, True, "even")
    broken = perm.clone()
    broken[3], broken[11] = -1, 2 ** 31 - 1
    zero = perm.clone()
    zero[3], zero[11] = 0, 0  # such a row is row 0
    assert torch.equal(fp8_run(T, d, E, k, N, (offsets, broken, A, As, W, Ws), F32),
                       fp8_run(T, d, E, k, N, (offsets, zero, A, As, W, Ws), F32))


def test_fp8_of_no_tokens():
    plan = binding.moe_plan(0, 128, 4, 2, 256)
    ws, st = buffers(plan)
    e8, f = torch.empty(0, 128, device=DEV).to(E4M3), torch.empty(0, 1, device=DEV)
    W, Ws = codes_of((4, 256, 128), 1), scales_of((4, 2, 1), 2, 1.0)
    binding.moe_grouped_gemm_fp8(plan, e8, f, None, torch.zeros(5, dtype=I32, device=DEV), W, Ws, torch.empty(0, 256, device=DEV), ws, st)
    assert binding.moe_read_status(st)[0] == 0


def test_fp8_is_the_same_in_a_graph_and_on_another_stream():
    T, d, E, k, N = 300, 512, 8, 2, 1024
    offsets, perm, A, As, W, Ws = operands(T, d, E, k, N, 1, True, "even")
    plan = binding.moe_plan(T, d, E, k, N)
    ws, st = buffers(plan)
    Y = torch.empty(T * k, N, device=DEV)
    binding.moe_grouped_gemm_fp8(plan, A, As, perm, offsets, W, Ws, Y, ws, st)
    first = Y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    binding.moe_grouped_gemm_fp8(plan, A, As, perm, offsets, W, Ws, Y, ws, st, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_grouped_gemm_fp8(plan, A, As, perm, offsets, W, Ws, Y, ws, st)
    for _ in range(2):
        Y.fill_(0)
        graph.replay()
        assert torch.equal(Y, first)
    A.copy_(codes_of(A.shape, 77))  # new inputs in the captured buffers
    graph.replay()
    ref, mag = product((offsets, perm, A, As, W, Ws), k, 1)
    within(Y, ref, product_rounds(d) * U * mag + 2.0 ** -126)


def test_operators_beyond_two_to_the_31_elements():
    """Offsets of rows and results that pass 32 bits: the last rows are right."""
    T, d, N = 1 << 20, 16, 2064
    ops = operands(T, d, 1, 1, N, 1, False, "even", seed=100)
    plan = binding.moe_plan(T, d, 1, 1, N, out_dtype=binding.MOE_OUT_BF16)
    Y = torch.empty(T, N, dtype=BF16, device=DEV)
    ws, st = buffers(plan)
    binding.moe_grouped_gemm_fp8(plan, *ops[2:4], None, ops[0], *ops[4:], Y, ws, st)
    assert binding.moe_read_status(st)[0] == 0
    last = (torch.tensor([0, 300], dtype=I32, device=DEV), None, ops[2][-300:], ops[3][-300:], ops[4], ops[5])
    ref, mag = product(last, 1, 1)
    within(Y[-300:], ref, product_rounds(d) * U * mag + 2.0 ** -8 * ref.abs() + 2.0 ** -126)
    del Y
    T, d = (1 << 17) + 5, 16400
    x = randn((T, d), 101, BF16)
    plan = binding.moe_plan(T, d, 1, 1, 256)
    y, codes, scales = torch.empty_like(x), torch.empty(T, d, dtype=E4M3, device=DEV), torch.empty(T, blocks(d), device=DEV)
    binding.moe_rmsnorm(plan, x, None, None, 1e-5, None, y, codes, scales)
    _, _, ref = rms_ref(x[-3:], None, None, BF16)
    err = ((d / 64 + 64) / 2 + 8) * U * ref.abs()
    within(y[-3:], ref, err + 2.0 ** -8 * ref.abs())
    check_8bit(codes[-3:], scales[-3:], ref, err)


@pytest.mark.parametrize("N,dtype", [((1 << 29) + 272, F32), ((1 << 30) + 272, BF16)])
def test_rows_of_two_to_the_31_bytes_and_more(N, dtype):
    """The bytes that are left of a row, from a tile's first column on, pass 32 bits."""
    plan = binding.moe_plan(1, 16, 1, 1, N, out_dtype=binding.MOE_OUT_F32 if dtype == F32 else binding.MOE_OUT_BF16)
    one = torch.full((1, 16), 0x38, dtype=torch.uint8, device=DEV)  # 1.0
    W = torch.full((1, N, 16), 0x38, dtype=torch.uint8, device=DEV)
    Ws = (1 + torch.arange(blocks(N), device=DEV) % 7).float().reshape(1, -1, 1)
    Y = nan((1, N), dtype)
    ws, st = buffers(plan)
    offsets = torch.tensor([0, 1], dtype=I32, device=DEV)
    binding.moe_grouped_gemm_fp8(plan, one, torch.ones(1, 1, device=DEV), None, offsets, W, Ws, Y, ws, st)
    assert binding.moe_read_status(st)[0] == 0
    del W
    want = (16 * Ws.reshape(-1)).to(dtype).repeat_interleave(128)[:N]
    assert torch.equal(Y[0], want)


def test_calls_on_two_streams_at_once():
    """The products keep nothing in the workspace or between calls: two at a time on one plan give what each gives alone."""
    T, d, E, k, N = 2000, 1024, 4, 2, 1024
    a, c = operands(T, d, E, k, N, 1, True, "even", seed=110), operands(T, d, E, k, N, 1, True, "skew", seed=120)
    plan = binding.moe_plan(T, d, E, k, N)
    ws, st = buffers(plan)
    alone, both = [], [torch.zeros(T * k, N, device=DEV) for _ in range(2)]
    for o in (a, c):
        Y = torch.zeros(T * k, N, device=DEV)
        binding.moe_grouped_gemm_fp8(plan, o[2], o[3], o[1], o[0], o[4], o[5], Y, ws, st)
        alone.append(Y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o, Y, s in zip((a, c), both, streams):
            binding.moe_grouped_gemm_fp8(plan, o[2], o[3], o[1], o[0], o[4], o[5], Y, ws, st, stream=s)
    torch.cuda.synchronize()
    assert binding.moe_read_status(st)[0] == 0
    for x, y in zip(alone, both):
        assert torch.equal(x, y)


def test_unaligned_scales_and_views():
    """Scales that start at any 4 bytes, and results that are views of larger buffers."""
    T, d, E, k, N = 300, 512, 4, 2, 256   # four k-blocks: the aligned form copies 16 bytes of scales at a time
    offsets, perm, A, As, W, Ws = operands(T, d, E, k, N, 1, True, "even", seed=130)
    want = fp8_run(T, d, E, k, N, (offsets, perm, A, As, W, Ws), F32)
    room = torch.empty(As.numel() + 1, device=DEV)
    room[1:] = As.reshape(-1)
    assert torch.equal(fp8_run(T, d, E, k, N, (offsets, perm, A, room[1:].reshape(As.shape), W, Ws), F32), want)
    wide = torch.empty(Ws.numel() + 3, device=DEV)
    wide[3:] = Ws.reshape(-1)
    assert torch.equal(fp8_run(T, d, E, k, N, (offsets, perm, A, As, W, wide[3:].reshape(Ws.shape)), F32), want)


def test_misaligned_operands_are_refused():
    T, d, E, k, N = 8, 128, 2, 1, 256
    offsets, perm, A, As, W, Ws = operands(T, d, E, k, N, 1, False, "even")
    plan = binding.moe_plan(T, d, E, k, N)
    ws, st = buffers(plan)
    room = torch.empty(A.numel() + 8, dtype=torch.uint8, device=DEV)[8:].view(E4M3).reshape(A.shape)
    Y = torch.full((T, N), 7.0, device=DEV)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):
        binding.moe_grouped_gemm_fp8(plan, room, As, perm, offsets, W, Ws, Y, ws, st)
    odd = binding.moe_plan(T, d, E, k, 272)
    H, Hs = torch.empty(T, 136, device=DEV).to(E4M3), torch.empty(T, 2, device=DEV)
    W, Ws = codes_of((E, 272, d), 1), scales_of((E, 4, 1), 2, 1.0)
    ws, st = buffers(odd)
    with pytest.raises(binding.MoeError, match="UNSUPPORTED"):
        binding.moe_grouped_gemm_fp8_swiglu(odd, A, As, perm, offsets, W, Ws, H, Hs, ws, st)
    with pytest.raises(binding.MoeError, match="UNSUPPORTED"):
        binding.moe_quantize_weights(odd, randn((E, d, 272), 1, BF16), W, Ws, halves=2)
    x = randn((T, d), 5)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):  # neither output
        binding.moe_rmsnorm(plan, x, None, None, 1e-5, None, None)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):  # codes without scales
        binding.moe_rmsnorm(plan, x, None, None, 1e-5, None, None, A)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):
        binding.moe_rmsnorm(plan, x, None, None, 0.0, None, x.to(BF16))
    torch.cuda.synchronize()
    assert (Y == 7.0).all()
