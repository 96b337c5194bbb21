"""The training operators' loops: every kernel with more work than its grid takes in two passes, with odd remainders, so
that strides, prefetched units and the shared arrays that rows take in turn are behind checked results; and tensors of
more than 2^31 elements.

Tolerances as in test_train_gpu.py, with the orders of summation that these sizes take.  A sum over the rows (dgamma,
dbeta) is at most T/8 terms in sequence (a warp of the widest rows' kernel takes every eighth row; the others less) and
64 joins of threads, row groups and CTAs.  The sigmoid's exponential is off by 2 + 1.173 |g| units, hence the magnitudes
with 1 + |g|.
"""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding
from tests.test_train_gpu import (BF16, DEV, F32, cb_ref, cb_run, check, ckpt_ref, ckpt_run, dgrad_ref, grad_setup,
                                  ln_back_ref, ln_back_run, ln_ref, ln_run, mma_rounds, nan, randn, restored, rounds,
                                  swiglu_back_ref, wgrad_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# (d, rows that the grid takes in a pass, for each SM): 8 to 256 threads a row, two rows at a time, 2048 threads an
# SM; one row at a time above 8192 columns; one row a CTA, one CTA an SM above 32768
@pytest.mark.parametrize("d,pass_rows", [(48, 512), (272, 256), (528, 128), (1040, 64), (4096, 32), (8192, 16), (12304, 4),
                                         (20496, 2), (32784, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layernorm_passes(sms, d, pass_rows, dtype):
    T = 2 * sms * pass_rows + 37
    x = (randn((T, d), 1) * 3 + randn((T, 1), 2)).to(dtype)
    gamma, beta = 1 + randn((d,), 3, scale=0.1), randn((d,), 4, scale=0.1)
    _, y, mean, rstd = ln_run(x, gamma, beta)
    for r in range(0, T, 20000):  # in parts, for the 64-bit copies' memory
        p = slice(r, r + 20000)
        ry, rmean, rrstd = ln_ref(x[p], gamma, beta, 1e-5)
        xa = x[p].double().abs().mean(1)
        check(mean[p], rmean[:, 0], xa, rounds(d), "mean")
        check(rstd[p], rrstd[:, 0], rrstd[:, 0] * (1 + xa * rrstd[:, 0]), rounds(d), "rstd")
        mag = (x[p].double().abs() + xa[:, None]) * rrstd * (1 + xa[:, None] * rrstd) * gamma.abs().double() + beta.abs().double()
        check(y[p], ry, mag, rounds(d), "y")


# 8 to 128 threads a row and 1024 an SM; a row a CTA of 256 to 1024; one CTA an SM above 8192
@pytest.mark.parametrize("d,pass_rows", [(64, 128), (128, 64), (256, 32), (272, 16), (1024, 8), (1040, 4), (2064, 2), (7168, 1),
                                         (12304, 1), (16400, 1)])
@pytest.mark.parametrize("x_dtype,dy_dtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
def test_layernorm_backward_passes(sms, d, pass_rows, x_dtype, dy_dtype):
    T = 2 * sms * pass_rows + 37
    x = (randn((T, d), 11) + randn((T, 1), 12)).to(x_dtype)
    dy, dres = randn((T, d), 13, dy_dtype), randn((T, d), 14, x_dtype)
    gamma = 1 + randn((d,), 15, scale=0.1)
    _, _, mean, rstd, dx, dg, db = ln_back_run(dy, x, gamma, dres)
    rdx, mdx, rdg, mdg, rdb, mdb = ln_back_ref(dy, x, gamma, mean, rstd, dres)
    check(dx, rdx, mdx, rounds(d), "dx")
    check(dg, rdg, mdg, T / 8 + 64, "dgamma")
    check(db, rdb, mdb, T / 8 + 64, "dbeta")


def test_layernorm_backward_of_many_wide_rows():
    T, d = 3001, 16400
    x, dy = randn((T, d), 21, BF16), randn((T, d), 22)
    _, _, mean, rstd, dx, dg, db = ln_back_run(dy, x, None, None)
    rdx, mdx, rdg, mdg, rdb, mdb = ln_back_ref(dy, x, None, mean, rstd, None)
    check(dx, rdx, mdx, rounds(d), "dx")
    check(dg, rdg, mdg, T / 8 + 64, "dgamma")
    check(db, rdb, mdb, T / 8 + 64, "dbeta")


# grids of 3 or 4 CTAs an SM, of 16 blocks (forward) or 256 units of 8 columns (backward)
@pytest.mark.parametrize("S,F", [(3001, 1408), (20011, 136), (320003, 8), (45, 65544)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu_checkpoint_passes(sms, S, F, dtype):
    assert S * binding.checkpoint_blocks(F) > 2 * sms * 4 * 16 and S * (F // 8) > 2 * sms * 4 * 256
    GU = randn((S, 2 * F), 40)
    GU[:, :: 7] *= 5
    GU = GU.to(dtype)
    plan, H, codes, scales = ckpt_run(GU)
    rc, rs = ckpt_ref(GU)
    assert torch.equal(codes.cpu(), rc) and torch.equal(scales.cpu(), rs)
    g, u = GU[:, :F].double(), GU[:, F:].double()
    want = g * torch.sigmoid(g) * u
    check(H, want, want.abs() * (1 + g.abs()), 16, "H")
    dH = randn((S, F), 44, dtype)
    H2, dGU = nan((S, F), BF16), nan((S, 2 * F), BF16)
    binding.moe_swiglu_checkpoint_backward(plan, dH, codes, scales, H2, dGU)
    g, u = restored(codes, scales)
    rd, rh = swiglu_back_ref(g, u, dH)
    s, d64 = torch.sigmoid(g), dH.double().abs()
    mag = torch.cat([d64 * u.abs() * s * (1 + g.abs()) ** 2, d64 * (g * s).abs() * (1 + g.abs())], 1)
    check(dGU, rd, mag, 32, "dGU")
    check(H2, rh, rh.abs() * (1 + g.abs()), 16, "H again")


# 32 CTAs an SM: of a token (rows of 2048 columns and more), or of eight, a warp each
@pytest.mark.parametrize("T,k,N", [(10007, 2, 2064), (10009, 12, 2064), (80009, 3, 64), (80021, 9, 32), (78001, 1, 1040)])
@pytest.mark.parametrize("y_dtype,dout_dtype", [(F32, BF16), (BF16, F32)])
def test_combine_backward_passes(sms, T, k, N, y_dtype, dout_dtype):
    assert T > 2 * 32 * sms * (1 if N >= 2048 else 8)
    dout, Y, w, dest, dY, dw = cb_run(T, k, N, y_dtype, dout_dtype)
    rY, rw, mw = cb_ref(dout, Y, w, dest)
    check(dY, rY, rY.abs(), 2, "dY")
    check(dw, rw, mw, rounds(N), "dw")


# ---------------------------------------------------------------- more than 2^31 elements

def base_rows(d, seed, dtype, n=997):
    return randn((n, d), seed, dtype)


def repeated(base, T):
    """[T][d]: row t is base row t mod n."""
    n = base.shape[0]
    return base.repeat(-(-T // n), 1)[:T]


def test_layernorm_beyond_2_31_elements():
    d, n = 4112, 997
    T = (1 << 31) // d + 2 * n
    base, dbase = base_rows(d, 1, BF16), base_rows(d, 2, BF16)
    x, dy = repeated(base, T), repeated(dbase, T)
    _, y, mean, rstd = ln_run(x, None, None)
    first = y[:n].clone()
    assert torch.equal(y[:n], ln_run(base, None, None)[1])
    for r in range(0, T, n):  # rows repeat, so results do, bit for bit
        assert torch.equal(y[r:r + n], first[:min(n, T - r)]), r
    plan = binding.moe_plan(T, d, 1, 1, 256)
    dg, db = nan((d,)), nan((d,))
    dx = y  # written over
    binding.moe_layernorm_backward(plan, dy, x, None, mean, rstd, None, dx, dg, db, binding.backward_scratch(plan))
    rdx, mdx, _, _, _, _ = ln_back_ref(dbase, base, None, mean[:n], rstd[:n], None)
    check(dx[:n], rdx, mdx, rounds(d), "dx")
    first = dx[:n].clone()
    for r in range(0, T, n):
        assert torch.equal(dx[r:r + n], first[:min(n, T - r)]), r
    times = torch.bincount(torch.arange(T, device=DEV) % n, minlength=n).double()[:, None]
    xh = (base.double() - mean[:n, None].double()) * rstd[:n, None].double()
    d64 = dbase.double()
    big = (base.double().abs() + mean[:n, None].double().abs()) * rstd[:n, None].double() + xh.abs()
    check(dg, (times * d64 * xh).sum(0), (times * d64.abs() * big).sum(0), T / 8 + 64, "dgamma")
    check(db, (times * d64).sum(0), (times * d64.abs()).sum(0), T / 8 + 64, "dbeta")


def test_swiglu_checkpoint_beyond_2_31_elements():
    F, n = 4104, 997
    S = (1 << 31) // (2 * F) + 2 * n
    base, hbase = base_rows(2 * F, 3, BF16), base_rows(F, 4, BF16)
    want = ckpt_run(base)
    want_h, want_d = nan((n, F), BF16), nan((n, 2 * F), BF16)
    binding.moe_swiglu_checkpoint_backward(want[0], hbase, want[2], want[3], want_h, want_d)
    plan, H, codes, scales = ckpt_run(repeated(base, S))
    H2, dGU = nan((S, F), BF16), nan((S, 2 * F), BF16)
    binding.moe_swiglu_checkpoint_backward(plan, repeated(hbase, S), codes, scales, H2, dGU)
    for got, ref in ((H, want[1]), (codes, want[2]), (scales, want[3]), (H2, want_h), (dGU, want_d)):
        for r in range(0, S, n):
            assert torch.equal(got[r:r + n], ref[:min(n, S - r)]), r


def test_combine_backward_beyond_2_31_elements():
    k, N = 8, 4112
    T = (1 << 31) // (k * N) + 501
    S = T * k
    plan = binding.moe_plan(T, 256, 8, k, N, out_dtype=binding.MOE_OUT_BF16)
    dout, Y, w = randn((T, N), 5), randn((S, N), 6, BF16), torch.softmax(randn((T, k), 7), 1)
    dest = torch.randperm(S, generator=torch.Generator(device=DEV).manual_seed(8), device=DEV).to(torch.int32)
    dY, dw = nan((S, N), BF16), nan((T, k))
    binding.moe_combine_backward(plan, dout, Y, w, dest, dY, dw)
    for t0 in list(range(0, T, T // 7)) + [T - 300]:
        t = slice(t0, min(T, t0 + 300))
        rows = dest.reshape(T, k)[t].long()
        terms = Y[rows].double() * dout[t].double()[:, None]
        check(dw[t], terms.sum(-1), terms.abs().sum(-1), rounds(N), "dw")
        want = w[t].double()[:, :, None] * dout[t].double()[:, None]
        check(dY[rows.reshape(-1)], want.reshape(-1, N), want.reshape(-1, N).abs(), 2, "dY")
    assert not torch.isnan(dY).any()


def test_grouped_gradients_beyond_2_31_elements_of_the_weights():
    d, N = 4112, 8208
    E = (1 << 31) // (d * N) + 3
    counts = [2] * (E - 1) + [131]
    plan, ws, st, off, A, dY, W = grad_setup(counts, d, N)
    dA = nan((sum(counts), d))
    binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
    dW = nan((E, d, N))
    binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
    assert binding.moe_read_status(st)[0] == 0
    for e in (0, E - 4, E - 2, E - 1):
        a = 2 * e
        b = a + counts[e]
        ref, mag = dgrad_ref([b - a], dY[a:b], W[e:e + 1])
        check(dA[a:b], ref, mag, mma_rounds(N), "dA")
        ref, mag = wgrad_ref([b - a], A[a:b], dY[a:b])
        check(dW[e:e + 1], ref, mag, mma_rounds(b - a), "dW")
    assert not torch.isnan(dW).any()


@pytest.mark.parametrize("d,N", [(16, 2064), (2064, 16)])
def test_grouped_gradients_beyond_2_31_elements_of_the_rows(d, N):
    S = (1 << 31) // 2064 + 4001
    counts = [S // 3, 0, S // 3 + 7, S - 2 * (S // 3) - 7]
    plan, ws, st, off, A, dY, W = grad_setup(counts, d, N)
    dA, dW = nan((S, d), BF16), nan((4, d, N))
    binding.moe_grouped_gemm_dgrad(plan, dY, off, W, dA, ws, st)
    binding.moe_grouped_gemm_wgrad(plan, A, dY, off, dW, ws, st)
    assert binding.moe_read_status(st)[0] == 0
    for e, a in ((0, 0), (0, counts[0] - 500), (2, counts[0]), (3, S - 500)):
        ref, mag = dgrad_ref([500], dY[a:a + 500], W[e:e + 1])
        check(dA[a:a + 500], ref, mag, mma_rounds(N), "dA")
    assert not torch.isnan(dA).any()
    a = S - counts[3]
    for r in range(3):  # the reference of the last expert in parts, for the 64-bit copies' memory
        part = slice(a + counts[3] * r // 3, a + counts[3] * (r + 1) // 3)
        one = wgrad_ref([part.stop - part.start], A[part], dY[part])
        ref, mag = one if r == 0 else (ref + one[0], mag + one[1])
    check(dW[3:], ref, mag, mma_rounds(counts[3]), "dW")


@pytest.mark.parametrize("d,ctas", [(16, 1), (512, 2), (1040, 4), (8192, 1), (16384, 1)])
def test_scratch_of_as_many_rows_as_a_plan_takes(sms, d, ctas):
    """Partial sums of the CTAs that are resident, however many rows there are."""
    for T in (1 << 20, (1 << 31) - 1):
        assert binding.moe_plan(T, d, 1, 1, 256).scratch_bytes == sms * ctas * 2 * d * 4
