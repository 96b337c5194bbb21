// The per-expert product in 8-bit floating point with a scale for each block of 128:
//   Y[i][n] = sum_b As[i][b] Ws[e(i)][n / 128][b] (sum over columns j of block b of A[i][j] W[e(i)][n][j])
// e4m3 codes; the tensor cores sum a block's products in fp32 (tcgen05 kind::f8f6f4, K = 32 a step), and the
// blocks' sums, times the product of their two scales, are added in fp32 registers.  Rows are in place (destination
// order) or gathered from the token rows by perm.  With SwiGLU, N = 2F and the result is
// H = silu(gate) up, stored as e4m3 codes with a scale for each row's 128 columns.
//
// A tile is 256 rows (a pair of CTAs, tcgen05 cta_group::2, 128 rows each) or 128 rows (one CTA) by 256 columns: two
// blocks of 128 rows of W, neighbours in N, or with SwiGLU a gate block and its up block.  A k-block is 128
// columns, one scale: 128 bytes of a row, one swizzle row.  Its products go to one of two TMEM accumulators of 256
// columns, and eight epilogue warps read it (lane = row, so a thread has one scale of A and one of each block
// of W) and add it to their 128 sums while the other accumulator is being filled.  That costs 512 bytes a cycle of TMEM
// reads and 128 multiply-adds a cycle: half of the time the tensor cores take for the block.
//
// Roles of a CTA (384 threads): warp 0 loads (one thread, or with gathered rows all lanes, four rows each),
// warp 1 issues the MMAs (the leader's), warps 4-11 are the epilogue, each with one TMEM lane quarter and half of
// the columns of both blocks.  Tile i of the list is the CTA's (or pair's) i mod grid: all tiles cost the same.
#include <algorithm>
#include <atomic>

#include "bounded_wait.cuh"
#include "moe_internal.cuh"
#include "serve.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kFp8Threads = 384;
constexpr int kBlk = kScaleBlock;           // columns of a k-block
constexpr int kOpBytes = 128 * kBlk;        // 16 KB: 128 rows of an operand
constexpr int kEpiFirst = 4, kEpiWarps = 8;
constexpr int kBand = 8;                    // row tiles per schedule band
constexpr int kFp8K = 32;                   // products of an MMA step
constexpr int kMaxStages = 6;
constexpr int kStageOut = 2048;             // a warp's 32 rows of 64 bytes on their way out

template <bool PAIR>
struct Cfg {
    static constexpr int kRowTile = PAIR ? 256 : 128;
    static constexpr int kStages = PAIR ? 6 : 4;
    static constexpr int kWBytes = PAIR ? kOpBytes : 2 * kOpBytes;  // this CTA's share of the 256 rows of W
    static constexpr int kStageBytes = kOpBytes + kWBytes;
};

struct Fp8Ctl {
    uint64_t full[kMaxStages];  // leader: the stage's loads of both CTAs
    uint64_t empty[kMaxStages];
    uint64_t tfull[2];
    uint64_t tempty[2];         // leader
    uint64_t mma_done;
    uint64_t amax_there;        // all epilogue warps have written a tile's amax
    uint32_t tmem_base;
    int abort;
    float amax[2][2][128];      // by tile parity and half of the columns: a row's largest magnitude
};

struct Fp8Params {
    CUtensorMap a_map;    // rows in place: boxes of 128 rows; gathered: of one row
    CUtensorMap a_part;   // rows in place: boxes of 32 rows
    CUtensorMap w_map;
    GroupedFp8Args a;
    int c_tiles, nkb;
    int w_blocks;         // scale blocks of an expert's rows of W
};

__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void umma_fp8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// TMA loads whose completion is signalled on an mbarrier of this CTA, or (PAIR) of either CTA of the pair
template <bool PAIR>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int row) {
    if (PAIR) tma_load_2d_pair(dst, map, bar, x, row);
    else tma_load_2d(dst, map, bar, x, row);
}
// four rows by index
template <bool PAIR>
__device__ __forceinline__ void gather_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, const int (&r)[4]) {
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void load_weights(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int row, int half,
                                             int e) {
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x),
            "r"(row), "r"(half), "r"(e)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x),
            "r"(row), "r"(half), "r"(e)
            : "memory");
}

// (a, b) += v * (s, s)
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n}\n" : "+l"(acc) : "r"(lo), "r"(hi), "l"(s));
}
__device__ __forceinline__ float2 unpack(uint64_t v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

struct Fp8Tile {
    int e, c, r;      // expert, column tile, row tile
    int seg0, rows;   // expert's first row; the tile's valid rows
};

// rows of CTA `rank` of the pair
__device__ __forceinline__ int cta_rows(const Fp8Tile& t, int rank) { return max(0, min(128, t.rows - 128 * rank)); }

template <bool PAIR>
__device__ __forceinline__ Fp8Tile tile_at(const Fp8Params& p, const int* off, const int* base, int i) {
    Fp8Tile t;
    const int u = i / p.c_tiles;
    int lo = 0, hi = p.a.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= u) lo = mid;
        else hi = mid;
    }
    t.e = lo;
    const int local = i - base[lo] * p.c_tiles, rt = base[lo + 1] - base[lo];
    // bands of kBand row tiles, all column tiles of a band together: each operand is read from DRAM about once
    const int band = local / (kBand * p.c_tiles);
    const int nr = min(kBand, rt - band * kBand);
    const int j = local - band * kBand * p.c_tiles;
    t.c = j / nr;
    t.r = band * kBand + j % nr;
    t.seg0 = off[lo];
    t.rows = min(Cfg<PAIR>::kRowTile, off[lo + 1] - off[lo] - Cfg<PAIR>::kRowTile * t.r);
    return t;
}

// A row of A that stands for destination row g (any row where perm is not one of the plan's)
__device__ __forceinline__ int source_row(const Fp8Params& p, int g) {
    if (!p.a.perm) return g;
    const unsigned s = (unsigned)__ldg(p.a.perm + g);
    return s < (unsigned)p.a.S ? (int)(s / (unsigned)p.a.k) : 0;
}

// Bytes of the k-block's rows of A that a CTA with `rows` valid ones loads: boxes of 32 rows, or four rows a gather.
__device__ __forceinline__ uint32_t a_bytes(const Fp8Params& p, int rows) {
    return p.a.perm ? (uint32_t)((rows + 3) & ~3) * kBlk : (uint32_t)((rows + 31) & ~31) * kBlk;
}

// Warp 0, all lanes.
template <bool PAIR>
__device__ void producer(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* stages, const int* off, const int* base, int total, int first,
                         int step, const Wait& w, bool leader, uint32_t lead, int rank) {
    using C = Cfg<PAIR>;
    const int lane = threadIdx.x & 31;
    const uint32_t full0 = smem_addr(&ctl->full[0]), empty0 = smem_addr(&ctl->empty[0]);
    const uint32_t full_lead = PAIR ? mapa_shared(full0, lead) : full0;
    int s = 0;
    uint32_t phase = 0, uses = 0;
    bool ok = true;
    for (int i = first; ok && i < total; i += step) {
        const Fp8Tile t = tile_at<PAIR>(p, off, base, i);
        const int mine = cta_rows(t, rank), row0 = t.seg0 + C::kRowTile * t.r + 128 * rank;
        const uint32_t bytes = PAIR ? a_bytes(p, cta_rows(t, 0)) + a_bytes(p, cta_rows(t, 1)) + 2u * C::kWBytes
                                    : a_bytes(p, mine) + (uint32_t)C::kWBytes;
        int src[4];
        if (p.a.perm) {
#pragma unroll
            for (int j = 0; j < 4; ++j) src[j] = 4 * lane < mine ? source_row(p, row0 + min(4 * lane + j, mine - 1)) : 0;
        }
        for (int kb = 0; kb < p.nkb; ++kb) {
            ok = bar_wait(empty0 + 8 * s, phase ^ 1u, w, 70);
            if (!(ok = __all_sync(kFull, ok))) break;
            const uint32_t dst = smem_addr(stages) + s * C::kStageBytes, bar = full_lead + 8 * s;
            const int x = kb * kBlk;
            if (lane == 0) {
                if (leader) mbar_arrive_expect_tx(full0 + 8 * s, bytes);
                for (int b = 0; b < (PAIR ? 1 : 2); ++b) {
                    const int blk = PAIR ? rank : b;
                    load_weights<PAIR>(dst + kOpBytes * (1 + b), &p.w_map, bar, x, p.a.glu ? kBlk * t.c : kBlk * (2 * t.c + blk),
                                       p.a.glu ? blk : 0, t.e);
                }
                if (!p.a.perm) {
                    if (mine > 96) load_rows<PAIR>(dst, &p.a_map, bar, x, row0);
                    else
                        for (int r = 0; r < mine; r += 32) load_rows<PAIR>(dst + r * kBlk, &p.a_part, bar, x, row0 + r);
                }
            }
            if (p.a.perm) {
                __syncwarp();
                if (4 * lane < mine) gather_rows<PAIR>(dst + 4 * lane * kBlk, &p.a_map, bar, x, src);
            }
            ++uses;
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    // no load may still be landing when the CTA leaves
    if (leader && lane == 0)
        for (uint32_t u = uses > C::kStages ? uses - C::kStages : 0; u < uses; ++u)
            bar_wait(full0 + 8 * (u % C::kStages), (u / C::kStages) & 1u, w, 71, false);
}

// Leader's warp 1, one thread.
template <bool PAIR>
__device__ void mma_role(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* stages, int total, int first, int step, uint32_t tmem,
                         const Wait& w) {
    using C = Cfg<PAIR>;
    // fp32 accumulator, e4m3 operands (format 0), both K-major; N = 256
    constexpr uint32_t kDesc = (1u << 4) | (256u >> 3) << 17 | (uint32_t)(C::kRowTile >> 4) << 24;
    const uint64_t ad0 = smem_desc_sw128(smem_addr(stages), 16, 1024), bd0 = smem_desc_sw128(smem_addr(stages) + kOpBytes, 16, 1024);
    const uint32_t full0 = smem_addr(&ctl->full[0]), empty0 = smem_addr(&ctl->empty[0]);
    const uint32_t tfull0 = smem_addr(&ctl->tfull[0]), tempty0 = smem_addr(&ctl->tempty[0]);
    const int last_steps = (p.a.d - kBlk * (p.nkb - 1) + kFp8K - 1) / kFp8K;  // columns past d are loaded as zeros
    int s = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    for (int i = first; ok && i < total; i += step) {
        for (int kb = 0; kb < p.nkb; ++kb, ++it) {
            const uint32_t buf = it & 1u;
            if (!(ok = bar_wait(tempty0 + 8 * buf, (it >> 1 & 1u) ^ 1u, w, 72))) break;
            if (!(ok = bar_wait(full0 + 8 * s, phase, w, 73))) break;
            tc_fence_after();
            const uint64_t ad = ad0 + (uint32_t)(s * (C::kStageBytes >> 4)), bd = bd0 + (uint32_t)(s * (C::kStageBytes >> 4));
            const uint32_t d = tmem + 256u * buf;
            const int steps = kb + 1 == p.nkb ? last_steps : kBlk / kFp8K;
#pragma unroll
            for (int k = 0; k < kBlk / kFp8K; ++k) {
                if (k < steps) {
                    if (PAIR) umma_fp8_pair(d, ad + 2 * k, bd + 2 * k, kDesc, k != 0);
                    else umma_fp8(d, ad + 2 * k, bd + 2 * k, kDesc, k != 0);
                }
            }
            if (PAIR) {
                umma_commit_pair_mc(empty0 + 8 * s, 0x3);
                umma_commit_pair_mc(tfull0 + 8 * buf, 0x3);
            } else {
                umma_commit(empty0 + 8 * s);
                umma_commit(tfull0 + 8 * buf);
            }
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    if (PAIR) umma_commit_pair(smem_addr(&ctl->mma_done));
    else umma_commit(smem_addr(&ctl->mma_done));
    bar_wait(smem_addr(&ctl->mma_done), 0u, w, 74, false);
}

// Puts 64 bytes of each lane's row into the warp's staging rows and writes them out, 16 bytes a lane, four lanes a
// row: `to` is the output's byte at the warp's first row and column, `rows` its valid rows, `bytes` the valid bytes of a row.
__device__ __forceinline__ void rows_out(uint8_t* staging, const uint4 (&v)[4], uint8_t* to, size_t pitch, int rows, int bytes) {
    const int lane = threadIdx.x & 31;
    // 16-byte column c of row r is at c ^ (r / 2 % 4): eight rows' stores and loads touch all banks once
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(staging + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = v[c];
    __syncwarp();
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        const uint4 x = *reinterpret_cast<const uint4*>(staging + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
        if (r < rows && 16 * c < bytes) __stcs(reinterpret_cast<uint4*>(to + r * pitch + 16 * c), x);
    }
    __syncwarp();
}

// g / (1 + e^-g) from e^-|g|, which does not overflow.  The exponential is within 2 + 1.173 |g| units in its last
// place and the quotient within 2, as the activation of the 8-bit checkpoint has it.
__device__ __forceinline__ float silu(float g) {
    const float e = __expf(-fabsf(g));
    return g * __fdividef(g >= 0.f ? 1.f : e, 1.f + e);
}

// Warps 4-11: TMEM lane quarter q = warp & 3 (rows) and half h of the columns of both blocks.
template <bool PAIR>
__device__ void epilogue_role(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* staging, const int* off, const int* base, int total,
                              int first, int step, uint32_t tmem, const Wait& w, bool leader, uint32_t lead, int rank) {
    using C = Cfg<PAIR>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = warp & 3, h = (warp - kEpiFirst) >> 2;
    const int nkb = p.nkb;
    staging += (warp - kEpiFirst) * kStageOut;
    const uint32_t tempty0 = PAIR && !leader ? mapa_shared(smem_addr(&ctl->tempty[0]), lead) : smem_addr(&ctl->tempty[0]);
    const uint32_t tfull0 = smem_addr(&ctl->tfull[0]);
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 64u * h;
    uint32_t it = 0;
    int turn = 0;
    for (int i = first; i < total; i += step, turn ^= 1) {
        const Fp8Tile t = tile_at<PAIR>(p, off, base, i);
        const int mine = cta_rows(t, rank) - 32 * q;  // this warp's valid rows, may be <= 0
        const size_t row0 = (size_t)t.seg0 + (size_t)(C::kRowTile * t.r + 128 * rank + 32 * q);
        const float* as = p.a.A_scales + (mine > 0 ? (size_t)source_row(p, (int)row0 + min(lane, mine - 1)) * nkb : 0);
        const int blk0 = p.a.glu ? t.c : 2 * t.c, blk1 = p.a.glu ? p.w_blocks / 2 + t.c : min(2 * t.c + 1, p.w_blocks - 1);
        const float* ws0 = p.a.W_scales + ((size_t)t.e * p.w_blocks + blk0) * nkb;
        const float* ws1 = p.a.W_scales + ((size_t)t.e * p.w_blocks + blk1) * nkb;
        uint64_t acc[64];  // columns 64 h .. of the first block, then of the second, in twos
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0;
        // a lane's scales of four k-blocks are on their way while the four before are used
        float cur[4], next[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) next[j] = j < nkb ? __ldg(as + j) : 0.f;
        float w0 = __ldg(ws0), w1 = __ldg(ws1);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
            if ((kb & 3) == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cur[j] = next[j];
                    next[j] = kb + 4 + j < nkb ? __ldg(as + kb + 4 + j) : 0.f;
                }
            }
            const float s0 = cur[0] * w0, s1 = cur[0] * w1;
            cur[0] = cur[1];
            cur[1] = cur[2];
            cur[2] = cur[3];
            if (kb + 1 < nkb) {
                w0 = __ldg(ws0 + kb + 1);
                w1 = __ldg(ws1 + kb + 1);
            }
            const uint32_t buf = it & 1u;
            const bool ready = bar_wait(tfull0 + 8 * buf, it >> 1 & 1u, w, 75);
            if (!__all_sync(kFull, ready)) return;
            tc_fence_after();
            if (mine > 0) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t v[32];
                    tmem_ld_32x32(lanes + 256u * buf + 128u * (g >> 1) + 32u * (g & 1), v);
                    tmem_ld_wait(v);
                    const uint32_t sb = __float_as_uint(g < 2 ? s0 : s1);
                    const uint64_t s = (uint64_t)sb << 32 | sb;
#pragma unroll
                    for (int j = 0; j < 16; ++j) fma2(acc[16 * g + j], v[2 * j], v[2 * j + 1], s);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && !leader) mbar_arrive_remote(tempty0 + 8 * buf);
                else mbar_arrive(tempty0 + 8 * buf);
            }
        }
        if (p.a.glu) {
            const int F = p.a.N / 2, col = kBlk * t.c + 64 * h;
            float hv[64];
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float2 g = unpack(acc[j]), u = unpack(acc[32 + j]);
                hv[2 * j] = silu(g.x) * u.x;
                hv[2 * j + 1] = silu(g.y) * u.y;
                amax = max(amax, max(__float_as_uint(hv[2 * j]) & 0x7FFFFFFFu, __float_as_uint(hv[2 * j + 1]) & 0x7FFFFFFFu));
            }
            ctl->amax[turn][h][32 * q + lane] = __uint_as_float(amax);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl->amax_there));
            const bool there = bar_wait(smem_addr(&ctl->amax_there), (uint32_t)turn, w, 76);
            if (!__all_sync(kFull, there)) return;
            amax = max(amax, __float_as_uint(ctl->amax[turn][h ^ 1][32 * q + lane]));
            const float inv = block_quotient(amax, true);
            if (mine <= 0) continue;
            if (h == 0 && lane < mine) p.a.H_scales[(row0 + lane) * scale_blocks(F) + t.c] = block_quotient(amax, false);
            uint4 v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                v[c].x = e4m3x4(hv[16 * c], hv[16 * c + 1], hv[16 * c + 2], hv[16 * c + 3], inv);
                v[c].y = e4m3x4(hv[16 * c + 4], hv[16 * c + 5], hv[16 * c + 6], hv[16 * c + 7], inv);
                v[c].z = e4m3x4(hv[16 * c + 8], hv[16 * c + 9], hv[16 * c + 10], hv[16 * c + 11], inv);
                v[c].w = e4m3x4(hv[16 * c + 12], hv[16 * c + 13], hv[16 * c + 14], hv[16 * c + 15], inv);
            }
            rows_out(staging, v, p.a.H + row0 * F + col, F, mine, F - col);
        } else if (mine > 0) {
            const size_t N = p.a.N;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int col = 256 * t.c + 128 * b + 64 * h;
                if (p.a.out_bf16) {
                    uint8_t* to = static_cast<uint8_t*>(p.a.Y) + (row0 * N + col) * 2;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = unpack(acc[32 * b + 16 * g + 4 * c + j]);
                                x[j] = bf16x2(f.x, f.y);
                            }
                            v[c] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                        rows_out(staging, v, to + 64 * g, 2 * N, mine, 2 * (p.a.N - col) - 64 * g);
                    }
                } else {
                    uint8_t* to = static_cast<uint8_t*>(p.a.Y) + (row0 * N + col) * 4;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint64_t lo = acc[32 * b + 8 * g + 2 * c], hi = acc[32 * b + 8 * g + 2 * c + 1];
                            v[c] = make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
                        }
                        rows_out(staging, v, to + 64 * g, 4 * N, mine, 4 * (p.a.N - col) - 64 * g);
                    }
                }
            }
        }
    }
}

template <bool PAIR>
__host__ __device__ constexpr uint32_t smem_bytes(int E) {
    return (uint32_t)(Cfg<PAIR>::kStages * Cfg<PAIR>::kStageBytes + kEpiWarps * kStageOut + (int)sizeof(Fp8Ctl) + 8 * (E + 1));
}
constexpr uint32_t kSmemMax = 232448;  // 227 KB
static_assert(smem_bytes<true>(kMaxE) <= kSmemMax && smem_bytes<false>(kMaxE) <= kSmemMax, "more than 227 KB of shared memory");
static_assert(Cfg<true>::kStages <= kMaxStages && Cfg<false>::kStages <= kMaxStages, "stages");

__device__ __forceinline__ uint32_t dynamic_smem_size() {
    uint32_t n;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(n));
    return n;
}

template <bool PAIR>
__device__ __forceinline__ void fp8_body(const Fp8Params& p) {
    using C = Cfg<PAIR>;
    // the swizzled stages need 1024 bytes' alignment, which shared memory starts with
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    if (pad + smem_bytes<PAIR>(p.a.E) > dynamic_smem_size()) {
        wait_for_kernel_before();
        if (threadIdx.x == 0) report_error(p.a.status, kStDevice, -3, (int)raw, 0);
        return;
    }
    uint8_t* stages = smem_raw + pad;
    uint8_t* staging = stages + C::kStages * C::kStageBytes;
    Fp8Ctl* ctl = reinterpret_cast<Fp8Ctl*>(staging + kEpiWarps * kStageOut);
    int* off = reinterpret_cast<int*>(ctl + 1);  // [E+1]
    int* base = off + p.a.E + 1;                 // [E+1] row tiles before expert e

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = PAIR ? cluster_ctarank() : 0u;
    const int rank = (int)(crank & 1u);
    const bool leader = rank == 0;
    const uint32_t lead = crank & ~1u;
    const int E = p.a.E;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_addr(&ctl->tfull[a]), 1);
            mbar_init(smem_addr(&ctl->tempty[a]), (PAIR ? 2 : 1) * kEpiWarps);
        }
        mbar_init(smem_addr(&ctl->mma_done), 1);
        mbar_init(smem_addr(&ctl->amax_there), kEpiWarps);
        ctl->abort = 0;
        mbar_fence_init();
    }
    if (warp == 2) {
        if (PAIR) {
            tmem_alloc_pair(smem_addr(&ctl->tmem_base), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(&ctl->tmem_base), 512);
            tmem_relinquish();
        }
    } else if (warp == 3 && lane == 0) {
        tma_prefetch_map(&p.a_map);
        tma_prefetch_map(&p.w_map);
    }
    // what is above runs beside the end of the kernel before this one in the stream
    wait_for_kernel_before();
    // offsets have to ascend from 0 to S: they bound every access
    int bad = 0;
    for (int e = tid; e <= E; e += kFp8Threads) {
        const int v = __ldg(p.a.offsets + e);
        off[e] = v;
        bad |= e == 0 ? v != 0 : v < __ldg(p.a.offsets + e - 1);
        bad |= e == E && v != p.a.S;
    }
    bad = __syncthreads_or(bad);
    if (warp == 0) {
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? (int)(((unsigned)(off[e + 1] - off[e]) + C::kRowTile - 1u) / (unsigned)C::kRowTile) : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < E) base[e] = run + incl - n;
            run += __shfl_sync(kFull, incl, 31);
        }
        if (lane == 0) base[E] = run;
    }
    if (bad && tid == 0) report_error(p.a.status, kStDevice, -2, off[E], 0);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // barriers and TMEM address of both CTAs are there
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const long long timeout = p.a.timeout_ns * 2 > 500000000LL ? p.a.timeout_ns * 2 : 500000000LL;
    const Wait w{&ctl->abort, p.a.status, timeout};
    const int total = bad ? 0 : base[E] * p.c_tiles;
    const int first = (int)(PAIR ? blockIdx.x / 2 : blockIdx.x), step = (int)(PAIR ? gridDim.x / 2 : gridDim.x);

    // 384 threads x 168 registers: the four warps that load and issue hand some to the epilogue's
    if (warp < kEpiFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) producer<PAIR>(p, ctl, stages, off, base, total, first, step, w, leader, lead, rank);
        else if (warp == 1 && leader && lane == 0) mma_role<PAIR>(p, ctl, stages, total, first, step, tmem, w);
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        epilogue_role<PAIR>(p, ctl, staging, off, base, total, first, step, tmem, w, leader, lead, rank);
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // no CTA leaves while its peer may still signal it
    if (warp == 2) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp8Threads, 1) grouped_fp8_pair_kernel(const __grid_constant__ Fp8Params p) {
    fp8_body<true>(p);
}
__global__ void __launch_bounds__(kFp8Threads, 1) grouped_fp8_kernel(const __grid_constant__ Fp8Params p) { fp8_body<false>(p); }

// CTAs (pairs of them) that are resident together on the current device; the kernels' attributes are set once per device.
template <bool PAIR>
cudaError_t resident(int device, int sm_count, int* n) {
    static std::atomic<int> known[64];
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    *n = known[device].load(std::memory_order_acquire);
    if (*n > 0) return cudaSuccess;
    const auto kernel = PAIR ? grouped_fp8_pair_kernel : grouped_fp8_kernel;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    if (e != cudaSuccess) return e;
    if (PAIR) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = 2;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kFp8Threads);
        cfg.dynamicSmemBytes = kSmemMax;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (*n < 1) return cudaErrorLaunchOutOfResources;
    } else {
        *n = sm_count;
    }
    known[device].store(*n, std::memory_order_release);
    return cudaSuccess;
}

template <bool PAIR>
cudaError_t launch(const Fp8Params& p, int device, int sm_count, cudaStream_t stream) {
    int n = 0;
    cudaError_t e = resident<PAIR>(device, sm_count, &n);
    if (e != cudaSuccess) return e;
    const long long tiles = ((long long)p.a.S / Cfg<PAIR>::kRowTile + p.a.E) * p.c_tiles;  // at most
    if (tiles >= (1LL << 31) - (1 << 20)) return cudaErrorInvalidValue;
    n = (int)std::min<long long>(n, tiles);
    return launch_after(PAIR ? grouped_fp8_pair_kernel : grouped_fp8_kernel, (PAIR ? 2u : 1u) * n, kFp8Threads,
                        smem_bytes<PAIR>(p.a.E), stream, p);
}

}  // namespace

cudaError_t launch_grouped_fp8(const GroupedFp8Args& a, int device, int sm_count, cudaStream_t stream) {
    Fp8Params p = {};
    p.a = a;
    const int halves = a.glu ? 2 : 1, n = a.N / halves;
    p.w_blocks = halves * scale_blocks(n);
    p.nkb = scale_blocks(a.d);
    p.c_tiles = a.glu ? scale_blocks(n) : (a.N + 255) / 256;
    const uint64_t rows = a.perm ? (uint64_t)a.T : (uint64_t)a.S;
    if (!map_e4m3_2d(&p.a_map, a.A, rows, (uint64_t)a.d, a.perm ? 1 : 128) || !map_e4m3_2d(&p.a_part, a.A, rows, (uint64_t)a.d, 32) ||
        !map_e4m3_weights(&p.w_map, a.W, (uint64_t)a.E, (uint64_t)halves, (uint64_t)n, (uint64_t)a.d))
        return cudaErrorInvalidValue;
    // pairs where the experts have that many rows on average
    return a.S >= 128LL * a.E ? launch<true>(p, device, sm_count, stream) : launch<false>(p, device, sm_count, stream);
}

}  // namespace moe
