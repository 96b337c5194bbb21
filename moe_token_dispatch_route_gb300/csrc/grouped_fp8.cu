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
// reads and 128 multiply-adds a cycle: half of the 512 cycles that the tensor cores take for the block.  The thread
// that issues the MMAs has as long, so its loop has two commits a k-block (the accumulator is there, the stage is free) and
// nothing that can be done elsewhere.  Bound by the two accumulators taking turns: an MMA's latency, the additions and the handing
// back are about 1500 cycles, 720 to 770 a k-block.
// One GB300: 16384 rows of 8 experts, 14336 x 4096, bf16 out: 782 to 817 us (2.46 to 2.36 PFLOP/s; 678 to 705 in loops of a few
// calls); SwiGLU, 65536 gathered rows of 64 experts, 2048 x 2 x 1408: 427 to 437 us; 512 rows of 128 experts, 1536 x 4096: 115 to 119 us
// (HBM: the weights).
//
// Roles of a CTA (512 threads): warp 0 loads W and, where its rows are in place, A (TMA); warp 1 issues the MMAs (the
// leader's) or tells the leader that gathered rows have landed (the peer's); warp 2 brings the scales; warps 4-7 copy
// gathered rows (16-byte cp.async: TMA's gather of four rows took three times as long); warps 8-15 are the epilogue, each
// with one TMEM lane quarter and half of the columns of both blocks.  Tile i of the list is the CTA's (or pair's) i mod
// grid: all tiles cost the same.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "bounded_wait.cuh"
#include "moe_internal.cuh"
#include "serve.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kFp8Threads = 512;
constexpr int kBlk = kScaleBlock;           // columns of a k-block
constexpr int kOpBytes = 128 * kBlk;        // 16 KB: 128 rows of an operand
constexpr int kEpiFirst = 8, kEpiWarps = 8;
constexpr int kBand = 8;                    // row tiles per schedule band
constexpr int kFp8K = 32;                   // products of an MMA step
constexpr int kMaxStages = 6;
constexpr int kStageOut = 2048;             // a warp's 32 rows of 64 bytes on their way out
constexpr int kScaleRing = 4;               // slots of four k-blocks' scales
constexpr int kGatherFirst = 4, kGatherWarps = 4;
constexpr int kGatherRows = 128 / kGatherWarps;  // of a warp

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
    uint64_t tfull[2];          // an accumulator has its k-block's products
    uint64_t tempty[2];         // leader: it has been read
    uint64_t mma_done;
    uint64_t amax_there[4];     // the two epilogue warps of a lane quarter have written a tile's amax
    uint64_t afull[kMaxStages]; // gathered rows, the pair's peer: its own have landed
    uint64_t sfull[kScaleRing], sempty[kScaleRing];
    uint32_t tmem_base;
    int abort;
    float amax[2][2][128];      // by tile parity and half of the columns: a row's largest magnitude
    float4 as[kScaleRing][128]; // four k-blocks' scales of each row
    float4 ws[kScaleRing][2];   // and of the two blocks of W
};

// Division of an int >= 0 by a number that the host knows: by ceil(2^64 / n), exact below 2^31.  (Three integer divisions were
// most of the thousand cycles that a tile's place took.)
struct Divisor {
    uint64_t inverse;  // 0: n is 1
    static Divisor of(int n) { return Divisor{n == 1 ? 0 : ~0ull / (uint64_t)n + 1}; }
    __device__ __forceinline__ int operator()(int v) const { return inverse ? (int)__umul64hi((uint64_t)v, inverse) : v; }
};
// v / n for 0 < n <= kBand and v below 2^26
__device__ __forceinline__ int divide_small(int v, int n) {
    static_assert(kBand == 8, "an inverse for each");
    constexpr uint32_t kInverse[9] = {0, 0, 0x80000000u, 0x55555556u, 0x40000000u, 0x33333334u, 0x2AAAAAABu, 0x24924925u, 0x20000000u};
    uint32_t inverse = 0;
#pragma unroll
    for (int i = 2; i <= 8; ++i) inverse = n == i ? kInverse[i] : inverse;
    return n == 1 ? v : (int)__umulhi((uint32_t)v, inverse);
}

struct Fp8Params {
    CUtensorMap a_map;    // rows in place: boxes of 128 rows
    CUtensorMap a_part;   // rows in place: boxes of 32 rows
    CUtensorMap w_map;
    GroupedFp8Args a;
    int c_tiles, nkb;
    Divisor by_c, by_band;  // c_tiles, and kBand times it
    int as_vec;           // rows of A's scales are whole 16 bytes
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

// 32 TMEM lanes x 16 consecutive columns, loaded and there.  (A wait in a statement of its own would take the registers as
// operands, and they would be copied.)
__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// One arrival of a converged warp, without a branch.  PAIR: `bar` is a shared::cluster address.
template <bool PAIR>
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
            "@p mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n}\n" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
            "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar)
            : "memory");
}

// A wait on a barrier whose arrivals hand over TMEM, which the tcgen05 fences order: acquired at CTA scope.
__device__ __forceinline__ bool tmem_wait(uint32_t bar, uint32_t parity, const Wait& w, int where) {
    return mbar_try_wait(bar, parity) || bar_wait_slow(bar, parity, w, where, true);
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
    const int u = p.by_c(i);
    int lo = 0, hi = p.a.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= u) lo = mid;
        else hi = mid;
    }
    t.e = lo;
    const int local = i - base[lo] * p.c_tiles, rt = base[lo + 1] - base[lo];
    // bands of kBand row tiles, all column tiles of a band together: each operand is read from DRAM about once
    const int band = p.by_band(local);
    const int nr = min(kBand, rt - band * kBand);
    const int j = local - band * kBand * p.c_tiles;
    t.c = divide_small(j, nr);
    t.r = band * kBand + j - t.c * nr;
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

// Bytes of the k-block's rows of A that a CTA with `rows` valid ones loads by TMA: boxes of 32 rows.
__device__ __forceinline__ uint32_t a_bytes(const Fp8Params& p, int rows) {
    return p.a.perm ? 0u : (uint32_t)((rows + 31) & ~31) * kBlk;
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e != 0;
}

// Warp 0.  All lanes run the loop and one issues: addresses are then known to be the warp's, not a lane's.
template <bool PAIR>
__device__ void producer(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* stages, const int* off, const int* base, int total, int first,
                         int step, const Wait& w, bool leader, uint32_t lead, int rank) {
    using C = Cfg<PAIR>;
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
        for (int kb = 0; kb < p.nkb; ++kb) {

            ok = bar_wait(empty0 + 8 * s, phase ^ 1u, w, 70);
            if (!(ok = __all_sync(kFull, ok))) break;

            if (elected()) {
                const uint32_t dst = smem_addr(stages) + s * C::kStageBytes, bar = full_lead + 8 * s;
                const int x = kb * kBlk;
                if (leader) mbar_arrive_expect_tx(full0 + 8 * s, bytes);
#pragma unroll
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
            __syncwarp();

            ++uses;
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    // no load may still be landing when the CTA leaves
    if (leader)
        for (uint32_t u = uses > C::kStages ? uses - C::kStages : 0; u < uses; ++u)
            bar_wait(full0 + 8 * (u % C::kStages), (u / C::kStages) & 1u, w, 71, false);
}

// Gathered rows, kGatherWarps warps: eight lanes copy the 128 bytes of a row, in the swizzled layout that TMA
// gives (16-byte column c of row r at c ^ (r % 8)).  Every lane's arrival on the stage's barrier follows its copies, so
// nobody waits for them here.
template <bool PAIR>
__device__ void gather_role(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* stages, const int* off, const int* base, int total, int first,
                            int step, const Wait& w, bool leader, int rank) {
    using C = Cfg<PAIR>;
    const int lane = threadIdx.x & 31, c = lane & 7, r_lane = lane >> 3, part = (int)(threadIdx.x >> 5) - kGatherFirst;
    const uint32_t empty0 = smem_addr(&ctl->empty[0]);
    const uint32_t landed0 = leader ? smem_addr(&ctl->full[0]) : smem_addr(&ctl->afull[0]);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = first; ok && i < total; i += step) {
        const Fp8Tile t = tile_at<PAIR>(p, off, base, i);
        const int mine = cta_rows(t, rank), row0 = t.seg0 + C::kRowTile * t.r + 128 * rank;
        // the source rows of this lane's rows kGatherRows part + 4 j + r_lane, first read by a lane each
        int src[kGatherRows / 4];
        {
            const int r = kGatherRows * part + lane;
            const int read = r < mine ? source_row(p, row0 + r) : -1;
#pragma unroll
            for (int j = 0; j < kGatherRows / 4; ++j) src[j] = __shfl_sync(kFull, read, 4 * j + r_lane);
        }
        for (int kb = 0; kb < p.nkb; ++kb) {
            ok = bar_wait(empty0 + 8 * s, phase ^ 1u, w, 77);
            if (!(ok = __all_sync(kFull, ok))) break;
            const uint32_t dst = smem_addr(stages) + s * C::kStageBytes;
            const int x = kb * kBlk + 16 * c;
            const int bytes = x < p.a.d ? 16 : 0;  // columns past d are zeros
            const uint8_t* col = p.a.A + (bytes ? x : 0);
#pragma unroll
            for (int j = 0; j < kGatherRows / 4; ++j) {
                const int r = kGatherRows * part + 4 * j + r_lane;
                if (src[j] >= 0)
                    cp_async16_cg_zfill(dst + (uint32_t)(r * kBlk + ((c ^ (r & 7)) << 4)), col + (size_t)src[j] * p.a.d, bytes);
            }
            cp_async_mbar_arrive_noinc(landed0 + 8 * s);
            if (++s == C::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
    cp_async_wait_all();  // no copy may still be landing when the CTA leaves
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Warp 2: the scales of four k-blocks at a time, four rows a lane, and those of the two blocks of W.  (Loaded by the
// epilogue's threads, even four k-blocks ahead, they held its loop up.)
template <bool PAIR>
__device__ void scales_role(const Fp8Params& p, Fp8Ctl* ctl, const int* off, const int* base, int total, int first, int step,
                            const Wait& w, int rank) {
    const int lane = threadIdx.x & 31;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = first; ok && i < total; i += step) {
        const Fp8Tile t = tile_at<PAIR>(p, off, base, i);
        const int mine = cta_rows(t, rank), row0 = t.seg0 + Cfg<PAIR>::kRowTile * t.r + 128 * rank;
        const float* as[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = lane + 32 * j;
            as[j] = r < mine ? p.a.A_scales + (size_t)source_row(p, row0 + r) * p.nkb : nullptr;
        }
        const int blk0 = p.a.glu ? t.c : 2 * t.c, blk1 = p.a.glu ? p.w_blocks / 2 + t.c : min(2 * t.c + 1, p.w_blocks - 1);
        const float* ws = p.a.W_scales + ((size_t)t.e * p.w_blocks + (lane < 4 ? blk0 : blk1)) * p.nkb + (lane & 3);
        for (int kb = 0; kb < p.nkb; kb += 4) {
            ok = bar_wait(smem_addr(&ctl->sempty[slot]), phase ^ 1u, w, 79);
            if (!(ok = __all_sync(kFull, ok))) break;
            const int n = min(4, p.nkb - kb);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!as[j]) continue;
                const uint32_t dst = smem_addr(&ctl->as[slot][lane + 32 * j]);
                if (p.as_vec) {
                    cp_async16_cg(dst, as[j] + kb);
                } else {
                    for (int k = 0; k < n; ++k) cp_async4(dst + 4 * k, as[j] + kb + k);
                }
            }
            if (lane < 8 && (lane & 3) < n) cp_async4(smem_addr(&ctl->ws[slot][0]) + 4 * lane, ws + kb);
            cp_async_mbar_arrive_noinc(smem_addr(&ctl->sfull[slot]));
            if (++slot == kScaleRing) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
    cp_async_wait_all();
}

// Gathered rows, the peer's warp 1, one thread: passes a stage whose rows have landed on to the leader.
template <bool PAIR>
__device__ void relay_role(const Fp8Params& p, Fp8Ctl* ctl, int total, int first, int step, const Wait& w, uint32_t lead) {
    const uint32_t full_lead = mapa_shared(smem_addr(&ctl->full[0]), lead), afull0 = smem_addr(&ctl->afull[0]);
    int s = 0;
    uint32_t phase = 0;
    for (int i = first; i < total; i += step) {
        for (int kb = 0; kb < p.nkb; ++kb) {
            if (!bar_wait(afull0 + 8 * s, phase, w, 78)) return;
            fence_proxy_async_smem();  // the copies, before the leader's MMAs read them
            mbar_arrive_remote(full_lead + 8 * s);
            if (++s == Cfg<PAIR>::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
}

// Leader's warp 1.  All lanes run the loop and one issues: descriptors and addresses are then known to be the warp's, not a
// lane's.  (Run by one lane alone, an MMA took some 75 cycles to issue.)
template <bool PAIR>
__device__ void mma_role(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* stages, int total, int first, int step, uint32_t tmem,
                         const Wait& w) {
    using C = Cfg<PAIR>;
    // fp32 accumulator, e4m3 operands (format 0), both K-major; N = 256
    constexpr uint32_t kDesc = (1u << 4) | (256u >> 3) << 17 | (uint32_t)(C::kRowTile >> 4) << 24;
    const uint64_t ad0 = smem_desc_sw128(smem_addr(stages), 16, 1024), bd0 = smem_desc_sw128(smem_addr(stages) + kOpBytes, 16, 1024);
    const uint32_t full0 = smem_addr(&ctl->full[0]), empty0 = smem_addr(&ctl->empty[0]);
    const uint32_t tfull0 = smem_addr(&ctl->tfull[0]), tempty0 = smem_addr(&ctl->tempty[0]);
    const bool gathered = p.a.perm != nullptr;
    const int last_steps = (p.a.d - kBlk * (p.nkb - 1) + kFp8K - 1) / kFp8K;  // columns past d are loaded as zeros
    int s = 0;
    uint32_t phase = 0, free_phase[2] = {1, 1};
    // a tile's k-blocks go to accumulator 0 and 1 in turn, from 0 on
    auto block = [&](int buf, int steps) {
        // (the loads are long there; the accumulator is what this warp waits for, so it is waited for last)
        const bool landed = bar_wait(full0 + 8 * s, phase, w, 73);
        if (gathered) fence_proxy_async_smem();  // this CTA's copies
        const uint64_t ad = ad0 + (uint32_t)(s * (C::kStageBytes >> 4)), bd = bd0 + (uint32_t)(s * (C::kStageBytes >> 4));
        const uint32_t d = tmem + 256u * buf;
        const bool there = landed && tmem_wait(tempty0 + 8 * buf, free_phase[buf], w, 72);
        if (!__all_sync(kFull, there)) return false;
        free_phase[buf] ^= 1u;
        tc_fence_after();
        if (elected()) {
#pragma unroll
            for (int k = 0; k < steps; ++k) {
                if (PAIR) umma_fp8_pair(d, ad + 2 * k, bd + 2 * k, kDesc, k != 0);
                else umma_fp8(d, ad + 2 * k, bd + 2 * k, kDesc, k != 0);
            }
            if (PAIR) {
                umma_commit_pair_mc(tfull0 + 8 * buf, 0x3);
                umma_commit_pair_mc(empty0 + 8 * s, 0x3);
            } else {
                umma_commit(tfull0 + 8 * buf);
                umma_commit(empty0 + 8 * s);
            }
        }
        __syncwarp();
        if (++s == C::kStages) {
            s = 0;
            phase ^= 1u;
        }
        return true;
    };
    bool ok = true;
    for (int i = first; ok && i < total; i += step) {
        int kb = 0;
        for (; ok && kb + 2 < p.nkb; kb += 2) ok = block(0, kBlk / kFp8K) && block(1, kBlk / kFp8K);
        if (ok && kb + 2 == p.nkb) ok = block(0, kBlk / kFp8K) && block(1, last_steps);
        else if (ok) ok = block(0, last_steps);
    }
    if (elected()) {
        if (PAIR) umma_commit_pair(smem_addr(&ctl->mma_done));
        else umma_commit(smem_addr(&ctl->mma_done));
    }
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

// u *= silu(g) for four values.  With e = e^-|g| and q = e / (1 + e), silu(g) = max(g, 0) - |g| q: nothing overflows, and far
// negative g keeps its small result (e is the square of e^(-|g| / 2), whose own fast form would flush it).  The four
// quotients share one reciprocal: the exponentials and reciprocals are what bounds the activation, five in place of
// eight.  A NaN makes NaN of all four, as its block's scale does in any case.
__device__ __forceinline__ void silu4(const float* g, float* u) {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(fabsf(g[i]) * -0.72134752f));  // log2(e) / 2
    float2 lo = make_float2(e[0], e[1]), hi = make_float2(e[2], e[3]);
    lo = __fmul2_rn(lo, lo);
    hi = __fmul2_rn(hi, hi);
    const float2 dl = __fadd2_rn(lo, make_float2(1.f, 1.f)), dh = __fadd2_rn(hi, make_float2(1.f, 1.f));
    const float pl = dl.x * dl.y, ph = dh.x * dh.y;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(pl * ph));
    const float rl = r * ph, rh = r * pl;
    const float2 ql = __fmul2_rn(lo, __fmul2_rn(make_float2(rl, rl), make_float2(dl.y, dl.x)));
    const float2 qh = __fmul2_rn(hi, __fmul2_rn(make_float2(rh, rh), make_float2(dh.y, dh.x)));
    const float q[4] = {ql.x, ql.y, qh.x, qh.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] *= fmaf(-fabsf(g[i]), q[i], g[i] < 0.f ? 0.f : g[i]);
}

// Warps 8-15: TMEM lane quarter q = warp & 3 (rows) and half h of the columns of both blocks.
template <bool PAIR>
__device__ void epilogue_role(const Fp8Params& p, Fp8Ctl* ctl, uint8_t* staging, const int* off, const int* base, int total,
                              int first, int step, uint32_t tmem, const Wait& w, bool leader, uint32_t lead, int rank) {
    using C = Cfg<PAIR>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = warp & 3, h = (warp - kEpiFirst) >> 2;
    const int nkb = p.nkb;
    staging += (warp - kEpiFirst) * kStageOut;
    const uint32_t tempty_own = smem_addr(&ctl->tempty[0]), tempty0 = PAIR ? mapa_shared(tempty_own, lead) : tempty_own;
    const uint32_t tfull0 = smem_addr(&ctl->tfull[0]);
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 64u * h;
    uint32_t ready_phase[2] = {0, 0}, sphase = 0;
    int turn = 0, slot = 0;
    for (int i = first; i < total; i += step, turn ^= 1) {
        const Fp8Tile t = tile_at<PAIR>(p, off, base, i);
        const int mine = cta_rows(t, rank) - 32 * q;  // this warp's valid rows, may be <= 0
        const size_t row0 = (size_t)t.seg0 + (size_t)(C::kRowTile * t.r + 128 * rank + 32 * q);
        float acc[2][64];  // columns 64 h .. of the two blocks
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[b][j] = 0.f;
        // The k-blocks of a warp with (LIVE) and without valid rows; false: a wait gave up.  FOURS: they are whole fours.
        // (A branch around the sums inside the loop would copy them.  16384 rows, 14336 x 4096: 757 us in twos, 727 in fours.)
        auto blocks = [&](auto live, auto fours) {
            constexpr bool LIVE = decltype(live)::value, FOURS = decltype(fours)::value;
            float sc[4][2];  // four k-blocks' scales, for either block of W
            auto block = [&](int buf, float s0, float s1) {
                const bool ready = tmem_wait(tfull0 + 8 * buf, ready_phase[buf], w, 75);
                if (!__all_sync(kFull, ready)) return false;
                ready_phase[buf] ^= 1u;
                tc_fence_after();
                if constexpr (LIVE) {
                    const uint32_t at = lanes + 256u * buf;
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        uint32_t v[16];
                        tmem_ld_32x16(at + 128 * (g >> 2) + 16 * (g & 3), v);
                        float* sum = acc[g >> 2] + 16 * (g & 3);
                        const float2 scale = g < 4 ? make_float2(s0, s0) : make_float2(s1, s1);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), scale,
                                                        make_float2(sum[j], sum[j + 1]));
                            sum[j] = r.x;
                            sum[j + 1] = r.y;
                        }
                    }
                }
                tc_fence_before();
                warp_arrive<PAIR>(tempty0 + 8 * buf);
                return true;
            };
            auto scales = [&]() {
                const bool there = bar_wait(smem_addr(&ctl->sfull[slot]), sphase, w, 80);
                if (!__all_sync(kFull, there)) return false;
                const float4 a4 = ctl->as[slot][32 * q + lane], w0 = ctl->ws[slot][0], w1 = ctl->ws[slot][1];
                sc[0][0] = a4.x * w0.x;
                sc[0][1] = a4.x * w1.x;
                sc[1][0] = a4.y * w0.y;
                sc[1][1] = a4.y * w1.y;
                sc[2][0] = a4.z * w0.z;
                sc[2][1] = a4.z * w1.z;
                sc[3][0] = a4.w * w0.w;
                sc[3][1] = a4.w * w1.w;
                return true;
            };
            auto read = [&]() {  // the scales are in registers
                __syncwarp();    // all lanes' reads, before one lane's arrival hands the slot back
                warp_arrive<false>(smem_addr(&ctl->sempty[slot]));
                if (++slot == kScaleRing) {
                    slot = 0;
                    sphase ^= 1u;
                }
            };
            if constexpr (FOURS) {
#pragma unroll 1
                for (int kb = 0; kb < nkb; kb += 4) {
                    if (!scales()) return false;
                    if (!block(0, sc[0][0], sc[0][1])) return false;
                    read();
                    if (!block(1, sc[1][0], sc[1][1])) return false;
                    if (!block(0, sc[2][0], sc[2][1])) return false;
                    if (!block(1, sc[3][0], sc[3][1])) return false;
                }
            } else {
#pragma unroll 1
                for (int kb = 0; kb < nkb; kb += 2) {
                    if ((kb & 3) == 0 && !scales()) return false;
                    if (!block(0, sc[0][0], sc[0][1])) return false;
                    if ((kb & 3) == 0) read();
                    if (kb + 1 == nkb) break;
                    if (!block(1, sc[1][0], sc[1][1])) return false;
                    sc[0][0] = sc[2][0];
                    sc[0][1] = sc[2][1];
                    sc[1][0] = sc[3][0];
                    sc[1][1] = sc[3][1];
                }
            }
            return true;
        };
        const bool ok = mine <= 0 ? blocks(std::false_type(), std::false_type())
                        : (nkb & 3) == 0 ? blocks(std::true_type(), std::true_type()) : blocks(std::true_type(), std::false_type());
        if (!ok) return;
        if (p.a.glu) {
            const int F = p.a.N / 2, col = kBlk * t.c + 64 * h;
            float(&hv)[64] = acc[1];
            float big = 0.f;
#pragma unroll
            for (int j = 0; j < 64; j += 4) silu4(acc[0] + j, hv + j);
#pragma unroll
            for (int j = 0; j < 64; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(big) : "f"(fabsf(hv[j])));
            uint32_t amax = __float_as_uint(big);
            ctl->amax[turn][h][32 * q + lane] = __uint_as_float(amax);
            __syncwarp();
            warp_arrive<false>(smem_addr(&ctl->amax_there[q]));
            const bool there = bar_wait(smem_addr(&ctl->amax_there[q]), (uint32_t)turn, w, 76);
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
                const int col = 256 * t.c + 128 * b + 64 * h, cols = min(p.a.N - col, 64);  // (a long row's bytes pass 32 bits)
                if (p.a.out_bf16) {
                    uint8_t* to = static_cast<uint8_t*>(p.a.Y) + (row0 * N + col) * 2;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[j] = bf16x2(acc[b][32 * g + 8 * c + 2 * j], acc[b][32 * g + 8 * c + 2 * j + 1]);
                            v[c] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                        rows_out(staging, v, to + 64 * g, 2 * N, mine, 2 * cols - 64 * g);
                    }
                } else {
                    uint8_t* to = static_cast<uint8_t*>(p.a.Y) + (row0 * N + col) * 4;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            v[c] = make_uint4(__float_as_uint(acc[b][16 * g + 4 * c]), __float_as_uint(acc[b][16 * g + 4 * c + 1]),
                                              __float_as_uint(acc[b][16 * g + 4 * c + 2]), __float_as_uint(acc[b][16 * g + 4 * c + 3]));
                        rows_out(staging, v, to + 64 * g, 4 * N, mine, 4 * cols - 64 * g);
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

    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const uint32_t crank = PAIR ? cluster_ctarank() : 0u;
    const int rank = (int)(crank & 1u);
    const bool leader = rank == 0;
    const uint32_t lead = crank & ~1u;
    const int E = p.a.E;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            // the loading thread, and with gathered rows the copying lanes and the peer's relay
            mbar_init(smem_addr(&ctl->full[s]), p.a.perm ? 1 + 32 * kGatherWarps + (PAIR ? 1 : 0) : 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
            mbar_init(smem_addr(&ctl->afull[s]), 32 * kGatherWarps);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_addr(&ctl->tfull[a]), 1);
            mbar_init(smem_addr(&ctl->tempty[a]), (PAIR ? 2 : 1) * kEpiWarps);
        }
        for (int r = 0; r < kScaleRing; ++r) {
            mbar_init(smem_addr(&ctl->sfull[r]), 32);
            mbar_init(smem_addr(&ctl->sempty[r]), kEpiWarps);
        }
        mbar_init(smem_addr(&ctl->mma_done), 1);
        for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&ctl->amax_there[i]), 2);
        ctl->abort = 0;
        mbar_fence_init();
    }
    if (warp == 3) {
        if (PAIR) {
            tmem_alloc_pair(smem_addr(&ctl->tmem_base), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(&ctl->tmem_base), 512);
            tmem_relinquish();
        }
    } else if (warp == 4 && lane == 0) {
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
    const uint32_t tmem = __shfl_sync(kFull, ctl->tmem_base, 0);  // the same for all, which the compiler cannot see
    const long long timeout = p.a.timeout_ns * 2 > 500000000LL ? p.a.timeout_ns * 2 : 500000000LL;
    const Wait w{&ctl->abort, p.a.status, timeout};
    const int total = bad ? 0 : base[E] * p.c_tiles;
    const int first = (int)(PAIR ? blockIdx.x / 2 : blockIdx.x), step = (int)(PAIR ? gridDim.x / 2 : gridDim.x);

    // 512 threads x 128 registers: the eight warps that load and issue hand some to the epilogue's
    if (warp < kEpiFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 0) {
            producer<PAIR>(p, ctl, stages, off, base, total, first, step, w, leader, lead, rank);
        } else if (warp == 1) {
            if (leader) mma_role<PAIR>(p, ctl, stages, total, first, step, tmem, w);
            else if (p.a.perm && lane == 0) relay_role<PAIR>(p, ctl, total, first, step, w, lead);
        } else if (warp == 2) {
            scales_role<PAIR>(p, ctl, off, base, total, first, step, w, rank);
        } else if (p.a.perm && warp >= kGatherFirst) {
            gather_role<PAIR>(p, ctl, stages, off, base, total, first, step, w, leader, rank);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        epilogue_role<PAIR>(p, ctl, staging, off, base, total, first, step, tmem, w, leader, lead, rank);
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // no CTA leaves while its peer may still signal it
    if (warp == 3) {
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
    p.as_vec = p.nkb % 4 == 0 && reinterpret_cast<uintptr_t>(a.A_scales) % 16 == 0;
    p.c_tiles = a.glu ? scale_blocks(n) : (a.N - 1) / 256 + 1;
    p.by_c = Divisor::of(p.c_tiles);
    p.by_band = Divisor::of(kBand * p.c_tiles);
    // Pairs of CTAs load half of W each, but waste more rows of an expert's last tile, and gathered rows reach the leader's
    // MMAs through one more thread.  us with one CTA a tile and in pairs: rows in place, 32 experts of 4096 x 4096, 256
    // rows each 161 and 178, 512 265 and 264, 768 417 and 379, 2048 983 and 941; gathered, 2048 x 2816 SwiGLU, 1024 rows
    // 433 and 459, 4096 x 8192, 2048 rows 500 and 493.
    const bool pair = a.S >= (a.perm ? 1536LL : 512LL) * a.E;
    const uint64_t rows = a.perm ? (uint64_t)a.T : (uint64_t)a.S;
    if (!map_e4m3_2d(&p.a_map, a.A, rows, (uint64_t)a.d, 128) || !map_e4m3_2d(&p.a_part, a.A, rows, (uint64_t)a.d, 32) ||
        !map_e4m3_weights(&p.w_map, a.W, (uint64_t)a.E, (uint64_t)halves, (uint64_t)n, (uint64_t)a.d))
        return cudaErrorInvalidValue;

    return pair ? launch<true>(p, device, sm_count, stream) : launch<false>(p, device, sm_count, stream);
}

}  // namespace moe
