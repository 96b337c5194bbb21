// The two gradients of the per-expert grouped product Y_i = A_i W_e(i), one persistent kernel:
//   input gradient   dA_i = dY_i W_e(i)^T            (i over expert e's rows)
//   weight gradient  dW_e = A_e^T dY_e               (summed over expert e's rows)
// bf16 operands, fp32 sums, output fp32 or bf16 (rounded once).
//
// Both are written as out[r][c] = sum_k Q[r][k] P[c][k] with c the contiguous axis of the output:
//   input gradient:  r = expert row, c = d, k = N;  P = W_e [d][N],   Q = dY [rows][N]  (K-major)
//   weight gradient: r = d,          c = N, k = row; P = dY [rows][N], Q = A [rows][d]  (MN-major)
// A tile is 256 c by up to 256 r, computed by a pair of CTAs (tcgen05 cta_group::2): P gives the
// 256 rows of the MMA (128 per CTA), Q its columns.  So
//  * the accumulator's TMEM lanes are consecutive c: the epilogue stores 128 contiguous bytes of
//    an output row per warp straight from registers, with no transposition;
//  * the ragged axis of the input gradient is the MMA's N, which goes in steps of 32: an expert
//    with few rows costs few columns, and a row past the segment is a column that is not stored.
// The weight gradient's ragged axis is the reduction.  Its last k-block is loaded in boxes of 16
// rows, the MMAs stop at the last 16, and a warp zeroes the rows past the segment (another
// expert's, whose NaN or infinity times zero would spread) in shared memory before the MMAs.
//
// Roles of a CTA (384 threads): warp 0 loads P and warp 2 loads Q, warp 1 issues the MMAs (leader)
// or claims the pair's tiles (peer), warp 3 zeroes the rows past a segment, warps 4-11 are the
// epilogue, each with one TMEM lane quarter and half of the columns.  A k-block is 512 cycles of
// the tensor cores; the loading threads have to issue theirs in less, so they do nothing else
// (claims and tails inside their loop cost 250 cycles more, and the weight gradient waited for
// loads 35% of the time).
//
// Few tiles and a long reduction (more than 32 or 64 k-blocks): it is cut into pieces of at least 16, at
// most two for each pair of CTAs, whose sums go to the workspace; a second kernel adds
// them in order (2 experts, 192 x 13808, 166 rows: 67 us whole, 19 in pieces).
//
// fp32 outputs: the tensor cores' running sum rounds towards zero at every step of 16 products,
// which over a long reduction is a bias (relative error 1e-6 at 1024 products, 1.6e-5 at 14336).
// So a sum runs in TMEM over 768 products (7e-7) and the epilogue adds these in registers; the two
// accumulators alternate, so the MMAs do not wait.  bf16 outputs (2e-3 apart) take one sum.
//
// Measured.  16384 rows of 8 experts, 4096 x 14336: input gradient bf16 1.12 ms (1.72 PFLOP/s), weight gradient bf16
// 1.11 and fp32 1.21 ms; after seconds at the power limit 1.29 and (fp32) 1.28.  65536 rows of 64 experts (Zipf),
// 2048 x 1408: weight gradient fp32 0.30 ms, with its 738 MB of stores.  512 rows of 128 experts, 4096 x 1536: input
// gradient 203 us, 7.0 TB/s of weights.
#include <algorithm>
#include <atomic>

#include "bounded_wait.cuh"
#include "moe_internal.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kGradThreads = 384;
constexpr int kMaxStages = 10;
constexpr int kGradRing = 4;
constexpr int kOpBytes = kTileM * kTileK * 2;  // 16 KB: one CTA's 128 rows (or columns) of an operand
constexpr int kEpiFirst = 4, kEpiWarps = 8;
constexpr int kBand = 8;       // row tiles per schedule band
constexpr int kChunkKb = 12;   // k-blocks (of 64) per TMEM sum of an fp32 output

// The forms of the kernel.  kNarrow is the input gradient for experts of few rows: row tiles
// of 64, whose smaller Q leaves shared memory for ten stages of loads in flight.  The seventh stage of the
// others fills the shared memory to the last KB, where the offsets of some 250 experts fit beside it: with more
// experts (the Many forms) there are six.  Stages are what hides the loads' latency (us with seven and six; fp32
// outputs): 64 experts of 512 rows, 4096 x 1536, input gradient 296 and 306, weight gradient 358 and 371; 8 experts of 2048
// rows, 4096 x 14336, weight gradient 1212 and 1244 (five: 4% more again, four: 12%).  bf16 weight gradients of few
// rows lose 2% by the smaller L1.
enum class Form { kInput, kInputMany, kNarrow, kWeight, kWeightMany };
template <Form F>
struct Cfg {
    static constexpr bool kWeight = F == Form::kWeight || F == Form::kWeightMany;
    static constexpr int kRowTile = F == Form::kNarrow ? 64 : 256;
    static constexpr int kQBytes = kRowTile / 2 * kTileK * 2;  // one CTA's half of Q
    static constexpr int kStages = F == Form::kNarrow ? 10 : F == Form::kInput || F == Form::kWeight ? 7 : 6;
    static constexpr int kWarpRows = kRowTile / 2;             // output rows of an epilogue warp
    // Splitting a reduction costs about as much as this many k-blocks (a second kernel) and as many
    // more for each piece; reductions of up to kMinSplit blocks stay whole (16 tiles of 41 blocks: 20 us
    // whole, 28 in two pieces).
    static constexpr int kSplitCost = F == Form::kNarrow ? 14 : 24;
    static constexpr int kPieceCost = F == Form::kNarrow ? 2 : 4;
    static constexpr int kMinSplit = F == Form::kNarrow ? 32 : 64;
};

// A tile as the roles take it from the ring: the scheduler has worked out what they need, since a
// tile's change costs the MMA thread's time (500 cycles of it when each role worked it out itself).
struct GradTile {
    int e, c, r;  // expert (-1: no more), column tile, row tile
    int seg0;     // expert's first row
    int nkb;      // k-blocks
    int rows;     // valid output rows
    int last;     // of the last k-block: MMA steps | rows to keep when they end inside a step << 8 | half of the MMA's N << 16
    int boxes;    // weight gradient: rows of P's boxes | of Q's << 8 | Q's chunks are paired << 16
    int kbeg;     // first k-block
    int slot;     // >= 0: a piece of a tile's reduction, whose sums go there
};

// A tile whose reduction is cut into pieces, for the joining kernel: its pieces are in slots
// slot0, slot0 + stride, ... (n of them).
struct SplitTile {
    long long out_row;  // of the tile's first row
    int c0, rows;
    int slot0, n, stride, pad;
};
// Whether a listed tile lies inside an output of `out_rows` rows, and its pieces inside `slots` slots.
// The list is the kernel's own, but one that ended early (a wait ran out, which the status says) leaves entries of
// an earlier call in it, of another output: the joining kernel passes over what it must not touch.
__host__ __device__ constexpr bool inside(long long out_row, int c0, int rows, int slot0, int n, int stride,
                                          long long out_rows, int row_tile, int slots) {
    return rows > 0 && rows <= row_tile && out_row >= 0 && out_row <= out_rows - rows && c0 >= 0 && n > 0 && n <= slots &&
           slot0 >= 0 && stride >= 0 && slot0 + (long long)(n - 1) * stride < slots;
}
static_assert(inside(0, 0, 256, 0, 2, 76, 256, 256, 152) && inside(744, 512, 256, 75, 2, 76, 1000, 256, 152), "in bounds");
static_assert(!inside(745, 0, 256, 0, 2, 76, 1000, 256, 152) && !inside(-1, 0, 16, 0, 2, 1, 1000, 256, 152) &&
                  !inside(1LL << 62, 0, 16, 0, 2, 1, 1000, 256, 152) && !inside(0, -256, 16, 0, 2, 1, 1000, 256, 152),
              "outside the output");
static_assert(!inside(0, 0, 0, 0, 2, 1, 1000, 256, 152) && !inside(0, 0, 257, 0, 2, 1, 1000, 256, 152) &&
                  !inside(0, 0, 65, 0, 2, 1, 1000, 64, 152),
              "no rows, or more than a tile's");
static_assert(!inside(0, 0, 16, 76, 2, 76, 1000, 256, 152) && !inside(0, 0, 16, -1, 2, 76, 1000, 256, 152) &&
                  !inside(0, 0, 16, 0, 153, 0, 1000, 256, 152) && !inside(0, 0, 16, 0, 152, 0x7FFFFFFF, 1000, 256, 152) &&
                  !inside(0, 0, 16, 0, 2, -1, 1000, 256, 152) && !inside(0, 0, 16, 0, 0, 1, 1000, 256, 152),
              "outside the slots");
constexpr int kMaxSplit = 256;    // split tiles: at most one for each pair of CTAs
constexpr int kMaxSplitExperts = 160;  // each has more than a pair's share of all the work: fewer than pairs
constexpr int kMinPieceKb = 16;   // shortest piece, in k-blocks
// The split area of a workspace: the number of split tiles, their list, the slots.
struct SplitArea {
    int count, pad[7];
    SplitTile tile[kMaxSplit];
};

struct GradCtl {
    uint64_t full[kMaxStages];   // leader: the stage's loads of both CTAs
    uint64_t empty[kMaxStages];
    uint64_t tail[kMaxStages];   // each CTA's own loads of a block to be zeroed
    uint64_t fixed[kMaxStages];  // leader: both CTAs have zeroed
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t sfull[kGradRing];
    uint64_t sempty[kGradRing];
    uint64_t mma_done;
    GradTile ring[kGradRing];
    uint32_t tmem_base;
    int abort;
    // Pieces of at most `limit` k-blocks.  Input gradient: every tile has `pieces`; weight gradient, where
    // no piece is longer than a pair's share of all the work: the first `split_experts` of
    // `order` have, expert k's from piece split_base[k] of an output tile on.
    int limit, pieces, split_experts, split_items;
    int total_kb;  // weight gradient: k-blocks of all experts
    int one_round;  // no more items than pairs: nothing is claimed, and the counters stay as they are
    short split_base[kMaxSplitExperts + 1];
};

struct GradParams {
    CUtensorMap p_map, q_map;      // whole blocks
    CUtensorMap q_tail;            // input gradient: boxes of 16 rows (q_map: of kRowTile / 2)
    // weight gradient, where rows are whole chunks of 64 columns: two chunks in one copy,
    // of 64, 32 and 16 rows
    CUtensorMap p_pair[3], q_pair[3];
    int p_paired, q_paired;
    GroupedGradArgs a;
    int c_tiles, r_tiles;          // r_tiles: weight gradient only
    int chunk_kb;
    int c_size;                    // extent of c: d or N
    SplitArea* split;              // null: no tile is split
    float* slots;
};

// The unpacked fields of a tile.
struct Shape {
    int seg0, nkb, rows;
    int ksteps;  // MMA steps of 16 in the last k-block
    int half;    // Q rows (columns) per CTA: half of the MMA's N
    int fix;     // rows of the last k-block that are the expert's, when they end inside a step; else 0
    // weight gradient, last k-block: rows of its boxes (a last block of one or two steps is loaded in
    // boxes of 16 or 32 rows where the columns are paired: an expert of a few rows costs few bytes)
    int p_box, q_box;
    bool q_paired;
    __device__ explicit Shape(const GradTile& t)
        : seg0(t.seg0), nkb(t.nkb), rows(t.rows), ksteps(t.last & 0xFF), half(t.last >> 16), fix(t.last >> 8 & 0xFF),
          p_box(t.boxes & 0xFF), q_box(t.boxes >> 8 & 0xFF), q_paired(t.boxes >> 16 != 0) {}
};

// v / step, rounded up, for every v that an int holds
__host__ __device__ constexpr int steps_of(int v, int step) { return (int)(((unsigned)v + (unsigned)step - 1u) / (unsigned)step); }
static_assert(steps_of(0, 64) == 0 && steps_of(64, 64) == 1 && steps_of(65, 64) == 2 && steps_of(0x7FFFFFFF, 256) == 1 << 23,
              "rounded up");

// k-blocks of a reduction, and of each of its pieces
template <Form F>
__device__ __forceinline__ int blocks_of(const GradParams& p, int rows) {
    return steps_of(Cfg<F>::kWeight ? rows : p.a.N, kTileK);
}
template <Form F>
__device__ __forceinline__ int piece_blocks(int nkb, int limit) {
    if (nkb <= limit || nkb <= Cfg<F>::kMinSplit) return nkb;
    const int n = (nkb + limit - 1) / limit;
    return (nkb + n - 1) / n;
}

template <Form F>
__device__ void fill_shape(const GradParams& p, const int* off, GradTile& t, int piece, int limit) {
    constexpr bool WG = Cfg<F>::kWeight;
    constexpr int kRow = Cfg<F>::kRowTile;
    t.seg0 = off[t.e];
    const int cnt = off[t.e + 1] - t.seg0;
    const int K = WG ? cnt : p.a.N;
    t.rows = min(kRow, (WG ? p.a.d : cnt) - kRow * t.r);
    const int half = ((t.rows + 31) & ~31) / 2;
    const int nkb = blocks_of<F>(p, cnt), len = piece_blocks<F>(nkb, limit);
    t.kbeg = piece * len;
    t.nkb = min(len, nkb - t.kbeg);
    const int last = t.kbeg + t.nkb == nkb ? K - kTileK * (nkb - 1) : kTileK;
    const int ksteps = (last + kUmmaK - 1) / kUmmaK;
    // (rows past the last one of all are read as zeros)
    const int fix = (WG && (last & (kUmmaK - 1)) && t.seg0 + cnt < p.a.S) ? last : 0;
    t.last = ksteps | fix << 8 | half << 16;
    t.boxes = 0;
    if (WG) {
        const bool paired = p.q_paired && half % 64 == 0;  // the peer's first column starts a chunk
        t.boxes = (p.p_paired && ksteps <= 2 ? kUmmaK * ksteps : kTileK) |
                  (paired && ksteps <= 2 ? kUmmaK * ksteps : kTileK) << 8 | (paired ? 1 : 0) << 16;
    }
}

// the next slot of the schedule ring
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ void next() {
        if (++slot == kGradRing) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

template <int kStages>
struct Stage {
    int s = 0;
    uint32_t phase = 0;
    __device__ void next() {
        if (++s == kStages) {
            s = 0;
            phase ^= 1u;
        }
    }
    __device__ void skip(int n) {
        s += n;
        phase ^= (uint32_t)(s / kStages) & 1u;
        s %= kStages;
    }
};

// True, once every word of the tile is in a register.  A slot may be handed back only then: a load of shared memory
// queues behind its warp's stores to global memory, microseconds of them in the epilogue, but an arrival on a
// barrier does not, and the scheduler's next tile would be read in the slot's place.  (No field but -1
// is negative, so the words' OR is never the lowest integer.)
__device__ __forceinline__ bool loaded(const GradTile& t) {
    return (t.e | t.c | t.r | t.seg0 | t.nkb | t.rows | t.last | t.boxes | t.kbeg | t.slot) != (int)0x80000000;
}

// Takes the next tile from the ring and hands the slot back to the scheduler in the peer CTA;
// called by one thread, or (WARP) by all lanes of a warp, which arrives once.
template <bool WARP>
__device__ __forceinline__ bool take(GradCtl* ctl, Ring& ring, GradTile& t, const Wait& w, int where, bool leader,
                                     uint32_t sched) {
    bool got = bar_wait(smem_addr(&ctl->sfull[ring.slot]), ring.phase, w, where);
    if (WARP) got = __all_sync(kFull, got);
    if (!got) return false;
    t = ctl->ring[ring.slot];
    bool read = loaded(t);
    if (WARP) read = __all_sync(kFull, read);
    if (read && (!WARP || (threadIdx.x & 31) == 0)) {
        const uint32_t se = smem_addr(&ctl->sempty[ring.slot]);
        if (leader) mbar_arrive_remote(mapa_shared(se, sched));
        else mbar_arrive(se);
    }
    ring.next();
    return true;
}

// Work item i: a tile, or a piece of one.  `note`: the first piece of a tile enters it in the list of split tiles.
template <Form F>
__device__ GradTile item_at(const GradParams& p, const GradCtl* ctl, const int* off, const int* base, const short* order,
                            uint32_t i, bool note) {
    constexpr bool WG = Cfg<F>::kWeight;
    GradTile t{-1, 0, 0, 0, 0, 0, 0, 0, 0, -1};
    int local, rt, piece = 0, n = 1, stride = 1, ordinal;
    if (WG) {
        const uint32_t per_expert = (uint32_t)p.c_tiles * (uint32_t)p.r_tiles;
        rt = p.r_tiles;
        if (i < (uint32_t)ctl->split_items) {
            int k = 0;
            while ((uint32_t)ctl->split_base[k + 1] * per_expert <= i) ++k;
            const uint32_t j = i - (uint32_t)ctl->split_base[k] * per_expert;
            t.e = order[k];
            piece = (int)(j / per_expert);
            local = (int)(j % per_expert);
            n = ctl->split_base[k + 1] - ctl->split_base[k];
            stride = (int)per_expert;
            ordinal = k * (int)per_expert + local;
        } else {
            const uint32_t j = i - (uint32_t)ctl->split_items;
            if (j >= (uint32_t)(p.a.E - ctl->split_experts) * per_expert) return t;
            t.e = order[ctl->split_experts + j / per_expert];
            local = (int)(j % per_expert);
            ordinal = 0;
        }
    } else {
        n = ctl->pieces;
        const uint32_t tile = i / (uint32_t)n;
        if (tile >= (uint32_t)base[p.a.E] * (uint32_t)p.c_tiles) return t;
        piece = (int)(i % (uint32_t)n);
        ordinal = (int)tile;
        const int u = (int)(tile / (uint32_t)p.c_tiles);
        int lo = 0, hi = p.a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (base[mid] <= u) lo = mid;
            else hi = mid;
        }
        t.e = lo;
        local = (int)(tile - (uint32_t)base[lo] * (uint32_t)p.c_tiles);
        rt = base[lo + 1] - base[lo];
    }
    // bands of kBand row tiles, all column tiles of a band together: about as many row as column
    // tiles run at a time, so each operand is read from DRAM about once
    const int band = local / (kBand * p.c_tiles);
    const int nr = min(kBand, rt - band * kBand);
    const int j = local - band * kBand * p.c_tiles;
    t.c = j / nr;
    t.r = band * kBand + j % nr;
    fill_shape<F>(p, off, t, piece, ctl->limit);
    if (n > 1) {
        t.slot = (int)i;
        if (note && piece == 0 && ordinal < kMaxSplit) {
            const long long row = (WG ? (long long)t.e * p.a.d : (long long)t.seg0) + (long long)Cfg<F>::kRowTile * t.r;
            p.split->tile[ordinal] = SplitTile{row, 256 * t.c, t.rows, t.slot, n, stride, 0};
        }
    }
    return t;
}

// How the reductions are cut, by one thread: see GradCtl.
template <Form F>
__device__ void plan_pieces(const GradParams& p, GradCtl* ctl, const int* off, const int* base, const short* order, bool write) {
    using C = Cfg<F>;
    constexpr bool WG = Cfg<F>::kWeight;
    ctl->limit = 1 << 30;
    ctl->pieces = 1;
    ctl->split_experts = ctl->split_items = 0;
    const int pairs = (int)(gridDim.x / 2);
    const long long per_expert = (long long)p.c_tiles * p.r_tiles;
    ctl->one_round = (WG ? p.a.E * per_expert : (long long)base[p.a.E] * p.c_tiles) <= pairs;
    if (!p.split) return;
    int split = 0;
    if (WG) {
        const long long total = ctl->total_kb * per_expert;
        const int limit = (int)min((long long)(1 << 30), max((long long)kMinPieceKb, (total + pairs - 1) / pairs));
        ctl->limit = limit;
        int k = 0, run = 0;
        for (; k < p.a.E && k < kMaxSplitExperts; ++k) {  // most rows first
            const int nkb = blocks_of<F>(p, off[order[k] + 1] - off[order[k]]), len = piece_blocks<F>(nkb, limit);
            if (len == nkb) break;
            ctl->split_base[k] = (short)run;
            run += (nkb + len - 1) / len;
        }
        ctl->split_base[k] = (short)run;
        ctl->split_experts = k;
        ctl->split_items = (int)(run * per_expert);
        split = (int)(k * per_expert);
        ctl->one_round = (p.a.E - k) * per_expert + ctl->split_items <= pairs;
    } else {
        // all tiles have the same reduction: the number of pieces whose rounds of pairs end first
        const int nkb = blocks_of<F>(p, 0), tiles = base[p.a.E] * p.c_tiles;
        int best = (tiles + pairs - 1) / pairs * nkb;
        for (int n = 2; nkb > C::kMinSplit && tiles * n <= 2 * pairs && n * kMinPieceKb <= nkb; ++n) {
            const int len = (nkb + n - 1) / n, cost = (tiles * n + pairs - 1) / pairs * len + C::kSplitCost + C::kPieceCost * n;
            if (cost < best) {
                best = cost;
                ctl->limit = len;
            }
        }
        const int len = piece_blocks<F>(nkb, ctl->limit);
        ctl->pieces = (nkb + len - 1) / len;
        if (ctl->pieces > 1) split = tiles;
        ctl->one_round = (long long)tiles * ctl->pieces <= pairs;
    }
    if (write) p.split->count = split;
}

// Peer CTA's warp 1, one thread: claims the items after a pair's first (which is its own number) and
// writes them into both CTAs' rings.
template <Form F>
__device__ void scheduler(const GradParams& p, GradCtl* ctl, const int* off, const int* base, const short* order, const Wait& w,
                          uint32_t lead) {
    Ring ring;
    const uint32_t pairs = gridDim.x / 2;
    bool more = ctl->ring[0].e >= 0;
    ring.next();  // the first item was put into both rings before the roles began
    while (more) {
        if (!bar_wait(smem_addr(&ctl->sempty[ring.slot]), ring.phase ^ 1u, w, 51)) return;
        const uint32_t next = ctl->one_round ? 0u : atomicAdd(p.a.hdr + kHdrTileCtr, 1u);
        const GradTile t = item_at<F>(p, ctl, off, base, order, pairs + next, true);
        ctl->ring[ring.slot] = t;
        const uint32_t dst = mapa_shared(smem_addr(&ctl->ring[ring.slot]), lead);
        const uint32_t bar = mapa_shared(smem_addr(&ctl->sfull[ring.slot]), lead);
        st_async_v2(dst, (uint32_t)t.e, (uint32_t)t.c, bar);
        st_async_v2(dst + 8, (uint32_t)t.r, (uint32_t)t.seg0, bar);
        st_async_v2(dst + 16, (uint32_t)t.nkb, (uint32_t)t.rows, bar);
        st_async_v2(dst + 24, (uint32_t)t.last, (uint32_t)t.boxes, bar);
        st_async_v2(dst + 32, (uint32_t)t.kbeg, (uint32_t)t.slot, bar);
        mbar_arrive(smem_addr(&ctl->sfull[ring.slot]));
        more = t.e >= 0;
        ring.next();
    }
}

// Loads of one operand of one k-block into `dst`.  K-major (input gradient): 64 k by `rows` rows
// from (x = k, y = row).
__device__ __forceinline__ void load_kmajor(uint32_t dst, const CUtensorMap* whole, const CUtensorMap* part,
                                            uint32_t bar, int k, int row, int rows, int whole_rows) {
    if (rows == whole_rows) {
        tma_load_2d_pair(dst, whole, bar, k, row);
    } else {
        for (int i = 0; i < rows; i += 16) tma_load_2d_pair(dst + i * 128, part, bar, k, row + i);
    }
}

// MN-major (weight gradient): one or two chunks of 64 columns by `box` rows, one after the other.
__device__ __forceinline__ void load_mnmajor(uint32_t dst, const CUtensorMap* whole, const CUtensorMap* pair, bool paired,
                                             uint32_t bar, int col, int row, int chunks, int box) {
    if (paired) {
        tma_load_3d_pair(dst, pair + (box == kTileK ? 0 : box == 32 ? 1 : 2), bar, 0, row, col >> 6);
    } else {
        tma_load_2d_pair(dst, whole, bar, col, row);
        if (chunks == 2) tma_load_2d_pair(dst + 8192, whole, bar, col + 64, row);
    }
}

// bytes of one CTA's Q loads of a k-block whose boxes are `box` rows
template <Form F>
__device__ __forceinline__ uint32_t q_bytes(const Shape& s, int box) {
    if (!Cfg<F>::kWeight) return (uint32_t)s.half * 128u;
    return s.q_paired || s.half > 64 ? (uint32_t)box * 256u : (uint32_t)box * 128u;
}

// Warp 0, one thread: this CTA's half of P, and the stage barriers' expected bytes.
template <Form F>
__device__ void producer_p(const GradParams& p, GradCtl* ctl, uint8_t* sP, const Wait& w, bool leader,
                           uint32_t peer, uint32_t lead, uint32_t rank) {
    using C = Cfg<F>;
    constexpr bool WG = C::kWeight;
    constexpr uint32_t kStages = C::kStages;
    const uint32_t full0 = smem_addr(&ctl->full[0]), empty0 = smem_addr(&ctl->empty[0]);
    const uint32_t full_lead = mapa_shared(full0, lead), dst0 = smem_addr(sP);
    const int side = 128 * (int)(rank & 1u);
    Ring ring;
    Stage<C::kStages> st;
    uint32_t uses = 0, tail_phase = 0, tail_used = 0;
    GradTile t;
    bool ok = true;
    for (bool first = true; ok; first = false) {
        if (leader && !first)  // the description comes from the peer's scheduler
            mbar_arrive_expect_tx(smem_addr(&ctl->sfull[ring.slot]), (uint32_t)sizeof(GradTile));
        if (!take<false>(ctl, ring, t, w, 52, leader, peer) || t.e < 0) break;
        const Shape s(t);
        const int c0 = 256 * t.c + side;
        const int whole = WG && s.nkb > 0 ? s.nkb - 1 : s.nkb;
        const int row0 = WG ? s.seg0 + t.kbeg * kTileK : t.e * p.a.d + c0, k0 = t.kbeg * kTileK;
        const uint32_t bytes = 2 * (kOpBytes + q_bytes<F>(s, kTileK));
        for (int kb = 0; kb < whole; ++kb) {
            if (!(ok = bar_wait(empty0 + 8 * st.s, st.phase ^ 1u, w, 53))) break;
            if (leader) mbar_arrive_expect_tx(full0 + 8 * st.s, bytes);
            if (WG) load_mnmajor(dst0 + st.s * kOpBytes, &p.p_map, p.p_pair, p.p_paired, full_lead + 8 * st.s, c0,
                                 row0 + kb * kTileK, 2, kTileK);
            else tma_load_2d_pair(dst0 + st.s * kOpBytes, &p.p_map, full_lead + 8 * st.s, k0 + kb * kTileK, row0);
            st.next();
            ++uses;
        }
        if (ok && whole < s.nkb) {  // weight gradient: the last block
            if (!(ok = bar_wait(empty0 + 8 * st.s, st.phase ^ 1u, w, 53))) break;
            const uint32_t last = (uint32_t)s.p_box * 256u + q_bytes<F>(s, s.q_box);
            const uint32_t tail = smem_addr(&ctl->tail[st.s]);
            // A block to be zeroed lands on each CTA's own tail barrier, which its warp 3 waits for:
            // a stage's next tail comes only after the MMAs have read this one, so that warp, which
            // skips the blocks in between, never falls a whole phase behind.  The leader's stage
            // barrier then gets its arrival alone and keeps its phase.
            if (s.fix) {
                mbar_arrive_expect_tx(tail, last);
                tail_used |= 1u << st.s;
                tail_phase ^= 1u << st.s;
            }
            if (leader) {
                if (s.fix) mbar_arrive(full0 + 8 * st.s);
                else mbar_arrive_expect_tx(full0 + 8 * st.s, 2 * last);
            }
            load_mnmajor(dst0 + st.s * kOpBytes, &p.p_map, p.p_pair, p.p_paired,
                         s.fix ? mapa_shared(tail, rank) : full_lead + 8 * st.s, c0, row0 + whole * kTileK, 2, s.p_box);
            st.next();
            ++uses;
        }
    }
    // no load may still be landing when the CTA leaves
    if (leader)
        for (uint32_t u = uses > kStages ? uses - kStages : 0; u < uses; ++u)
            bar_wait(full0 + 8 * (u % kStages), (u / kStages) & 1u, w, 54, false);
    for (uint32_t i = 0; i < kStages; ++i)
        if (tail_used >> i & 1u) bar_wait(smem_addr(&ctl->tail[i]), (tail_phase >> i & 1u) ^ 1u, w, 55, false);
}

// Warp 2, one thread: this CTA's half of Q.
template <Form F>
__device__ void producer_q(const GradParams& p, GradCtl* ctl, uint8_t* sQ, const Wait& w, bool leader,
                           uint32_t peer, uint32_t lead, uint32_t rank) {
    using C = Cfg<F>;
    constexpr bool WG = C::kWeight;
    const uint32_t empty0 = smem_addr(&ctl->empty[0]), full_lead = mapa_shared(smem_addr(&ctl->full[0]), lead);
    const uint32_t dst0 = smem_addr(sQ);
    Ring ring;
    Stage<C::kStages> st;
    GradTile t;
    for (;;) {
        if (!take<false>(ctl, ring, t, w, 56, leader, peer) || t.e < 0) return;
        const Shape s(t);
        const int r0 = C::kRowTile * t.r + s.half * (int)(rank & 1u);
        const int whole = WG && s.nkb > 0 ? s.nkb - 1 : s.nkb;
        const int chunks = s.half > 64 ? 2 : 1;
        const int k0 = t.kbeg * kTileK;
        for (int kb = 0; kb < whole; ++kb) {
            if (!bar_wait(empty0 + 8 * st.s, st.phase ^ 1u, w, 57)) return;
            if (WG) load_mnmajor(dst0 + st.s * C::kQBytes, &p.q_map, p.q_pair, s.q_paired, full_lead + 8 * st.s, r0,
                                 s.seg0 + k0 + kb * kTileK, chunks, kTileK);
            else load_kmajor(dst0 + st.s * C::kQBytes, &p.q_map, &p.q_tail, full_lead + 8 * st.s, k0 + kb * kTileK, s.seg0 + r0, s.half, C::kRowTile / 2);
            st.next();
        }
        if (whole < s.nkb) {
            if (!bar_wait(empty0 + 8 * st.s, st.phase ^ 1u, w, 57)) return;
            load_mnmajor(dst0 + st.s * C::kQBytes, &p.q_map, p.q_pair, s.q_paired,
                         s.fix ? mapa_shared(smem_addr(&ctl->tail[st.s]), rank) : full_lead + 8 * st.s, r0,
                         s.seg0 + k0 + whole * kTileK, chunks, s.q_box);
            st.next();
        }
    }
}

// Warp 3 (weight gradient): zeroes the rows of a last k-block that are not the expert's, up to
// the end of its last step of 16, in both operands.
template <Form F>
__device__ void zero_rows(const GradParams& p, GradCtl* ctl, uint8_t* sP, uint8_t* sQ, const Wait& w,
                          bool leader, uint32_t peer, uint32_t lead) {
    using C = Cfg<F>;
    const int lane = threadIdx.x & 31;
    Ring ring;
    Stage<C::kStages> st;
    uint32_t tail_phase = 0;
    GradTile t;
    for (;;) {
        if (!take<true>(ctl, ring, t, w, 58, leader, peer) || t.e < 0) return;
        const Shape s(t);
        if (s.fix) {
            Stage<C::kStages> at = st;
            at.skip(s.nkb - 1);
            const bool landed = bar_wait(smem_addr(&ctl->tail[at.s]), tail_phase >> at.s & 1u, w, 59);
            if (!__all_sync(kFull, landed)) return;
            tail_phase ^= 1u << at.s;
            // eight lanes for each chunk of 64 columns (128 bytes a row): P's two, then Q's two
            const int chunk = lane >> 3;
            uint8_t* op = (chunk < 2 ? sP + chunk * s.p_box * 128 : sQ + (chunk - 2) * s.q_box * 128) +
                          at.s * kOpBytes + (lane & 7) * 16;
            if (chunk < 3 || s.half > 64)  // a narrow Q has one chunk
                for (int r = s.fix; r < s.ksteps * kUmmaK; ++r) *reinterpret_cast<uint4*>(op + r * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();  // before the MMAs read it
            __syncwarp();
            const uint32_t fixed = smem_addr(&ctl->fixed[at.s]);
            // The zeros stay in this CTA's shared memory and the proxy fence has made them visible to the
            // tensor cores before the arrival is sent; a release at cluster scope on top of it
            // waits another 0.5 us (3% of a weight gradient with odd counts).
            if (lane == 0) {
                if (leader) mbar_arrive(fixed);
                else mbar_arrive_remote(mapa_shared(fixed, lead));
            }
        }
        st.skip(s.nkb);
    }
}

template <Form F>
__device__ void mma_role(const GradParams& p, GradCtl* ctl, uint8_t* sP, uint8_t* sQ, uint32_t tmem,
                         const Wait& w, uint32_t peer) {
    using C = Cfg<F>;
    constexpr bool WG = C::kWeight;
    // fp32 accumulator, bf16 operands; MN-major operands for the weight gradient; M = 256
    constexpr uint32_t kDesc = (1u << 4) | (1u << 7) | (1u << 10) | (WG ? (1u << 15) | (1u << 16) : 0u) | (16u << 24);
    constexpr uint32_t kLbo = WG ? 8192 : 16, kStep = WG ? 2048 : 32;
    Ring ring;
    Stage<C::kStages> st;
    uint32_t fixed_phase = 0;
    const uint64_t pd0 = smem_desc_sw128(smem_addr(sP), kLbo, 1024), qd0 = smem_desc_sw128(smem_addr(sQ), kLbo, 1024);
    const uint32_t full0 = smem_addr(&ctl->full[0]), empty0 = smem_addr(&ctl->empty[0]);
    int acc = 0;
    uint32_t aphase = 0;
    GradTile t;
    bool ok = true;
    while (ok) {
        // the slot is handed back after the tile's first sum is issued, off the path from tile to tile
        if (!bar_wait(smem_addr(&ctl->sfull[ring.slot]), ring.phase, w, 61)) break;
        t = ctl->ring[ring.slot];
        const uint32_t taken = mapa_shared(smem_addr(&ctl->sempty[ring.slot]), peer);
        ring.next();
        const bool read = loaded(t);
        if (t.e < 0 || t.nkb == 0) {
            if (read) mbar_arrive_remote(taken);
            if (t.e < 0) break;
            continue;
        }
        const Shape s(t);
        const uint32_t idesc = kDesc | ((uint32_t)(2 * s.half) >> 3) << 17;
        for (int kb0 = 0; ok && kb0 < s.nkb; kb0 += p.chunk_kb) {
            if (!(ok = bar_wait(smem_addr(&ctl->tempty[acc]), aphase ^ 1u, w, 62))) break;
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(acc * 256);
            // blocks of four steps in the loop (this thread's issue rate bounds the kernel), a
            // short or zeroed last block after it
            const int end = min(s.nkb - kb0, p.chunk_kb);
            const bool tail = kb0 + end == s.nkb && (s.ksteps < kTileK / kUmmaK || (WG && s.fix));
            const int whole = tail ? end - 1 : end;
            for (int i = 0; i < whole; ++i) {
                if (!(ok = bar_wait(full0 + st.s * 8, st.phase, w, 63))) break;
                tc_fence_after();
                const uint64_t pd = pd0 + (uint32_t)(st.s * (kOpBytes >> 4)), qd = qd0 + (uint32_t)(st.s * (C::kQBytes >> 4));
                umma_bf16_pair(d, pd, qd, idesc, i != 0);
#pragma unroll
                for (int kk = 1; kk < kTileK / kUmmaK; ++kk)
                    umma_bf16_pair(d, pd + kk * (kStep >> 4), qd + kk * (kStep >> 4), idesc, 1u);
                umma_commit_pair_mc(empty0 + st.s * 8, 0x3);
                st.next();
            }
            if (!ok) break;
            if (tail) {
                if (WG && s.fix) {
                    ok = bar_wait(smem_addr(&ctl->fixed[st.s]), fixed_phase >> st.s & 1u, w, 64);
                    fixed_phase ^= 1u << st.s;
                } else {
                    ok = bar_wait(full0 + st.s * 8, st.phase, w, 63);
                }
                if (!ok) break;
                tc_fence_after();
                const uint64_t pd = smem_desc_sw128(smem_addr(sP) + st.s * kOpBytes, WG ? s.p_box * 128 : kLbo, 1024);
                const uint64_t qd = smem_desc_sw128(smem_addr(sQ) + st.s * C::kQBytes, WG ? s.q_box * 128 : kLbo, 1024);
                for (int kk = 0; kk < s.ksteps; ++kk)
                    umma_bf16_pair(d, pd + kk * (kStep >> 4), qd + kk * (kStep >> 4), idesc, (whole | kk) != 0);
                umma_commit_pair_mc(empty0 + st.s * 8, 0x3);
                st.next();
            }
            umma_commit_pair_mc(smem_addr(&ctl->tfull[acc]), 0x3);
            if (kb0 == 0 && read) mbar_arrive_remote(taken);
            if ((acc ^= 1) == 0) aphase ^= 1u;
        }
    }
    umma_commit_pair(smem_addr(&ctl->mma_done));
    bar_wait(smem_addr(&ctl->mma_done), 0u, w, 65, false);
}

// visit(address, i, rows left) for i = 0, STEP, ... below ROWS, addresses `pitch` bytes apart for each
// step.  n of the lane's rows are to be visited: n - i are left, and where every lane of the warp has all of
// its rows STEP is passed, a constant, so that the visits' tests vanish.  The address is stepped, not multiplied
// out: 128 products in flight spilled, and the whole epilogue ran at 2.6 TB/s.
template <int ROWS, int STEP, class Visit>
__device__ __forceinline__ void walk_rows(uint8_t* at, size_t pitch, int n, Visit visit) {
    constexpr int kAll = STEP == 4 ? ROWS - 2 : ROWS;  // (of four rows a lane stores two)
    if (__all_sync(kFull, n >= kAll)) {
#pragma unroll
        for (int i = 0; i < ROWS; i += STEP) {
            visit(at, i, STEP);
            asm volatile("add.u64 %0, %0, %1;" : "+l"(at) : "l"(pitch));
        }
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; i += STEP) {
            visit(at, i, n - i);
            asm volatile("add.u64 %0, %0, %1;" : "+l"(at) : "l"(pitch));
        }
    }
}

// Warps 4-11: lane quarter q = warp & 3 (c) and half h of the rows.  All sums of a thread, one c by
// up to 128 r, are in registers before the first store, so the accumulator is handed
// back while the stores are still leaving.
template <Form F>
__device__ void epilogue_role(const GradParams& p, GradCtl* ctl, uint32_t tmem, const Wait& w,
                              bool leader, uint32_t peer, uint32_t lead, uint32_t rank) {
    using C = Cfg<F>;
    constexpr bool WG = C::kWeight;
    constexpr int kRows = C::kWarpRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = warp & 3, h = (warp - kEpiFirst) >> 2;
    Ring ring;
    int acc = 0;
    uint32_t aphase = 0;
    GradTile t;
    for (;;) {
        if (!take<true>(ctl, ring, t, w, 66, leader, peer) || t.e < 0) return;
        const Shape s(t);
        const int cols = min(kRows, s.rows - kRows * h);  // this warp's valid rows, may be <= 0
        const int c = 256 * t.c + 128 * (int)(rank & 1u) + 32 * q + lane;
        const int mine = c < p.c_size ? cols : 0;  // this lane's valid rows
        // This lane's first result and the bytes from row to row.  A piece's sums go to [slot][row][256
        // columns].  bf16: even lanes store columns c, c + 1 of two rows of four, odd lanes c - 1, c of the
        // other two.
        const int odd = lane & 1;
        const bool low = p.a.out_bf16 && t.slot < 0;
        const size_t row0 = (WG ? (size_t)t.e * p.a.d : (size_t)s.seg0) + (size_t)(C::kRowTile * t.r + kRows * h);
        uint8_t* at;
        size_t pitch;
        if (t.slot >= 0) {
            at = reinterpret_cast<uint8_t*>(p.slots + ((size_t)t.slot * C::kRowTile + kRows * h) * 256 + (c & 255));
            pitch = 1024;
        } else if (low) {
            at = static_cast<uint8_t*>(p.a.out) + ((row0 + 2 * odd) * p.c_size + (c - odd)) * 2;
            pitch = (size_t)p.c_size * 2;
        } else {
            at = static_cast<uint8_t*>(p.a.out) + (row0 * p.c_size + c) * 4;
            pitch = (size_t)p.c_size * 4;
        }
        const bool add = WG && p.a.accumulate && t.slot < 0;
        if (add && s.nkb == 0) continue;  // nothing to add
        uint32_t sum[kRows / 32][32];  // fp32 bits
        if (s.nkb == 0) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) sum[i / 32][i % 32] = 0u;
        }
        for (int kb = 0; kb < s.nkb; kb += p.chunk_kb) {
            const bool ready = bar_wait(smem_addr(&ctl->tfull[acc]), aphase, w, 67);
            if (!__all_sync(kFull, ready)) return;
            tc_fence_after();
            const uint32_t base = tmem + (uint32_t)(acc * 256 + kRows * h) + ((uint32_t)(32 * q) << 16);
            if (kb == 0) {  // the first sum is loaded where it stays, all of it in flight
#pragma unroll
                for (int g = 0; g < kRows / 32; ++g)
                    if (32 * g < cols) tmem_ld_32x32(base + 32 * g, sum[g]);
#pragma unroll
                for (int g = 0; g < kRows / 32; ++g) tmem_ld_wait(sum[g]);
            } else {
#pragma unroll
                for (int g = 0; g < kRows / 32; ++g) {
                    if (32 * g < cols) {
                        uint32_t v[32];
                        tmem_ld_32x32(base + 32 * g, v);
                        tmem_ld_wait(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sum[g][i] = __float_as_uint(__uint_as_float(sum[g][i]) + __uint_as_float(v[i]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t te = smem_addr(&ctl->tempty[acc]);
                if (leader) mbar_arrive(te);
                else mbar_arrive_remote(mapa_shared(te, lead));
            }
            if ((acc ^= 1) == 0) aphase ^= 1u;
        }
        if (low) {
            // Four rows at a time.  A lane rounds and packs two rows of its column, so one exchange serves
            // four rows; the exchanges share a pipe with the stores (decode-sized weight gradient: 405 us with one
            // for two rows, 354 with one for four).
            const uint32_t lo = odd ? 0x1054u : 0x5410u, hi = odd ? 0x3276u : 0x7632u;  // (mine, other) or (other, mine)
            walk_rows<kRows, 4>(at, 4 * pitch, mine - 2 * odd, [&](uint8_t* at, int i, int n) {
                const uint32_t a = bf16x2(__uint_as_float(sum[i / 32][i % 32]), __uint_as_float(sum[i / 32][i % 32 + 1]));
                const uint32_t b = bf16x2(__uint_as_float(sum[i / 32][i % 32 + 2]), __uint_as_float(sum[i / 32][i % 32 + 3]));
                const uint32_t other = __shfl_xor_sync(kFull, odd ? a : b, 1), own = odd ? b : a;
                if (n > 0) __stcs(reinterpret_cast<uint32_t*>(at), __byte_perm(own, other, lo));
                if (n > 1) __stcs(reinterpret_cast<uint32_t*>(at + pitch), __byte_perm(own, other, hi));
            });
        } else if (add) {
            // Added in L2, once for each element, so in no order that could change: to read the sums first takes these
            // warps a round trip a tile (64 experts of 64 rows, 4096 x 1536: 693 us, 596 added in L2; 2048
            // rows, 4096 x 14336: 1376 and 1321).  The reduction takes subnormal values as zeros.
            walk_rows<kRows, 1>(at, pitch, mine, [&](uint8_t* at, int i, int n) {
                if (n > 0) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(at), "f"(__uint_as_float(sum[i / 32][i % 32])) : "memory");
            });
        } else {
            walk_rows<kRows, 1>(at, pitch, mine, [&](uint8_t* at, int i, int n) {
                if (n > 0) __stcs(reinterpret_cast<uint32_t*>(at), sum[i / 32][i % 32]);
            });
        }
    }
}

constexpr uint32_t kSmemMax = 232448;  // 227 KB
template <Form F>
__host__ __device__ constexpr uint32_t smem_bytes(int E) {
    return (uint32_t)(Cfg<F>::kStages * (kOpBytes + Cfg<F>::kQBytes) + (int)sizeof(GradCtl) +
                      (Cfg<F>::kWeight ? 4 * (E + 1) + 2 * E : 8 * (E + 1)));
}
static_assert(smem_bytes<Form::kInputMany>(kMaxE) <= kSmemMax && smem_bytes<Form::kWeightMany>(kMaxE) <= kSmemMax &&
                  smem_bytes<Form::kNarrow>(kMaxE) <= kSmemMax,
              "more than 227 KB of shared memory per CTA");
static_assert(smem_bytes<Form::kInput>(256) <= kSmemMax && smem_bytes<Form::kWeight>(256) <= kSmemMax, "seven stages");
static_assert(Cfg<Form::kInput>::kStages <= kMaxStages && Cfg<Form::kNarrow>::kStages <= kMaxStages, "stages");
static_assert(sizeof(GradTile) == 40, "a tile travels as five 8-byte stores");

__device__ __forceinline__ uint32_t dynamic_smem_size() {
    uint32_t n;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(n));
    return n;
}

template <Form F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    grouped_grad_kernel(const __grid_constant__ GradParams p) {
    using C = Cfg<F>;
    constexpr bool WG = C::kWeight;
    constexpr int kStages = C::kStages;
    // The swizzled stages need 1024 bytes' alignment.  Shared memory starts with that, and nothing is left to
    // align it with, so a start that has not is refused.  (Declared with the alignment, it compiles to a
    // kernel that takes 10% longer.)
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    if (pad + smem_bytes<F>(p.a.E) > dynamic_smem_size()) {
        wait_for_kernel_before();
        if (threadIdx.x == 0) report_error(p.a.status, kStDevice, -3, (int)raw, 0);
        if (threadIdx.x == 0 && blockIdx.x == 0 && p.split) p.split->count = 0;
        return;
    }
    uint8_t* sP = smem_raw + pad;
    uint8_t* sQ = sP + kStages * kOpBytes;
    GradCtl* ctl = reinterpret_cast<GradCtl*>(sQ + kStages * C::kQBytes);
    int* off = reinterpret_cast<int*>(ctl + 1);        // [E+1]
    int* base = off + p.a.E + 1;                       // [E+1] row tiles before expert e (input gradient)
    short* order = reinterpret_cast<short*>(base);     // [E] experts, most rows first (weight gradient)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = (rank & 1u) == 0u;
    const uint32_t lead = rank & ~1u, sched = rank | 1u;
    const int E = p.a.E;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
            mbar_init(smem_addr(&ctl->tail[s]), 1);
            mbar_init(smem_addr(&ctl->fixed[s]), 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_addr(&ctl->tfull[a]), 1);
            mbar_init(smem_addr(&ctl->tempty[a]), 2 * kEpiWarps);
        }
        for (int r = 0; r < kGradRing; ++r) {
            mbar_init(smem_addr(&ctl->sfull[r]), 1);
            // (the peer's) the leader's MMA thread, and of both CTAs warps 0, 2, the epilogue and warp 3
            mbar_init(smem_addr(&ctl->sempty[r]), 1 + 2 * (2 + kEpiWarps + (WG ? 1 : 0)));
        }
        mbar_init(smem_addr(&ctl->mma_done), 1);
        ctl->abort = 0;
        ctl->total_kb = 0;
        mbar_fence_init();
    }
    if (warp == 2) {
        tmem_alloc_pair(smem_addr(&ctl->tmem_base), 512);
        tmem_relinquish_pair();
    } else if (warp == 3 && lane == 0) {
        tma_prefetch_map(&p.p_map);
        tma_prefetch_map(&p.q_map);
    }
    // what is above runs beside the end of the kernel before this one in the stream
    wait_for_kernel_before();
    // offsets have to ascend from 0 to S: they bound every access
    int bad = 0;
    for (int e = tid; e <= E; e += kGradThreads) {
        const int v = __ldg(p.a.offsets + e);
        off[e] = v;
        bad |= e == 0 ? v != 0 : v < __ldg(p.a.offsets + e - 1);
        bad |= e == E && v != p.a.S;
    }
    bad = __syncthreads_or(bad);
    if (WG) {
        // longest reductions first, so that none is left for the end
        for (int e = tid; e < E; e += kGradThreads) {
            const int cnt = off[e + 1] - off[e];
            if (cnt > 0) atomicAdd(&ctl->total_kb, blocks_of<F>(p, cnt));
            int before = 0, prev = off[0];
            for (int f = 0; f < E; ++f) {
                const int nx = off[f + 1], n = nx - prev;
                prev = nx;
                before += (n > cnt) || (n == cnt && f < e);
            }
            order[before] = (short)e;
        }
    } else if (warp == 0) {
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? steps_of(off[e + 1] - off[e], C::kRowTile) : 0;
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
    __syncthreads();
    if (tid == 0) {  // a pair's first item is its own number: both CTAs know it without a claim
        plan_pieces<F>(p, ctl, off, base, order, blockIdx.x == 0 && !bad);
        if (bad && p.split && blockIdx.x == 0) p.split->count = 0;
        if (!bad) ctl->ring[0] = item_at<F>(p, ctl, off, base, order, blockIdx.x / 2, leader);
        mbar_arrive(smem_addr(&ctl->sfull[0]));
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers and TMEM address of both CTAs are there
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const long long timeout = p.a.timeout_ns * 2 > 500000000LL ? p.a.timeout_ns * 2 : 500000000LL;
    const Wait w{&ctl->abort, p.a.status, timeout};

    // 384 threads x 168 registers: the four warps of single threads hand some to the epilogue's
    if (warp < kEpiFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (!bad) {
            if (warp == 0) {
                if (lane == 0) producer_p<F>(p, ctl, sP, w, leader, sched, lead, rank);
            } else if (warp == 1) {
                if (lane == 0) {
                    if (leader) mma_role<F>(p, ctl, sP, sQ, tmem, w, sched);
                    else scheduler<F>(p, ctl, off, base, order, w, lead);
                }
            } else if (warp == 2) {
                if (lane == 0) producer_q<F>(p, ctl, sQ, w, leader, sched, lead, rank);
            } else if (WG) {
                zero_rows<F>(p, ctl, sP, sQ, w, leader, sched, lead);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        if (!bad) epilogue_role<F>(p, ctl, tmem, w, leader, sched, lead, rank);
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its peer may still signal it
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    // (the wait for the last claim's return, 0.7 us, is what a small product's end would otherwise be)
    if (tid == 0 && !ctl->one_round) {
        __threadfence();
        const uint32_t prev = atomicAdd(p.a.hdr + kHdrDoneCtr, 1u);
        if (prev == gridDim.x - 1) {  // every CTA has finished with the counters
            __threadfence();
            p.a.hdr[kHdrTileCtr] = 0u;
            p.a.hdr[kHdrDoneCtr] = 0u;
            __threadfence();
        }
    }
}

// Adds the pieces of the split tiles in their order and stores (or adds) the results: 64 threads a
// row of 256 columns, four rows a CTA at a time.
constexpr int kJoinThreads = 256;
template <Form F>
__global__ void __launch_bounds__(kJoinThreads) join_pieces_kernel(const SplitArea* split, const float* slots, void* out,
                                                                   long long out_rows, int n_slots, int c_size,
                                                                   int out_bf16, int accumulate) {
    constexpr int kRow = Cfg<F>::kRowTile;
    wait_for_kernel_before();
    const int count = min(__ldcg(&split->count), kMaxSplit);
    const int c = (threadIdx.x & 63) * 4;
    for (int u = blockIdx.x; u < count * (kRow / 4); u += gridDim.x) {
        const SplitTile* t = split->tile + u / (kRow / 4);
        const int row = u % (kRow / 4) * 4 + (threadIdx.x >> 6);
        const long long out_row = __ldcg(&t->out_row);
        const int c0 = __ldcg(&t->c0), rows = __ldcg(&t->rows), slot0 = __ldcg(&t->slot0), n = __ldcg(&t->n), stride = __ldcg(&t->stride);
        if (!inside(out_row, c0, rows, slot0, n, stride, out_rows, kRow, n_slots)) continue;
        const int col = c0 + c;
        if (row >= rows || col >= c_size) continue;  // c_size % 16 == 0
        const size_t step = (size_t)stride * kRow * 256;
        const float* at = slots + ((size_t)slot0 * kRow + row) * 256 + c;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(at + i * step));
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
        }
        const size_t o = (size_t)(out_row + row) * c_size + col;
        if (out_bf16) {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
        } else {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
            if (accumulate) {
                const float4 x = *dst;
                v = make_float4(x.x + v.x, x.y + v.y, x.z + v.z, x.w + v.w);
            }
            *dst = v;
        }
    }
}

// Pairs of CTAs that are resident together on the current device; the kernel's attributes are set once per device.
template <Form F>
cudaError_t resident_pairs(int device, int* pairs) {
    static std::atomic<int> known[64];
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    *pairs = known[device].load(std::memory_order_acquire);
    if (*pairs > 0) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(grouped_grad_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kGradThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(pairs, grouped_grad_kernel<F>, &cfg);
    if (e != cudaSuccess) return e;
    if (*pairs < 1) return cudaErrorLaunchOutOfResources;
    known[device].store(*pairs, std::memory_order_release);
    return cudaSuccess;
}

template <Form F>
cudaError_t launch(GradParams& p, const GroupedGradArgs& a, bool may_split, int device, int sm_count, long long max_tiles,
                   cudaStream_t stream) {
    p.a = a;
    p.chunk_kb = a.out_bf16 ? 1 << 30 : kChunkKb;
    int pairs = 0;
    cudaError_t e = resident_pairs<F>(device, &pairs);
    if (e != cudaSuccess) return e;
    if (may_split && a.split) {
        p.split = static_cast<SplitArea*>(a.split);
        p.slots = reinterpret_cast<float*>(p.split + 1);
    } else {
        pairs = (int)std::min<long long>(pairs, max_tiles);
    }
    e = launch_after(grouped_grad_kernel<F>, 2u * pairs, kGradThreads, smem_bytes<F>(a.E), stream, (const GradParams&)p);
    if (e == cudaSuccess && p.split)
        e = launch_after(join_pieces_kernel<F>, (unsigned)sm_count, kJoinThreads, 0, stream, (const SplitArea*)p.split,
                         (const float*)p.slots, a.out, Cfg<F>::kWeight ? (long long)a.E * a.d : (long long)a.S, sm_count,
                         p.c_size, a.out_bf16, a.accumulate);
    return e;
}

// Row tiles of 64 where that is an expert's mean or more: the ten stages in flight read the weights faster (64
// experts of 2048 x 2048 with 64 rows each: 92 us, 94 in tiles of 256; with 8 rows 86 and 89), and with more rows
// they are read twice (80 rows: 118 and 96).  These are equal loads: the mean decides for all experts, and one with more than
// 64 rows beside many with few reads its weights once for each 64 of them.
bool narrow_rows(long long S, int E) { return S <= 64LL * E; }
// Whether an input (weight) gradient of this shape may have fewer tiles than pairs of CTAs and a reduction long
// enough to be split.
bool dgrad_may_split(long long S, int d, int E, int N, int sm_count) {
    const long long rows = narrow_rows(S, E) ? 64 : 256, tiles = (S + rows - 1) / rows * ((d + 255) / 256);
    return N > (narrow_rows(S, E) ? Cfg<Form::kNarrow>::kMinSplit : Cfg<Form::kInput>::kMinSplit) * kTileK && tiles < sm_count / 2;
}
bool wgrad_may_split(long long S, int d, int N, int sm_count) {
    const long long tiles = (long long)((d + 255) / 256) * ((N + 255) / 256);
    return S > Cfg<Form::kWeight>::kMinSplit * kTileK && tiles < sm_count / 2;
}

template <Form F>
cudaError_t dgrad(const GroupedGradArgs& a, int device, int sm_count, cudaStream_t stream) {
    GradParams p = {};
    p.c_size = a.d;
    p.c_tiles = (a.d + 255) / 256;
    const uint64_t S = (uint64_t)a.S, N = (uint64_t)a.N, wrows = (uint64_t)a.E * a.d;
    if (!map_bf16_2d(&p.p_map, a.W, wrows, N, kTileK, kTileM) ||
        !map_bf16_2d(&p.q_map, a.dY, S, N, kTileK, Cfg<F>::kRowTile / 2) || !map_bf16_2d(&p.q_tail, a.dY, S, N, kTileK, 16))
        return cudaErrorInvalidValue;
    return launch<F>(p, a, dgrad_may_split(a.S, a.d, a.E, a.N, sm_count), device, sm_count,
                     ((long long)a.S / Cfg<F>::kRowTile + a.E) * p.c_tiles, stream);
}

}  // namespace

// Workspace bytes for the pieces of split reductions: no piece is longer than a pair's share of all the work, so
// there are at most two for each pair of CTAs.
size_t grouped_grad_split_bytes(long long S, int d, int E, int N, int sm_count) {
    size_t tile = 0;
    if (dgrad_may_split(S, d, E, N, sm_count)) tile = narrow_rows(S, E) ? 64 : 256;
    if (wgrad_may_split(S, d, N, sm_count)) tile = 256;
    return tile == 0 ? 0 : sizeof(SplitArea) + (size_t)sm_count * tile * 256 * 4;
}

cudaError_t launch_grouped_dgrad(const GroupedGradArgs& a, int device, int sm_count, cudaStream_t stream) {
    if (narrow_rows(a.S, a.E)) return dgrad<Form::kNarrow>(a, device, sm_count, stream);
    return smem_bytes<Form::kInput>(a.E) <= kSmemMax ? dgrad<Form::kInput>(a, device, sm_count, stream)
                                                     : dgrad<Form::kInputMany>(a, device, sm_count, stream);
}

cudaError_t launch_grouped_wgrad(const GroupedGradArgs& a, int device, int sm_count, cudaStream_t stream) {
    GradParams p = {};
    p.c_size = a.N;
    p.c_tiles = (a.N + 255) / 256;
    p.r_tiles = (a.d + 255) / 256;
    const uint64_t S = (uint64_t)a.S, N = (uint64_t)a.N, d = (uint64_t)a.d;
    if (!map_bf16_2d(&p.p_map, a.dY, S, N, 64, kTileK) || !map_bf16_2d(&p.q_map, a.A, S, d, 64, kTileK))
        return cudaErrorInvalidValue;
    p.p_paired = p.q_paired = 1;
    for (int i = 0; i < 3; ++i) {
        p.p_paired &= map_bf16_chunks(&p.p_pair[i], a.dY, S, N, kTileK >> i);
        p.q_paired &= map_bf16_chunks(&p.q_pair[i], a.A, S, d, kTileK >> i);
    }
    const long long tiles = (long long)a.E * p.c_tiles * p.r_tiles;
    if (tiles >= (1LL << 31)) return cudaErrorInvalidValue;
    const bool split = wgrad_may_split(a.S, a.d, a.N, sm_count);
    return smem_bytes<Form::kWeight>(a.E) <= kSmemMax ? launch<Form::kWeight>(p, a, split, device, sm_count, tiles, stream)
                                                      : launch<Form::kWeightMany>(p, a, split, device, sm_count, tiles, stream);
}

}  // namespace moe
