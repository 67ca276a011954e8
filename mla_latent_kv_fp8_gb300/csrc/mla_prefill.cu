// mla_prefill.cu -- attention of many new tokens per sequence over up-projected
// keys and values (device side), for sm_103a (GB300).
//
//   s_ij = sm_scale * (q_nope_i . k_nope_j + q_pe_i . k_pe_j), capped to
//   cap * tanh(s / cap) where a cap is given; out_i = sum_j softmax(s_i)_j v_j
//   and lse_i = ln sum_j exp(s_ij) over the keys that row i sees.
//
// A work item is 256 query rows of one head (two tiles of 128) and the key
// blocks (128 keys) that any of them sees, or one of n_splits parts of those.
// The rotated key part is shared by the heads, so a key block is three 64-dim
// chunks -- two of the head's own part, one of the shared part -- that meet in
// one score tile; no 192-wide key tensor is ever made.
//   * TMA brings 16 KB chunks (128 keys x 64 dims, 128-byte swizzle) into a ring
//     of eight, three for a block's keys and two for its values, each such group
//     with one full and one empty barrier; the query tiles stay in shared memory.
//   * tcgen05.mma: S_t = Q_t K^T (12 steps of 16 dims) and O_t += P_t V (8 steps
//     of 16 keys), P_t read from tensor memory.  While one tile's softmax runs,
//     the other tile's products run.
//   * One thread issues all copies and one thread per tile its products.  (All
//     by whole warps with warp-wide waits for each chunk: 5,800 cycles for a pair
//     of tile blocks whose products take 2,560; one thread for both tiles 3,700.)
//   * A softmax warpgroup per tile, one row per thread: no shuffles.  P replaces
//     S in tensor memory, and its first 64 keys are multiplied while the others
//     are still exponentials.  Online softmax with a reference that moves only
//     when a score exceeds it by 8 (log2 units), so the accumulated O_t is rarely
//     rescaled; probabilities are at most 2^8 and are rounded to bf16 for the
//     product (off by at most 2^-8 of their value, like the output itself); their
//     sum is taken in fp32 before the rounding.
//   * Four output warps scale and write an item's answer while the softmax and
//     the products of the next item run.
//   * An item with at most 128 rows would leave a tile idle and run the other one
//     without overlap: both tiles then take the same rows, tile 0 the even and
//     tile 1 the odd entries of the block list, and the output warps join the two
//     answers ("halves").
//   * TMEM: 2 x 128 columns of scores + 2 x 128 of output = all 512.
//   * The grid has one CTA per item, but a running CTA takes the next item itself
//     by cancelling the launch of a CTA that has not started, so that the start
//     of an item overlaps the end of the one before and the SMs stay busy
//     whatever the items' lengths.  A planner warp turns item numbers into
//     sequences and key ranges, one ahead of the other warps.
// Warps: 0 TMA producer, 1 and 3 MMA issuers, 2 planner, 4-7 and 8-11 softmax,
// 12-15 output.  A softmax thread holds a row of 128 scores: the other warps
// hand registers over (128 x 64 + 128 x 80 + 256 x 184 = 512 x 128, what the
// launch has; with 72 and 72 the output warps spilled: 4 x 1,000 tokens x 12
// heads 28.8 us, with 64 and 80 28.0.  The kernel with packed caps still spills
// five registers, the others none).
// Every wait is bounded; on a timeout the kernel sets the error word, drains
// its copies and products, frees its tensor memory and returns.
//
// Measured on a GB300 (bursts of graph replays; the products alone at the rate of
// a large library product, 1,861 TFLOP/s, would take 554 us in the first case):
// 16,384 causal tokens x 12 heads 560 us (1,840 TFLOP/s, bound by the tensor core
// and the power limit, which makes it 630 in calls back to back); 16 documents, 8,192 tokens 48 us, 4,000 tokens 50
// and 300 tokens over 98,000 191: bound by the chain score - softmax - product of
// a tile block, ~2,850 cycles of which the products are 1,280, and by the start
// and end of items; with a cap by a chain of twice that length, 2,000 cycles of it
// for the cap (8,192 tokens x 12 heads 276 us, without the cap 159).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "mla_host.h"
#include "mla_prefill.cuh"
#include "mla_ragged.cuh"
#include "mla_tc_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;                    // rows of a query tile
constexpr int kKeys = kPfBlock;               // keys of a block
constexpr int kChunk = kKeys * 64 * 2;        // 16,384 bytes: 128 rows x 64 dims
constexpr int kQChunks = kPfHead / 64;        // 3
constexpr int kVChunks = kPfV / 64;           // 2
constexpr int kPerBlock = kQChunks + kVChunks;
constexpr int kSlots = 8;
// Chunk groups (a block's keys, or its values) in the order of their use.  Any
// three in a row have at most eight chunks, so a group's chunks lie where those
// of the groups up to the third before it were: three barriers of each kind.
constexpr int kGroups = 3;
constexpr int kPlans = 2;                     // plans in flight
constexpr int kReaders = 15;                  // producer, two issuers, eight softmax and four output warps
// Blocks before an item's end at which the next item is asked for: asking and
// planning take 1.6 us, a block of two tiles 1.3 and one of an item in halves
// 0.8.  Asking sooner would hand the items out before it is known which SM is
// free first: 2,000 causal tokens x 12 heads took 28.6 us with the question at
// an item's start and take 24.1.
constexpr int kAskAhead = 4, kAskAheadHalves = 6;
constexpr uint32_t kCols = 512;
constexpr uint32_t kOCol = 256;               // O tile t at 256 + 128 t, S tile t at 128 t
constexpr float kHeadroom = 8.f;
constexpr uint32_t kLayoutSw128 = 2;

// One work item, as the planner lays it out for the other warps.
struct Plan {
    int h;                                    // head; -1: no more items
    int split;
    int q0, i0, rows, nq;                     // first row of the sequence, of the item in it; rows; the sequence's
    int k0, nk, prefix;
    int it0, n;                               // first entry of the block list, entries
    int n_first, lo;                          // entry e is block e < n_first ? e : e - n_first + lo
    int lo0, hi0, lo1, hi1;                   // the tiles' block ranges (besides the prefix)
    int halves;                               // both tiles take the same rows, entries in turn
    __device__ __forceinline__ int block(int e) const { return e < n_first ? e : e - n_first + lo; }
    __device__ __forceinline__ bool need(int t, int e) const {
        if (halves) return ((e - it0) & 1) == t;
        const int blk = block(e);
        return blk * kKeys < prefix || (blk >= (t ? lo1 : lo0) && blk < (t ? hi1 : hi0));
    }
};

struct PfSmem {
    uint8_t q[2][kQChunks][kChunk];
    uint8_t ring[kSlots][kChunk];
    Plan plan[kPlans];
    float row_m[2][kRows], row_l[2][kRows];   // an item's references and sums, for the output warps
    alignas(16) uint4 next;                   // answer to the request for another item
    uint64_t next_full;
    uint64_t plan_full[kPlans], plan_empty[kPlans];
    uint64_t q_full[2], q_empty[2];
    uint64_t full[kGroups], empty[kGroups];
    uint64_t s_full[2];                       // scores of the tile's next block are in TMEM
    uint64_t p_half[2], p_full[2];            // its probabilities are (64 keys, all), and O may be accumulated
    uint64_t o_done[2];                       // its PV product is done
    uint64_t o_ready[2], o_free[2];           // O is the item's answer / may be written again
    uint64_t rows_full[2], rows_free[2];      // row_m and row_l likewise
    uint64_t mma_done[2];
    uint64_t ask;                             // an item nears its end: time to ask for another
    uint32_t tmem_base;
    int abort;
};
constexpr int kSmemBytes = sizeof(PfSmem);   // no static shared memory: the dynamic part starts on 1 KB
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct Maps {
    CUtensorMap q, kn, kp, v;
};

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Instruction descriptor, kind::f16, A = B = bf16, D = f32, A K-major.
constexpr uint32_t idesc_bf16(int M, int N, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A from tensor memory: row = lane, two bf16 per column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 32 bytes to a 32-byte boundary in one access: a warp whose lanes write rows
// of their own needs half as many accesses.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// The n lowest bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Asks for a CTA of this grid that has not started yet; the answer (16 bytes)
// lands at `dst` and completes `bar`.
__device__ __forceinline__ void request_item(uint4* dst, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(dst)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The index of the CTA taken over, or -1: none was left.
__device__ __forceinline__ int64_t taken_item(const uint4* src) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
        "ld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(smem_u32(src))
        : "memory");
    return ok ? static_cast<int64_t>(x) : -1;
}

// As wait_bounded, for waits that may last as long as an item (the longest
// sequences that fit the memory take a few seconds).
__device__ __forceinline__ bool wait_item(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if ((it & 127u) == 127u && global_ns() - t0 > 30 * kTimeoutNs) {
            *abort = 1;
            atomicCAS(err, 0, kErrWaitTimeout);
            return false;
        }
    }
}

// ---------------------------------------------------------------- work items

__device__ __forceinline__ int row_tiles(const PrefillParams& p, const PrefillSeq& s) {
    return p.tile == kPfTile ? (s.nq + kPfTile - 1) / kPfTile : (s.nq + kPfTile / 2 - 1) / (kPfTile / 2);
}

// Item numbers run over the heads first, then the row tiles.  Row tiles of up
// to 32 sequences come in falling order of their place in the sequence (under
// a causal mask those with the most keys first), so that the last items are
// short; those of more sequences come sequence by sequence.  Parts (n_splits >
// 1) run over the row tiles first, then the heads: items that read the same
// keys run together and find them in L2.
struct Planner {
    int base = 0, before = 0;  // more than 32 sequences: the 32 last looked at, row tiles before them
    // up to 32 sequences: lane b keeps sequence b and its row tiles
    PrefillSeq kept{};
    int mine = 0, tiles = 0, most = 0;

    __device__ __forceinline__ Planner(const PrefillParams& p, int lane, bool used) {
        if (p.B > 32 || !used) return;
        if (lane < p.B) {
            kept = prefill_seq(p, lane, false);
            mine = row_tiles(p, kept);
        }
        tiles = __reduce_add_sync(0xffffffffu, mine);
        most = __reduce_max_sync(0xffffffffu, mine);
    }

    // Sequence b, in every lane.
    __device__ __forceinline__ PrefillSeq sequence(const PrefillParams& p, int b) const {
        if (p.B > 32) return prefill_seq(p, b, false);
        PrefillSeq s;
        s.q0 = __shfl_sync(0xffffffffu, kept.q0, b);
        s.k0 = __shfl_sync(0xffffffffu, kept.k0, b);
        s.nq = __shfl_sync(0xffffffffu, kept.nq, b);
        s.nk = __shfl_sync(0xffffffffu, kept.nk, b);
        s.prefix = __shfl_sync(0xffffffffu, kept.prefix, b);
        s.ok = true;
        return s;
    }

    // Head, part and row tile number of an item; false: there is no such item.
    __device__ __forceinline__ bool place(const PrefillParams& p, int64_t id, int* h, int* split, int* k) const {
        if (p.B > 32) {
            const int w = static_cast<int>(id / p.H);
            *h = static_cast<int>(id - (int64_t)w * p.H);
            *split = w % p.n_splits;
            *k = w / p.n_splits;
            return true;
        }
        if (id >= (int64_t)tiles * p.n_splits * p.H) return false;
        const int w = static_cast<int>(id);
        if (p.n_splits == 1) {
            *h = w % p.H;
            *k = w / p.H;
            *split = 0;
        } else {
            *k = w % tiles;
            *h = w / tiles % p.H;
            *split = w / tiles / p.H;
        }
        return true;
    }

    // The sequence and row tile of the k-th row tile; false: there is none.
    __device__ __forceinline__ bool find(const PrefillParams& p, int k, int lane, int* seq, int* tile) {
        if (p.B <= 32) {
            if (k >= tiles) return false;
            auto from = [&](int t) {  // row tiles with a place >= t
                return __reduce_add_sync(0xffffffffu, max(0, mine - t));
            };
            int lo = 0, hi = most;  // from(lo) > k >= from(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (from(mid) > k)
                    lo = mid;
                else
                    hi = mid;
            }
            // the nth of the sequences with a row tile there
            const int nth = k - from(lo + 1);
            const unsigned m = __ballot_sync(0xffffffffu, mine > lo);
            const bool me = mine > lo && __popc(m & ((1u << lane) - 1u)) == nth;
            *seq = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
            *tile = lo;
            return true;
        }
        if (k < before) base = before = 0;  // (items come in rising order)
        while (base < p.B) {
            const int b = base + lane;
            const int mine = b < p.B ? row_tiles(p, prefill_seq(p, b, false)) : 0;
            int sum = mine;  // inclusive prefix sum
#pragma unroll
            for (int sh = 1; sh < 32; sh <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, sh);
                if (lane >= sh) sum += up;
            }
            const int all = __shfl_sync(0xffffffffu, sum, 31);
            if (k < before + all) {
                const unsigned m = __ballot_sync(0xffffffffu, k < before + sum);
                const int at = __ffs(m) - 1;
                *seq = base + at;
                *tile = k - before - __shfl_sync(0xffffffffu, sum - mine, at);
                return true;
            }
            before += all;
            base += 32;
        }
        return false;
    }
};

__device__ __forceinline__ void block_range(const PrefillParams& p, const PrefillSeq& s, int i0, int rows, int* lo,
                                            int* hi) {
    *lo = *hi = 0;
    if (rows <= 0) return;
    int l, h, unused;
    prefill_range(p, s, i0, &l, &unused);              // the first row's start
    prefill_range(p, s, i0 + rows - 1, &unused, &h);   // the last row's end
    if (l < h) *lo = l / kKeys, *hi = (h + kKeys - 1) / kKeys;
}

__device__ __forceinline__ Plan make_plan(const PrefillParams& p, const PrefillSeq& s, int tile, int split, int h) {
    Plan a;
    a.h = h;
    a.split = split;
    a.q0 = s.q0;
    a.i0 = tile * p.tile;
    a.rows = min(p.tile, s.nq - a.i0);
    a.nq = s.nq;
    a.k0 = s.k0;
    a.nk = s.nk;
    a.prefix = s.prefix;
    a.halves = a.rows <= kRows;
    block_range(p, s, a.i0, min(a.rows, kRows), &a.lo0, &a.hi0);
    block_range(p, s, a.i0 + kRows, a.rows - kRows, &a.lo1, &a.hi1);
    // blocks of either tile: the ranges of neighbouring rows touch or overlap
    const bool any0 = a.hi0 > a.lo0, any1 = a.hi1 > a.lo1;
    a.lo = any0 ? a.lo0 : (any1 ? a.lo1 : 0);
    int hi = any1 ? max(a.hi1, a.hi0) : (any0 ? a.hi0 : 0);
    const int pre = (s.prefix + kKeys - 1) / kKeys;
    a.n_first = min(pre, a.lo);
    if (pre > a.lo) hi = max(hi, pre);
    const int all = a.n_first + max(0, hi - a.lo);
    const int part = p.n_splits == 1 ? all : (all + p.n_splits - 1) / p.n_splits;
    a.it0 = min(all, split * part);
    a.n = min(all, a.it0 + part) - a.it0;
    return a;
}

// An item without a block: its rows see no key (of their part).  The other
// warps never hear of it.
__device__ __forceinline__ void write_empty(const PrefillParams& p, const Plan& a, int lane) {
    if (p.n_splits > 1) {  // the join does not read the values of such a part
        for (int r = lane; r < a.rows; r += 32)
            p.part_lse[((int64_t)a.split * p.Nq + a.q0 + a.i0 + r) * p.H + a.h] = -INFINITY;
        return;
    }
    for (int r = lane >> 4; r < a.rows; r += 2) {
        const int64_t row = (int64_t)a.q0 + a.i0 + r;
        reinterpret_cast<uint4*>(p.out + row * p.out_tok + a.h * p.out_head)[lane & 15] = make_uint4(0, 0, 0, 0);
        if (p.lse && (lane & 15) == 0) p.lse[row * p.H + a.h] = -INFINITY;
    }
}

// ---------------------------------------------------------------- kernel

// How scores are capped.  The packed form is off by up to softcap * 2^-20 and
// holds a score as a difference to the cap, so it serves caps up to 64 (6e-5);
// beyond, each score is taken through tanhf, whose error goes by the score.
// Both on 8,192 causal tokens x 12 heads: 281 and 425 us (169 without a cap).
// lse off by up to 4e-6 at a cap of 64 (packed), 2.6e-4 at 4,096 by the packed
// form and 1e-6 by tanhf.
constexpr int kCapNone = 0, kCapPacked = 1, kCapTanh = 2;
constexpr float kPackedCapMost = 64.f;

template <int kCap>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ Maps maps, const PrefillParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    PfSmem& S = *reinterpret_cast<PfSmem*>(smem_raw);
    if (smem_u32(smem_raw) & 1023) {  // the swizzled tiles need it; never seen
        if (threadIdx.x == 0) atomicCAS(p.err, 0, kErrWaitTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &S.abort;

    if (tid == 0) {
        mbar_init(&S.next_full, 1);
        for (int i = 0; i < kPlans; ++i) {
            mbar_init(&S.plan_full[i], 1);
            mbar_init(&S.plan_empty[i], kReaders);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&S.q_full[t], 1);
            mbar_init(&S.q_empty[t], 2 - t);
            mbar_init(&S.mma_done[t], 1);
            mbar_init(&S.s_full[t], 1);
            mbar_init(&S.p_half[t], 4);
            mbar_init(&S.p_full[t], 4);
            mbar_init(&S.o_done[t], 1);
            mbar_init(&S.o_ready[t], 1);
            mbar_init(&S.o_free[t], 4);
            mbar_init(&S.rows_full[t], 4);
            mbar_init(&S.rows_free[t], 4);
        }
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 2);
        }
        mbar_init(&S.ask, 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&maps.q);
        if (p.Nk > 0) {
            prefetch_map(&maps.kn);
            prefetch_map(&maps.kp);
            prefetch_map(&maps.v);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)),
                     "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Up to here nothing was read: this much overlaps the stream's previous kernel.
    wait_for_previous();
    Planner planner(p, lane, warp == 2);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ======================= TMA producer =======================
        if (elect_one()) {
            int g = 0, s = 0;              // next group and slot
            int used0 = 0, used1 = 0;      // loads of each query tile
            bool ok = true;
            auto next_slot = [&] {
                const uint32_t dst = smem_u32(S.ring[s]);
                s = (s + 1) % kSlots;
                return dst;
            };
            for (int item = 0; ok && !p.test_stall_copies; ++item) {
                const int sl = item % kPlans;
                if (!wait_bounded(&S.plan_full[sl], (item / kPlans) & 1, abort, p.err)) break;
                const Plan a = S.plan[sl];
                mbar_arrive(&S.plan_empty[sl]);
                if (a.h < 0) break;
                auto load_q = [&](int t, int used) {
                    if (!wait_bounded(&S.q_empty[t], (used & 1) ^ 1, abort, p.err)) return false;
                    mbar_expect_tx(&S.q_full[t], kQChunks * kChunk);
                    for (int d = 0; d < kQChunks; ++d)
                        tma_load3(smem_u32(S.q[t][d]), &maps.q, 64 * d, a.h, a.q0 + a.i0 + kRows * t, &S.q_full[t]);
                    return true;
                };
                auto load_k = [&](int i) {
                    if (!wait_bounded(&S.empty[g % kGroups], ((g / kGroups) & 1) ^ 1, abort, p.err)) return false;
                    const int key = a.k0 + a.block(a.it0 + i) * kKeys;
                    uint64_t* bar = &S.full[g % kGroups];
                    mbar_expect_tx(bar, kQChunks * kChunk);
                    tma_load3(next_slot(), &maps.kn, 0, a.h, key, bar);
                    tma_load3(next_slot(), &maps.kn, 64, a.h, key, bar);
                    tma_load3(next_slot(), &maps.kp, 0, 0, key, bar);
                    ++g;
                    return true;
                };
                auto load_v = [&](int i) {
                    if (!wait_bounded(&S.empty[g % kGroups], ((g / kGroups) & 1) ^ 1, abort, p.err)) return false;
                    const int key = a.k0 + a.block(a.it0 + i) * kKeys;
                    uint64_t* bar = &S.full[g % kGroups];
                    mbar_expect_tx(bar, kVChunks * kChunk);
                    tma_load3(next_slot(), &maps.v, 0, a.h, key, bar);
                    tma_load3(next_slot(), &maps.v, 64, a.h, key, bar);
                    ++g;
                    return true;
                };
                // the ring's first groups are free before the query tiles are
                ok = load_k(0);
                ok = ok && load_q(0, used0);
                used0 += ok;
                if (!a.halves) {
                    ok = ok && load_q(1, used1);
                    used1 += ok;
                    for (int i = 0; i < a.n && ok; ++i) ok = (i == 0 || load_k(i)) && load_v(i);
                } else {
                    if (a.n > 1) ok = ok && load_k(1);
                    for (int i = 0; i < a.n && ok; ++i) ok = load_v(i) && (i + 2 >= a.n || load_k(i + 2));
                }
            }
            // never leave with a copy in flight into this CTA's shared memory
            const uint64_t t0 = global_ns();
            while (used0 > 0 && !mbar_try_wait(&S.q_full[0], (used0 - 1) & 1) && global_ns() - t0 < kTimeoutNs) {
            }
            while (used1 > 0 && !mbar_try_wait(&S.q_full[1], (used1 - 1) & 1) && global_ns() - t0 < kTimeoutNs) {
            }
            for (int i = max(0, g - kGroups); i < g; ++i)
                while (!mbar_try_wait(&S.full[i % kGroups], (i / kGroups) & 1) && global_ns() - t0 < kTimeoutNs) {
                }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ======================= MMA issuers =======================
        // One thread for each tile.  Both walk all groups of the ring in order and
        // release each (a group is free when both have); products of one tile are
        // issued by one thread and so run in the order of their issue.
        const int t = warp >> 1;
        if (elect_one()) {
            constexpr uint32_t kIdQk = idesc_bf16(kRows, kKeys, false);
            constexpr uint32_t kIdPv = idesc_bf16(kRows, kPfV, true);
            constexpr uint32_t kIdPvHalf = idesc_bf16(kRows, 64, true);
            const uint64_t ring = smem_desc(smem_u32(S.ring[0]), kChunk, 1024, kLayoutSw128);
            const uint64_t queries = smem_desc(smem_u32(S.q[0][0]), kChunk, 1024, kLayoutSw128);
            constexpr uint64_t kStep = kChunk >> 4;  // a chunk, in descriptor units
            const uint32_t ts = tmem + kRows * t, to = tmem + kOCol + kPfV * t;
            int g = 0, s = 0;             // next group and slot
            int used0 = 0, used1 = 0;     // loads of each query buffer
            int taken = 0;                // blocks whose probabilities were taken
            int answers = 0;              // items done
            auto group_full = [&] { return wait_bounded(&S.full[g % kGroups], (g / kGroups) & 1, abort, p.err); };
            auto pass = [&](bool used, int chunks) {  // release the group
                if (used)
                    mma_commit(&S.empty[g % kGroups]);
                else
                    mbar_arrive(&S.empty[g % kGroups]);
                ++g;
                s = (s + chunks) % kSlots;
            };
            // S = Q K^T of the query tile in buffer `buf` and the key chunks at slot s
            auto qk = [&](int buf) {
                const uint64_t ad = queries + (buf ? kQChunks * kStep : 0);
#pragma unroll
                for (int d = 0; d < kQChunks; ++d) {
                    const uint64_t bd = ring + kStep * ((s + d) % kSlots);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ss(ts, ad + kStep * d + 2 * k, bd + 2 * k, kIdQk, d > 0 || k > 0);
                }
                mma_commit(&S.s_full[t]);
            };
            // O += P V of the value chunks at slot s, 64 keys (half `half`) at a time
            auto pv = [&](int half, bool first) {
                // MN-major: 64 values of a key are one 128-byte row, 8 keys an
                // atom of 1 KB; SBO = next 8 keys, LBO = the other 64 values.
                const uint64_t b0 = ring + kStep * s + 512 * half, b1 = ring + 512 * half;
                const uint32_t pr = ts + 32 * half;
                if (s != kSlots - 1) {  // the two chunks are neighbours
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ts(to, pr + 8 * k, b0 + 128 * k, kIdPv, !first || k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma_bf16_ts(to, pr + 8 * k, b0 + 128 * k, kIdPvHalf, !first || k > 0);
                        mma_bf16_ts(to + 64, pr + 8 * k, b1 + 128 * k, kIdPvHalf, !first || k > 0);
                    }
                }
            };
            // One group of keys: scores if the tile needs the block.
            auto keys = [&](bool need, int buf) {
                if (!group_full()) return false;
                if (need) qk(buf);
                pass(need, kQChunks);
                return true;
            };
            // One group of values; the item's first one waits until the last item's
            // output was read (whether the tile needs the block or not: a parity
            // tells a phase from its neighbours only).
            auto values = [&](bool need, bool begins, bool& first) {
                if (begins && !wait_bounded(&S.o_free[t], (answers & 1) ^ 1, abort, p.err)) return false;
                if (!group_full()) return false;
                if (need) {
                    if (!wait_bounded(&S.p_half[t], taken & 1, abort, p.err)) return false;
                    tc_fence_after();
                    pv(0, first);
                    if (!wait_bounded(&S.p_full[t], taken & 1, abort, p.err)) return false;
                    tc_fence_after();
                    pv(1, false);
                    mma_commit(&S.o_done[t]);
                    ++taken;
                    first = false;
                }
                pass(need, kVChunks);
                return true;
            };
            // After the item's last product.
            auto answer = [&] {
                mma_commit(&S.o_ready[t]);
                ++answers;
            };
            bool ok = true;
            int item = 0;
            // the next item (h < 0: there is none)
            auto fetch = [&] {
                const int sl = item % kPlans;
                ok = wait_bounded(&S.plan_full[sl], (item / kPlans) & 1, abort, p.err);
                Plan a;
                a.h = -1;
                if (ok) {
                    a = S.plan[sl];
                    mbar_arrive(&S.plan_empty[sl]);
                    ++item;
                }
                return a;
            };
            // Waits for the item's queries (thread 1 for every load of buffer 0 too: a
            // parity tells a phase from its neighbours only).
            auto start = [&](const Plan& a) {
                ok = wait_bounded(&S.q_full[0], used0++ & 1, abort, p.err);
                if (ok && !a.halves && t == 1) {
                    mbar_arrive(&S.q_empty[0]);
                    ok = wait_bounded(&S.q_full[1], used1++ & 1, abort, p.err);
                }
                return ok;
            };
            // After the tile's last scores of the item its query buffer is free: buffer
            // 1 is thread 1's alone, buffer 0 thread 0's and, in halves, both threads'
            // (else thread 1 lets go of it at once; it cannot be a phase ahead, because
            // it waits for every load of buffer 0).
            auto finish = [&](const Plan& a) {
                if (t == 0 || a.halves) mma_commit(&S.q_empty[0]);
                if (t == 1 && !a.halves) mma_commit(&S.q_empty[1]);
            };
            Plan a = fetch();
            bool primed = false;  // the first scores of `a` were issued with the item before
            while (ok && a.h >= 0) {
                bool first = true;
                Plan b;
                if (a.halves) {
                    // Tile e & 1 takes entry e of the list; keys run two entries ahead.
                    if (!start(a) || !keys(t == 0, 0)) break;
                    if (a.n > 1 && !keys(t == 1, 0)) break;
                    if (a.n <= 2) finish(a);
                    for (int i = 0; i < a.n && ok; ++i) {
                        const bool mine = (i & 1) == t;
                        if (t == 0 && i == max(0, a.n - kAskAheadHalves)) mbar_arrive(&S.ask);
                        ok = values(mine, i == 0, first) && (i + 2 >= a.n || keys(mine, 0));
                        if (ok && i + 3 == a.n) finish(a);  // the last scores were issued
                    }
                    if (!ok) break;
                    answer();
                    a = fetch();
                    continue;
                }
                bool now = a.need(t, a.it0), next = now;
                if (!primed) {
                    if (!start(a) || !keys(now, t)) break;
                    if (a.n == 1) finish(a);
                }
                // Step i multiplies block i's probabilities and scores block i + 1; after
                // the item's last block come the first scores of the next item, so that
                // its softmax need not wait for this one's output.
                for (int i = 0; i < a.n; ++i) {
                    if (t == 0 && i == max(0, a.n - kAskAhead)) mbar_arrive(&S.ask);
                    const bool inside = i + 1 < a.n;
                    if (inside) {
                        next = a.need(t, a.it0 + i + 1);
                    } else {
                        b = fetch();
                        if (!ok) break;
                        primed = b.h >= 0 && !b.halves;
                        if (primed) next = b.need(t, b.it0);
                    }
                    if (!(ok = values(now, i == 0, first))) break;
                    if (!inside) answer();
                    if (inside) {
                        if (!(ok = keys(next, t))) break;
                        if (i + 2 == a.n) finish(a);
                    } else if (primed) {
                        if (!start(b) || !(ok = keys(next, t))) break;
                        if (b.n == 1) finish(b);
                    }
                    now = next;
                }
                if (!ok) break;
                a = b;
            }
            mma_commit(&S.mma_done[t]);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(&S.mma_done[t], 0) && global_ns() - t0 < kTimeoutNs) {
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ======================= planner =======================
        int64_t id = blockIdx.x;
        int published = 0;
        auto publish = [&](const Plan& a) {
            const int sl = published % kPlans;
            const bool ok = __all_sync(0xffffffffu, wait_item(&S.plan_empty[sl], ((published / kPlans) & 1) ^ 1, abort, p.err));
            if (ok && lane == 0) {
                S.plan[sl] = a;
                mbar_arrive(&S.plan_full[sl]);
            }
            __syncwarp();
            ++published;
            return ok;
        };
        bool ok = true;
        for (int n = 0; ok; ++n) {
            int h, split, k, seq, tile;
            bool some = planner.place(p, id, &h, &split, &k) && planner.find(p, k, lane, &seq, &tile);
            if (some) {
                const Plan a = make_plan(p, planner.sequence(p, seq), tile, split, h);
                some = a.n > 0;
                if (some)
                    ok = publish(a);
                else
                    write_empty(p, a, lane);
            }
            if (id == 0)  // one CTA reports the sequences that are left out
                for (int b = lane; b < p.B; b += 32) prefill_seq(p, b, true);
            __syncwarp();
            if (some && ok) ok = __all_sync(0xffffffffu, wait_item(&S.ask, (published - 1) & 1, abort, p.err));
            if (!ok) break;
            if (lane == 0) {
                fence_async_smem();  // the last answer was read
                mbar_expect_tx(&S.next_full, 16);
                request_item(&S.next, &S.next_full);
            }
            // (the answer is a copy into shared memory: never left in flight)
            if (!warp_wait(&S.next_full, n & 1, abort, p.err)) {
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(&S.next_full, n & 1) && global_ns() - t0 < kTimeoutNs) {
                }
                break;
            }
            id = taken_item(&S.next);
            __syncwarp();
            if (id < 0) break;
        }
        Plan end;
        end.h = -1;
        publish(end);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ======================= softmax warpgroups =======================
        const int t = (warp - 4) >> 2, quad = warp & 3;  // a warp reads the TMEM lanes 32 (warp % 4) ..
        const int r = 32 * quad + lane;                  // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const uint32_t ts = tmem + lanes + kRows * t, to = tmem + lanes + kOCol + kPfV * t;
        const float scale = kCap == kCapPacked ? 2.f * kLog2e * p.cap : kCap == kCapTanh ? kLog2e : p.scale_log2;
        // argument of the cap: 2 s / cap in log2 units, or s / cap
        const float cap_in = kCap == kCapPacked ? 2.f * p.scale_log2 / p.cap : kCap == kCapTanh ? p.scale_log2 * kLn2 / p.cap : 0.f;
        int n = 0;         // blocks of this tile so far, over all items
        int entries = 0;   // entries of both tiles
        bool fail = false;
        for (int item = 0; !fail; ++item) {
            const int sl = item % kPlans;
            if (!warp_wait(&S.plan_full[sl], (item / kPlans) & 1, abort, p.err)) break;
            const Plan a = S.plan[sl];
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.plan_empty[sl]);
            if (a.h < 0) break;
            const int row0 = a.halves ? 0 : kRows * t;           // first row of the tile in the item
            const int tile_rows = min(kRows, a.rows - row0);     // >= 1
            PrefillSeq q;
            q.nq = a.nq;
            q.nk = a.nk;
            int row_lo, row_hi, lo_max, hi_min, unused;
            prefill_range(p, q, a.i0 + row0 + min(r, tile_rows - 1), &row_lo, &row_hi);
            prefill_range(p, q, a.i0 + row0, &unused, &hi_min);
            prefill_range(p, q, a.i0 + row0 + tile_rows - 1, &lo_max, &unused);
            float m = -INFINITY, l = 0.f;  // reference (in units of the loaded score) and sum
            const int n0 = n;
            for (int e = a.it0; e < a.it0 + a.n; ++e) {
                if (!a.need(t, e)) continue;
                const int key0 = a.block(e) * kKeys;
                if (!warp_wait(&S.s_full[t], n & 1, abort, p.err)) {
                    fail = true;
                    break;
                }
                tc_fence_after();
                if constexpr (kCap == kCapTanh) {
                    // in place, a few scores at a time: the registers are for the row below
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        uint32_t x[16];
                        tmem_ld16(ts + 16 * j, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(p.cap * tanhf(__uint_as_float(x[k]) * cap_in));
                        tmem_st16(ts + 16 * j, x);
                    }
                    tmem_wait_st();
                }
                uint32_t sv[4][32];
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld32(ts + 32 * j, sv[j]);
                tmem_wait_ld();
                // the tile row's visible keys among the 32 of group j, as bits
                auto visible = [&](int j) {
                    const int at = key0 + 32 * j;
                    return (low_bits(row_hi - at) & ~low_bits(row_lo - at)) | low_bits(a.prefix - at);
                };
                if constexpr (kCap == kCapPacked) {
                    // The cap below would make a number of a NaN.  A NaN or an infinity in a
                    // query makes every score of its row one, so one score tells whether to
                    // look at all; a visible NaN then goes into the sum and so into out and lse.
                    if (__any_sync(0xffffffffu, !(fabsf(__uint_as_float(sv[0][0])) < INFINITY))) {
                        bool bad = false;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t see = visible(j);
#pragma unroll
                            for (int k = 0; k < 32; ++k) bad |= (see >> k & 1) && isnan(__uint_as_float(sv[j][k]));
                        }
                        if (bad) l = NAN;
                    }
                    // cap tanh(s / cap) = cap + 2 cap u with u = -1 / (1 + e^(2 s / cap)): u is
                    // the score from here on, scale 2 cap, and the constant joins lse at
                    // the end (u is off by up to 7 2^-24).  One reciprocal serves four scores
                    // (1 / a = b c d / (a b c d)): 226 -> 219 us with a window, against one
                    // for two.  The exponent is held at 30, where u is below half a step of
                    // the values around it, so that the product of four stays finite.
                    const uint64_t in2 = pair(cap_in, cap_in), one2 = pair(1.f, 1.f);
#pragma unroll
                    for (int c = 0; c < 128; c += 4) {
                        float e[4];
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            float x, y;
                            split(mul2(pair(__uint_as_float(sv[c >> 5][(c & 31) + k]), __uint_as_float(sv[c >> 5][(c & 31) + k + 1])),
                                       in2), x, y);
                            split(add2(pair(ex2(fminf(x, 30.f)), ex2(fminf(y, 30.f))), one2), e[k], e[k + 1]);
                        }
                        const float ab = e[0] * e[1], cd = e[2] * e[3], z = -rcp(ab * cd), zab = z * cd, zcd = z * ab;
                        float x, y;
                        split(mul2(pair(zab, zab), pair(e[1], e[0])), x, y);
                        sv[c >> 5][c & 31] = __float_as_uint(x);
                        sv[c >> 5][(c & 31) + 1] = __float_as_uint(y);
                        split(mul2(pair(zcd, zcd), pair(e[3], e[2])), x, y);
                        sv[c >> 5][(c & 31) + 2] = __float_as_uint(x);
                        sv[c >> 5][(c & 31) + 3] = __float_as_uint(y);
                    }
                }
                const bool clear = (key0 >= lo_max && key0 + kKeys <= hi_min) || key0 + kKeys <= a.prefix;
                if (!clear) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t see = visible(j);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(see >> k & 1)) sv[j][k] = __float_as_uint(-INFINITY);
                    }
                }
                // Rows of V past the sequence may hold anything, and 0 * NaN is NaN:
                // zero them (each tile before its own product; the second one writes
                // zeros over zeros).  That block is the last of the item's list, its
                // values the last group.
                if (key0 + kKeys > a.nk) {
                    const int all = entries + a.n, g = 2 * all - 1, c = kPerBlock * all - kVChunks;
                    if (!warp_wait(&S.full[g % kGroups], (g / kGroups) & 1, abort, p.err)) {
                        fail = true;
                        break;
                    }
                    // (a chunk's rows are 128 bytes each, one after the other)
#pragma unroll 1
                    for (int i = (a.nk - key0) * 8 + r; i < kKeys * 8; i += kRows) {
                        *reinterpret_cast<uint4*>(S.ring[c % kSlots] + 16 * i) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(S.ring[(c + 1) % kSlots] + 16 * i) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                // Probabilities of 32 keys against the reference `ref` (log2 units).
                const uint64_t scale2 = pair(scale, scale);
                uint64_t sum[2];
                auto probs = [&](int j, float ref, uint32_t(&pk)[16]) {
                    const uint64_t ref2 = pair(-ref, -ref);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float x, y;
                        split(fma2(pair(__uint_as_float(sv[j][2 * k]), __uint_as_float(sv[j][2 * k + 1])), scale2, ref2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sum[k & 1] = add2(sum[k & 1], pair(x, y));
                        pk[k] = pack_bf16(x, y);
                    }
                };
                float mx[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mx[j] = fmaxf(__uint_as_float(sv[j][0]), __uint_as_float(sv[j][1]));
#pragma unroll
                    for (int k = 2; k < 32; k += 2)
                        mx[j] = max3(mx[j], __uint_as_float(sv[j][k]), __uint_as_float(sv[j][k + 1]));
                }
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                // m = -inf: any visible score moves it
                const bool move = top > -INFINITY && !((top - m) * scale <= kHeadroom);
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? ex2((m - top) * scale) : 1.f;
                    if (move) m = top;
                    l *= f;
                    if (n > n0) {
                        if (!warp_wait(&S.o_done[t], (n - 1) & 1, abort, p.err)) {
                            fail = true;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < 8; ++j) {
                            uint32_t o[16];
                            tmem_ld16(to + 16 * j, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st16(to + 16 * j, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m * scale;
                sum[0] = sum[1] = 0ull;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t pk[16];
                    probs(j, ref, pk);
                    tmem_st16(ts + 16 * j, pk);
                    if (j == 1) {  // the product's first half may start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&S.p_half[t]);
                    }
                }
                float s0, s1;
                split(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[t]);
                ++n;
            }
            entries += a.n;
            if (fail || !warp_wait(&S.rows_free[t], (item & 1) ^ 1, abort, p.err)) break;
            S.row_m[t][r] = m;
            S.row_l[t][r] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.rows_full[t]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // ======================= output warps =======================
        const int quad = warp & 3, r = 32 * quad + lane;
        const uint32_t to = tmem + (static_cast<uint32_t>(32 * quad) << 16) + kOCol;
        const float scale = kCap == kCapPacked ? 2.f * kLog2e * p.cap : kCap == kCapTanh ? kLog2e : p.scale_log2;
        for (int item = 0;; ++item) {
            const int sl = item % kPlans;
            if (!warp_wait(&S.plan_full[sl], (item / kPlans) & 1, abort, p.err)) break;
            const Plan& plan = S.plan[sl];
            const int h = plan.h, split = plan.split, q0 = plan.q0 + plan.i0, rows = plan.rows;
            const bool halves = plan.halves;
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.plan_empty[sl]);
            if (h < 0) break;
            bool ok = true;
            float m_odd = -INFINITY, l_odd = 0.f;
            // tile 1 first where it only adds to tile 0's rows
            for (int u = 0; u < 2 && ok; ++u) {
                const int t = halves ? 1 - u : u;
                // (this wait lasts as long as the item)
                ok = __all_sync(0xffffffffu, wait_item(&S.rows_full[t], item & 1, abort, p.err));
                float m = S.row_m[t][r], l = S.row_l[t][r];
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.rows_free[t]);
                ok = ok && warp_wait(&S.o_ready[t], item & 1, abort, p.err);
                if (!ok) break;
                tc_fence_after();
                if (halves && t == 1) {
                    m_odd = m;
                    l_odd = l;
                    continue;
                }
                // O of the tile times f0 plus, in halves, O of tile 1 times f1.  (A sum is 0
                // for a row that saw no key; a NaN is an answer and stays one.)
                float f0 = 1.f, f1 = 0.f;
                const bool join = __any_sync(0xffffffffu, l_odd != 0.f), some = __any_sync(0xffffffffu, l != 0.f);
                if (join) {
                    const float top = fmaxf(m, m_odd);
                    if (top > -INFINITY) {
                        f0 = ex2((m - top) * scale);
                        f1 = ex2((m_odd - top) * scale);
                    }
                    l = l * f0 + l_odd * f1;
                    m = top;
                }
                const float inv = l != 0.f ? 1.f / l : 0.f;
                const float lse2 = l != 0.f ? m * scale + (kCap == kCapPacked ? kLog2e * p.cap : 0.f) + log2f(l) : -INFINITY;
                f0 *= inv;
                f1 *= inv;
                const int at = kRows * t + r;
                const int64_t row = (int64_t)q0 + at;
                const bool mine = at < rows;
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    uint32_t o[32];
                    if (some) {
                        tmem_ld32(to + kPfV * t + 32 * j, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0u;
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f0);
                    if (join) {
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            uint32_t o1[16];
                            tmem_ld16(to + kPfV + 32 * j + 16 * v, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[16 * v + k] = __float_as_uint(
                                    fmaf(__uint_as_float(o1[k]), f1, __uint_as_float(o[16 * v + k])));
                        }
                    }
                    if (mine && p.n_splits == 1) {
                        uint16_t* dst = p.out + row * p.out_tok + h * p.out_head + 32 * j;
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] = pack_bf16(__uint_as_float(o[16 * v + 2 * k]), __uint_as_float(o[16 * v + 2 * k + 1]));
                            if (p.out_wide) {
                                store32(dst + 16 * v, w);
                            } else {
                                reinterpret_cast<uint4*>(dst)[2 * v] = make_uint4(w[0], w[1], w[2], w[3]);
                                reinterpret_cast<uint4*>(dst)[2 * v + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    } else if (mine) {
                        float* dst = p.part_out + (((int64_t)split * p.Nq + row) * p.H + h) * kPfV + 32 * j;
#pragma unroll
                        for (int v = 0; v < 4; ++v) store32(dst + 8 * v, reinterpret_cast<uint32_t(&)[8]>(o[8 * v]));
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&S.o_free[t]);
                    if (halves) mbar_arrive(&S.o_free[1]);
                }
                if (mine) {
                    if (p.n_splits > 1)
                        p.part_lse[((int64_t)split * p.Nq + row) * p.H + h] = lse2;
                    else if (p.lse)
                        p.lse[row * p.H + h] = lse2 * kLn2;
                }
            }
            if (!ok) break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

// The parts of each (row, head), merged by their normalisers (log2 units): one
// warp per (row, head), 4 dims per lane; a part that saw no key weighs nothing
// and its values are not used.  Rows of no (valid) sequence were written by no
// part and are left alone.
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillParams p) {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= p.Nq * p.H) return;
    const int64_t row = w / p.H;
    const RaggedRow rr = ragged_find(p.cu_q, nullptr, p.B, row, lane);
    if (rr.seq < 0 || !prefill_seq(p, rr.seq, false).ok) return;
    const int64_t step = p.Nq * p.H;
    float top = -INFINITY;
    for (int s = lane; s < p.n_splits; s += 32) top = fmaxf(top, p.part_lse[s * step + w]);
#pragma unroll
    for (int sh = 16; sh >= 1; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int s = 0; s < p.n_splits; ++s) {
        const float e = p.part_lse[s * step + w];
        if (e == -INFINITY) continue;
        const float a = ex2(e - top);  // (a part that is NaN stays NaN: the maximum passes over it)
        const float4 v = reinterpret_cast<const float4*>(p.part_out + (s * step + w) * kPfV)[lane];
        acc.x = fmaf(a, v.x, acc.x);
        acc.y = fmaf(a, v.y, acc.y);
        acc.z = fmaf(a, v.z, acc.z);
        acc.w = fmaf(a, v.w, acc.w);
        sum += a;
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int h = static_cast<int>(w - row * p.H);
    *reinterpret_cast<uint2*>(p.out + row * p.out_tok + h * p.out_head + 4 * lane) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (p.lse && lane == 0) p.lse[w] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

// [tokens][heads][dims] as boxes of 128 tokens x 64 dims of one head, 128-byte
// swizzle; tokens past the tensor read as zeros.
bool encode_map(CUtensorMap* map, const uint16_t* data, int64_t tokens, int64_t heads, int dims, int64_t tok_stride,
                int64_t head_stride) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t size[3] = {(cuuint64_t)dims, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t stride[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)tok_stride * 2};
    cuuint32_t box[3] = {64, 1, kRows}, step[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(data), size, stride, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int64_t prefill_ctas(const PrefillParams& p) {
    // every row tile of every sequence: a sequence's last one may be short
    const int64_t tiles = std::min(((p.max_q + (int64_t)p.tile - 1) / p.tile) * p.B, p.Nq / p.tile + p.B);
    return tiles * p.n_splits * p.H;
}

cudaError_t launch_prefill(const PrefillParams& p, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static bool ready[64];
    static std::mutex mu;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!ready[dev]) {
            for (auto* k : {prefill_kernel<kCapNone>, prefill_kernel<kCapPacked>, prefill_kernel<kCapTanh>})
                if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)) != cudaSuccess)
                    return e;
            ready[dev] = true;
        }
    }
    Maps maps{};
    if (!encode_map(&maps.q, p.q, p.Nq, p.H, kPfHead, p.q_tok, p.q_head)) return cudaErrorInvalidValue;
    if (p.Nk > 0 &&  // without a key the kernel copies nothing
        (!encode_map(&maps.kn, p.k_nope, p.Nk, p.H, kPfNope, p.kn_tok, p.kn_head) ||
         !encode_map(&maps.kp, p.k_pe, p.Nk, 1, kPfRope, p.kp_tok, p.kp_tok) ||
         !encode_map(&maps.v, p.v, p.Nk, p.H, kPfV, p.v_tok, p.v_head)))
        return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(prefill_ctas(p));
    auto* kernel = p.cap == 0.f              ? prefill_kernel<kCapNone>
                   : p.cap <= kPackedCapMost ? prefill_kernel<kCapPacked>
                                             : prefill_kernel<kCapTanh>;
    e = launch_dependent(kernel, grid, kThreads, kSmemBytes, stream, maps, p);
    if (e == cudaSuccess && p.n_splits > 1)
        e = launch_dependent(prefill_join_kernel, static_cast<unsigned>((p.Nq * p.H + 7) / 8), 256, 0, stream, p);
    return e;
}

}  // namespace mla
