// mla_prefill.cuh -- parameters and masks of the ragged prefill attention,
// shared by its kernels (internal; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mla_internal.cuh"

namespace mla {

constexpr int kPfNope = 128;             // query/key dims of a head's own part
constexpr int kPfRope = 64;              // shared, rotated key dims
constexpr int kPfHead = kPfNope + kPfRope;
constexpr int kPfV = 128;                // value dims

struct PrefillParams {
    const uint16_t* q;                   // bf16 [Nq][H][192]
    const uint16_t* k_nope;              // bf16 [Nk][H][128]
    const uint16_t* k_pe;                // bf16 [Nk][64]
    const uint16_t* v;                   // bf16 [Nk][H][128]
    int64_t q_tok, q_head, kn_tok, kn_head, kp_tok, v_tok, v_head;  // strides
    int64_t Nq, Nk;
    const int32_t* cu_q;                 // [B + 1]
    const int32_t* cu_k;                 // [B + 1]
    int B, H;
    int max_q, max_k;
    int tile;                            // query rows of a work item: 128 or 256
    int n_splits;                        // partitions of every tile's key blocks (>= 1)
    float scale_log2;                    // sm_scale * log2(e)
    float cap;                           // score cap (0: none)
    int causal;
    int window;                          // 0: none
    const int32_t* prefix;               // [B] or null
    uint16_t* out;                       // bf16 [Nq][H][128]
    int64_t out_tok, out_head;
    int out_wide;                        // every row of out starts on 32 bytes
    float* lse;                          // [Nq][H] or null
    // n_splits > 1: fp32 partials [n_splits][Nq][H][128] and [n_splits][Nq][H]
    float* part_out;
    float* part_lse;
    int* err;
    int test_stall_copies;               // failure-detection tests only: issue no copies
};

// One sequence of the batch: its rows and lengths.  ok is false, and the
// device error word set, when its offsets lie outside the tensors, run
// backwards or exceed max_q / max_k; its rows are then left as they were.
struct PrefillSeq {
    int q0, k0, nq, nk, prefix;
    bool ok;
};

__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillParams& p, int b, bool report) {
    PrefillSeq s;
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
    const int k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    s.ok = q0 >= 0 && q1 >= q0 && q1 <= p.Nq && k0 >= 0 && k1 >= k0 && k1 <= p.Nk && q1 - q0 <= p.max_q &&
           k1 - k0 <= p.max_k;
    if (!s.ok && report) atomicCAS(p.err, 0, kErrSeqRange);
    s.q0 = q0;
    s.k0 = k0;
    s.nq = s.ok ? q1 - q0 : 0;
    s.nk = s.ok ? k1 - k0 : 0;
    const int pre = p.prefix && s.ok ? p.prefix[b] : 0;
    s.prefix = pre < 0 ? 0 : (pre > s.nk ? s.nk : pre);
    return s;
}

// Keys that query i of a sequence sees: [0, s.prefix) and [lo, hi).  Query i
// stands at position i + nk - nq (the queries are the last of the sequence),
// which is negative for the first rows of a sequence with fewer keys than
// queries: such a row sees nothing but the prefix.
__device__ __forceinline__ void prefill_range(const PrefillParams& p, const PrefillSeq& s, int i, int* lo, int* hi) {
    const int64_t pos = (int64_t)i + s.nk - s.nq;
    int64_t h = p.causal ? pos + 1 : s.nk;
    h = h < 0 ? 0 : (h > s.nk ? s.nk : h);
    int64_t l = p.window > 0 ? pos - p.window + 1 : 0;
    l = l < 0 ? 0 : (l > h ? h : l);
    *lo = static_cast<int>(l);
    *hi = static_cast<int>(h);
}

// CTAs of one call (the caller checks that they fit a grid), and the launch.
int64_t prefill_ctas(const PrefillParams& p);
cudaError_t launch_prefill(const PrefillParams& p, cudaStream_t stream);

// The most query rows of an item and the keys of one block.
constexpr int kPfTile = 256;
constexpr int kPfBlock = 128;

}  // namespace mla
