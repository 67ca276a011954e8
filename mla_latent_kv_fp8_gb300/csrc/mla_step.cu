// mla_step.cu -- the memory-bound operators around a decode or prefill call on
// packed (ragged) batches:
//   mla_append_rotated  norm + rotation + E4M3FN quantisation of new latents
//                       into their paged cache slots
//   mla_rotate_query    per-head norm + rotation of the query heads
//   mla_gather_latent   a history read back from its pages as bf16 rows
//
// The rotation turns pair i of the 64 positional dims by the angle of the
// position: (a, b) -> (a c - b s, b c + a s) with c = cos_sin[pos][i] and
// s = cos_sin[pos][32 + i]; pair i is (x[i], x[i + 32]), or (x[2i], x[2i + 1])
// in the interleaved layout.  The norm is x * rsqrt(mean(x^2) + eps) * weight.
// Both are computed in fp32; a value is rounded once, to what is stored.
//
// In all three eight lanes hold a 64-dim positional part, lane l pairs
// 4l .. 4l + 3: one 16-byte load in the interleaved layout, two 8-byte loads
// otherwise, and one float4 of cosines and of sines either way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cstdio>

#include "mla_host.h"
#include "mla_ragged.cuh"

namespace mla {
namespace {

constexpr int kRope = 64;
constexpr int kNope = 128;
constexpr int kHead = kNope + kRope;

// bf16 pair <-> floats
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = lo_f(w[j]), x[2 * j + 1] = hi_f(w[j]);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ float sum_squares(const uint4& v) {
    float x[8], s = 0.f;
    unpack8(v, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
    return s;
}
// Makes the compiler unpack the values again where they are used next instead
// of keeping eight registers for them.
__device__ __forceinline__ void keep_packed(uint4& v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }

// Eight consecutive norm weights, bf16 or fp32.
__device__ __forceinline__ void load_weight8(const void* w, bool f32, int at, float (&x)[8]) {
    if (f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
        const float4 a = p[0], b = p[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at), x);
    }
}

__device__ __forceinline__ void load_weight4(const void* w, bool f32, int at, float* x) {
    if (f32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    } else {
        const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + at);
        x[0] = lo_f(a.x), x[1] = hi_f(a.x), x[2] = lo_f(a.y), x[3] = hi_f(a.y);
    }
}

// The four pairs of lane l (< 8): a[j], b[j] are pair 4l + j.  The raw loads
// and stores keep the layout's order: 16 bytes interleaved, 8 + 8 bytes
// otherwise.
template <bool kInter>
__device__ __forceinline__ uint4 load_pairs(const uint16_t* x, int l) {
    if constexpr (kInter) return *reinterpret_cast<const uint4*>(x + 8 * l);
    const uint2 a = *reinterpret_cast<const uint2*>(x + 4 * l);
    const uint2 b = *reinterpret_cast<const uint2*>(x + kRope / 2 + 4 * l);
    return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool kInter>
__device__ __forceinline__ void split_pairs(const float (&x)[8], float (&a)[4], float (&b)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a[j] = kInter ? x[2 * j] : x[j];
        b[j] = kInter ? x[2 * j + 1] : x[4 + j];
    }
}
template <bool kInter>
__device__ __forceinline__ void join_pairs(const float (&a)[4], const float (&b)[4], float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[kInter ? 2 * j : j] = a[j];
        x[kInter ? 2 * j + 1 : 4 + j] = b[j];
    }
}
template <bool kInter>
__device__ __forceinline__ void store_pairs(uint16_t* x, int l, const uint4& v) {
    if constexpr (kInter) {
        *reinterpret_cast<uint4*>(x + 8 * l) = v;
    } else {
        *reinterpret_cast<uint2*>(x + 4 * l) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(x + kRope / 2 + 4 * l) = make_uint2(v.z, v.w);
    }
}
// Turns the lane's pairs by the angles c[j], s[j].
__device__ __forceinline__ void rotate4(float (&a)[4], float (&b)[4], const float4& c4, const float4& s4) {
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float u = a[j] * c[j] - b[j] * s[j];
        b[j] = b[j] * c[j] + a[j] * s[j];
        a[j] = u;
    }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xffffu) | (hi << 16);
}

// ---------------------------------------------------------------- append

struct AppendParams {
    const uint16_t* latent;  // [N] rows of 576
    int64_t stride;
    int64_t rows;
    const void* weight;      // [512] or null
    float eps;
    const float* cos_sin;    // [positions][64]
    int64_t positions;
    const int32_t* cu;       // [B + 1]
    const int32_t* start;    // [B]
    int B;
    const float* kv_scale;
    const int32_t* block_table;
    int64_t bt_stride;
    int max_pages;
    uint8_t* kv;
    int64_t num_pages;
    uint16_t* keep;          // bf16 [N] rows of 576, or null
    int64_t keep_stride;
    int* err;
};

// x / s with the E4M3FN code of the correctly rounded quotient.  For a divisor
// of ordinary size: q = x * RN(1 / s) and one correction, c = RN(q + (x - q s)
// RN(1 / s)).  A quotient of 2^10 or more saturates as it is, and one below
// 2^-10 becomes the code 0; between them nothing over- or underflows.
// q is up to 1.5 ulp off, the remainder and RN(1 / s) up to 2^-24 of themselves,
// so before its rounding c is within 3.01 * 2^-24 ulp of x / s: c can differ
// from RN(x / s) only where x / s lies that near to the middle of two floats,
// and their codes only where one of the two is a border between codes, a
// number T = t 2^a with 16 <= t < 32.  With s = S 2^b, 2^23 <= S < 2^24, x a
// multiple of 2^(a + b + 3) and the middle at 2^a (t +- 2^-20) (or, below t = 16,
// 2^a (16 - 2^-21)), that needs an S within 12 of a multiple of 2^20.  All such S
// with all t and the x around s T were tried (tests/test_packed_division.py): c
// is RN(x / s) for each.
// 18 divisions a lane by the library's general one bound the kernel (16,384
// rows: 14.6 us, now 11.9).
struct Divider {
    float s, inv;
    bool plain;
    __device__ __forceinline__ explicit Divider(float scale)
        : s(scale), inv(1.f / scale), plain(scale >= 0x1p-90f && scale <= 0x1p90f) {}
    __device__ __forceinline__ float operator()(float x) const {
        if (!plain) return __fdiv_rn(x, s);
        const float q = x * inv;
        // (the remainder with this sign: of a signed zero it is +0 and its negative -0, which keeps q's sign)
        return fabsf(q) < 1024.f ? fmaf(-fmaf(q, s, -x), inv, q) : q;
    }
};

// One warp per new position: lane l holds latent dims [8l, 8l + 8) and
// [256 + 8l, 256 + 8l + 8), lanes 0..7 also the positional pairs, so a row is
// read with three and written with three coalesced accesses.  Everything is
// read before anything is written: `keep` may be `latent` itself.
// kNorm as below.
template <bool kInter, int kNorm>
__global__ void __launch_bounds__(256, 5) append_rotated_kernel(const AppendParams p) {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    // the row's values do not depend on its sequence: their loads go out first
    const uint16_t* src = p.latent + row * p.stride;
    uint4 v0 = *reinterpret_cast<const uint4*>(src + 8 * lane);
    uint4 v1 = *reinterpret_cast<const uint4*>(src + 256 + 8 * lane);
    const uint4 vr = lane < 8 ? load_pairs<kInter>(src + kDv, lane) : make_uint4(0, 0, 0, 0);
    const Divider by_scale(*p.kv_scale);
    const RaggedRow r = ragged_find(p.cu, p.start, p.B, row, lane);
    if (r.seq < 0) return;
    const int64_t pos = (int64_t)r.start + r.at;
    if (pos < 0 || pos >= (int64_t)p.max_pages * kPage || pos >= p.positions) {
        if (lane == 0) atomicCAS(p.err, 0, kErrSeqRange);
        return;
    }
    const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + pos * kRope);
    const float4 c4 = cs[lane & 7], s4 = cs[8 + (lane & 7)];
    const int32_t page = p.block_table[r.seq * p.bt_stride + pos / kPage];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicCAS(p.err, 0, kErrPageRange);
        return;
    }
    float inv = 1.f;
    if constexpr (kNorm != 0) {
        float ss = sum_squares(v0) + sum_squares(v1);
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, sh);
        inv = rsqrtf(ss * (1.f / kDv) + p.eps);
        keep_packed(v0);
        keep_packed(v1);
    }
    uint8_t* dst = p.kv + ((int64_t)page * kPage + pos % kPage) * kDqk;
    uint16_t* keep = p.keep ? p.keep + row * p.keep_stride : nullptr;
    // code = e4m3fn(x / scale)
    auto codes = [&](const float (&x)[8]) {
        return make_uint2(e4m3x4(by_scale(x[0]), by_scale(x[1]), by_scale(x[2]), by_scale(x[3])),
                          e4m3x4(by_scale(x[4]), by_scale(x[5]), by_scale(x[6]), by_scale(x[7])));
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int d = 256 * u + 8 * lane;
        float x[8];
        unpack8(u ? v1 : v0, x);
        if constexpr (kNorm != 0) {
            float weight[8];
            load_weight8(p.weight, kNorm == 2, d, weight);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * weight[j];
        }
        reinterpret_cast<uint2*>(dst + d)[0] = codes(x);
        if (keep) *reinterpret_cast<uint4*>(keep + d) = pack8(x);
    }
    if (lane < 8) {
        float x[8], a[4], b[4];
        unpack8(vr, x);
        split_pairs<kInter>(x, a, b);
        rotate4(a, b, c4, s4);
        join_pairs<kInter>(a, b, x);
        const uint2 c = codes(x);
        if constexpr (kInter) {
            reinterpret_cast<uint2*>(dst + kDv)[lane] = c;
        } else {
            reinterpret_cast<uint32_t*>(dst + kDv)[lane] = c.x;
            reinterpret_cast<uint32_t*>(dst + kDv + kRope / 2)[lane] = c.y;
        }
        if (keep) store_pairs<kInter>(keep + kDv, lane, pack8(x));
    }
}

// ---------------------------------------------------------------- query heads

struct RotateParams {
    const uint16_t* q;       // [N][H][192]
    int64_t q_tok, q_head;   // strides
    int64_t rows;
    int H;
    const void* weight;      // [192] or null
    float eps;
    const float* cos_sin;
    int64_t positions;
    const int32_t* cu;
    const int32_t* start;
    int B;
    uint16_t* nope;          // [N][H][128] or null
    int64_t nope_tok, nope_head;
    uint16_t* pe;            // [N][H][64]
    int64_t pe_tok, pe_head;
    int* err;
};

// A warp takes four heads of one token, eight lanes each: lane l of a head
// holds its dims [8l, 8l + 8), [64 + 8l, 64 + 8l + 8) and the positional pairs
// 4l .. 4l + 3.  Everything of a head is read before any of it is written, by
// the same lane at the same place, so the outputs may be the input's own dims.
// Bound by memory (it reads and writes the same bytes, like a copy): 8,191
// tokens x 96 heads with a norm 93 us, 6.5 TB/s, in both layouts; 48 registers
// and 40 warps an SM (64 registers 107 us, 40 with spills 100; the interleaved
// layout with a norm spills four to six of the 48).  Without a norm only a third
// of each head is read, 128 of 384 bytes, and written as 128-byte rows of a wider
// tensor: 53 us for the 203 MB, 3.8 TB/s.
// kNorm: 0 none, 1 with bf16 weights, 2 with fp32 weights.
template <bool kInter, int kNorm>
__global__ void __launch_bounds__(256, 5) rotate_query_kernel(const RotateParams p) {
    wait_for_previous();
    const int lane = threadIdx.x & 31, l = lane & 7;
    // (rows x groups < 2^32: a 64-bit division costs more than the rest of the address)
    const unsigned groups = (p.H + 3) >> 2, w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const unsigned row = w / groups;
    if (row >= p.rows) return;
    const int h = static_cast<int>(w - row * groups) * 4 + (lane >> 3);
    const bool live = h < p.H;
    const uint16_t* src = p.q + row * p.q_tok + h * p.q_head;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0, vr = v0;
    if (live) {
        if (kNorm != 0 || p.nope) {
            v0 = *reinterpret_cast<const uint4*>(src + 8 * l);
            v1 = *reinterpret_cast<const uint4*>(src + 64 + 8 * l);
        }
        vr = load_pairs<kInter>(src + kNope, l);
    }
    const RaggedRow r = ragged_find(p.cu, p.start, p.B, row, lane);
    if (r.seq < 0) return;
    const int64_t pos = (int64_t)r.start + r.at;
    if (pos < 0 || pos >= p.positions) {
        if (lane == 0) atomicCAS(p.err, 0, kErrSeqRange);
        return;
    }
    const float4* cs = reinterpret_cast<const float4*>(p.cos_sin + pos * kRope);
    const float4 c4 = cs[l], s4 = cs[8 + l];
    float xr[8];
    if constexpr (kNorm != 0) {
        // The values stay packed between the sum of squares and their scaling, which
        // is what lets 48 registers do.
        float x[8], weight[8];
        float ss = sum_squares(v0) + sum_squares(v1) + sum_squares(vr);
#pragma unroll
        for (int sh = 4; sh >= 1; sh >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, sh);
        const float inv = rsqrtf(ss * (1.f / kHead) + p.eps);
        keep_packed(v0);
        keep_packed(v1);
        keep_packed(vr);
        load_weight8(p.weight, kNorm == 2, 8 * l, weight);
        unpack8(v0, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * weight[j];
        v0 = pack8(x);
        load_weight8(p.weight, kNorm == 2, 64 + 8 * l, weight);
        unpack8(v1, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * weight[j];
        v1 = pack8(x);
        if constexpr (kInter) {
            load_weight8(p.weight, kNorm == 2, kNope + 8 * l, weight);
        } else {
            load_weight4(p.weight, kNorm == 2, kNope + 4 * l, weight);
            load_weight4(p.weight, kNorm == 2, kNope + kRope / 2 + 4 * l, weight + 4);
        }
        unpack8(vr, xr);
#pragma unroll
        for (int j = 0; j < 8; ++j) xr[j] = xr[j] * inv * weight[j];
    } else {
        unpack8(vr, xr);
    }
    float a[4], b[4];
    split_pairs<kInter>(xr, a, b);
    rotate4(a, b, c4, s4);
    join_pairs<kInter>(a, b, xr);
    if (!live) return;
    if (kNorm != 0 || p.nope) {
        uint16_t* o = p.nope + row * p.nope_tok + h * p.nope_head;
        *reinterpret_cast<uint4*>(o + 8 * l) = v0;
        *reinterpret_cast<uint4*>(o + 64 + 8 * l) = v1;
    }
    store_pairs<kInter>(p.pe + row * p.pe_tok + h * p.pe_head, l, pack8(xr));
}

// ---------------------------------------------------------------- gather

struct GatherParams {
    const uint8_t* kv;
    int64_t num_pages;
    const float* kv_scale;
    const int32_t* block_table;
    int64_t bt_stride;
    int max_pages;
    const int32_t* cu;
    const int32_t* start;    // or null: histories from position 0
    int B;
    int64_t rows;
    uint16_t* latent;        // [N] rows of 512
    int64_t latent_stride;
    uint16_t* pe;            // [N] rows of 64
    int64_t pe_stride;
    int* err;
};

// One warp per row: 36 chunks of 16 codes, loaded as 16 and stored as 32 bytes.
// Bound by its stores at large sizes (262,144 rows: 302 MB, 76 us; a plain fill
// of that size takes 76).  Two, four and eight rows a warp measured no faster
// there (85 us) and slower below (20,000 rows: 9.8, 10.3, 12.3 us, against 8.2).
__global__ void gather_latent_kernel(const GatherParams p) {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const float scale = *p.kv_scale;
    const RaggedRow r = ragged_find(p.cu, p.start, p.B, row, lane);
    if (r.seq < 0) return;
    const int64_t pos = (int64_t)r.start + r.at;
    const uint8_t* src = nullptr;  // null: the row is written as zeros
    if (pos < 0 || pos >= (int64_t)p.max_pages * kPage) {
        if (lane == 0) atomicCAS(p.err, 0, kErrSeqRange);
    } else {
        const int32_t page = p.block_table[r.seq * p.bt_stride + pos / kPage];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicCAS(p.err, 0, kErrPageRange);
        } else {
            src = p.kv + ((int64_t)page * kPage + pos % kPage) * kDqk;
        }
    }
    constexpr int kChunks = kDqk / 16;
    uint4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v[i] = src && 32 * i + lane < kChunks ? reinterpret_cast<const uint4*>(src)[32 * i + lane]
                                              : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 32 * i + lane;
        if (c >= kChunks) break;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>((w[j >> 1] >> (16 * (j & 1))) & 0xffffu), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            o[j] = pack_bf16(f.x * scale, f.y * scale);
        }
        uint16_t* dst = c < kDv / 16 ? p.latent + row * p.latent_stride + 16 * c
                                     : p.pe + row * p.pe_stride + 16 * (c - kDv / 16);
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Warps per CTA: small calls spread over the SMs one warp each.
unsigned warps_per_cta(int64_t warps, int sm_count) { return warps <= 8 * (int64_t)sm_count ? 1 : 4; }

// Grid of `warps` warps; the caller has checked that it fits.
struct Launch {
    unsigned grid, block;
};
bool plan_launch(int64_t warps, int sm_count, Launch* l) {
    const unsigned w = warps_per_cta(warps, sm_count);
    const int64_t grid = (warps + w - 1) / w;
    if (grid > 0x7fffffff) return false;
    l->grid = static_cast<unsigned>(grid);
    l->block = 32 * w;
    return true;
}

// ---------------------------------------------------------------- host checks

mla_status_t check_norm(const mla_tensor_t* w, int64_t n, float eps) {
    if (!w) return MLA_OK;
    mla_status_t st;
    const int dt = w->dtype == MLA_DTYPE_F32 ? MLA_DTYPE_F32 : MLA_DTYPE_BF16;
    if ((st = internal_check_tensor(w, "norm_weight", 1, dt, true, 16)) != MLA_OK) return st;
    if (w->shape[0] != n) return internal_fail(MLA_ERR_INVALID_ARG, "norm_weight: wrong number of weights");
    if (!(eps >= 0.f)) return internal_fail(MLA_ERR_INVALID_ARG, "eps must be >= 0");
    return MLA_OK;
}

mla_status_t check_cos_sin(const mla_tensor_t* t) {
    mla_status_t st;
    if ((st = internal_check_tensor(t, "cos_sin", 2, MLA_DTYPE_F32, true, 16)) != MLA_OK) return st;
    if (t->shape[1] != kRope) return internal_fail(MLA_ERR_INVALID_ARG, "cos_sin: must be [positions, 64]");
    return MLA_OK;
}

mla_status_t check_style(int32_t interleaved) {
    if (interleaved != 0 && interleaved != 1)
        return internal_fail(MLA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    return MLA_OK;
}

// kv_cache, kv_scale and block_table of B requests.
mla_status_t check_cache(const mla_tensor_t* kv_cache, const float* kv_scale, const mla_tensor_t* block_table,
                         int64_t B) {
    mla_status_t st;
    if ((st = internal_check_tensor(kv_cache, "kv_cache", 3, MLA_DTYPE_E4M3FN, true, 16)) != MLA_OK) return st;
    if (kv_cache->shape[1] != kPage || kv_cache->shape[2] != kDqk)
        return internal_fail(MLA_ERR_UNSUPPORTED, "kv_cache: must be [num_pages, 64, 576]");
    if (!kv_scale) return internal_fail(MLA_ERR_INVALID_ARG, "kv_scale: null pointer");
    if ((st = internal_check_tensor(block_table, "block_table", 2, MLA_DTYPE_I32, false, 4)) != MLA_OK) return st;
    if (block_table->shape[0] != B) return internal_fail(MLA_ERR_INVALID_ARG, "block_table: first dim must be B");
    const int64_t max_pages = block_table->shape[1];
    if (max_pages > 1 && block_table->stride[1] != 1)
        return internal_fail(MLA_ERR_UNSUPPORTED, "block_table: rows must be contiguous");
    if (B > 1 && block_table->stride[0] < max_pages)
        return internal_fail(MLA_ERR_UNSUPPORTED, "block_table: rows must be contiguous");
    if (max_pages > (1 << 24)) return internal_fail(MLA_ERR_UNSUPPORTED, "block_table: too many pages");
    return MLA_OK;
}

}  // namespace

mla_status_t internal_check_offsets(const mla_tensor_t* cu, const char* name, int64_t* B) {
    char msg[96];
    mla_status_t st;
    if ((st = internal_check_tensor(cu, name, 1, MLA_DTYPE_I32, true, 4)) != MLA_OK) return st;
    if (cu->shape[0] < 1) {
        snprintf(msg, sizeof msg, "%s: needs B + 1 entries", name);
        return internal_fail(MLA_ERR_INVALID_ARG, msg);
    }
    if (cu->shape[0] > 65536) {
        snprintf(msg, sizeof msg, "%s: more than 65535 sequences", name);
        return internal_fail(MLA_ERR_UNSUPPORTED, msg);
    }
    *B = cu->shape[0] - 1;
    return MLA_OK;
}

mla_status_t internal_check_rows(const mla_tensor_t* t, const char* name, int ndim, int dtype, int64_t width,
                                 int64_t step, size_t align, int64_t stride[2]) {
    char msg[128];
    mla_status_t st;
    if ((st = internal_check_tensor(t, name, ndim, dtype, false, align)) != MLA_OK) return st;
    if (t->shape[ndim - 1] != width) {
        snprintf(msg, sizeof msg, "%s: last dim must be %lld", name, (long long)width);
        return internal_fail(MLA_ERR_INVALID_ARG, msg);
    }
    if (t->stride[ndim - 1] != 1) {
        snprintf(msg, sizeof msg, "%s: the last dim must be contiguous", name);
        return internal_fail(MLA_ERR_UNSUPPORTED, msg);
    }
    // Rows may lie anywhere, in either order of the outer dims, as long as they
    // do not overlap and start on `step` elements; a dim of size 1 has no stride.
    int64_t n[2] = {t->shape[0], ndim == 3 ? t->shape[1] : 1};
    int64_t s[2] = {t->stride[0], ndim == 3 ? t->stride[1] : width};
    if (n[0] == 0 || n[1] == 0) n[0] = n[1] = 0;  // no rows
    if (n[0] <= 1) s[0] = n[1] > 1 && s[1] > 0 ? n[1] * s[1] : width;
    if (n[1] <= 1) s[1] = width;
    const int in = (n[1] > 1 && (n[0] <= 1 || s[1] <= s[0])) ? 1 : 0, out = 1 - in;
    const bool fits = (n[in] <= 1 || s[in] >= width) && (n[out] <= 1 || s[out] >= (n[in] - 1) * s[in] + width);
    if (!fits || s[0] % step != 0 || s[1] % step != 0) {
        snprintf(msg, sizeof msg, "%s: rows must not overlap and their strides must be multiples of %lld", name,
                 (long long)step);
        return internal_fail(MLA_ERR_UNSUPPORTED, msg);
    }
    stride[0] = s[0];
    stride[1] = s[1];
    return MLA_OK;
}

}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_append_rotated(const mla_tensor_t* latent, const mla_tensor_t* norm_weight, float eps,
                                const mla_tensor_t* cos_sin, int32_t interleaved, const mla_tensor_t* cu_tokens,
                                const float* kv_scale, const mla_tensor_t* block_table,
                                const mla_tensor_t* start_pos, const mla_tensor_t* kv_cache,
                                const mla_tensor_t* latent_out, void* stream) {
    internal_clear_error();
    mla_status_t st;
    int64_t ls[2] = {0, 0}, ks[2] = {0, 0}, B = 0;
    if ((st = internal_check_rows(latent, "latent", 2, MLA_DTYPE_BF16, kDqk, 8, 16, ls)) != MLA_OK) return st;
    const int64_t N = latent->shape[0];
    if ((st = check_norm(norm_weight, kDv, eps)) != MLA_OK) return st;
    if ((st = check_cos_sin(cos_sin)) != MLA_OK) return st;
    if ((st = check_style(interleaved)) != MLA_OK) return st;
    if ((st = internal_check_offsets(cu_tokens, "cu_tokens", &B)) != MLA_OK) return st;
    if ((st = check_cache(kv_cache, kv_scale, block_table, B)) != MLA_OK) return st;
    if ((st = internal_check_tensor(start_pos, "start_pos", 1, MLA_DTYPE_I32, true, 4)) != MLA_OK) return st;
    if (start_pos->shape[0] != B) return internal_fail(MLA_ERR_INVALID_ARG, "start_pos: must have B entries");
    if (latent_out) {
        if ((st = internal_check_rows(latent_out, "latent_out", 2, MLA_DTYPE_BF16, kDqk, 8, 16, ks)) != MLA_OK)
            return st;
        if (latent_out->shape[0] != N) return internal_fail(MLA_ERR_INVALID_ARG, "latent_out: must be [N, 576]");
    }
    if (N == 0 || B == 0) return MLA_OK;
    AppendParams p{};
    int sm_count = 0;
    if ((st = internal_device(&p.err, &sm_count)) != MLA_OK) return st;
    p.latent = static_cast<const uint16_t*>(latent->data);
    p.stride = ls[0];
    p.rows = N;
    p.weight = norm_weight ? norm_weight->data : nullptr;
    p.eps = eps;
    p.cos_sin = static_cast<const float*>(cos_sin->data);
    p.positions = cos_sin->shape[0];
    p.cu = static_cast<const int32_t*>(cu_tokens->data);
    p.start = static_cast<const int32_t*>(start_pos->data);
    p.B = static_cast<int>(B);
    p.kv_scale = kv_scale;
    p.block_table = static_cast<const int32_t*>(block_table->data);
    p.bt_stride = block_table->stride[0];
    p.max_pages = static_cast<int>(block_table->shape[1]);
    p.kv = static_cast<uint8_t*>(kv_cache->data);
    p.num_pages = kv_cache->shape[0];
    p.keep = latent_out ? static_cast<uint16_t*>(latent_out->data) : nullptr;
    p.keep_stride = ks[0];
    Launch l;
    if (!plan_launch(N, sm_count, &l)) return internal_fail(MLA_ERR_UNSUPPORTED, "latent: too many rows");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int norm = norm_weight ? (norm_weight->dtype == MLA_DTYPE_F32 ? 2 : 1) : 0;
    auto* kernel = interleaved ? (norm == 0   ? append_rotated_kernel<true, 0>
                                  : norm == 1 ? append_rotated_kernel<true, 1>
                                              : append_rotated_kernel<true, 2>)
                               : (norm == 0   ? append_rotated_kernel<false, 0>
                                  : norm == 1 ? append_rotated_kernel<false, 1>
                                              : append_rotated_kernel<false, 2>);
    const cudaError_t e = launch_dependent(kernel, l.grid, l.block, 0, s, p);
    return e == cudaSuccess ? MLA_OK : internal_cuda_fail(e, "rotated append launch");
}

mla_status_t mla_rotate_query(const mla_tensor_t* q, const mla_tensor_t* norm_weight, float eps,
                              const mla_tensor_t* cos_sin, int32_t interleaved, const mla_tensor_t* cu_tokens,
                              const mla_tensor_t* start_pos, const mla_tensor_t* nope_out,
                              const mla_tensor_t* pe_out, void* stream) {
    internal_clear_error();
    mla_status_t st;
    int64_t qs[2] = {0, 0}, ns[2] = {0, 0}, ps[2] = {0, 0}, B = 0;
    if ((st = internal_check_rows(q, "q", 3, MLA_DTYPE_BF16, kHead, 8, 16, qs)) != MLA_OK) return st;
    const int64_t N = q->shape[0], H = q->shape[1];
    if ((st = check_norm(norm_weight, kHead, eps)) != MLA_OK) return st;
    if ((st = check_cos_sin(cos_sin)) != MLA_OK) return st;
    if ((st = check_style(interleaved)) != MLA_OK) return st;
    if ((st = internal_check_offsets(cu_tokens, "cu_tokens", &B)) != MLA_OK) return st;
    if ((st = internal_check_tensor(start_pos, "start_pos", 1, MLA_DTYPE_I32, true, 4)) != MLA_OK) return st;
    if (start_pos->shape[0] != B) return internal_fail(MLA_ERR_INVALID_ARG, "start_pos: must have B entries");
    if (norm_weight && !nope_out)
        return internal_fail(MLA_ERR_INVALID_ARG, "nope_out: required with norm_weight (the norm changes every dim)");
    if (nope_out) {
        if ((st = internal_check_rows(nope_out, "nope_out", 3, MLA_DTYPE_BF16, kNope, 8, 16, ns)) != MLA_OK) return st;
        if (nope_out->shape[0] != N || nope_out->shape[1] != H)
            return internal_fail(MLA_ERR_INVALID_ARG, "nope_out: must be [N, H, 128]");
    }
    if ((st = internal_check_rows(pe_out, "pe_out", 3, MLA_DTYPE_BF16, kRope, 8, 16, ps)) != MLA_OK) return st;
    if (pe_out->shape[0] != N || pe_out->shape[1] != H)
        return internal_fail(MLA_ERR_INVALID_ARG, "pe_out: must be [N, H, 64]");
    if (H > (1 << 20)) return internal_fail(MLA_ERR_UNSUPPORTED, "q: too many heads");
    if (N == 0 || H == 0 || B == 0) return MLA_OK;
    RotateParams p{};
    int sm_count = 0;
    if ((st = internal_device(&p.err, &sm_count)) != MLA_OK) return st;
    p.q = static_cast<const uint16_t*>(q->data);
    p.q_tok = qs[0];
    p.q_head = qs[1];
    p.rows = N;
    p.H = static_cast<int>(H);
    p.weight = norm_weight ? norm_weight->data : nullptr;
    p.eps = eps;
    p.cos_sin = static_cast<const float*>(cos_sin->data);
    p.positions = cos_sin->shape[0];
    p.cu = static_cast<const int32_t*>(cu_tokens->data);
    p.start = static_cast<const int32_t*>(start_pos->data);
    p.B = static_cast<int>(B);
    p.nope = nope_out ? static_cast<uint16_t*>(nope_out->data) : nullptr;
    p.nope_tok = ns[0];
    p.nope_head = ns[1];
    p.pe = static_cast<uint16_t*>(pe_out->data);
    p.pe_tok = ps[0];
    p.pe_head = ps[1];
    Launch l;
    if (N > 0xffffff00 / ((H + 3) / 4) || !plan_launch(N * ((H + 3) / 4), sm_count, &l))
        return internal_fail(MLA_ERR_UNSUPPORTED, "q: too many rows");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int norm = norm_weight ? (norm_weight->dtype == MLA_DTYPE_F32 ? 2 : 1) : 0;
    auto* kernel = interleaved ? (norm == 0   ? rotate_query_kernel<true, 0>
                                  : norm == 1 ? rotate_query_kernel<true, 1>
                                              : rotate_query_kernel<true, 2>)
                               : (norm == 0   ? rotate_query_kernel<false, 0>
                                  : norm == 1 ? rotate_query_kernel<false, 1>
                                              : rotate_query_kernel<false, 2>);
    const cudaError_t e = launch_dependent(kernel, l.grid, l.block, 0, s, p);
    return e == cudaSuccess ? MLA_OK : internal_cuda_fail(e, "query rotation launch");
}

mla_status_t mla_gather_latent(const mla_tensor_t* kv_cache, const float* kv_scale, const mla_tensor_t* block_table,
                               const mla_tensor_t* cu_tokens, const mla_tensor_t* start_pos,
                               const mla_tensor_t* latent_out, const mla_tensor_t* pe_out, void* stream) {
    internal_clear_error();
    mla_status_t st;
    int64_t ls[2] = {0, 0}, ps[2] = {0, 0}, B = 0;
    if ((st = internal_check_offsets(cu_tokens, "cu_tokens", &B)) != MLA_OK) return st;
    if ((st = check_cache(kv_cache, kv_scale, block_table, B)) != MLA_OK) return st;
    if (start_pos) {
        if ((st = internal_check_tensor(start_pos, "start_pos", 1, MLA_DTYPE_I32, true, 4)) != MLA_OK) return st;
        if (start_pos->shape[0] != B) return internal_fail(MLA_ERR_INVALID_ARG, "start_pos: must have B entries");
    }
    if ((st = internal_check_rows(latent_out, "latent_out", 2, MLA_DTYPE_BF16, kDv, 8, 16, ls)) != MLA_OK) return st;
    if ((st = internal_check_rows(pe_out, "pe_out", 2, MLA_DTYPE_BF16, kRope, 8, 16, ps)) != MLA_OK) return st;
    const int64_t N = latent_out->shape[0];
    if (pe_out->shape[0] != N) return internal_fail(MLA_ERR_INVALID_ARG, "pe_out: must be [N, 64]");
    if (N == 0 || B == 0) return MLA_OK;
    GatherParams p{};
    int sm_count = 0;
    if ((st = internal_device(&p.err, &sm_count)) != MLA_OK) return st;
    p.kv = static_cast<const uint8_t*>(kv_cache->data);
    p.num_pages = kv_cache->shape[0];
    p.kv_scale = kv_scale;
    p.block_table = static_cast<const int32_t*>(block_table->data);
    p.bt_stride = block_table->stride[0];
    p.max_pages = static_cast<int>(block_table->shape[1]);
    p.cu = static_cast<const int32_t*>(cu_tokens->data);
    p.start = start_pos ? static_cast<const int32_t*>(start_pos->data) : nullptr;
    p.B = static_cast<int>(B);
    p.rows = N;
    p.latent = static_cast<uint16_t*>(latent_out->data);
    p.latent_stride = ls[0];
    p.pe = static_cast<uint16_t*>(pe_out->data);
    p.pe_stride = ps[0];
    Launch l;
    if (!plan_launch(N, sm_count, &l)) return internal_fail(MLA_ERR_UNSUPPORTED, "latent_out: too many rows");
    const cudaError_t e = launch_dependent(gather_latent_kernel, l.grid, l.block, 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? MLA_OK : internal_cuda_fail(e, "history gather launch");
}

}  // extern "C"
