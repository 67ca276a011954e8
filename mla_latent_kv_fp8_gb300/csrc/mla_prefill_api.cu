// mla_prefill_api.cu -- host side of mla_prefill_ragged: argument checks, the
// split count and the split scratch.
#include <algorithm>
#include <cmath>

#include "mla_host.h"
#include "mla_prefill.cuh"

using namespace mla;

extern "C" {

// The plan of a call: query rows of an item (256, or 128 taken in halves) and
// parts of its keys.  256-row items read the keys half as often; 128-row ones
// are shorter, so that few sequences spread over the SMs better.  Both sides
// measured on a GB300, us (256 / 128 rows): 4,000 causal tokens x 12 heads 62 /
// 52, 2,048 without a mask 42 / 36, 300 over 98,000 256 / 194, 6,000 causal 91 /
// 98, 16,384 569 / 611, 4,096 x 96 heads, whose keys do not fit L2, 359 / 435.
//
// Costs in microseconds from the same runs: a key block of a 256-row item and
// of a 128-row one, an item's start and end that nothing hides, how much longer
// a 256-row item takes where each has an SM to itself (its two tiles start in
// step and take some eight blocks to drift apart, and its output is twice as
// long), the start of the joining kernel and each part in it, bytes per
// microsecond of partials written and read back, and of keys and values where
// they exceed L2.
namespace {
constexpr double kBlockUs = 1.6, kHalfBlockUs = 0.87, kItemUs = 1.0, kFillUs = 6.0, kJoinUs = 5.0, kPartUs = 0.15;
constexpr double kPartBytesPerUs = 2.2e6, kKeyBytesPerUs = 6e6, kL2Bytes = 110e6;

struct PrefillPlan {
    int32_t tile, splits;
};

PrefillPlan plan_prefill(int64_t Nq, int32_t B, int32_t H, int32_t max_q, int32_t max_k, int32_t causal, int32_t window,
                         int32_t sm_count, int32_t want_splits) {
    PrefillPlan plan{kPfTile / 2, std::max(1, want_splits)};
    if (Nq <= 0 || B <= 0 || H <= 0 || max_q <= 0 || max_k <= 0) return plan;
    double best = -1;
    for (const int32_t tile : {kPfTile, kPfTile / 2}) {
        if (tile == kPfTile && max_q <= kPfTile / 2) continue;  // no such item
        const double block_us = tile == kPfTile ? kBlockUs : kHalfBlockUs;
        const double items = (double)H * std::min<int64_t>((max_q + (int64_t)tile - 1) / tile * B, Nq / tile + B);
        // blocks of an item: the most, and the average over a causal sequence's items
        double most = max_k, mean = causal ? std::max(max_k - max_q / 2.0, max_k / 2.0) : max_k;
        if (window > 0) {
            most = std::min(most, (double)window + std::min<int32_t>(max_q, tile));
            mean = std::min(mean, most);
        }
        most = std::ceil(most / kPfBlock);
        mean = std::max(1.0, mean / kPfBlock);
        // keys and values that one head's items read from memory: each item its own
        // where all heads' together exceed L2, once in the order of split items
        const double block_bytes = kPfBlock * (kPfNope + kPfV) * 2.0;
        const double reach = window > 0 ? std::min<double>(max_k, (double)window + max_q) : max_k;
        const double all_bytes = std::ceil(reach / kPfBlock) * B * H * block_bytes;
        const bool even = mean >= 0.95 * most;  // items of about one length run in whole rounds
        for (int32_t s = 1; s <= 256; ++s) {
            if (want_splits > 0) s = want_splits;
            const double longest = std::ceil(most / s);
            // parts of at least 512 keys, and not more items than eight rounds
            if (s > 1 && want_splits <= 0 && (longest < 4 || items * s > 8.0 * sm_count)) break;
            const double n = items * s, each = mean / s * block_us + kItemUs;
            // The items start in turn on the SM that is free first, the longest first: half
            // of a mean one is idle at the end.
            double cost = even ? std::ceil(n / sm_count) * (longest * block_us + kItemUs)
                               : std::max(longest * block_us + kItemUs, n * each / sm_count + (n > sm_count ? each / 2 : 0.0));
            const double bytes = all_bytes <= kL2Bytes ? 0.0 : (s > 1 ? all_bytes : items * mean * block_bytes);
            const double busy = even ? n / sm_count / std::ceil(n / sm_count) : std::min(1.0, n / sm_count);  // SMs
            cost = std::max(cost, bytes / kKeyBytesPerUs / busy);
            if (tile == kPfTile && n <= sm_count) cost += kFillUs;
            if (s > 1)
                cost += kJoinUs + kPartUs * s + 2.0 * s * (double)mla_prefill_workspace_bytes(Nq, H, 2) / 2 / kPartBytesPerUs;
            if (best < 0 || cost < 0.97 * best) {  // nearly equal: larger items, fewer parts
                best = cost;
                plan = {tile, s};
            }
            if (want_splits > 0) break;
        }
    }
    return plan;
}

int resolve_sm_count(int32_t sm_count) {
    if (sm_count > 0) return sm_count;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sm_count = 148;
    }
    return sm_count;
}
}  // namespace

int32_t mla_prefill_auto_splits(int64_t Nq, int32_t B, int32_t H, int32_t max_q, int32_t max_k, int32_t causal,
                                int32_t window, int32_t sm_count) {
    return plan_prefill(Nq, B, H, max_q, max_k, causal, window, resolve_sm_count(sm_count), 0).splits;
}

size_t mla_prefill_workspace_bytes(int64_t Nq, int32_t H, int32_t n_splits) {
    if (n_splits <= 1 || Nq <= 0 || H <= 0) return 0;
    const size_t rows = (size_t)n_splits * Nq * H;
    return rows * kPfV * sizeof(float) + rows * sizeof(float);
}

mla_status_t mla_prefill_ragged(const mla_tensor_t* q, const mla_tensor_t* k_nope, const mla_tensor_t* k_pe,
                                const mla_tensor_t* v, const mla_tensor_t* cu_q, const mla_tensor_t* cu_k,
                                int32_t max_q, int32_t max_k, int32_t n_splits, float sm_scale, float softcap,
                                int32_t causal, int32_t window, const mla_tensor_t* prefix_lens,
                                const mla_tensor_t* out, const mla_tensor_t* lse, void* stream) {
    internal_clear_error();
    mla_status_t st;
    int64_t qs[2], kns[2], kps[2], vs[2], os[2], B = 0, Bk = 0;
    if ((st = internal_check_rows(q, "q", 3, MLA_DTYPE_BF16, kPfHead, 8, 16, qs)) != MLA_OK) return st;
    if ((st = internal_check_rows(k_nope, "k_nope", 3, MLA_DTYPE_BF16, kPfNope, 8, 16, kns)) != MLA_OK) return st;
    if ((st = internal_check_rows(k_pe, "k_pe", 2, MLA_DTYPE_BF16, kPfRope, 8, 16, kps)) != MLA_OK) return st;
    if ((st = internal_check_rows(v, "v", 3, MLA_DTYPE_BF16, kPfV, 8, 16, vs)) != MLA_OK) return st;
    const int64_t Nq = q->shape[0], H = q->shape[1], Nk = k_nope->shape[0];
    if (k_nope->shape[1] != H || v->shape[1] != H)
        return internal_fail(MLA_ERR_INVALID_ARG, "k_nope and v must have as many heads as q");
    if (v->shape[0] != Nk || k_pe->shape[0] != Nk)
        return internal_fail(MLA_ERR_INVALID_ARG, "k_nope, k_pe and v must have as many rows");
    if ((st = internal_check_offsets(cu_q, "cu_q", &B)) != MLA_OK) return st;
    if ((st = internal_check_offsets(cu_k, "cu_k", &Bk)) != MLA_OK) return st;
    if (B != Bk) return internal_fail(MLA_ERR_INVALID_ARG, "cu_q and cu_k must have as many entries");
    if (prefix_lens) {
        if ((st = internal_check_tensor(prefix_lens, "prefix_lens", 1, MLA_DTYPE_I32, true, 4)) != MLA_OK) return st;
        if (prefix_lens->shape[0] != B) return internal_fail(MLA_ERR_INVALID_ARG, "prefix_lens: must have B entries");
    }
    if ((st = internal_check_rows(out, "out", 3, MLA_DTYPE_BF16, kPfV, 8, 16, os)) != MLA_OK) return st;
    if (out->shape[0] != Nq || out->shape[1] != H)
        return internal_fail(MLA_ERR_INVALID_ARG, "out: must be [Nq, H, 128]");
    if (lse) {
        if ((st = internal_check_tensor(lse, "lse", 2, MLA_DTYPE_F32, true, 4)) != MLA_OK) return st;
        if (lse->shape[0] != Nq || lse->shape[1] != H) return internal_fail(MLA_ERR_INVALID_ARG, "lse: must be [Nq, H]");
    }
    if (max_q < 0 || max_k < 0) return internal_fail(MLA_ERR_INVALID_ARG, "max_q and max_k must be >= 0");
    if (n_splits < 0 || n_splits > 256) return internal_fail(MLA_ERR_INVALID_ARG, "n_splits must lie in [0, 256]");
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale))
        return internal_fail(MLA_ERR_INVALID_ARG, "sm_scale must be finite and > 0");
    // A row's largest score times log2(e) is held in fp32; beyond 2^31 its rounding exceeds what an exponential can
    // take, and the answer is not a number (scores of 2^30 are told apart by 64, which is a weight of 0 or 1).
    if (sm_scale > 0x1p20f) return internal_fail(MLA_ERR_UNSUPPORTED, "sm_scale must be at most 2^20");
    if (!(softcap >= 0.f)) return internal_fail(MLA_ERR_INVALID_ARG, "softcap must be >= 0");
    if (softcap != 0.f && (softcap < 0x1p-10f || softcap > 4096.f))
        return internal_fail(MLA_ERR_UNSUPPORTED, "softcap must be 0 (none) or lie in [2^-10, 4096]");
    if (causal != 0 && causal != 1) return internal_fail(MLA_ERR_INVALID_ARG, "causal must be 0 or 1");
    if (window < 0) return internal_fail(MLA_ERR_INVALID_ARG, "window must be >= 0");
    if (H > 65535) return internal_fail(MLA_ERR_UNSUPPORTED, "more than 65535 heads");
    if (Nq > 0x7fffff00 || Nk > 0x7fffff00) return internal_fail(MLA_ERR_UNSUPPORTED, "2^31 rows or more");
    const int64_t far[] = {qs[0], qs[1], kns[0], kns[1], kps[0], vs[0], vs[1]};
    for (int64_t f : far)
        if (f >= (int64_t(1) << 39))  // a copy's strides are below 2^40 bytes
            return internal_fail(MLA_ERR_UNSUPPORTED, "strides of 2^39 elements or more");
    if (max_q == 0 || max_q > Nq) max_q = static_cast<int32_t>(Nq);
    if (max_k == 0 || max_k > Nk) max_k = static_cast<int32_t>(Nk);
    if (Nq == 0 || H == 0 || B == 0) return MLA_OK;
    PrefillParams p{};
    int sm_count = 0;
    if ((st = internal_device(&p.err, &sm_count)) != MLA_OK) return st;
    p.q = static_cast<const uint16_t*>(q->data);
    p.k_nope = static_cast<const uint16_t*>(k_nope->data);
    p.k_pe = static_cast<const uint16_t*>(k_pe->data);
    p.v = static_cast<const uint16_t*>(v->data);
    p.q_tok = qs[0], p.q_head = qs[1];
    p.kn_tok = kns[0], p.kn_head = kns[1];
    p.kp_tok = kps[0];
    p.v_tok = vs[0], p.v_head = vs[1];
    p.Nq = Nq;
    p.Nk = Nk;
    p.cu_q = static_cast<const int32_t*>(cu_q->data);
    p.cu_k = static_cast<const int32_t*>(cu_k->data);
    p.B = static_cast<int>(B);
    p.H = static_cast<int>(H);
    p.max_q = max_q;
    p.max_k = max_k;
    const PrefillPlan plan = plan_prefill(Nq, p.B, p.H, max_q, max_k, causal, window, sm_count, n_splits);
    p.tile = plan.tile;
    p.n_splits = plan.splits;
    p.scale_log2 = sm_scale * kLog2e;
    p.cap = softcap;
    p.causal = causal;
    p.window = window;
    p.prefix = prefix_lens ? static_cast<const int32_t*>(prefix_lens->data) : nullptr;
    p.out = static_cast<uint16_t*>(out->data);
    p.out_tok = os[0], p.out_head = os[1];
    p.out_wide = reinterpret_cast<uintptr_t>(out->data) % 32 == 0 && os[0] % 16 == 0 && os[1] % 16 == 0;
    p.lse = lse ? static_cast<float*>(lse->data) : nullptr;
    if (prefill_ctas(p) > 0x7fffffff || Nq * H > (int64_t(1) << 33))
        return internal_fail(MLA_ERR_UNSUPPORTED, "too many query rows for one launch");
    p.test_stall_copies = internal_test_stall();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.n_splits > 1) {
        void* ws = nullptr;
        if ((st = internal_scratch(mla_prefill_workspace_bytes(Nq, p.H, p.n_splits), s, &ws)) != MLA_OK) return st;
        p.part_out = static_cast<float*>(ws);
        p.part_lse = p.part_out + (size_t)p.n_splits * Nq * H * kPfV;
    }
    const cudaError_t e = launch_prefill(p, s);
    return e == cudaSuccess ? MLA_OK : internal_cuda_fail(e, "prefill launch");
}

}  // extern "C"
