// What the eviction kernels share: page tables in CSR form on the device and the parameters
// of the gathered weights.
#pragma once

#include <climits>
#include <cstdint>

#include "bsp_internal.h"
#include "device_common.cuh"

namespace bsp {
namespace evict {

constexpr uint32_t kNoRow = ~0u;  // a token that is not there, or whose page id is outside the pool

// The page table of a batch. Values out of range are read as the nearest in range, so that a
// malformed table reads and writes nothing outside the arrays.
struct Csr {
    const int32_t *kv_indptr, *kv_indices, *last_page_len;
    int max_pages;  // entries of kv_indices
    int batch, ps, num_pages;
    uint32_t div_mul;  // t / ps = t * div_mul >> div_shift for 0 <= t < 2^31
    int div_shift;
};

struct Request {
    int p0, len;  // first table entry, tokens
};

__device__ __forceinline__ int clamp_page(const Csr &c, int i) { return min(max(__ldg(c.kv_indptr + i), 0), c.max_pages); }

__device__ __forceinline__ Request request(const Csr &c, int b) {
    const int p0 = clamp_page(c, b), n = clamp_page(c, b + 1) - p0;
    const int last = min(max(__ldg(c.last_page_len + b), 0), c.ps);
    return {p0, n > 0 ? (int)min((long long)(n - 1) * c.ps + last, (long long)INT_MAX) : 0};
}

__device__ __forceinline__ int div_ps(const Csr &c, int t) { return (int)(((uint64_t)(uint32_t)t * c.div_mul) >> c.div_shift); }

// Slot of token t of a request, or kNoRow (host: num_pages * ps < 2^32 - 1).
__device__ __forceinline__ uint32_t slot_of(const Csr &c, const Request &r, int t, int &page, int &place) {
    const int col = div_ps(c, t);
    place = t - col * c.ps;
    page = __ldg(c.kv_indices + r.p0 + col);
    return (unsigned)page < (unsigned)c.num_pages ? (uint32_t)page * (uint32_t)c.ps + (uint32_t)place : kNoRow;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct WeightsParams {
    Csr csr;
    const int32_t *qo_indptr;  // or null: one query per request
    const void *q, *k;
    const float *lse, *lam;
    const int8_t *k_exp;
    float *weights;
    int n_tokens, H_qo, H_kv, g;
    float scale_log2, cap_in, cap_out, decay;
    int soft_cap_on, window;
    long long wait_limit;  // kStall alone: SM clock cycles
};

// Every wait of these kernels is bounded. One that gives up (a fault, not a stall) ends the CTA's work, and what it had
// not summed yet becomes NaN, so that no weight is left as it was unnoticed. kStall: the self-test's instantiations, where
// the warps that bring the keys stop after the first few.
constexpr long long kWaitLimitCycles = 4000000000ll;  // about 2 s at 2 GHz

// Virtual blocks of kTokens tokens: request b's begin at floor(kv_indptr[b] * ps / kTokens) + b, which
// leaves room for ceil(len / kTokens) of them without a prefix sum over the requests. The first is
// block_start(0), which is not 0 where the table is a part of another (kv_indptr[0] > 0).
template <int kTokens>
__device__ __forceinline__ long long block_start(const Csr &c, int b) {
    return (long long)clamp_page(c, b) * c.ps / kTokens + b;
}

// A warp: the request of virtual block x (the last that begins at or before it).
template <int kTokens>
__device__ __forceinline__ int find_request(const Csr &c, long long x, int lane) {
    int lo = 0, hi = c.batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, m = lo + (lane + 1) * step;
        const unsigned le = __ballot_sync(0xffffffffu, m < hi && block_start<kTokens>(c, m) <= x);
        lo += __popc(le) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

struct Queries {
    int q0, n;  // first row of q, queries of the request
};

__device__ __forceinline__ Queries queries(const WeightsParams &p, int b) {
    if (!p.qo_indptr) return {min(b, p.n_tokens), b < p.n_tokens ? 1 : 0};
    const int a = min(max(__ldg(p.qo_indptr + b), 0), p.n_tokens), e = min(max(__ldg(p.qo_indptr + b + 1), a), p.n_tokens);
    return {a, e - a};
}

}  // namespace evict

// csrc/weights_prefill.cu: whether its kernel takes a call, and its launch.
bool weights_prefill_takes(const bsp_problem *problem, int64_t num_pages, int64_t n_tokens, int32_t batch, const int32_t *qo_indptr);
int launch_weights_prefill(const bsp_problem *problem, const evict::WeightsParams &w, int64_t num_pages, int64_t max_table_pages,
                           int sms, cudaStream_t stream);  // (w.wait_limit > 0: the self-test)

}  // namespace bsp
