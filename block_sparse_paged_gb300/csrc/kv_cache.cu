// The paged KV cache beside the attention that reads it: the page table and the
// slots of a step's new tokens from request lengths, and the append that
// quantises new keys and values into an e4m3 cache with one power-of-two
// exponent per (page, kv head).
#include <algorithm>
#include <climits>

#include <cuda_fp16.h>

#include "bsp_internal.h"
#include "device_common.cuh"

namespace bsp {
namespace {

// ---------------------------------------------------------------- page tables
// For request b with c cached and m new tokens: old = ceil(c / ps) entries of its
// table row hold pages, all = ceil((c + m) / ps) shall; the all - old missing ones
// come from the free list, requests in order. Three exclusive sums over the
// requests (pages, free pages taken, new tokens) place everything.
//
// Every CTA computes the sums of all requests for itself, in shared memory, and
// then expands its share of the entries and tokens: one launch, no pass over
// global memory between the sums and their use, no atomics. The lengths are at
// most 128 KB, read from L2. Bound by the latency of that chain (lengths, sums, search,
// entry): 4.9 us for 4 requests, 10.3-10.9 us for 0.8 M entries and as many slots (20 MB).
// A thread's entries are addressed first, loaded together and then stored: 0.5-0.8 us less
// than one after the other. 2 to 8 CTAs per SM, 128 to 512 threads and eight entries per
// thread measured equal or slower.
constexpr int kTabThreads = 256;
constexpr int kTabUnit = 4;  // consecutive entries (tokens) per thread: one search, vector stores
constexpr int kTabMaxBatch = 16384;

struct TableParams {
    const int32_t *cached, *fresh;
    const int32_t *free_pages, *num_free;
    long long free_capacity;
    int32_t *table;
    long long table_stride;
    int width, batch, ps;
    int32_t *kv_indptr, *last_page_len, *kv_indices, *qo_indptr, *positions, *counts;
    long long *slots;
    long long cap_pages, cap_tokens;
};

// Lengths of one request: negative ones read as 0, pages clipped to the row.
struct TableRow {
    int cached, fresh, old_pages, all_pages;
    int flags;
};
__device__ __forceinline__ TableRow table_row(const TableParams &p, int b) {
    TableRow r;
    const int c = __ldg(p.cached + b), m = __ldg(p.fresh + b);
    r.flags = (c < 0 || m < 0) ? BSP_TABLES_BAD_LENGTH : 0;
    r.cached = max(c, 0);
    r.fresh = max(m, 0);
    const uint32_t ps = (uint32_t)p.ps, total = (uint32_t)r.cached + (uint32_t)r.fresh;  // at most 2^32 - 2
    const uint32_t all = total ? (total - 1) / ps + 1 : 0;
    if (all > (uint32_t)p.width) r.flags |= BSP_TABLES_OVER_CAPACITY;
    r.all_pages = (int)min(all, (uint32_t)p.width);
    r.old_pages = min((int)(r.cached ? ((uint32_t)r.cached - 1) / ps + 1 : 0), r.all_pages);
    return r;
}

// The pages alone, out of line (used where sums are saturated).
__device__ __noinline__ int table_row_pages(const TableParams &p, int b, int &old_pages) {
    const TableRow r = table_row(p, b);
    old_pages = r.old_pages;
    return r.all_pages;
}

// Largest b with start[b] <= x, for x in [0, start[n]).
__device__ __forceinline__ int find_row(const int *start, int n, int x) {
    int lo = 0, hi = n;  // start[lo] <= x < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const TableParams p) {
    extern __shared__ int sm[];
    const int B = p.batch;
    int *s_pages = sm, *s_take = sm + (B + 1), *s_tok = sm + 2 * (B + 1);
    __shared__ long long s_part[3][kTabThreads / 32];
    __shared__ int s_flags;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_flags = 0;
    const int n_free = (int)max(0ll, min((long long)__ldg(p.num_free), p.free_capacity));
    __syncthreads();

    // exclusive sums in 64 bits, kept saturated to int32 (an output that needs more
    // is over its capacity anyway)
    long long base[3] = {0, 0, 0};
    for (int b0 = 0; b0 < B; b0 += kTabThreads) {
        const int b = b0 + tid;
        long long v[3] = {0, 0, 0};
        if (b < B) {
            const TableRow r = table_row(p, b);
            v[0] = r.all_pages;
            v[1] = r.all_pages - r.old_pages;
            v[2] = r.fresh;
            if (r.flags) atomicOr(&s_flags, r.flags);
        }
        long long inc[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            inc[j] = v[j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, inc[j], o);
                if (lane >= o) inc[j] += up;
            }
            if (lane == 31) s_part[j][warp] = inc[j];
        }
        __syncthreads();
        long long sum[3] = {0, 0, 0};
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            long long before = base[j];
#pragma unroll
            for (int w = 0; w < kTabThreads / 32; ++w) {
                before += w < warp ? s_part[j][w] : 0;
                sum[j] += s_part[j][w];
            }
            if (b < B) sm[j * (B + 1) + b] = (int)min(before + inc[j] - v[j], (long long)INT32_MAX);
            base[j] += sum[j];
        }
        __syncthreads();
    }
    if (tid == 0) {
#pragma unroll
        for (int j = 0; j < 3; ++j) sm[j * (B + 1) + B] = (int)min(base[j], (long long)INT32_MAX);
    }
    __syncthreads();
    const int n_pages = s_pages[B], n_tok = s_tok[B];

    if (blockIdx.x == 0) {
        for (int b = tid; b <= B; b += kTabThreads) {
            p.kv_indptr[b] = s_pages[b];
            p.qo_indptr[b] = s_tok[b];
            if (b < B) {
                const TableRow r = table_row(p, b);
                const long long total = min((long long)r.cached + r.fresh, (long long)r.all_pages * p.ps);
                p.last_page_len[b] = r.all_pages > 0 ? (int)((total - 1) % p.ps) + 1 : 0;
            }
        }
        if (tid == 0) {
            int f = s_flags;
            if (s_take[B] > n_free) f |= BSP_TABLES_OUT_OF_PAGES;
            if (base[0] > p.cap_pages || base[2] > p.cap_tokens) f |= BSP_TABLES_OVER_CAPACITY;
            p.counts[0] = n_pages;
            p.counts[1] = n_tok;
            p.counts[2] = min(s_take[B], n_free);
            p.counts[3] = f;
        }
    }

    // pages of request b, and how many of them its row held, from the sums (unless they
    // are saturated)
    auto pages_of = [&](int b, int &old_pages) -> int {
        if (n_pages == INT32_MAX) return table_row_pages(p, b, old_pages);
        const int all = s_pages[b + 1] - s_pages[b];
        old_pages = all - (s_take[b + 1] - s_take[b]);
        return all;
    };
    // where column i of request b stands: in the row, or in the free list (null: none left)
    auto place = [&](int b, int old_pages, int i) -> const int32_t * {
        if (i < old_pages) return p.table + (long long)b * p.table_stride + i;
        const uint32_t k = (uint32_t)s_take[b] + (uint32_t)(i - old_pages);  // (s_take saturates at 2^31 - 1)
        return k < (uint32_t)n_free ? p.free_pages + k : nullptr;
    };

    // One index space: groups of kTabUnit table entries, then groups of tokens, so that
    // a small step's entries and tokens are worked on at the same time.
    const long long n_ent = max((long long)n_pages, p.cap_pages);
    const long long g_ent = (n_ent + kTabUnit - 1) / kTabUnit, g_all = g_ent + (p.cap_tokens + kTabUnit - 1) / kTabUnit;
    for (long long gi = (long long)blockIdx.x * kTabThreads + tid; gi < g_all; gi += (long long)gridDim.x * kTabThreads) {
        if (gi < g_ent) {
            // table entries: CSR copy of every row, new entries also into the row; the CSR
            // tail up to its capacity is 0
            const long long e0 = gi * kTabUnit;
            // (addresses of all entries first, then their loads together, then the stores)
            const int32_t *from[kTabUnit];
            int32_t *to[kTabUnit];  // where a new entry goes
            int id[kTabUnit];
            int b = e0 < n_pages ? find_row(s_pages, B, (int)e0) - 1 : 0, old_pages = 0, end = -1, begin = 0;
#pragma unroll
            for (int u = 0; u < kTabUnit; ++u) {
                const long long e = e0 + u;
                from[u] = nullptr;
                to[u] = nullptr;
                if (e < n_pages) {
                    if ((int)e >= end) {
                        do ++b;
                        while (s_pages[b + 1] <= (int)e);  // (passes rows without pages)
                        begin = s_pages[b];
                        end = s_pages[b + 1];
                        pages_of(b, old_pages);
                    }
                    const int i = (int)e - begin;
                    from[u] = place(b, old_pages, i);
                    if (i >= old_pages) to[u] = p.table + (long long)b * p.table_stride + i;
                }
            }
#pragma unroll
            for (int u = 0; u < kTabUnit; ++u) id[u] = from[u] ? *from[u] : -1;
#pragma unroll
            for (int u = 0; u < kTabUnit; ++u) {
                if (to[u]) *to[u] = id[u];
                id[u] = max(id[u], 0);
            }
            if (e0 + kTabUnit <= p.cap_pages) {
                *reinterpret_cast<int4 *>(p.kv_indices + e0) = make_int4(id[0], id[1], id[2], id[3]);
            } else {
#pragma unroll
                for (int u = 0; u < kTabUnit; ++u)
                    if (e0 + u < p.cap_pages) p.kv_indices[e0 + u] = id[u];
            }
            continue;
        }
        // tokens: slot and position of every new token; the tail is -1 and 0
        const long long t0 = (gi - g_ent) * kTabUnit;
        const int32_t *from[kTabUnit];
        int offs[kTabUnit], pos[kTabUnit];
        long long slot[kTabUnit];
        int b = t0 < n_tok ? find_row(s_tok, B, (int)t0) - 1 : 0, end = -1, begin = 0;
        uint32_t col = 0;  // (past 2^31 with pages of one token)
        int off = 0, cached = 0, all_pages = 0, old_pages = 0;
#pragma unroll
        for (int u = 0; u < kTabUnit; ++u) {
            const long long t = t0 + u;
            from[u] = nullptr;
            offs[u] = 0;
            pos[u] = 0;
            if (t < n_tok) {
                if ((int)t >= end) {
                    do ++b;
                    while (s_tok[b + 1] <= (int)t);  // (passes requests without new tokens)
                    begin = s_tok[b];
                    end = s_tok[b + 1];
                    all_pages = pages_of(b, old_pages);
                    cached = max(__ldg(p.cached + b), 0);
                    const uint32_t x = (uint32_t)cached + (uint32_t)((int)t - begin);
                    col = x / (uint32_t)p.ps;
                    off = (int)(x - col * (uint32_t)p.ps);
                } else if (++off == p.ps) {
                    off = 0;
                    ++col;
                }
                pos[u] = (int)min((long long)cached + ((int)t - begin), (long long)INT32_MAX);
                offs[u] = off;
                if (col < (uint32_t)all_pages) from[u] = place(b, old_pages, (int)col);
            }
        }
#pragma unroll
        for (int u = 0; u < kTabUnit; ++u) {
            const int pg = from[u] ? *from[u] : -1;
            slot[u] = pg >= 0 ? (long long)pg * p.ps + offs[u] : -1;
        }
        if (t0 + kTabUnit <= p.cap_tokens) {
            *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            reinterpret_cast<longlong2 *>(p.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2 *>(p.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int u = 0; u < kTabUnit; ++u)
                if (t0 + u < p.cap_tokens) {
                    p.slots[t0 + u] = slot[u];
                    p.positions[t0 + u] = pos[u];
                }
        }
    }
}

// ---------------------------------------------------------------- append
// A page's exponent for one kv head is the least e with amax <= 448 * 2^e over the
// tokens that the page holds (448: the largest e4m3 value), within [kExpMin,
// kExpMax], where every code * 2^e is a normal bf16 value. A power of two costs an
// e4m3 code no precision against amax / 448, and moving stored codes to a larger
// exponent only shifts them.
//
// One CTA per (window of 128 tokens, kv head, K or V); its 8 (bf16) or 16 (fp32) warps
// hold the tokens in registers from the first read to the stored codes, so keys and
// values are read once: HBM-bound, the heads of a window in neighbouring CTAs so that whole
// token rows are read together. The tokens of a page stand next to each other (a run):
// token maxima meet in shared memory per run. A run that goes past the window is
// measured by every CTA that holds a part of it (its outside tokens are read for their
// maximum alone, from L2); all get the same exponent, and the CTA with the run's first
// token writes it and rescales the codes that the page held before. A CTA that
// reads the exponent after that write gets max(need, e) = e: the same.
// 24k ragged bf16 tokens x 8 heads 36 us (149 MB); with 37.5 us then: 64 and 256 tokens per
// window 38.9, 41.6; 3, 5 and 6 CTAs per SM 43.5, 40.7, 42.9 (spills from 5 on).
constexpr int kAppTokens = 128;
constexpr int kExpMin = -117, kExpMax = 119;
constexpr int kCacheD = 128;

struct AppendParams {
    const char *k, *v;             // new keys, values
    long long k_tok, k_head, v_tok, v_head;  // byte strides
    uint8_t *k_codes, *v_codes;
    int8_t *k_exp, *v_exp;
    const long long *slots;
    long long n, rows;             // tokens; slots of the pool
    int ps, H;
    int ps_shift;                  // log2(ps), or -1
};

// 2^e for e in [-149, 127]
__device__ __forceinline__ float pow2i(int e) {
    return __int_as_float(e >= -126 ? (e + 127) << 23 : 0x00400000 >> (-127 - e));
}

// Least e with amax <= 448 * 2^e for the bits of a finite amax >= 0, clamped.
__device__ __forceinline__ int exponent_for(uint32_t amax_bits) {
    // amax = 1.f * 2^(x - 127) for normal values; 448 = 1.75 * 2^8. Subnormal maxima
    // have x = 0 and clamp to kExpMin like every value below 448 * 2^kExpMin.
    const int x = (int)(amax_bits >> 23);
    const int e = x - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(kExpMin, min(kExpMax, e));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// max(|a|, |b|) per half (signs: the product's), of bf16 values; a NaN gives the other operand
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// lo * s and hi * s as two e4m3 codes
__device__ __forceinline__ uint32_t e4m3x2_scaled(float lo, float hi, float s) {
    asm("{ .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mul.rn.f32x2 a, a, b;\n"
        " mov.b64 {%0, %1}, a;\n}"
        : "+f"(lo), "+f"(hi)
        : "f"(s));
    return e4m3x2(lo, hi);
}

// One lane's piece of a token row: 8 values of 128, 16 lanes to a row, as one (bf16) or
// two (fp32) 16-byte vectors.
constexpr int kPieceLanes = 16, kPer = 32 / kPieceLanes;  // lanes per row, rows per warp-wide load
template <bool kF32>
struct Piece {
    static constexpr int kVecs = kF32 ? 2 : 1;
    static constexpr int kLoads = kF32 ? 4 : 8;               // rows in flight per lane: 32 registers
    static constexpr int kPerWarp = kLoads * kPer;            // tokens per warp
    static constexpr int kWarps = kAppTokens / kPerWarp;      // 8 (bf16), 16 (fp32)
    uint4 w[kVecs];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    // Maxima of |value| are kept as bits: fp32 ones, or two bf16 ones (even and odd values).
    // An infinity gives a maximum that is not finite(), so do values that are all NaN (fp32:
    // one NaN).
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return kF32 ? max(a, b) : max2(a, b); }
    static __device__ __forceinline__ bool finite(uint32_t m) {
        return kF32 ? m < 0x7f800000u : ((m + 0x00800080u) & 0x80008000u) == 0;
    }
    static __device__ __forceinline__ uint32_t fp32_bits(uint32_t m) { return kF32 ? m : max(m << 16, m & 0xffff0000u); }
    __device__ __forceinline__ uint32_t amax() const {
        if constexpr (kF32) {
            constexpr uint32_t m = 0x7fffffffu;
            return max(max(max(w[0].x & m, w[0].y & m), max(w[0].z & m, w[0].w & m)),
                       max(max(w[1].x & m, w[1].y & m), max(w[1].z & m, w[1].w & m)));
        } else {
            return absmax_bf16x2(absmax_bf16x2(w[0].x, w[0].y), absmax_bf16x2(w[0].z, w[0].w)) & 0x7fff7fffu;
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kF32) {
                    f[4 * v + i] = __uint_as_float(u[i]);
                } else {
                    f[2 * i] = dev::bf16_lo(u[i]);
                    f[2 * i + 1] = dev::bf16_hi(u[i]);
                }
            }
        }
    }
    // infinities become NaN (the format has none)
    __device__ __forceinline__ void no_infinities() {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kF32) {
                    if ((u[i] & 0x7fffffffu) == 0x7f800000u) u[i] = 0x7fffffffu;
                } else {
                    if ((u[i] & 0x7fffu) == 0x7f80u) u[i] |= 0x7fu;
                    if ((u[i] & 0x7fff0000u) == 0x7f800000u) u[i] |= 0x7f0000u;
                }
            }
            w[v] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
    // codes of the piece at scale s = 2^-e (lowest first)
    __device__ __forceinline__ uint2 codes(float s) const {
        float f[8];
        values(f);
        return make_uint2(e4m3x2_scaled(f[0], f[1], s) | (e4m3x2_scaled(f[2], f[3], s) << 16),
                          e4m3x2_scaled(f[4], f[5], s) | (e4m3x2_scaled(f[6], f[7], s) << 16));
    }
};
// the same maximum over the finite values
template <bool kF32>
__device__ __noinline__ uint32_t amax_finite(Piece<kF32> x) {
    float f[8];
    x.values(f);
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(f[i]) & 0x7fffffffu;
        if (a < 0x7f800000u) r = max(r, a);
    }
    return kF32 ? r : r >> 16;
}

// Maxima of a lane's pieces, over their finite values; pieces with an infinity lose it. The
// pieces that are not finite are looked at one by one.
template <bool kF32, int kN>
__device__ __forceinline__ void piece_maxima(Piece<kF32> (&w)[kN], uint32_t (&v)[kN]) {
    using PC = Piece<kF32>;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        v[i] = w[i].amax();
        top = PC::larger(top, v[i]);
    }
    if (PC::finite(top)) return;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (!PC::finite(v[i])) {
            v[i] = amax_finite(w[i]);
            w[i].no_infinities();
        }
}

// Four stored codes times s (a power of two <= 1), rounded to nearest even.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float s) {
    uint32_t h0, h1;
    dev::e4m3x4_to_f16x4(w, h0, h1);
    const __half2 a = *reinterpret_cast<__half2 *>(&h0), b = *reinterpret_cast<__half2 *>(&h1);
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    return e4m3x2(fa.x * s, fa.y * s) | (e4m3x2(fb.x * s, fb.y * s) << 16);
}

// Page and place of token t's slot; page -1 outside the pool or the list.
__device__ __forceinline__ int place_of(const AppendParams &p, long long t, int &off) {
    off = 0;
    if (t < 0 || t >= p.n) return -1;
    const long long sl = __ldg(p.slots + t);
    if (sl < 0 || sl >= p.rows) return -1;
    // (rows fit 32 bits: checked by the caller)
    const uint32_t pg = p.ps_shift >= 0 ? (uint32_t)sl >> p.ps_shift : (uint32_t)sl / (uint32_t)p.ps;
    off = (int)((uint32_t)sl - pg * (uint32_t)p.ps);
    return (int)pg;
}

// A warp: codes of rows 0 .. held - 1 of a page whose exponent rose by -drop, four rows of
// 8 lanes x 16 bytes at a time. page: the page's codes of this kv head.
__device__ __forceinline__ void rescale_rows(uint8_t *page, uint32_t row_bytes, int held, int drop, int lane) {
    const float s = pow2i(max(drop, -126));
    for (int r = lane >> 3; r < held; r += 4) {
        uint4 *at = reinterpret_cast<uint4 *>(page + (uint64_t)r * row_bytes) + (lane & 7);
        uint4 c = *at;
        c.x = rescale_codes(c.x, s);
        c.y = rescale_codes(c.y, s);
        c.z = rescale_codes(c.z, s);
        c.w = rescale_codes(c.w, s);
        *at = c;
    }
}

// Maxima of a warp's tokens: v[i] is this lane's part of load i. The values are halved
// while the lanes are folded (then plain folds): lane l of a row ends with the maximum of
// load (l / (kPieceLanes / kN)) of its row.
template <class PC, int kN>
__device__ __forceinline__ uint32_t fold_max(uint32_t (&v)[kN], int piece) {
#pragma unroll
    for (int n = kN / 2, o = kPieceLanes / 2; n >= 1; n >>= 1, o >>= 1) {
        const bool up = piece & o;  // keeps the upper half of the values
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
            v[i] = PC::larger(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
#pragma unroll
    for (int o = kPieceLanes / kN / 2; o >= 1; o >>= 1) v[0] = PC::larger(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    return PC::fp32_bits(v[0]);
}

template <bool kF32>
__global__ void __launch_bounds__(32 * Piece<kF32>::kWarps, kF32 ? 2 : 4) append_kernel(const AppendParams p) {
    using PC = Piece<kF32>;
    constexpr int kTok = kAppTokens, kWords = kTok / 32, kWarps = PC::kWarps;
    __shared__ int s_page[kTok];         // page of each token, or -1
    __shared__ int s_off[kTok];          // its place in the page
    __shared__ int s_had[kTok];          // the page's exponent before (of first tokens)
    __shared__ uint32_t s_lead[kWords];  // tokens that begin a run in this window
    __shared__ uint32_t s_tmax[kTok];    // token maxima
    __shared__ uint32_t s_max[kTok];     // maxima of runs, by their first token in the window
    __shared__ int s_left, s_right;      // tokens of the first / last run outside the window
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long win = blockIdx.x / (2 * p.H);
    const int hv = (int)(blockIdx.x - win * (2 * p.H));
    const bool is_v = hv >= p.H;
    const int h = is_v ? hv - p.H : hv;
    const long long T0 = win * kTok;
    const int nt = (int)min((long long)kTok, p.n - T0);
    const long long tb = is_v ? p.v_tok : p.k_tok;
    const char *x = is_v ? p.v + h * p.v_head : p.k + h * p.k_head;
    int8_t *exps = (is_v ? p.v_exp : p.k_exp) + h;
    constexpr int kLoads = PC::kLoads, kBytes = 16 * PC::kVecs;  // bytes of a piece
    const int sub = lane / kPieceLanes, piece = lane % kPieceLanes;
    const int t_first = warp * PC::kPerWarp + sub;  // token of this lane's load i: t_first + i * kPer

    PC w[kLoads];
    const char *src = x + (T0 + t_first) * tb + piece * kBytes;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        w[i].clear();
        if (t_first + i * kPer < nt) w[i].load(src + i * kPer * tb);
    }
    if (tid < kTok) {
        int off = 0, off_before;
        const int page = tid < nt ? place_of(p, T0 + tid, off) : -1;
        // (of token 0 the run may begin before the window: s_left tells)
        const bool lead = page >= 0 && (tid == 0 || place_of(p, T0 + tid - 1, off_before) != page);
        s_page[tid] = page;
        s_off[tid] = off;
        s_max[tid] = 0;
        if (lead) s_had[tid] = *reinterpret_cast<volatile int8_t *>(exps + (long long)page * p.H);
        const uint32_t m = __ballot_sync(0xffffffffu, lead);
        if (lane == 0) s_lead[warp] = m;
    } else if (warp >= kWarps - 2) {
        // how far the first (last) run goes on before (behind) the window
        const bool left = warp == kWarps - 2;
        int got = 0, off;
        const int pg = place_of(p, left ? T0 : T0 + nt - 1, off);
        if (pg >= 0) {
            for (;;) {
                const long long t = left ? T0 - 1 - got - lane : T0 + nt + got + lane;
                const bool same = place_of(p, t, off) == pg;
                const uint32_t m = __ballot_sync(0xffffffffu, same);
                const int k = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
                got += k;
                if (k < 32) break;
            }
        }
        if (lane == 0) (left ? s_left : s_right) = got;
    }
    {
        uint32_t v[kLoads];
        piece_maxima(w, v);
        const uint32_t m = fold_max<PC>(v, piece);
        constexpr int kShare = kPieceLanes / kLoads;  // lanes that hold the same maximum
        if (piece % kShare == 0) s_tmax[t_first + piece / kShare * kPer] = m;
    }
    __syncthreads();
    // first token of the run that token t (with a page) belongs to, within the window
    auto run_of = [&](int t) -> int {
        int k = t >> 5;
        uint32_t m = s_lead[k] & (0xffffffffu >> (31 - (t & 31)));
        while (m == 0) m = s_lead[--k];
        return 32 * k + 31 - __clz(m);
    };
    if (tid < kTok && s_page[tid] >= 0) atomicMax(&s_max[run_of(tid)], s_tmax[tid]);
    if (s_left | s_right) {
        const int outside = s_left + s_right, last_run = s_page[nt - 1] >= 0 ? run_of(nt - 1) : 0;
        constexpr int kStep = kWarps * kPer, kFly = 2;
        for (int j = warp * kPer + sub; j - sub < outside; j += kFly * kStep) {
            PC y[kFly];
#pragma unroll
            for (int f = 0; f < kFly; ++f) {
                const int jj = j + f * kStep;
                y[f].clear();
                if (jj < outside) y[f].load(x + (jj < s_left ? T0 - 1 - jj : T0 + nt + (jj - s_left)) * tb + piece * kBytes);
            }
#pragma unroll
            for (int f = 0; f < kFly; ++f) {
                const int jj = j + f * kStep;
                uint32_t m = y[f].amax();
                if (!PC::finite(m)) m = amax_finite(y[f]);
                m = PC::fp32_bits(m);
#pragma unroll
                for (int o = kPieceLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (piece == 0 && jj < outside) atomicMax(&s_max[jj < s_left ? 0 : last_run], m);
            }
        }
    }
    __syncthreads();
    // Lane l < kPerWarp: the exponent of the warp's token l and where its codes go
    uint8_t *codes = (is_v ? p.v_codes : p.k_codes) + (long long)h * kCacheD;
    const uint32_t row_bytes = (uint32_t)p.H * kCacheD;
    constexpr uint32_t kNoRow = ~0u;
    uint32_t row = kNoRow;
    float scale = 0.f;
    bool grow = false;
    int drop = 0, held = 0;
    if (lane < PC::kPerWarp) {
        const int t = warp * PC::kPerWarp + lane, page = s_page[t];
        if (page >= 0) {
            row = (uint32_t)page * (uint32_t)p.ps + (uint32_t)s_off[t];
            const int r = run_of(t), need = exponent_for(s_max[r]);
            const bool inside = r > 0 || s_left == 0;  // the run's first token is in this window
            held = s_off[r];
            if (!inside) place_of(p, T0 - s_left, held);
            const int e = held > 0 ? max(need, s_had[r]) : need;
            scale = pow2i(-e);
            if (inside && r == t) {
                drop = s_had[t] - e;
                grow = held > 0 && drop < 0;
                exps[(long long)page * p.H] = (int8_t)e;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint32_t to = __shfl_sync(0xffffffffu, row, i * kPer + sub);
        const float sc = __shfl_sync(0xffffffffu, scale, i * kPer + sub);
        if (to != kNoRow) *reinterpret_cast<uint2 *>(codes + (uint64_t)to * row_bytes + piece * 8) = w[i].codes(sc);
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, grow); m; m &= m - 1) {  // codes that such a page held before
        const int l = __ffs(m) - 1;
        const int rows = __shfl_sync(0xffffffffu, held, l);
        uint8_t *page = codes + (uint64_t)(__shfl_sync(0xffffffffu, row, l) - rows) * row_bytes;
        rescale_rows(page, row_bytes, rows, __shfl_sync(0xffffffffu, drop, l), lane);
    }
}

// The same by runs: a warp owns the runs that begin among its 16 tokens, for one kv head's
// K or V, and reads exactly their tokens. Everything meets by shuffles, no barrier, and no
// token is read twice where runs have at most 16 tokens; a longer run is read once for its
// maximum and once more (from L2) for its codes, 16 tokens at a time. 24k ragged bf16
// tokens x 8 heads 27.1 us (5.5 TB/s, 0.81 of the measured copy bandwidth): instructions
// and load latency. Each trimmed piece showed: infinities looked at once per lane instead of
// per row, maxima as bf16 pairs (max.xorsign.abs), the last row again instead of zeros 31.4
// -> 29.7; exponents read only where a run begins inside its page, runs from the ballot
// instead of shuffled pages -> 27.7; shifts for pages of a power of two and 32-bit row bytes
// -> 27.1.
// CTA: 8 warps on neighbouring heads of the same tokens.
constexpr int kSeg = 16;

template <bool kF32>
__global__ void __launch_bounds__(256, kF32 ? 2 : 4) append_runs_kernel(const AppendParams p) {
    using PC = Piece<kF32>;
    constexpr int kLoads = kSeg / kPer, kBytes = 16 * PC::kVecs;
    const int lane = threadIdx.x & 31;
    const int units = 2 * p.H;  // of a segment: K heads, then V heads
    const uint32_t gw = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const uint32_t seg = gw / (uint32_t)units;
    const int hv = (int)(gw - seg * (uint32_t)units);
    const long long T0 = (long long)seg * kSeg;
    if (T0 >= p.n) return;
    // lane l: token T0 - 1 + l
    int off;
    const int page = place_of(p, T0 - 1 + lane, off);
    const int before = __shfl_up_sync(0xffffffffu, page, 1);
    const uint32_t change = __ballot_sync(0xffffffffu, lane > 0 && page != before);
    const uint32_t lead = __ballot_sync(0xffffffffu, lane > 0 && page >= 0 && page != before);
    const uint32_t mine = lead & 0x1fffeu;  // runs that begin at tokens T0 .. T0 + 15
    if (mine == 0) return;
    const int last = 31 - __clz(mine);  // lane of the last of them; it ends at the next change
    const uint32_t after = change & ~((2u << last) - 1u);
    int end = after ? __ffs(after) - 1 : 32;  // lanes [first, end) are this warp's tokens,
    long long tail = 0;                        // and `tail` more tokens behind lane 31
    if (!after) {
        const int pg = __shfl_sync(0xffffffffu, page, 31);
        for (;;) {
            int o;
            const uint32_t m = __ballot_sync(0xffffffffu, place_of(p, T0 + 31 + tail + lane, o) == pg);
            const int k = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            tail += k;
            if (k < 32) break;
        }
    }
    const bool is_v = hv >= p.H;
    const int h = is_v ? hv - p.H : hv;
    const long long tb = is_v ? p.v_tok : p.k_tok;
    const int sub = lane / kPieceLanes, piece = lane % kPieceLanes;
    const char *x = (is_v ? p.v + h * p.v_head : p.k + h * p.k_head) + (T0 - 1 + sub) * tb + piece * kBytes;
    int8_t *exps = (is_v ? p.v_exp : p.k_exp) + h;
    uint8_t *codes = (is_v ? p.v_codes : p.k_codes) + (long long)h * kCacheD;
    const uint32_t row_bytes = (uint32_t)p.H * kCacheD;
    constexpr uint32_t kNoRow = ~0u;

    PC w[kLoads];
    // tokens T0 - 1 + at .. + count - 1 into w (the last one again where there are fewer than
    // 16); lane l < 16: the maximum of token l
    auto read = [&](long long at, int count) -> uint32_t {
        const char *src = x + at * tb;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) w[i].load(src + (min(i * kPer + sub, count - 1) - sub) * tb);
        uint32_t v[kLoads];
        piece_maxima(w, v);
        const uint32_t m = fold_max<PC>(v, piece);  // lane (sub, piece): token 2 (piece / 2) + sub
        static_assert(kPieceLanes / kLoads == 2 && kPer == 2, "eight loads of two rows");
        return __shfl_sync(0xffffffffu, m, (lane & 1) * kPieceLanes + (lane & 14));
    };
    // codes of the tokens in w: lane l < 16 has token l's row (kNoRow: none) and 2^-e
    auto write = [&](uint32_t row, float scale) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t to = __shfl_sync(0xffffffffu, row, i * kPer + sub);
            const float sc = __shfl_sync(0xffffffffu, scale, i * kPer + sub);
            if (to != kNoRow) *reinterpret_cast<uint2 *>(codes + (uint64_t)to * row_bytes + piece * 8) = w[i].codes(sc);
        }
    };
    // exponent of a run that begins at place `held` of its page; writes it
    auto exponent = [&](uint32_t amax, int pg, int held, int had, int &drop) -> int {
        const int need = exponent_for(amax), e = held > 0 ? max(need, had) : need;
        drop = held > 0 ? had - e : 0;
        exps[(long long)pg * p.H] = (int8_t)e;
        return e;
    };
    auto rescale = [&](int pg, int held, int drop) {
        rescale_rows(codes + (uint64_t)pg * p.ps * row_bytes, row_bytes, held, drop, lane);
    };

    for (int at = __ffs(mine) - 1; at < end;) {
        // up to 16 tokens that end with a run
        const uint32_t upto = at + kSeg >= 31 ? ~0u : (2u << (at + kSeg)) - 1u;  // lanes up to at + 16
        uint32_t stops = change & upto & ~((2u << at) - 1u);                     // run ends in (at, at + 16]
        if (end <= at + kSeg && end < 32) stops |= 1u << end;
        int stop = stops ? 31 - __clz(stops) : 0;
        if (end == 32 && tail == 0 && at + kSeg >= 32) stop = 32;
        if (stop > end) stop = end;
        if (stop > at) {
            // lane l < 16: token lane at + l
            const int src = min(at + lane, 31);
            int pg = __shfl_sync(0xffffffffu, page, src);
            const int o = __shfl_sync(0xffffffffu, off, src);
            const int count = stop - at;
            if (lane >= count) pg = -1;
            const bool begins = pg >= 0 && (lead >> src & 1);
            int had = 0;
            if (begins && o > 0) had = *reinterpret_cast<volatile int8_t *>(exps + (long long)pg * p.H);
            const uint32_t first = __ballot_sync(0xffffffffu, begins);
            const uint32_t next = change >> at & ~((2u << lane) - 1u);  // where this lane's run ends
            const int run_end = next ? min(__ffs(next) - 1, count) : count;
            uint32_t m = read(at, count);
            // maximum of the run at its first token: fold over the following tokens of the page
#pragma unroll
            for (int d = 1; d < kSeg; d <<= 1) {
                const uint32_t mu = __shfl_down_sync(0xffffffffu, m, d);
                if (lane + d < run_end) m = max(m, mu);
            }
            const uint32_t upto_me = first & (0xffffffffu >> (31 - lane));
            const int head = pg >= 0 && upto_me ? 31 - __clz(upto_me) : lane;
            int drop = 0, e = 0;
            if (pg >= 0 && head == lane) e = exponent(m, pg, o, had, drop);
            e = __shfl_sync(0xffffffffu, e, head);
            write(pg >= 0 ? (uint32_t)pg * (uint32_t)p.ps + (uint32_t)o : kNoRow, pow2i(-e));
            for (uint32_t g = __ballot_sync(0xffffffffu, drop < 0); g; g &= g - 1) {
                const int l = __ffs(g) - 1;
                rescale(__shfl_sync(0xffffffffu, pg, l), __shfl_sync(0xffffffffu, o, l), __shfl_sync(0xffffffffu, drop, l));
            }
            at = stop;
            continue;
        }
        // a run of more than 16 tokens, [at, at + len)
        const uint32_t more = change & ~((2u << at) - 1u);
        const long long len = more ? __ffs(more) - 1 - at : 32 - at + tail;
        const int pg = __shfl_sync(0xffffffffu, page, at), held = __shfl_sync(0xffffffffu, off, at);
        const int had = held > 0 ? *reinterpret_cast<volatile int8_t *>(exps + (long long)pg * p.H) : 0;
        uint32_t m = 0;
        for (long long t = 0; t < len; t += kSeg) m = max(m, read(at + t, (int)min((long long)kSeg, len - t)));
#pragma unroll
        for (int d = kSeg / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        m = __shfl_sync(0xffffffffu, m, 0);
        int drop = 0, e = 0;
        if (lane == 0) e = exponent(m, pg, held, had, drop);
        e = __shfl_sync(0xffffffffu, e, 0);
        drop = __shfl_sync(0xffffffffu, drop, 0);
        const float scale = pow2i(-e);
        for (long long n_seg = (len + kSeg - 1) / kSeg, j = n_seg - 1; j >= 0; --j) {  // the last 16 are still there
            const int count = (int)min((long long)kSeg, len - j * kSeg);
            if (j != n_seg - 1) read(at + j * kSeg, count);
            int o;
            const int q = lane < count ? place_of(p, T0 - 1 + at + j * kSeg + lane, o) : -1;
            write(q >= 0 ? (uint32_t)q * (uint32_t)p.ps + (uint32_t)o : kNoRow, scale);
        }
        if (drop < 0) rescale(pg, held, drop);
        at = more ? at + (int)len : 32;
    }
}

int current_sms(int *dev_out) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        return -1;
    if (dev_out) *dev_out = dev;
    return sms;
}

}  // namespace

int launch_page_tables(int32_t batch, int32_t page_size, const int32_t *cached_lens, const int32_t *new_lens,
                       const int32_t *free_pages, int64_t free_capacity, const int32_t *num_free, int32_t *block_table,
                       int64_t block_table_stride, int32_t max_pages_per_request, int32_t *kv_indptr,
                       int32_t *last_page_len, int32_t *kv_indices, int64_t cap_pages, int32_t *qo_indptr,
                       int64_t *slot_map, int32_t *positions, int64_t cap_tokens, int32_t *counts,
                       cudaStream_t stream) {
    if (batch > kTabMaxBatch)
        return fail(BSP_ERR_UNSUPPORTED, "build_page_tables takes at most " + std::to_string(kTabMaxBatch) + " requests");
    int dev = 0;
    const int sms = current_sms(&dev);
    if (sms < 0) return fail(BSP_ERR_CUDA, "no current CUDA device");
    TableParams p;
    p.cached = cached_lens;
    p.fresh = new_lens;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.free_capacity = free_capacity;
    p.table = block_table;
    p.table_stride = block_table_stride;
    p.width = max_pages_per_request;
    p.batch = batch;
    p.ps = page_size;
    p.kv_indptr = kv_indptr;
    p.last_page_len = last_page_len;
    p.kv_indices = kv_indices;
    p.qo_indptr = qo_indptr;
    p.positions = positions;
    p.counts = counts;
    p.slots = reinterpret_cast<long long *>(slot_map);
    p.cap_pages = cap_pages;
    p.cap_tokens = cap_tokens;
    const size_t smem = 3 * sizeof(int) * (size_t)(batch + 1);
    static bool configured[64] = {false};
    if (!configured[dev]) {  // (the default limit counts the kernel's static shared memory too)
        cudaError_t e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(3 * sizeof(int) * (kTabMaxBatch + 1)));
        if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("page tables smem attribute: ") + cudaGetErrorString(e));
        configured[dev] = true;
    }
    const int64_t groups = (cap_pages + kTabUnit - 1) / kTabUnit + (cap_tokens + kTabUnit - 1) / kTabUnit;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((groups + kTabThreads - 1) / kTabThreads, 4ll * sms));
    page_tables_kernel<<<(unsigned)grid, kTabThreads, smem, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("page tables launch: ") + cudaGetErrorString(e));
    return BSP_OK;
}

int launch_append_kv(const void *k, const void *v, int64_t k_token_stride, int64_t k_head_stride,
                     int64_t v_token_stride, int64_t v_head_stride, int32_t dtype, int64_t n_tokens,
                     const int64_t *slot_map, void *k_pages, void *v_pages, int8_t *k_exp, int8_t *v_exp,
                     int64_t num_pages, int32_t page_size, int32_t num_kv_heads, cudaStream_t stream) {
    const int64_t elem = dtype == BSP_DTYPE_F32 ? 4 : 2;
    // By runs: pages of up to 16 tokens (24k ragged bf16 tokens into 16-token pages 27.5 us
    // against 36.1 by windows, single-token pages 28.0 / 37.7, fp32 46.1 / 58.3; 256 tokens 3.5 /
    // 3.7), and larger ones where their runs, each read by one warp, fill the GPU: 24k tokens
    // into 64- and 128-token pages 36.1 / 38.4 and 42.3 / 46.3, 49k fp32 tokens into 64-token
    // pages 101 / 116; about even at 3,100 runs (6.2k bf16 tokens into 32-token pages 10.5 /
    // 10.5) and at half as many of fp32 (6.2k tokens into 64-token pages 16.3 / 16.5). Windows
    // below that: 3.1k bf16 tokens into 32-token pages 8.1 / 5.8, one prompt of 256 tokens into
    // 128-token pages 16.1 / 3.7. (Each window of a page reads the whole run: 32k tokens into one
    // page of 4,096 / 16,384 / 32,768 tokens after the other take 0.8 / 3.4 / 7.6 ms.)
    const int64_t warps = (n_tokens + kSeg - 1) / kSeg * 2 * num_kv_heads;
    const bool runs = page_size <= kSeg || n_tokens * 2 * num_kv_heads / page_size * elem >= 3000 * 2;
    const int64_t ctas = runs ? (warps + 7) / 8 : (n_tokens + kAppTokens - 1) / kAppTokens * 2 * num_kv_heads;
    if (ctas > INT32_MAX / 8) return fail(BSP_ERR_UNSUPPORTED, "too many tokens for one append");
    AppendParams p;
    p.k = static_cast<const char *>(k);
    p.v = static_cast<const char *>(v);
    p.k_tok = k_token_stride * elem;
    p.k_head = k_head_stride * elem;
    p.v_tok = v_token_stride * elem;
    p.v_head = v_head_stride * elem;
    p.k_codes = static_cast<uint8_t *>(k_pages);
    p.v_codes = static_cast<uint8_t *>(v_pages);
    p.k_exp = k_exp;
    p.v_exp = v_exp;
    p.slots = reinterpret_cast<const long long *>(slot_map);
    p.n = n_tokens;
    p.rows = (long long)num_pages * page_size;
    p.ps = page_size;
    p.H = num_kv_heads;
    p.ps_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (page_size == 1 << i) p.ps_shift = i;
    if (runs) {
        if (dtype == BSP_DTYPE_F32) append_runs_kernel<true><<<(unsigned)ctas, 256, 0, stream>>>(p);
        else append_runs_kernel<false><<<(unsigned)ctas, 256, 0, stream>>>(p);
    } else if (dtype == BSP_DTYPE_F32) append_kernel<true><<<(unsigned)ctas, 32 * Piece<true>::kWarps, 0, stream>>>(p);
    else append_kernel<false><<<(unsigned)ctas, 32 * Piece<false>::kWarps, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("append launch: ") + cudaGetErrorString(e));
    return BSP_OK;
}

}  // namespace bsp
