// Eviction of cached tokens by the attention weight that they gathered (no counterpart on
// the pages): the weights' update after an attention run, the choice of the tokens to keep,
// and the move of their rows to the front of their request's pages.
//
// Gathered weights: float [num_pages][H_kv][page_size], one per cached token and kv head.
// Requests come as a page table in CSR form on the device (kv_indptr, kv_indices,
// last_page_len), as bsp_build_page_tables writes it; nothing is planned on the host.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "bsp_internal.h"
#include "device_common.cuh"
#include "evict.cuh"
#include "sm100.cuh"

namespace bsp {
namespace {

using namespace dev;
using namespace evict;
namespace cg = cooperative_groups;

// 2^e for e in [-149, 127]
__device__ __forceinline__ float pow2i(int e) { return __int_as_float(e >= -126 ? (e + 127) << 23 : 0x00400000 >> (-127 - e)); }

// ---------------------------------------------------------------- gathered weights
// For each key j of a request and kv head h:
//   w[j, h] = base + sum over queries i that see j, heads r of h: p,   p = exp(s_ijr - LSE_ir)
// (differential: p = |p1 - lam_r p2|), base = decay * w[j, h], or 0 for the last qo_len keys,
// the queries' own. Every key is summed by one thread group in one order: no atomics, the
// same result every time.
// bf16 pools (and e4m3 ones with exponents), few queries per request: bound by the read of K.
// One persistent CTA per SM takes a contiguous run of tasks (32 keys of one kv head, in the order
// request, head, keys), so that every SM reads the same number of keys and a query's fragments
// stay in a warp's registers from task to task.
//   6 warps (8 over rows of 128 bytes) look tokens up, a task each in turn, and leave rows, weights
//     and exponents in a ring: the chain of dependent reads (request, page id, weight) runs ahead of
//     the warps that need it (with 4 of them 9 us more in both forms below)
//   12 (16) warps compute, a task each in turn: 16-byte asynchronous copies bring the rows of the
//     next task into the warp's own two buffers (any page size alike) while one is worked on;
//     S = K Q^T by m16n8k16, keys on the M side, queries on the N side. The order of the head
//     dimension inside a product is free, so a lane's 16 adjacent bytes of a K row are fragment
//     words as they are, and q is read the same way.
// 64 requests up to 8192 tokens, us: warps that look up their own keys and load them into
// registers 120, with a ring of bulk copies per warp 153, loader warps and bulk copies 198 (one
// bulk copy per row: an SM starts one in about 25 cycles, whatever its size), now 97-99 (5.8-5.9 TB/s);
// 32 x 4096 tokens of an 8-bit cache 34.6 (4.1 TB/s).
constexpr int kTaskTokens = 32;

template <int D, bool kE4m3>
struct StreamLayout {
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);      // bytes of a K row
    static constexpr int kLoaders = kRow == 256 ? 6 : 8, kCompute = 2 * kLoaders, kThreads = 32 * (kLoaders + kCompute);
    static constexpr int kBufs = 2;                       // tasks' rows per compute warp
    static constexpr int kBuf = kTaskTokens * kRow;
    // ring of looked-up tasks: per token its weight's index, row, old weight and 2^exp; then
    // request, head, first key, tokens
    static constexpr int kStages = kBufs * kCompute + 2 * kLoaders;
    static constexpr int kStageBytes = kTaskTokens * 20 + 16;
    // A stage's look-ups have one order, and a barrier is never asked about a phase but the next: the
    // stage always has the same loader, and a compute warp's task before comes from that loader too
    // and not before the stage's previous one. (With 19 stages a loader could pass another one that
    // still waited for the same stage.) A compute warp holds kBufs stages.
    static_assert(kStages % kLoaders == 0 && kCompute % kLoaders == 0 && kStages >= kBufs * kCompute, "order of a stage's look-ups");
    static constexpr int kRingOff = kCompute * kBufs * kBuf;
    static constexpr int kBarOff = kRingOff + kStages * kStageBytes;
    static constexpr int kSmem = kBarOff + 2 * kStages * 8 + 8;
    static_assert(kSmem <= 227 * 1024, "weights ring exceeds shared memory");
};

// The queries' side of up to 8 columns: (query, head) pairs, differential 4 pairs of maps.
template <int kSteps>
struct Columns {
    uint32_t q[kSteps][2];
    float lse[2], scale[2], lam;  // of this lane's accumulator columns 2c, 2c + 1
    int pos[2];                   // keys up to this place see them; -1: none
};

template <int D, bool kE4m3, bool kDiff>
__device__ __forceinline__ void load_columns(const WeightsParams &p, const Queries &qs, int off, int h, int col, int col_hi,
                                             int lane, Columns<D / 16> &x) {
    constexpr int kJ = D * (kE4m3 ? 1 : 2) / 64, kSteps = D / 16;
    const int c = lane & 3, n = lane >> 2, g = p.g;
    // this lane's column of Q^T, n: its query row, and the half of it (differential)
    const int cn = col + (kDiff ? n >> 1 : n);
    const int qi = cn / g, r = cn - qi * g;
    const bool in = cn < col_hi;
    const size_t qrow = (size_t)(qs.q0 + (in ? qi : 0)) * p.H_qo + (size_t)h * g + (in ? r : 0);
    float lse2 = in ? __ldg(p.lse + (kDiff ? 2 * qrow + (n & 1) : qrow)) : -INFINITY;
    const bool live = lse2 != -INFINITY;
    lse2 *= kLog2e;
    const float lam = kDiff && in ? __ldg(p.lam + h * g + r) : 0.f;
    float scale = p.soft_cap_on ? p.cap_in : p.scale_log2;
    const uint4 *qp = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + qrow * D) + (kE4m3 ? 2 * c : c);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const bool mine = in && (!kDiff || (j >= kJ / 2) == (n & 1));
#pragma unroll
        for (int e = 0; e < (kE4m3 ? 2 : 1); ++e) {
            const uint4 w = mine ? __ldg(qp + j * (kE4m3 ? 8 : 4) + e) : make_uint4(0, 0, 0, 0);
            const int st = kE4m3 ? 4 * j + 2 * e : 2 * j;
            x.q[st][0] = w.x; x.q[st][1] = w.y;
            x.q[st + 1][0] = w.z; x.q[st + 1][1] = w.w;
        }
    }
    if constexpr (kE4m3) {
        // bf16 -> f16: the row times the power of two that takes its largest value to 2^14 .. 2^15
        // (values from 2^-31 of the largest on are exact); rows with an infinity or NaN as they are
        uint32_t mx = 0;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) mx = __vmaxu2(mx, __vmaxu2(x.q[st][0] & 0x7fff7fffu, x.q[st][1] & 0x7fff7fffu));
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int E = (int)(mx >> 7), up = E == 255 ? 0 : min(120, 141 - E);
        const float f = pow2i(up);
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float lo = bf16_lo(x.q[st][e]) * f, hi = bf16_hi(x.q[st][e]) * f;
                asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(x.q[st][e]) : "f"(hi), "f"(lo));
            }
        scale *= pow2i(-up);
    }
    // of the columns 2c and 2c + 1 of the product
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int from = 4 * (2 * c + e);
        x.lse[e] = __shfl_sync(0xffffffffu, lse2, from);
        x.scale[e] = __shfl_sync(0xffffffffu, scale, from);
        const int i = __shfl_sync(0xffffffffu, qi, from);
        const bool l = __shfl_sync(0xffffffffu, (int)live, from);
        x.pos[e] = l ? off + i : -1;
    }
    x.lam = kDiff ? __shfl_sync(0xffffffffu, lam, 8 * c) : 0.f;
}

// Where task x of a run's order (request, head, keys) lies; in range for tables that do not ascend. All lanes of a warp.
struct Task {
    int b, h, blk, nblk;  // request, head, block of keys, blocks of the request
};
__device__ __forceinline__ int blocks_of(const Csr &c, int b) {
    return (int)max(1ll, block_start<kTaskTokens>(c, b + 1) - block_start<kTaskTokens>(c, b));
}
__device__ __forceinline__ Task find_task(const WeightsParams &p, long long start0, long long x, int lane) {
    Task t;
    t.b = find_request<kTaskTokens>(p.csr, start0 + x / p.H_kv, lane);
    t.nblk = blocks_of(p.csr, t.b);
    const long long in = max(0ll, x - (block_start<kTaskTokens>(p.csr, t.b) - start0) * p.H_kv);
    t.h = (int)min(in / t.nblk, (long long)p.H_kv - 1);
    t.blk = (int)(in % t.nblk);
    return t;
}

// kVar: window and soft-cap compiled in.
template <int D, bool kE4m3, bool kDiff, bool kVar, bool kStall>
__global__ void __launch_bounds__(StreamLayout<D, kE4m3>::kThreads, 1) weights_kernel(const WeightsParams p) {
    using LY = StreamLayout<D, kE4m3>;
    constexpr int kJ = LY::kRow / 64;           // 16-byte chunks of a row per lane
    constexpr int kStages = LY::kStages;
    constexpr int kCols = kDiff ? 4 : 8;        // (query, head) pairs per column tile
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = p.H_kv, g = p.g, ps = p.csr.ps;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + LY::kBarOff + 2 * kStages * 8);
    const uint32_t full0 = smem_u32(smem) + LY::kBarOff, empty0 = full0 + kStages * 8;
    const long long start0 = block_start<kTaskTokens>(p.csr, 0);
    const long long tasks = (block_start<kTaskTokens>(p.csr, p.csr.batch) - start0) * H;
    const long long task0 = tasks * blockIdx.x / gridDim.x, task1 = tasks * (blockIdx.x + 1) / gridDim.x;
    const int count = (int)(task1 - task0);
    if (count <= 0) return;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * kStages; ++s) sm100::mbar_init(full0 + 8 * s, 1);
        *abort_flag = 0;
        sm100::fence_barrier_init();
    }
    __syncthreads();
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool ok = __all_sync(0xffffffffu, sm100::mbar_wait_spin(bar, parity, kStall ? p.wait_limit : kWaitLimitCycles, abort_flag));
        if (!ok) *abort_flag = 1;
        return ok;
    };

    if (warp < LY::kLoaders) {
        // this warp's place in the run: request, head, block of keys
        const Task first = find_task(p, start0, min(task0 + warp, tasks - 1), lane);
        int b = first.b, h = first.h, blk = first.blk, nblk = first.nblk;
        Request rq = request(p.csr, b);
        // two tasks on their way: asked for (page ids), then looked up (weights, exponents); each
        // step's reads are in flight for a turn of the loop
        struct { int b, h, t0, len, id, place; } ask = {0, 0, -1, 0, 0, 0};
        struct { int b, h, t0, len, exp; uint32_t row; long long at; float old; } got = {0, 0, -1, 0, 0, kNoRow, -1, 0.f};
        for (int k = warp - 2 * LY::kLoaders; k < count; k += LY::kLoaders) {
            if (k >= 0) {
                const int s = k % kStages;
                if (kStall && warp == 0 && k >= LY::kLoaders) return;
                if (!wait(empty0 + 8 * s, ((k / kStages) & 1) ^ 1)) return;
                uint8_t *stage = smem + LY::kRingOff + s * LY::kStageBytes;
                reinterpret_cast<long long *>(stage)[lane] = got.at;
                reinterpret_cast<uint32_t *>(stage)[64 + lane] = got.row;
                reinterpret_cast<float *>(stage)[96 + lane] = got.old;
                reinterpret_cast<float *>(stage)[128 + lane] = kE4m3 ? pow2i(got.exp) : 1.f;
                if (lane == 0) *reinterpret_cast<int4 *>(stage + kTaskTokens * 20) = make_int4(got.b, got.h, got.t0, got.len);
                __syncwarp();
                if (lane == 0) sm100::mbar_arrive(full0 + 8 * s);
            }
            // the page ids are here: rows, weights and exponents
            got = {ask.b, ask.h, ask.t0, ask.len, 0, kNoRow, -1, 0.f};
            if (ask.t0 >= 0 && ask.t0 + lane < ask.len && (unsigned)ask.id < (unsigned)p.csr.num_pages) {
                got.row = (uint32_t)ask.id * (uint32_t)ps + (uint32_t)ask.place;
                got.at = ((long long)ask.id * H + ask.h) * ps + ask.place;
                if (kE4m3) got.exp = __ldg(p.k_exp + (size_t)ask.id * H + ask.h);
                if (p.decay != 0.f) got.old = p.weights[got.at];  // (not used for the queries' own keys)
            }
            // the next task's page ids
            ask.t0 = -1;
            if (k + 2 * LY::kLoaders >= count || b >= p.csr.batch) continue;
            const int t0 = blk * kTaskTokens, t = t0 + lane;
            if (t0 < rq.len) {
                const int col = div_ps(p.csr, t);
                ask = {b, h, t0, rq.len, t < rq.len ? __ldg(p.csr.kv_indices + rq.p0 + col) : 0, t - col * ps};
            }
            blk += LY::kLoaders;
            while (blk >= nblk && b < p.csr.batch) {
                blk -= nblk;
                if (++h == H) {
                    h = 0;
                    if (++b < p.csr.batch) {
                        rq = request(p.csr, b);
                        nblk = blocks_of(p.csr, b);
                    }
                }
            }
        }
        return;
    }

    const int c = lane & 3, n = lane >> 2;
    int qb = -1, qh = -1;
    Queries qs = {0, 0};
    Columns<D / 16> x;
    const uint32_t bufs = smem_u32(smem) + (warp - LY::kLoaders) * LY::kBufs * LY::kBuf;
    // the rows of task k into buffer u, one group of copies (none behind the last task)
    auto copy = [&](int k, int u) -> bool {
        if (k < count) {
            const int s = k % kStages;
            if (!wait(full0 + 8 * s, (k / kStages) & 1)) return false;
            const uint32_t *row = reinterpret_cast<const uint32_t *>(smem + LY::kRingOff + s * LY::kStageBytes) + 64;
            const int h = *reinterpret_cast<const int *>(smem + LY::kRingOff + s * LY::kStageBytes + kTaskTokens * 20 + 4);
            constexpr int kC = LY::kRow / 16, kT = 32 / kC;  // chunks of a row, rows per instruction
            const int ch = lane % kC, sub = lane / kC;
            const char *base = static_cast<const char *>(p.k) + (size_t)h * LY::kRow + ch * 16;
            const size_t stride = (size_t)H * LY::kRow;
#pragma unroll
            for (int i = 0; i < kTaskTokens / kT; ++i) {
                const int t = i * kT + sub;
                const uint32_t r = row[t];
                // (chunks of odd rows in the other half of their 128 bytes: the reads below meet no bank twice)
                if (r != kNoRow) cp_async_16(bufs + u * LY::kBuf + t * LY::kRow + ((ch ^ ((t & 1) << 2)) << 4), base + r * stride, 16);
            }
        }
        cp_async_commit();
        return true;
    };
    int k = warp - LY::kLoaders;
    bool ok = copy(k, 0);
    for (int u = 0; k < count && ok; k += LY::kCompute, u ^= 1) {
        if (!(ok = copy(k + LY::kCompute, u ^ 1))) break;
        cp_async_wait<1>();
        __syncwarp();
        const int s = k % kStages;
        const uint8_t *stage = smem + LY::kRingOff + s * LY::kStageBytes;
        const int4 m = *reinterpret_cast<const int4 *>(stage + kTaskTokens * 20);
        const int b = m.x, h = m.y, t0 = m.z, len = m.w;
        // 2^exponent of the rows n + 8 i, and this lane's own key, n + 8 c
        float kf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kf[i] = kE4m3 ? reinterpret_cast<const float *>(stage)[128 + n + 8 * i] : 1.f;
        const long long at = reinterpret_cast<const long long *>(stage)[n + 8 * c];
        const float old = reinterpret_cast<const float *>(stage)[96 + n + 8 * c];
        __syncwarp();  // the stage is read
        if (lane == 0) sm100::mbar_arrive(empty0 + 8 * s);
        const uint32_t rows = bufs + u * LY::kBuf + n * LY::kRow + ((c ^ ((n & 1) << 2)) << 4);
        if (t0 < 0) continue;  // an empty block of the table

        if (b != qb) qs = queries(p, b);
        const int off = len - qs.n;  // position of the first query
        // columns (query i, head r) = i * g + r that any of the 32 keys can see
        const int i_lo = max(0, t0 - off);
        const int i_hi = kVar && p.window > 0 ? (int)min((long long)qs.n, (long long)t0 + kTaskTokens + p.window - off) : qs.n;
        const bool one = qs.n * g <= kCols;  // all in one tile, kept from task to task
        const int col_lo = one ? 0 : i_lo * g / kCols * kCols, col_hi = one ? qs.n * g : i_hi * g;
        if (one && (b != qb || h != qh)) load_columns<D, kE4m3, kDiff>(p, qs, off, h, 0, col_hi, lane, x);
        qb = b;
        qh = h;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int col = col_lo; col < col_hi; col += kCols) {
            if (!one) load_columns<D, kE4m3, kDiff>(p, qs, off, h, col, col_hi, lane, x);
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                uint4 kw[2][kJ];  // rows n + 16 sb and 8 further
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < kJ; ++j) kw[i][j] = sm100::ld_shared_v4((rows + 8 * (2 * sb + i) * LY::kRow) ^ (j * 64));
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const uint4 u = kw[0][j], v = kw[1][j];
                    if constexpr (kE4m3) {
                        const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t a[4];
                            e4m3x4_to_f16x4(us[e], a[0], a[2]);
                            e4m3x4_to_f16x4(vs[e], a[1], a[3]);
                            mma_f16_16816(d[e & 1], a, x.q[4 * j + e][0], x.q[4 * j + e][1]);
                        }
                    } else {
                        const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                        mma_bf16_16816(d[0], a0, x.q[2 * j][0], x.q[2 * j][1]);
                        mma_bf16_16816(d[1], a1, x.q[2 * j + 1][0], x.q[2 * j + 1][1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // rows n + 8 (2 sb + i)
                    const int row = 2 * sb + i, tok = t0 + n + 8 * row;
                    float pe[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = kE4m3 ? x.scale[e] * kf[row] : x.scale[e];
                        float y = d[0][2 * i + e] + d[1][2 * i + e];
                        if (kVar && p.soft_cap_on) y = fmaf(tanh_f32(y * f), p.cap_out, -x.lse[e]);
                        else y = fmaf(y, f, -x.lse[e]);
                        const bool see = tok <= x.pos[e] && (!kVar || p.window <= 0 || tok >= x.pos[e] - p.window);
                        pe[e] = see ? ex2(y) : 0.f;
                    }
                    sum[row] += kDiff ? fabsf(pe[0] - x.lam * pe[1]) : pe[0] + pe[1];
                }
            }
        }
        float own = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
            if (i == c) own = sum[i];
        }
        __syncwarp();  // the buffer is read
        if (at >= 0) p.weights[at] = t0 + n + 8 * c < off && p.decay != 0.f ? fmaf(p.decay, old, own) : own;
    }
    cp_async_wait<0>();  // nothing in flight at exit
    for (; !ok && k < count; k += LY::kCompute) {  // a wait gave up
        const Task task = find_task(p, start0, task0 + k, lane);
        const Request rq = request(p.csr, task.b);
        const long long t = (long long)task.blk * kTaskTokens + lane;
        int page, place;
        if (t < rq.len && slot_of(p.csr, rq, (int)t, page, place) != kNoRow) p.weights[((size_t)page * H + task.h) * ps + place] = NAN;
    }
}

// fp32 pools: a warp takes a task's 32 keys, eight at a time (8 lanes per row, two rows a lane group),
// fp32 products on the CUDA cores.
template <int D>
__global__ void __launch_bounds__(256) weights_f32_kernel(const WeightsParams p) {
    constexpr int kJ = D / 32;
    const int lane = threadIdx.x & 31, l8 = lane & 7, sub = lane >> 3;
    const int H = p.H_kv, g = p.g;
    const long long start0 = block_start<kTaskTokens>(p.csr, 0), blocks = block_start<kTaskTokens>(p.csr, p.csr.batch) - start0;
    const long long nwarps = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long task = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); task < blocks * H; task += nwarps) {
        const long long blk = start0 + task / H;
        const int h = (int)(task % H);
        const int b = find_request<kTaskTokens>(p.csr, blk, lane);
        const Request rq = request(p.csr, b);
        const long long first = (blk - block_start<kTaskTokens>(p.csr, b)) * kTaskTokens;
        if (first < 0 || first >= rq.len) continue;  // (below 0: a table that does not ascend)
        const Queries qs = queries(p, b);
        const int off = rq.len - qs.n;
        for (int t0 = (int)first; t0 < min(rq.len, (int)first + kTaskTokens); t0 += 8) {
            float4 kw[2][kJ];
            uint32_t slot[2];
            int tok[2], page[2] = {0, 0}, place[2] = {0, 0};
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                tok[u] = t0 + sub + 4 * u;
                slot[u] = tok[u] < rq.len ? slot_of(p.csr, rq, tok[u], page[u], place[u]) : kNoRow;
                const float4 *kr = reinterpret_cast<const float4 *>(static_cast<const float *>(p.k) + ((size_t)(slot[u] != kNoRow ? slot[u] : 0) * H + h) * D) + l8;
#pragma unroll
                for (int j = 0; j < kJ; ++j) kw[u][j] = slot[u] != kNoRow ? __ldg(kr + 8 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const int i_lo = max(0, t0 - off), i_hi = p.window > 0 ? (int)min((long long)qs.n, (long long)t0 + 8 + p.window - off) : qs.n;
            for (int i = i_lo; i < i_hi; ++i)
                for (int r = 0; r < g; ++r) {
                    const size_t qrow = (size_t)(qs.q0 + i) * p.H_qo + (size_t)h * g + r;
                    const float4 *qp = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + qrow * D) + l8;
                    const float lse = __ldg(p.lse + qrow);
                    float d[2] = {0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const float4 x = __ldg(qp + 8 * j);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            d[u] = fmaf(x.x, kw[u][j].x, fmaf(x.y, kw[u][j].y, fmaf(x.z, kw[u][j].z, fmaf(x.w, kw[u][j].w, d[u]))));
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) d[u] += __shfl_xor_sync(0xffffffffu, d[u], o);
                        const float x = p.soft_cap_on ? tanh_f32(d[u] * p.cap_in) * p.cap_out : d[u] * p.scale_log2;
                        const bool see = tok[u] <= off + i && (p.window <= 0 || tok[u] >= off + i - p.window) && lse != -INFINITY;
                        if (see) sum[u] += exp2f(x - lse * kLog2e);
                    }
                }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (slot[u] != kNoRow && l8 == 0) {
                    float *at = p.weights + ((size_t)page[u] * H + h) * p.csr.ps + place[u];
                    const float old = tok[u] < off && p.decay != 0.f ? *at : 0.f;
                    *at = fmaf(p.decay, old, sum[u]);
                }
        }
    }
}

// ---------------------------------------------------------------- choice of the tokens to keep
// Per (request, kv head) the n = min(tokens, budget, max_keep) tokens of the largest weights,
// protected ones (the first `sinks`, the last `recent`) counting as +inf, NaN as -inf, equal
// weights by the lower position; written as ascending positions. A radix selection of the n-th
// largest key over 11 + 11 + 10 bits, then one stable compaction. A cluster of CTAs takes one
// row of tokens, a contiguous part each; a thread holds 16 of its part's keys in registers (parts
// beyond 8192 tokens are read again in every pass). The first CTA of the cluster adds up the
// others' bins that are not empty and finds the digit (every CTA reading all histograms instead
// took 60 of 91 thousand cycles: an SM reads others' shared memory at 10 bytes a cycle or so).
//
// Bound by instructions and latency, not by the 4 bytes per token: 64 requests x 8 heads x 5100
// tokens on average, us: keys in shared memory and one read at a time 33, all reads of a thread in
// flight together 25, keys in registers 19; one request of 131,072 tokens 57, 28, 19.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 16;                       // keys per thread
constexpr int kSelChunk = kSelThreads * kSelKeys;  // tokens of a part in registers
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;
static_assert(kBins == 4 * kSelThreads, "four bins per thread");

struct SelectParams {
    Csr csr;
    const float *weights;
    const int32_t *budget;
    int32_t *kept, *new_lens;
    int H, max_keep, sinks, recent;
};

// kOne: a CTA per row.
template <bool kOne>
struct SelectShared {
    int hist[kBins];
    int all[kOne ? 1 : 3][kOne ? 4 : kBins];  // the cluster's, per pass (of the first CTA)
    int counts[2];             // keys above the threshold and equal to it, this CTA
    int warp_sum[kSelWarps];
    uint32_t totals[kSelKeys * kSelWarps];  // of a chunk, by group and warp: above | equal << 16
    int2 found[3];  // digit of the n-th largest key, keys above it, per pass
};

// Order-preserving whole number of a weight; never 0
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Conditional additions to shared memory and stores as predicated instructions (as branches they
// took three times the instructions; an SM's instructions are what the many rows wait for).
__device__ __forceinline__ void add_shared_if(bool cond, uint32_t addr, int x) {
    asm volatile("{ .reg .pred p;\n setp.ne.s32 p, %0, 0;\n @p red.shared.add.s32 [%1], %2;\n}" ::"r"((int)cond), "r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void store_if(bool cond, int32_t *p, int x) {
    asm volatile("{ .reg .pred p;\n setp.ne.s32 p, %0, 0;\n @p st.global.s32 [%1], %2;\n}" ::"r"((int)cond), "l"(p), "r"(x) : "memory");
}

// kV: tokens per load, 4 (page sizes that are multiples of 4) or 1
template <int kV, bool kOne>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelectParams p) {
    constexpr int kGroups = kSelKeys / kV;
    __shared__ __align__(16) SelectShared<kOne> sh;
    cg::cluster_group cl = cg::this_cluster();
    const int C = kOne ? 1 : (int)cl.num_blocks(), rank = kOne ? 0 : (int)cl.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / C, b = row / p.H, h = row - b * p.H;
    const Request rq = request(p.csr, b);
    const int n = min(min(rq.len, max(__ldg(p.budget + b), 0)), p.max_keep);
    int32_t *kept = p.kept + (size_t)row * p.max_keep;
    if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = n;
    const int gt = rank * kSelThreads + tid, gn = C * kSelThreads;
    for (int j = n + gt; j < p.max_keep; j += gn) kept[j] = -1;
    if (n == rq.len || n == 0) {  // the same for the whole cluster
        for (int j = gt; j < n; j += gn) kept[j] = j;
        return;
    }
    const int part = ((rq.len + C - 1) / C + 31) & ~31;  // tokens per CTA
    const int t_lo = min(rank * part, rq.len), m = min(part, rq.len - t_lo);
    const int chunks = (m + kSelChunk - 1) / kSelChunk;
    // groups of chunk c that hold a token (the same for all threads: the others are skipped)
    auto groups = [&](int c) { return min(kGroups, (m - c * kSelChunk + kSelThreads * kV - 1) / (kSelThreads * kV)); };
    reinterpret_cast<int4 *>(sh.hist)[tid] = make_int4(0, 0, 0, 0);
    if (!kOne && rank == 0) {
        for (int i = tid; i < 3 * kBins / 4; i += kSelThreads) reinterpret_cast<int4 *>(&sh.all[0][0])[i] = make_int4(0, 0, 0, 0);
    }
    // a chunk's keys: group u of this thread begins at token (u * threads + tid) * kV of it (the kV tokens
    // lie in one page); 0 behind the part
    uint32_t key[kSelKeys];
    auto load = [&](int c) {
        const int i0 = c * kSelChunk + tid * kV;
        int page[kGroups], place[kGroups];
        bool in[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            const int i = i0 + u * kSelThreads * kV;
            page[u] = place[u] = 0;
            in[u] = i < m && slot_of(p.csr, rq, t_lo + i, page[u], place[u]) != kNoRow;
        }
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            const float *w = p.weights + ((size_t)page[u] * p.H + h) * p.csr.ps + place[u];
            float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (in[u]) {
                if (kV == 4) x = __ldg(reinterpret_cast<const float4 *>(w));
                else x.x = __ldg(w);
            }
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int v = 0; v < kV; ++v) key[u * kV + v] = __float_as_uint(xs[v]);
        }
        const int lo = p.sinks - t_lo, hi = min(m, rq.len - p.recent - t_lo);  // protected: i < lo or i >= hi
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            const int i = i0 + u * kSelThreads * kV;
#pragma unroll
            for (int v = 0; v < kV; ++v) key[u * kV + v] = order_key(__uint_as_float(key[u * kV + v]));
            if (i < lo || i + kV > hi) {
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    if (i + v < lo || i + v >= hi) key[u * kV + v] = order_key(INFINITY);
                    if (i + v >= m) key[u * kV + v] = 0u;
                }
            }
        }
    };
    if (chunks) load(0);
    if (kOne) __syncthreads();
    else cl.sync();

    uint32_t prefix = 0;
    int need = n;  // how many of the keys that match the prefix are still to be taken
    auto run_pass = [&](auto number) {
        constexpr int pass = decltype(number)::value, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        int *hist = sh.hist;
        const uint32_t hist_at = smem_u32(hist);
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1 && (pass > 0 || c > 0)) load(c);
            const int G = groups(c);
            const uint32_t lo = pass == 0 ? 0u : prefix << ((shift + bits) & 31);  // keys from lo on, of this prefix
#pragma unroll
            for (int u = 0; u < kGroups; ++u) {
                if (u >= G) break;
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const uint32_t k = key[u * kV + v], d = k - lo;
                    // (a key behind the part, 0, is below every prefix, and in bin 0 it counts for nothing)
                    if (pass == 0) atomicAdd(&hist[k >> 21], 1);
                    else add_shared_if(d >> ((shift + bits) & 31) == 0, hist_at + (d >> shift) * 4, 1);
                }
            }
        }
        __syncthreads();
        // four bins per thread, the highest first; zero again for the next pass
        const int lo_bin = kBins - 4 - 4 * tid;
        int4 c4 = *reinterpret_cast<const int4 *>(hist + lo_bin);
        *reinterpret_cast<int4 *>(hist + lo_bin) = make_int4(0, 0, 0, 0);
        if constexpr (!kOne) {
            int *all = cl.map_shared_rank(sh.all[pass], 0) + lo_bin;
            if (c4.x) atomicAdd(all, c4.x);
            if (c4.y) atomicAdd(all + 1, c4.y);
            if (c4.z) atomicAdd(all + 2, c4.z);
            if (c4.w) atomicAdd(all + 3, c4.w);
            cl.sync();
            c4 = rank == 0 ? *reinterpret_cast<const int4 *>(sh.all[pass] + lo_bin) : make_int4(0, 0, 0, 0);
        }
        const int cnt[4] = {c4.w, c4.z, c4.y, c4.x};
        const int mine = (cnt[0] + cnt[1]) + (cnt[2] + cnt[3]);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) sh.warp_sum[warp] = inc;
        __syncthreads();
        int before = inc - mine + __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane & (kSelWarps - 1)] : 0);
        if (before < need && before + mine >= need) {
            int at = lo_bin + 3;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (before + cnt[i] < need && at == lo_bin + 3 - i) {
                    before += cnt[i];
                    --at;
                }
            sh.found[pass] = make_int2(at, before);
        }
        if (kOne) __syncthreads();
        else cl.sync();
        const int2 found = kOne ? sh.found[pass] : *cl.map_shared_rank(&sh.found[pass], 0);
        prefix = (prefix << bits) | (uint32_t)found.x;
        need -= found.y;
    };
    run_pass(std::integral_constant<int, 0>{});
    run_pass(std::integral_constant<int, 1>{});
    run_pass(std::integral_constant<int, 2>{});
    // prefix: the n-th largest key; `need` of those equal to it are taken, the lowest positions
    uint32_t sum[kGroups];  // of a chunk: keys above | equal << 16, by group, in the threads up to this one
    auto count = [&](int c) {
        if (chunks > 1) load(c);
        uint32_t own[kGroups];
        const int G = groups(c);
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            if (u >= G) {
                if (lane == 31) sh.totals[u * kSelWarps + warp] = 0;
                continue;
            }
            own[u] = 0;
#pragma unroll
            for (int v = 0; v < kV; ++v) own[u] += (key[u * kV + v] > prefix ? 1u : 0u) + (key[u * kV + v] == prefix ? 0x10000u : 0u);
            sum[u] = own[u];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, sum[u], o);
                if (lane >= o) sum[u] += x;
            }
            if (lane == 31) sh.totals[u * kSelWarps + warp] = sum[u];
            sum[u] -= own[u];
        }
        __syncthreads();
    };
    // (above, equal) over the first `upto` entries of totals, the same in every lane of a warp
    auto total = [&](int upto) -> int2 {
        int2 r = make_int2(0, 0);
#pragma unroll
        for (int e = 0; e < kGroups * kSelWarps; e += 32) {
            const uint32_t x = e + lane < upto ? sh.totals[e + lane] : 0u;
            r.x += x & 0xffff;
            r.y += x >> 16;
        }
        return make_int2(__reduce_add_sync(0xffffffffu, r.x), __reduce_add_sync(0xffffffffu, r.y));
    };
    int above = 0, equal = 0;
    if constexpr (!kOne) {  // what the CTAs before hold
        int2 all = make_int2(0, 0);
        for (int c = 0; c < chunks; ++c) {
            count(c);
            const int2 t = total(kGroups * kSelWarps);
            all.x += t.x;
            all.y += t.y;
            if (chunks > 1) __syncthreads();
        }
        if (tid == 0) {
            sh.counts[0] = all.x;
            sh.counts[1] = all.y;
        }
        cl.sync();
        int g = 0, e = 0;
        if (lane < rank) {
            g = *cl.map_shared_rank(&sh.counts[0], lane);
            e = *cl.map_shared_rank(&sh.counts[1], lane);
        }
        above = __reduce_add_sync(0xffffffffu, g);
        equal = __reduce_add_sync(0xffffffffu, e);
        cl.sync();  // nobody's shared memory is read behind this
    }
    for (int c = 0; c < chunks; ++c) {
        if (kOne || chunks > 1) count(c);
        // by group: the chunk's groups and warps before this one
        int2 at = total(warp);
        const int G = groups(c);
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
            if (u >= G) break;
            int e = equal + at.y + (sum[u] >> 16);
            int32_t *to = kept + (above + at.x + (sum[u] & 0xffff) + min(e, need));
            const int t = t_lo + c * kSelChunk + (u * kSelThreads + tid) * kV;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const uint32_t k = key[u * kV + v];
                const bool is_eq = k == prefix, take = k > prefix || (is_eq && e < need);
                store_if(take, to, t + v);
                to += take;
                e += is_eq;
            }
            if (u + 1 < G) {  // the rest of this group's warps, then the next group's before this one
                const uint32_t x = lane < kSelWarps ? sh.totals[(u + (lane < warp)) * kSelWarps + lane] : 0u;
                at.x += __reduce_add_sync(0xffffffffu, x & 0xffff);
                at.y += __reduce_add_sync(0xffffffffu, x >> 16);
            }
        }
        if (c + 1 < chunks) {
            const int2 t = total(kGroups * kSelWarps);
            above += t.x;
            equal += t.y;
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- the move of the kept rows
// Row kept[j] of a request and kv head goes to place j. Places ascend, so kept[j] >= j: tiles of
// rows taken in order never overwrite a row that a later tile reads, and inside a tile every row
// is read before the first is written. One CTA takes one stream of rows: (request, kv head,
// 128-byte slice of K or V, or the weights). Where the rows lie is looked up for 4096 rows at a
// time, all reads of a thread in flight together; then the rows go through a ring of four tiles
// in shared memory, filled by asynchronous copies. 512 threads and tiles of 16 KB, two CTAs to an
// SM, or 1024 threads and tiles of 32 KB where there is a CTA per SM at most. Bound by the copy's
// bandwidth where there are many streams, 64 requests x 2048 rows of 1 KB: 175 us (floor 160);
// by a stream's own chain of reads, barriers and writes where there are few: four 8-bit prompts,
// 96 streams, 17 us (floor 6; 39 with look-ups and copies one tile at a time, 26 with 256 threads
// and a ring of ten tiles).
constexpr int kMoveRows = 4096;                       // rows looked up at a time

struct MoveParams {
    Csr csr;
    const int32_t *kept, *new_lens;
    uint8_t *k, *v;
    int8_t *k_exp, *v_exp;
    float *weights;
    int H, max_keep, row_bytes, slices;
};

// Four codes times s (a power of two <= 1), rounded to nearest even.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float s) {
    uint32_t h0, h1;
    e4m3x4_to_f16x4(w, h0, h1);
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&h0)), b = __half22float2(*reinterpret_cast<__half2 *>(&h1));
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(a.y * s), "f"(a.x * s));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(b.y * s), "f"(b.x * s));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// kExp: e4m3 codes with an exponent per (page, kv head). A page's exponent becomes the largest
// of those that its rows had; codes are scaled by the difference and rounded to nearest even.
template <bool kExp, int kThreads>
struct MoveLayout {
    static constexpr int kTile = kThreads / 4, kStages = 4;  // rows of a tile: two 16-byte pieces per thread
    static constexpr int kTileBytes = kTile * 128;
    static constexpr int kSrcOff = kStages * kTileBytes;  // behind the ring: source and destination slots
    static constexpr int kFactorOff = kSrcOff + 8 * kMoveRows;
    static constexpr int kSmem = kFactorOff + (kExp ? kMoveRows : 0);
    static_assert(kSmem <= 227 * 1024 && kStages * kTileBytes >= 4 * kMoveRows, "the ring holds a largest exponent per row too");
};

template <bool kExp, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) compact_kernel(const MoveParams p) {
    using LY = MoveLayout<kExp, kThreads>;
    constexpr int kU = kMoveRows / kThreads;  // rows looked up per thread
    constexpr int kTile = LY::kTile, kStages = LY::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t *s_src = reinterpret_cast<uint32_t *>(smem + LY::kSrcOff), *s_dst = s_src + kMoveRows;
    int8_t *factor = reinterpret_cast<int8_t *>(smem + LY::kFactorOff);  // kExp: of the rows' codes
    const int tid = threadIdx.x, H = p.H, ps = p.csr.ps;
    const int h = blockIdx.y, b = blockIdx.z;
    const Request rq = request(p.csr, b);
    const int n = min(min(max(__ldg(p.new_lens + b), 0), p.max_keep), rq.len);
    if (n == 0) return;
    const int32_t *kept = p.kept + ((size_t)b * H + h) * p.max_keep;
    const int slices = p.slices;

    // this thread's rows r0 + tid + kThreads u, below r1: the slots of their source and their place, or kNoRow.
    // (A position below the place, one behind the request, or a page outside the pool: the row stays.)
    auto look_up = [&](int r0, int r1, uint32_t (&src)[kU], uint32_t (&dst)[kU], int (&page)[kU]) {
        int at[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = r0 + tid + u * kThreads;
            at[u] = j < r1 ? __ldg(kept + j) : -1;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int j = r0 + tid + u * kThreads;
            int place, to;
            src[u] = at[u] >= j && at[u] < rq.len ? slot_of(p.csr, rq, at[u], page[u], place) : kNoRow;
            dst[u] = j < r1 ? slot_of(p.csr, rq, j, to, place) : kNoRow;
            if (src[u] == kNoRow || dst[u] == kNoRow) {  // stays: its source is its place
                src[u] = dst[u];
                page[u] = to;
            }
        }
    };
    if ((int)blockIdx.x == 2 * slices) {
        // ---- weights: one value per row
        auto at = [&](uint32_t s) -> float * {
            const uint32_t pg = s / (uint32_t)ps;
            return p.weights + ((size_t)pg * H + h) * ps + (s - pg * (uint32_t)ps);
        };
        for (int r0 = 0; r0 < n; r0 += kMoveRows) {
            uint32_t src[kU], dst[kU];
            int page[kU];
            float x[kU];
            look_up(r0, min(n, r0 + kMoveRows), src, dst, page);
#pragma unroll
            for (int u = 0; u < kU; ++u) x[u] = src[u] != dst[u] ? __ldcg(at(src[u])) : 0.f;
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (src[u] != dst[u]) *at(dst[u]) = x[u];
            __syncthreads();
        }
        return;
    }
    const bool is_v = (int)blockIdx.x >= slices;
    const int slice = (int)blockIdx.x - (is_v ? slices : 0);
    const int off = slice * 128 + (tid & 7) * 16;  // this thread's piece of a row
    const bool live = off < p.row_bytes;
    uint8_t *base = (is_v ? p.v : p.k) + (size_t)h * p.row_bytes + off;
    const size_t stride = (size_t)H * p.row_bytes;
    int8_t *exps = is_v ? p.v_exp : p.k_exp;
    const int chunk = kExp ? kMoveRows / ps * ps : kMoveRows;  // (host: ps <= kMoveRows)
    for (int r0 = 0; r0 < n; r0 += chunk) {
        const int r1 = min(n, r0 + chunk);
        {
            uint32_t src[kU], dst[kU];
            int page[kU], f[kU];
            look_up(r0, r1, src, dst, page);
            if constexpr (kExp) {
                // the rows' exponents, each page's largest (in the ring, which is not used yet), the pages' new
                // exponents. (Pages of this chunk's places are read by no later chunk: its rows come from places
                // at or behind its own.)
                int *most = reinterpret_cast<int *>(smem);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    f[u] = src[u] != kNoRow ? exps[(size_t)page[u] * H + h] : -128;
                    most[tid + u * kThreads] = -128;
                }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int j = tid + u * kThreads;
                    if (r0 + j < r1) atomicMax(most + div_ps(p.csr, j), f[u]);
                }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int j = tid + u * kThreads, q = div_ps(p.csr, j);
                    if (r0 + j >= r1) continue;
                    const int e = most[q];
                    f[u] = max(f[u] - e, -100);
                    factor[j] = (int8_t)f[u];
                    if (j == q * ps && dst[u] != kNoRow) exps[(size_t)(dst[u] / (uint32_t)ps) * H + h] = (int8_t)e;
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = r0 + tid + u * kThreads;
                const bool moves = src[u] != dst[u] || (kExp && j < r1 && f[u] != 0);
                s_src[j - r0] = moves ? src[u] : kNoRow;
                s_dst[j - r0] = dst[u];
            }
        }
        __syncthreads();
        const uint32_t ring = smem_u32(smem) + tid * 16;
        const int nt = (r1 - r0 + kTile - 1) / kTile;
        auto fetch = [&](int t) {  // a tile's pieces of this thread into its stage, one group of copies
            if (t < nt && live) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t s = s_src[t * kTile + (tid >> 3) + u * (kThreads / 8)];
                    if (s != kNoRow) cp_async_16(ring + t % kStages * LY::kTileBytes + u * kThreads * 16, base + (size_t)s * stride, 16);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int t = 0; t < kStages - 1; ++t) fetch(t);
        for (int t = 0; t < nt; ++t) {
            fetch(t + kStages - 1);
            cp_async_wait<kStages - 1>();
            __syncthreads();  // every row of the tile is read
            if (live) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int jl = t * kTile + (tid >> 3) + u * (kThreads / 8);
                    if (s_src[jl] == kNoRow) continue;
                    uint4 x = sm100::ld_shared_v4(ring + t % kStages * LY::kTileBytes + u * kThreads * 16);
                    if constexpr (kExp) {
                        const int f = factor[jl];
                        if (f != 0) {
                            const float s = pow2i(f);
                            x.x = rescale_codes(x.x, s);
                            x.y = rescale_codes(x.y, s);
                            x.z = rescale_codes(x.z, s);
                            x.w = rescale_codes(x.w, s);
                        }
                    }
                    *reinterpret_cast<uint4 *>(base + (size_t)s_dst[jl] * stride) = x;
                }
            }
        }
        __syncthreads();  // the slots are used
    }
}

int current_sms(int *dev_out = nullptr) {
    static int sms[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
    if (!sms[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
        sms[dev] = n;
    }
    if (dev_out) *dev_out = dev;
    return sms[dev];
}

int launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? BSP_OK : fail(BSP_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
}

Csr make_csr(const int32_t *kv_indptr, const int32_t *kv_indices, const int32_t *last_page_len, int64_t max_pages, int batch,
             int ps, int64_t num_pages) {
    // ceil(2^(31 + k) / ps), k = ceil(log2(ps)): its excess over 2^(31 + k) / ps is below 1, so that t * excess stays
    // below 2^31 <= 2^(31 + k) / ps * (distance of t / ps to the next whole number)
    int k = 0;
    while ((int64_t{1} << k) < ps) ++k;
    const uint32_t mul = (uint32_t)(((uint64_t{1} << (31 + k)) + ps - 1) / ps);
    return {kv_indptr, kv_indices, last_page_len, (int)max_pages, batch, ps, (int)num_pages, mul, 31 + k};
}

template <int D, bool kE4m3, bool kDiff, bool kVar, bool kStall = false>
int launch_weights_kernel(const WeightsParams &p, int64_t tasks, int sms, cudaStream_t stream) {
    using LY = StreamLayout<D, kE4m3>;
    static bool configured[64] = {false};
    int dev = 0;
    if (current_sms(&dev) < 0) return fail(BSP_ERR_CUDA, "no current CUDA device");
    auto kern = weights_kernel<D, kE4m3, kDiff, kVar, kStall>;
    if (!configured[dev]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::kSmem);
        if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("weights smem attribute: ") + cudaGetErrorString(e));
        configured[dev] = true;
    }
    // (small calls: four tasks per CTA, so that every loader's first look-up runs at once)
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((tasks + 3) / 4, sms));
    kern<<<grid, LY::kThreads, LY::kSmem, stream>>>(p);
    return launched("weights");
}

template <int D, bool kE4m3>
int launch_weights(const WeightsParams &p, int64_t tasks, int sms, cudaStream_t stream) {
    const bool var = p.window > 0 || p.soft_cap_on;
    if (p.lam)
        return var ? launch_weights_kernel<D, kE4m3, true, true>(p, tasks, sms, stream)
                   : launch_weights_kernel<D, kE4m3, true, false>(p, tasks, sms, stream);
    return var ? launch_weights_kernel<D, kE4m3, false, true>(p, tasks, sms, stream)
               : launch_weights_kernel<D, kE4m3, false, false>(p, tasks, sms, stream);
}

template <bool kExp, int kThreads>
int launch_compact(const MoveParams &p, dim3 grid, cudaStream_t stream) {
    using LY = MoveLayout<kExp, kThreads>;
    static bool configured[64] = {false};
    int dev = 0;
    if (current_sms(&dev) < 0) return fail(BSP_ERR_CUDA, "no current CUDA device");
    if (!configured[dev]) {
        cudaError_t e = cudaFuncSetAttribute(compact_kernel<kExp, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::kSmem);
        if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("compact smem attribute: ") + cudaGetErrorString(e));
        configured[dev] = true;
    }
    compact_kernel<kExp, kThreads><<<grid, kThreads, LY::kSmem, stream>>>(p);
    return launched("compact");
}

}  // namespace

int launch_accumulate_weights(const bsp_problem *P, const void *q, const float *lse, int64_t n_tokens, const void *k_pages,
                              const int8_t *k_exp, int64_t num_pages, float *weights, int32_t batch,
                              const int32_t *qo_indptr, const int32_t *kv_indptr, const int32_t *kv_indices,
                              int64_t max_table_pages, const int32_t *last_page_len, float sm_scale, float decay,
                              const float *lambda, int64_t stall_limit, cudaStream_t stream) {
    WeightsParams p;
    p.wait_limit = stall_limit;
    p.csr = make_csr(kv_indptr, kv_indices, last_page_len, max_table_pages, batch, P->page_size, num_pages);
    p.qo_indptr = qo_indptr;
    p.q = q;
    p.k = k_pages;
    p.lse = lse;
    p.lam = lambda;
    p.k_exp = k_exp;
    p.weights = weights;
    p.n_tokens = (int)n_tokens;
    p.H_qo = P->num_qo_heads;
    p.H_kv = P->num_kv_heads;
    p.g = p.H_qo / p.H_kv;
    p.scale_log2 = sm_scale * kLog2e;
    p.soft_cap_on = P->logits_soft_cap > 0.f;
    p.cap_in = p.soft_cap_on ? sm_scale / P->logits_soft_cap : 0.f;
    p.cap_out = P->logits_soft_cap * kLog2e;
    p.decay = decay;
    p.window = P->window_left;
    const int sms = current_sms();
    if (sms < 0) return fail(BSP_ERR_CUDA, "no current CUDA device");
    if (!k_exp && weights_prefill_takes(P, num_pages, n_tokens, batch, qo_indptr))
        return launch_weights_prefill(P, p, num_pages, max_table_pages, sms, stream);
    const int64_t tasks = (max_table_pages * P->page_size / kTaskTokens + batch) * P->num_kv_heads;
    const int D = P->head_dim;
    if (P->dtype == BSP_DTYPE_F32) {
        const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((tasks + 7) / 8, (int64_t)sms * 4));
        switch (D) {
            case 32: weights_f32_kernel<32><<<grid, 256, 0, stream>>>(p); break;
            case 64: weights_f32_kernel<64><<<grid, 256, 0, stream>>>(p); break;
            case 128: weights_f32_kernel<128><<<grid, 256, 0, stream>>>(p); break;
            default: weights_f32_kernel<256><<<grid, 256, 0, stream>>>(p); break;
        }
        return launched("weights");
    }
    if (stall_limit > 0)
        return k_exp ? launch_weights_kernel<128, true, false, false, true>(p, tasks, sms, stream)
                     : launch_weights_kernel<128, false, false, false, true>(p, tasks, sms, stream);
    if (k_exp) return launch_weights<128, true>(p, tasks, sms, stream);
    return D == 128 ? launch_weights<128, false>(p, tasks, sms, stream) : launch_weights<64, false>(p, tasks, sms, stream);
}

int launch_select_tokens(const float *weights, int64_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t batch,
                         const int32_t *kv_indptr, const int32_t *kv_indices, int64_t max_table_pages,
                         const int32_t *last_page_len, const int32_t *budget, int32_t max_keep, int32_t sinks,
                         int32_t recent, int32_t *kept, int32_t *new_lens, cudaStream_t stream) {
    SelectParams p;
    p.csr = make_csr(kv_indptr, kv_indices, last_page_len, max_table_pages, batch, page_size, num_pages);
    p.weights = weights;
    p.budget = budget;
    p.kept = kept;
    p.new_lens = new_lens;
    p.H = num_kv_heads;
    p.max_keep = max_keep;
    p.sinks = sinks;
    p.recent = recent;
    int dev = 0;
    const int sms = current_sms(&dev);
    if (sms < 0) return fail(BSP_ERR_CUDA, "no current CUDA device");
    // CTAs per row: enough to hold the mean row in registers, more where rows are few. (The mean over kv_indices' room,
    // all that the host knows: a table with room, or one long row among many short ones, gets other clusters than it
    // would need, and is slower.)
    const int64_t rows = (int64_t)batch * num_kv_heads, mean = max_table_pages * page_size / batch;
    int C = 1;
    while (C < kMaxCluster && (mean > (int64_t)C * kSelChunk || (rows * C * 2 <= 2 * (int64_t)sms && mean / C >= 4096))) C *= 2;
    const bool one = C == 1, vec = page_size % 4 == 0 && reinterpret_cast<uintptr_t>(weights) % 16 == 0;
    auto kern = one ? (vec ? select_kernel<4, true> : select_kernel<1, true>) : (vec ? select_kernel<4, false> : select_kernel<1, false>);
    static bool configured[4][64] = {{false}};
    bool &done = configured[(one ? 2 : 0) + (vec ? 1 : 0)][dev];
    if (!done) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("select cluster attribute: ") + cudaGetErrorString(e));
        done = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("select launch: ") + cudaGetErrorString(e));
    return launched("select");
}

int launch_compact_cache(const int32_t *kept, const int32_t *new_lens, int32_t max_keep, int32_t batch,
                         const int32_t *kv_indptr, const int32_t *kv_indices, int64_t max_table_pages,
                         const int32_t *last_page_len, void *k_pages, void *v_pages, int8_t *k_exp, int8_t *v_exp,
                         float *weights, int64_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t row_bytes,
                         cudaStream_t stream) {
    MoveParams p;
    p.csr = make_csr(kv_indptr, kv_indices, last_page_len, max_table_pages, batch, page_size, num_pages);
    p.kept = kept;
    p.new_lens = new_lens;
    p.k = static_cast<uint8_t *>(k_pages);
    p.v = static_cast<uint8_t *>(v_pages);
    p.k_exp = k_exp;
    p.v_exp = v_exp;
    p.weights = weights;
    p.H = num_kv_heads;
    p.max_keep = max_keep;
    p.row_bytes = row_bytes;
    p.slices = (row_bytes + 127) / 128;
    const dim3 grid(2 * p.slices + (weights ? 1 : 0), num_kv_heads, batch);
    if (k_exp && page_size > kMoveRows) return fail(BSP_ERR_UNSUPPORTED, "compacting the 8-bit cache takes pages of at most 4096 tokens");
    const int sms = current_sms();
    if (sms < 0) return fail(BSP_ERR_CUDA, "no current CUDA device");
    const bool few = (int64_t)grid.x * grid.y * grid.z <= sms;
    if (k_exp) return few ? launch_compact<true, 1024>(p, grid, stream) : launch_compact<true, 512>(p, grid, stream);
    return few ? launch_compact<false, 1024>(p, grid, stream) : launch_compact<false, 512>(p, grid, stream);
}

}  // namespace bsp
