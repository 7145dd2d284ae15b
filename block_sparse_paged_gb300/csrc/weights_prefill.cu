// Gathered attention weights of keys that many queries see (whole prompts, chunks, observation
// windows), on the tcgen05 tensor cores: bf16 pools, head_dim 128, pages of a power of two from 8
// tokens on. (What is summed: csrc/evict.cu, whose warp-level kernel takes everything else.)
//
// The score tile is transposed, S^T = K Q^T: 128 keys on the accumulator's lanes, 128 query rows
// (positions x the g heads of the kv head) on its columns. A thread then owns a key and sums
// exp(scale s - LSE) along its lane, so that a key's sum has one order without any exchange per
// tile. LSE, a value per column, goes into the accumulator: x = -LSE / scale as three bf16 values
// (24 bits together) in three columns of one more product, of K = 16, whose other operand is 1 there.
// It is added last, so that the scores round as without it; exp2((s + x) scale log2 e) remains. No
// maximum is searched (LSE is given) and nothing is multiplied by P: half a multiplication, one
// exponential and half an addition per element. (A soft-cap stands between s and LSE, and LSE / scale
// must not overflow: kVar subtracts LSE in registers, from shared memory.)
//
// A unit of work is 256 keys of one kv head and all query tiles that see any of them. 18 warps:
//   warp 0      TMA: the unit's K (page boxes, 64 KB a stage) and the Q tiles (32 KB a stage); the
//               columns' values and which of them saw no key (8 slots)
//   warp 1      TMEM owner; one thread issues S^T of both 128-key halves per Q tile
//   warps 2-9   keys 0..127, warps 10-17 keys 128..255: two threads per key, 64 columns of a tile
//               each
// Each half has two accumulators, so that the tensor core fills one while the other is summed
// (differential weights need both for the two maps of a tile); one is free again before its last
// columns are summed. Two prompts of about 7k, 32 / 8 heads, us: one thread per key (8 warps) 543, two
// 512, fewer instructions for waits and masks 497, MMAs by an elected thread 478, LSE in the
// accumulator 396, early release and first load 370, look-up a unit ahead 357 (on other boxes 377-390). Bound by the sum
// warps' instructions and their waits at a tile's begin (exponentials alone 230, products 255); one
// accumulator of 256 columns per half was 507 (against 478), the next tile awaited inside a tile 397.
// Units go to CTAs in the order of the table; a request's first units have the most queries
// under the causal mask. Long units run one per CTA, so that the block scheduler levels them.
// Every wait is bounded; one that gives up makes NaN of the weights that its CTA has not summed by then.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "bsp_internal.h"
#include "device_common.cuh"
#include "evict.cuh"
#include "sm100.cuh"

namespace bsp {
namespace {

using namespace sm100;
using namespace evict;

constexpr int kD = 128;
constexpr int kRows = 128;                 // keys of a half, query rows of a tile
constexpr int kUnit = 256;                 // keys of a unit
constexpr int kThreads = 576;
constexpr int kSlab = 16384;               // [128 rows][64 bf16], 128-byte swizzle
constexpr int kTile = 2 * kSlab;
// Six tiles: long units have one stage of K (two tiles) and four of Q, so that Q's latency is
// covered; short ones two of each, so that the next unit's K is.
constexpr int kMaxKStages = 2, kMaxQStages = 4;
constexpr int kSlots = 8;                                  // tiles whose column values lie in shared memory
static_assert(kSlots >= kMaxQStages + 3, "a slot is written again when its tile's sums are done");
constexpr int kOffK = 0;
constexpr int kAug = kRows * 16;                           // 8 columns of bf16, no swizzle
constexpr int kOffAug = 6 * kTile;                         // per Q stage and map: -LSE / scale in three parts
constexpr int kOffLam = kOffAug + kMaxQStages * 2 * kAug;  // per slot: -lambda of the columns
constexpr int kOffL = kOffAug;                             // soft-cap, instead: per slot -LSE log2 e (both maps), -lambda
constexpr int kOffOnes = kOffLam + kSlots * kRows * 4;     // 1, 1, 1, 0 .. in every row
constexpr int kOffZeros = kOffOnes + kAug;
static_assert(kOffL + kSlots * 3 * kRows * 4 <= kOffOnes, "both uses fit");
constexpr int kOffBar = kOffZeros + kAug;
enum Bar {
    kKFull0 = 0, kKEmpty0 = kKFull0 + kMaxKStages, kQFull0 = kKEmpty0 + kMaxKStages, kQEmpty0 = kQFull0 + kMaxQStages,
    kSFull0 = kQEmpty0 + kMaxQStages,  // [half][accumulator]
    kSEmpty0 = kSFull0 + 4, kMeet0 = kSEmpty0 + 4,  // [half][lane quarter]
    kNumBars = kMeet0 + 8
};
constexpr int kOffMisc = kOffBar + kNumBars * 8;           // TMEM slot, abort flag
constexpr int kOddWords = 12;                              // any, (3 free), columns without keys: map 1, map 2
constexpr int kOffOdd = kOffMisc + 8;
constexpr int kOffPart = kOffOdd + kSlots * kOddWords * 4;  // [2 units][256 keys]: the second warps' sums
constexpr int kSmemBytes = kOffPart + 2 * kUnit * 4 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "tiles exceed shared memory");
constexpr uint32_t kTmemCols = 512;

struct PrefillWeights {
    WeightsParams w;
    int box_rows;
};

// What every warp needs of a unit.
struct Unit {
    int b, h, t0;         // request, kv head, first key
    Request rq;
    Queries qs;
    int off;              // position of the first query
    int tile0, tiles;     // query tiles that see a key of the unit
};

// a / b for a >= 0 and b a power of two: by a shift where it is done often (the other form leaves the long
// tiles' loop its registers)
template <bool kLong>
__device__ __forceinline__ int over(int a, int b) {
    return kLong ? a / b : a >> (31 - __clz(b));
}

// A CTA's units: u = blockIdx.x, blockIdx.x + gridDim.x, .. in the order (virtual block, head). Where there are
// many (kLong false) they are walked without a division or, as a rule, a search per unit, which take 2,000 cycles
// (64 requests x 4096 tokens with 16 queries 196 -> 170 us); where there is one, all that a warp keeps is u (two
// prompts of about 7k 357 us, with the walk's registers 370, on one box).
template <bool kLong>
struct Walk {
    uint32_t u;
    int h, b;             // kv head, request
    long long blk, next;  // virtual block; the first one behind its request's (kLong: neither kept)

    __device__ __forceinline__ void find(const WeightsParams &p, int lane) {
        blk = block_start<kUnit>(p.csr, 0) + (long long)u / p.H_kv;
        h = (int)((long long)u % p.H_kv);
        b = find_request<kUnit>(p.csr, blk, lane);
    }
    __device__ __forceinline__ void end(const WeightsParams &p) {
        next = b + 1 < p.csr.batch ? block_start<kUnit>(p.csr, b + 1) : LLONG_MAX;
    }
    __device__ __forceinline__ Walk(const WeightsParams &p, int lane) : u(blockIdx.x) {
        if constexpr (!kLong) {
            find(p, lane);
            end(p);
        }
    }
    __device__ __forceinline__ void on(const WeightsParams &p, int lane) {
        u += gridDim.x;
        if constexpr (!kLong) {
            blk += gridDim.x / (uint32_t)p.H_kv;
            h += (int)(gridDim.x % (uint32_t)p.H_kv);
            if (h >= p.H_kv) {
                h -= p.H_kv;
                ++blk;
            }
            if (blk >= next) {
                ++b;
                end(p);
                if (blk >= next) {
                    b = find_request<kUnit>(p.csr, blk, lane);
                    end(p);
                }
            }
        }
    }
    // the unit here, or false where the table's virtual block is empty
    __device__ __forceinline__ bool unit(const WeightsParams &p, int lane, Unit &x) {
        if constexpr (kLong) find(p, lane);
        x.h = h;
        x.b = b;
        x.rq = request(p.csr, b);
        const long long first = (blk - block_start<kUnit>(p.csr, b)) * kUnit;
        if (first < 0 || first >= x.rq.len) return false;  // (below 0: a table that does not ascend)
        x.t0 = (int)first;
        x.qs = queries(p, b);
        x.off = x.rq.len - x.qs.n;
        const int ppt = kRows / p.g;  // positions per tile
        const int i_lo = max(0, x.t0 - x.off);
        const int i_hi = p.window > 0 ? (int)min((long long)x.qs.n, (long long)x.t0 + kUnit + p.window - x.off) : x.qs.n;
        x.tile0 = over<kLong>(i_lo, ppt);
        x.tiles = i_hi > i_lo ? over<kLong>(i_hi - x.tile0 * ppt + ppt - 1, ppt) : 0;
        return true;
    }
};

__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b, float c0, float c1) {
    asm("{ .reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %4};\n mov.b64 rc, {%5, %6};\n"
        " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b) {
    asm("{ .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %4};\n mul.rn.f32x2 rd, ra, rb;\n"
        " mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b));
}
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1) {
    asm("{ .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rd, ra, rb;\n"
        " mov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1)
        : "f"(d0), "f"(d1), "f"(a0), "f"(a1));
}
// lse * f as a sum of three bf16 values (of 24 bits together); 0 where no key was seen.
__device__ __forceinline__ uint4 three_parts(float lse, float f) {
    const float x = lse == -INFINITY ? 0.f : lse * f;
    const uint32_t h = dev::pack_bf16(x, 0.f);
    const float r = fabsf(dev::bf16_lo(h)) < INFINITY ? x - dev::bf16_lo(h) : 0.f;  // exact; (NaN and infinities: in the first part)
    const uint32_t m = dev::pack_bf16(r, 0.f);
    return make_uint4((h & 0xffffu) | (m << 16), dev::pack_bf16(r - dev::bf16_lo(m), 0.f), 0u, 0u);
}
// kVar: soft-cap compiled in. kDiff: differential weights. kLong: units of many query tiles.
template <bool kVar, bool kDiff, bool kLong, bool kStall = false>
__global__ void __launch_bounds__(kThreads, 1)
    weights_prefill_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const PrefillWeights pp) {
    constexpr int kKStages = kLong ? 1 : 2, kQStages = kLong ? 4 : 2, kOffQ = kOffK + kKStages * 2 * kTile;
    const WeightsParams &p = pp.w;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = dev::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t units = (uint32_t)max(0ll, (block_start<kUnit>(p.csr, p.csr.batch) - block_start<kUnit>(p.csr, 0)) * p.H_kv);
    // leave before anything is set up if no unit of this CTA holds a key
    bool any = false;
    Unit x;
    for (Walk<kLong> w(p, lane); w.u < units && !any; w.on(p, lane)) any = w.unit(p, lane, x);
    if (!any) return;  // (the same for every warp)

    auto bar = [&](int i) { return sb + kOffBar + 8u * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i)
            mbar_init(bar(i), i >= kMeet0 ? 64 : i >= kSEmpty0 ? 8 : i >= kSFull0 || i >= kQEmpty0 ? 2 : i >= kQFull0 ? 33 : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    for (int i = tid; i < 2 * kRows; i += kThreads)  // bf16 1, 1, 1, 0, ..; zeros behind
        reinterpret_cast<uint4 *>(smem + kOffOnes)[i] = make_uint4(i < kRows ? 0x3f803f80u : 0u, i < kRows ? 0x3f80u : 0u, 0u, 0u);
    fence_proxy_async_smem();
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tq);
        prefetch_tmap(&tk);
    }
    if (warp == 1) {
        tmem_alloc(dev::smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait1 = [&](uint32_t b, uint32_t parity) -> bool {
        if (mbar_wait_spin(b, parity, kStall ? p.wait_limit : kWaitLimitCycles, abort_flag)) return true;
        *abort_flag = 1;
        return false;
    };
    // (the first try alone where it succeeds: a sum warp's own instructions are what a tile waits for)
    auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_try_wait(b, parity)) || __all_sync(0xffffffffu, wait1(b, parity));
    };
    const int g = p.g, ppt = kRows / g;  // (powers of two)

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        int kn = 0, n = 0;  // units and tiles so far
        const int g_shift = 31 - __clz(g);
        const float neg_inv_scale = -dev::kLog2e / p.scale_log2;
        (void)neg_inv_scale;
        bool ok = true;
        // the next unit with tiles, from u on; its page under this lane's box: l of the unit, box_rows keys of a page
        Walk<kLong> w(p, lane);
        Unit next;
        int page = -1;
        auto look_up = [&]() -> bool {
            for (; w.u < units; w.on(p, lane)) {
                if (!w.unit(p, lane, next) || next.tiles == 0) continue;
                const int t = next.t0 + lane * pp.box_rows;
                page = lane * pp.box_rows < kUnit && t < next.rq.len ? __ldg(p.csr.kv_indices + next.rq.p0 + div_ps(p.csr, t)) : -1;
                w.on(p, lane);
                return true;
            }
            return false;
        };
        bool more = look_up();
        while (more && ok) {
            x = next;
            const int ks = kn % kKStages;
            uint32_t slot = kNoRow;
            if ((unsigned)page < (unsigned)p.csr.num_pages) {
                const int t = x.t0 + lane * pp.box_rows;
                slot = (uint32_t)page * (uint32_t)p.csr.ps + (uint32_t)(t - div_ps(p.csr, t) * p.csr.ps);
            }
            const int boxes = __popc(__ballot_sync(0xffffffffu, slot != kNoRow));
            more = look_up();  // (the next unit's page is on its way during this one's tiles)
            if (!(ok = wait(bar(kKEmpty0 + ks), ((kn / kKStages) & 1) ^ 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(kKFull0 + ks), (uint32_t)boxes * pp.box_rows * 256);
            __syncwarp();
            if (slot != kNoRow) {
                const int key = lane * pp.box_rows;  // (a box lies in one half: box_rows <= 128)
                const uint32_t d = sb + kOffK + ks * 2 * kTile + (key >> 7) * kTile + (key & 127) * 128;
                tma_load_3d(d, &tk, bar(kKFull0 + ks), 0, x.h, (int)slot);
                tma_load_3d(d + kSlab, &tk, bar(kKFull0 + ks), 64, x.h, (int)slot);
            }
            ++kn;
            // -LSE log2 e of a tile's columns, read a tile ahead
            float a[4], a2[4], lm[4];
            auto columns = [&](int i) {
                const int pos0 = (x.tile0 + i) * ppt, rows = min(kRows, (x.qs.n - pos0) * g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = lane + 32 * j, i_c = c >> g_shift, r = c & (g - 1);
                    const size_t row = (size_t)(x.qs.q0 + pos0 + i_c) * p.H_qo + (size_t)x.h * g + r;
                    a[j] = a2[j] = lm[j] = 0.f;
                    if (i < x.tiles && c < rows) {
                        if (kDiff) {
                            const float2 z = __ldg(reinterpret_cast<const float2 *>(p.lse) + row);
                            a[j] = z.x;
                            a2[j] = z.y;
                            lm[j] = __ldg(p.lam + x.h * g + r);
                        } else {
                            a[j] = __ldg(p.lse + row);
                        }
                    }
                }
            };
            columns(0);
            for (int i = 0; i < x.tiles && ok; ++i, ++n) {
                const int qst = n % kQStages, sl = n % kSlots, pos0 = (x.tile0 + i) * ppt;
                if (kStall && n == 3) {
                    ok = false;
                    break;
                }
                if (!(ok = wait(bar(kQEmpty0 + qst), ((n / kQStages) & 1) ^ 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(kQFull0 + qst), kTile);
                    const uint32_t d = sb + kOffQ + qst * kTile;
                    tma_load_3d(d, &tq, bar(kQFull0 + qst), 0, x.h * g, x.qs.q0 + pos0);
                    tma_load_3d(d + kSlab, &tq, bar(kQFull0 + qst), 64, x.h * g, x.qs.q0 + pos0);
                }
                uint32_t *od = reinterpret_cast<uint32_t *>(smem + kOffOdd) + sl * kOddWords;
                uint32_t strange = 0;  // queries that saw no key
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = lane + 32 * j;
                    const uint32_t o1 = __ballot_sync(0xffffffffu, a[j] == -INFINITY);
                    const uint32_t o2 = kDiff ? __ballot_sync(0xffffffffu, a2[j] == -INFINITY) : 0;
                    strange |= o1 | o2;
                    if (lane == 0) {
                        od[4 + j] = o1;
                        od[8 + j] = o2;
                    }
                    if constexpr (kVar) {
                        float *l = reinterpret_cast<float *>(smem + kOffL) + sl * 3 * kRows;
                        l[c] = a[j] * -dev::kLog2e;
                        if constexpr (kDiff) {
                            l[kRows + c] = a2[j] * -dev::kLog2e;
                            l[2 * kRows + c] = -lm[j];
                        }
                    } else {
                        uint4 *aug = reinterpret_cast<uint4 *>(smem + kOffAug + qst * 2 * kAug);
                        aug[c] = three_parts(a[j], neg_inv_scale);
                        if constexpr (kDiff) {
                            aug[kRows + c] = three_parts(a2[j], neg_inv_scale);
                            reinterpret_cast<float *>(smem + kOffLam)[sl * kRows + c] = -lm[j];
                        }
                    }
                }
                if (lane == 0) od[0] = strange;
                fence_proxy_async_smem();
                mbar_arrive(bar(kQFull0 + qst));
                columns(i + 1);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        constexpr uint32_t id = idesc_bf16_f32(kRows, kRows, false, false);
        int kn = 0, n = 0;
        bool ok = true;
        for (Walk<kLong> w(p, lane); w.u < units && ok; w.on(p, lane)) {
            if (!w.unit(p, lane, x) || x.tiles == 0) continue;
            if (elect_one()) {
                const int ks = kn % kKStages;
                ok = wait1(bar(kKFull0 + ks), (kn / kKStages) & 1);
                for (int i = 0; i < x.tiles && ok; ++i) {
                    const int m = n + i, qst = m % kQStages;
                    if (!(ok = wait1(bar(kQFull0 + qst), (m / kQStages) & 1))) break;
                    const uint64_t dq = smem_desc_sw128(sb + kOffQ + qst * kTile, 16, 1024);
                    const uint64_t dk = smem_desc_sw128(sb + kOffK + ks * 2 * kTile, 16, 1024);
                    // (the second 8 of an operand's 16 columns: the zeros)
                    const uint32_t aug = kOffAug + qst * 2 * kAug;
                    [[maybe_unused]] const uint64_t d_ones = smem_desc_plain(sb + kOffOnes, kOffZeros - kOffOnes, 128);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // accumulator m & 1 of the half; differential: both, one per map
                        const int acc = kDiff ? 0 : m & 1, use = kDiff ? m : m >> 1;
                        if (!(ok = wait1(bar(kSEmpty0 + 2 * half + acc), (use & 1) ^ 1))) break;
                        tc_fence_after();
                        const uint32_t d = tmem + half * 256 + acc * 128;
                        mbar_arrive(bar(kSFull0 + 2 * half + acc));  // (hands on what warp 0 wrote for the tile)
#pragma unroll
                        for (int kk = 0; kk < kD / 16; ++kk) {
                            const uint32_t o = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
                            mma_bf16_ss(kDiff ? d + (kk >> 2) * 128 : d, dk + half * (kTile >> 4) + o, dq + o, id,
                                        kDiff ? (kk & 3) > 0 : kk > 0);
                        }
                        if constexpr (!kVar) {  // last, so that LSE goes through one addition
#pragma unroll
                            for (int map = 0; map < (kDiff ? 2 : 1); ++map) {
                                const uint32_t o = aug + map * kAug;
                                mma_bf16_ss(d + map * 128, d_ones, smem_desc_plain(sb + o, kOffZeros - o, 128), id, 1);
                            }
                        }
                        mma_commit(bar(kSFull0 + 2 * half + acc));
                    }
                    if (ok) {
                        mbar_arrive(bar(kQEmpty0 + qst));
                        mma_commit(bar(kQEmpty0 + qst));
                    }
                }
                if (ok) mma_commit(bar(kKEmpty0 + ks));
            }
            ok = __all_sync(0xffffffffu, ok);
            n += x.tiles;
            ++kn;
        }
    } else {
        // ------------------------------------------------------------ sums
        const int half = (warp - 2) >> 3, q4 = warp & 3, col0 = ((warp - 2) >> 2 & 1) * 64;
        const int key = half * kRows + q4 * 32 + lane;
        const uint32_t tS = tmem + ((uint32_t)(q4 * 32) << 16) + half * 256;
        int n = 0, meet = 0;
        bool ok = true;
        for (Walk<kLong> w(p, lane); w.u < units; w.on(p, lane)) {  // (behind a wait that gave up: NaN, without waiting)
            if (!w.unit(p, lane, x)) continue;
            const int t = x.t0 + key;
            int page = 0, place = 0;
            const uint32_t slot = t < x.rq.len ? slot_of(p.csr, x.rq, t, page, place) : kNoRow;
            float *at = p.weights + ((size_t)page * p.H_kv + x.h) * p.csr.ps + place;
            const float old = !col0 && slot != kNoRow && t < x.off && p.decay != 0.f ? *at : 0.f;
            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
            // tiles all of whose queries see all keys of the unit
            const int full_lo = p.window > 0 ? x.tiles : over<kLong>(max(0, x.t0 + kUnit - 1 - x.off) + ppt - 1, ppt) - x.tile0;
            const int full_hi = over<kLong>(x.qs.n, ppt) - x.tile0;
            const bool live = ok;
            for (int i = 0; i < x.tiles && ok; ++i, ++n) {
                const int acc = kDiff ? 0 : n & 1, use = kDiff ? n : n >> 1, sl = n % kSlots;
                if (!(ok = wait(bar(kSFull0 + 2 * half + acc), use & 1))) break;
                tc_fence_after();
                [[maybe_unused]] float va[32];
                if constexpr (!kDiff) tmem_ld32(tS + acc * 128 + col0, va);
                [[maybe_unused]] const float4 *lse = reinterpret_cast<const float4 *>(smem + kOffL) + sl * 3 * kRows / 4;
                [[maybe_unused]] const float4 *lam4 =
                    kVar ? lse + 2 * kRows / 4 : reinterpret_cast<const float4 *>(smem + kOffLam) + sl * kRows / 4;
                const uint32_t *od = reinterpret_cast<const uint32_t *>(smem + kOffOdd) + sl * kOddWords;
                const bool full = i >= full_lo && i < full_hi && od[0] == 0;
                int c_lo = 0;
                unsigned width = kRows;
                if (!full) {  // columns that see this key: positions t .. t + window
                    const int pos0 = (x.tile0 + i) * ppt, rows = min(kRows, (x.qs.n - pos0) * g);
                    c_lo = max(0, t - x.off - pos0) * g;
                    int c_hi = rows;
                    if (p.window > 0) c_hi = (int)max(0ll, min((long long)rows, ((long long)t - x.off - pos0 + p.window + 1) * g));
                    width = (unsigned)max(0, c_hi - c_lo);
                }
                const float scale = kVar && p.soft_cap_on ? p.cap_out : p.scale_log2;
                // 32 columns from c on: v (and v2, the second map's)
                auto add32 = [&](auto whole, int c, float (&v)[32], float (&v2)[kDiff ? 32 : 1]) {
                    constexpr bool kFull = decltype(whole)::value;
                    if (kVar && p.soft_cap_on) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            v[j] = dev::tanh_f32(v[j] * p.cap_in);
                            if constexpr (kDiff) v2[j] = dev::tanh_f32(v2[j] * p.cap_in);
                        }
                    }
                    // all loads before the first use
                    [[maybe_unused]] float4 lr[kVar ? 8 : 1], l2r[kVar && kDiff ? 8 : 1], lmr[kDiff ? 8 : 1];
                    if constexpr (kVar || kDiff) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if constexpr (kVar) lr[j] = lse[c / 4 + j];
                            if constexpr (kVar && kDiff) l2r[j] = lse[(kRows + c) / 4 + j];
                            if constexpr (kDiff) lmr[j] = lam4[c / 4 + j];
                        }
                    }
                    [[maybe_unused]] uint32_t see1 = 0, see2 = 0;  // of these columns: those that see the key in map 1, 2
                    if constexpr (!kFull) {
                        const int lo = min(max(c_lo - c, 0), 32), hi = min(max(c_lo + (int)width - c, 0), 32);
                        const uint32_t in = hi > lo ? (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo) : 0;
                        see1 = in & ~od[4 + c / 32];
                        if constexpr (kDiff) see2 = in & ~od[8 + c / 32];
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        // scale * s - LSE, base 2 (kVar false: LSE went into s)
                        auto exponents = [&](float *x, const float4 &l) {
                            if constexpr (kVar) {
                                fma2(x[0], x[1], x[0], x[1], scale, l.x, l.y);
                                fma2(x[2], x[3], x[2], x[3], scale, l.z, l.w);
                            } else {
                                mul2(x[0], x[1], x[0], x[1], scale);
                                mul2(x[2], x[3], x[2], x[3], scale);
                            }
                        };
                        exponents(v + j, lr[kVar ? j / 4 : 0]);
                        float e[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            e[k] = ex2(v[j + k]);
                            if constexpr (!kFull) e[k] = see1 >> (j + k) & 1 ? e[k] : 0.f;
                        }
                        if constexpr (kDiff) {
                            exponents(v2 + j, l2r[kVar ? j / 4 : 0]);
                            const float4 lm = lmr[j / 4];
                            const float lam[4] = {lm.x, lm.y, lm.z, lm.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float e2 = ex2(v2[j + k]);
                                if constexpr (!kFull) e2 = see2 >> (j + k) & 1 ? e2 : 0.f;
                                e[k] = fabsf(fmaf(lam[k], e2, e[k]));
                            }
                        }
                        add2(s0, s1, e[0], e[1]);
                        add2(s2, s3, e[2], e[3]);
                    }
                };
                const uint32_t tA = tS + acc * 128;
                // the accumulator is read, before the last 32 columns are summed
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kSEmpty0 + 2 * half + acc));
                };
                // (two copies of the loop: with a branch per group of columns 756 us instead of 543)
                auto add_tile = [&](auto whole) {
                    if constexpr (kDiff) {
#pragma unroll 1
                        for (int c = col0; c < col0 + 64; c += 32) {
                            float v[32], v2[32];
                            tmem_ld32(tS + c, v);
                            tmem_ld32(tS + 128 + c, v2);
                            tmem_wait_ld();
                            if (c > col0) release();
                            add32(whole, c, v, v2);
                        }
                    } else {
                        float vb[32], none[1];
                        tmem_wait_ld();
                        tmem_ld32(tA + col0 + 32, vb);  // read while the first 32 are summed
                        add32(whole, col0, va, none);
                        tmem_wait_ld();
                        release();
                        add32(whole, col0 + 32, vb, none);
                    }
                };
                if (full) add_tile(std::true_type{});
                else add_tile(std::false_type{});
            }
            // the columns' two halves
            float *part = reinterpret_cast<float *>(smem + kOffPart) + (meet & 1) * kUnit + key;
            const float sum = (s0 + s1) + (s2 + s3);
            if (live) {
                if (col0) *part = ok ? sum : NAN;
                mbar_arrive(bar(kMeet0 + half * 4 + q4));
                ok = ok && wait(bar(kMeet0 + half * 4 + q4), meet & 1);
                ++meet;
            }
            if (!col0 && slot != kNoRow) *at = ok ? fmaf(p.decay, old, sum + *part) : NAN;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // let copies and MMAs already in flight finish before TMEM is released
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

// From 32 query rows per request on (mean). Measured, 32 / 8 heads, us (warp-level kernel / this one): 8 requests x
// 4096 tokens, 6 queries (24 rows) 26 / 32, 8 queries 30 / 32, 16 queries 48 / 32; 8 x 16384, 6 queries 81 / 85, 8
// queries 96 / 85, 16 queries 166 / 86; 64 x 4096, 6 queries 157 / 169, 8 queries 189 / 170, 16 queries 326 / 170.
bool weights_prefill_takes(const bsp_problem *P, int64_t num_pages, int64_t n_tokens, int32_t batch, const int32_t *qo_indptr) {
    const int g = P->num_qo_heads / P->num_kv_heads, ps = P->page_size;
    return qo_indptr && P->dtype == BSP_DTYPE_BF16 && P->head_dim == kD && kRows % g == 0 && ps >= 8 && (ps & (ps - 1)) == 0 &&
           num_pages * (int64_t)ps <= INT32_MAX && n_tokens * g >= (int64_t)batch * 32;
}

int launch_weights_prefill(const bsp_problem *P, const evict::WeightsParams &w, int64_t num_pages, int64_t max_table_pages,
                           int sms, cudaStream_t stream) {
    PrefillWeights p;
    p.w = w;
    p.box_rows = std::min(P->page_size, kRows);
    CUtensorMap tq, tk;
    std::memset(&tq, 0, sizeof(tq));
    std::memset(&tk, 0, sizeof(tk));
    int rc = make_tmap_bf16(&tq, w.q, kD, P->num_qo_heads, (uint64_t)w.n_tokens, w.g, kRows / w.g);
    if (rc == BSP_OK) rc = make_tmap_bf16(&tk, w.k, kD, P->num_kv_heads, (uint64_t)num_pages * P->page_size, 1, p.box_rows);
    if (rc != BSP_OK) return rc;
    const bool diff = w.lam != nullptr;
    // LSE / scale must not overflow nor vanish: other scales take the variant that subtracts LSE from scaled scores
    const float size = std::fabs(w.scale_log2);
    const bool var = w.soft_cap_on || !(size > 1e-10f && size < 1e10f);
    // units of many tiles: a CTA each; of few: persistent CTAs, whose next unit's K is on its way
    const int64_t units = (max_table_pages * P->page_size / kUnit + w.csr.batch) * P->num_kv_heads;
    const bool longer = (int64_t)w.n_tokens * w.g / w.csr.batch >= 8 * kRows;
    auto pick = [&](auto l) {
        constexpr bool kLong = decltype(l)::value;
        return diff ? (var ? weights_prefill_kernel<true, true, kLong> : weights_prefill_kernel<false, true, kLong>)
                    : (var ? weights_prefill_kernel<true, false, kLong> : weights_prefill_kernel<false, false, kLong>);
    };
    const bool stall = w.wait_limit > 0;
    auto kern = stall ? (longer ? weights_prefill_kernel<false, false, true, true> : weights_prefill_kernel<false, false, false, true>)
                      : longer ? pick(std::true_type{}) : pick(std::false_type{});
    static bool configured[10][64] = {{false}};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(BSP_ERR_CUDA, "no current CUDA device");
    bool &done = configured[stall ? (longer ? 9 : 8) : (longer ? 4 : 0) + (diff ? 2 : 0) + (var ? 1 : 0)][dev];
    if (!done) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("weights smem attribute: ") + cudaGetErrorString(e));
        done = true;
    }
    const unsigned grid = (unsigned)std::max<int64_t>(1, longer ? units : std::min<int64_t>(units, sms));
    kern<<<grid, kThreads, kSmemBytes, stream>>>(tq, tk, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("weights launch: ") + cudaGetErrorString(e));
    return BSP_OK;
}

}  // namespace bsp
