// C-ABI entry points of libbsp.so other than the planner: argument checks,
// launch of the run kernels, merge_state, error reporting.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <string>

#include "bsp_internal.h"

namespace bsp {

namespace {
thread_local std::string g_msg;
thread_local int g_code = BSP_OK;
}  // namespace

int fail(int code, const std::string &msg) {
    g_code = code;
    g_msg = msg;
    return code;
}

void clear_error() {
    g_code = BSP_OK;
    g_msg.clear();
}

int last_code() { return g_code == BSP_OK ? BSP_ERR_INVALID_ARG : g_code; }

int check_aligned16(const void *q, const void *k, const void *v, const void *o, const void *workspace) {
    const void *ptr[5] = {q, k, v, o, workspace};
    const char *name[5] = {"q", "k_pages", "v_pages", "o", "workspace"};
    for (int i = 0; i < 5; ++i)
        if (reinterpret_cast<uintptr_t>(ptr[i]) % 16 != 0)
            return fail(BSP_ERR_INVALID_ARG, std::string(name[i]) + " is not 16-byte aligned");
    return BSP_OK;
}

namespace {

int check_plan(const bsp_plan_info *plan, int mode, const void *workspace) {
    if (!plan || plan->valid != 1) return fail(BSP_ERR_INVALID_ARG, "plan is NULL or was not produced by bsp_plan");
    if (plan->problem.mode != mode)
        return fail(BSP_ERR_INVALID_ARG, mode == BSP_MODE_DECODE ? "plan was made for prefill, not decode"
                                                                 : "plan was made for decode, not prefill");
    if (!workspace) return fail(BSP_ERR_INVALID_ARG, "workspace is NULL");
    Layout l;
    if (!compute_layout(&plan->problem, &plan->capacity, &l)) return last_code();
    if (l.total != plan->workspace_bytes || l.off_partial_o != plan->off_partial_o)
        return fail(BSP_ERR_INVALID_ARG, "plan info is inconsistent with its problem and capacity");
    return BSP_OK;
}

}  // namespace
}  // namespace bsp

using namespace bsp;

extern "C" const char *bsp_last_error(void) { return g_msg.c_str(); }

extern "C" const char *bsp_version(void) { return "bsp 0.1 (sm_103a)"; }

extern "C" int bsp_default_num_ctas(int32_t mode, int32_t device, int32_t *num_ctas_out) {
    clear_error();
    if (!num_ctas_out) return fail(BSP_ERR_INVALID_ARG, "num_ctas_out is NULL");
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
    if (mode == BSP_MODE_DECODE) *num_ctas_out = sms * decode_ctas_per_sm(128, BSP_DTYPE_BF16);
    else if (mode == BSP_MODE_PREFILL) *num_ctas_out = sms;
    else return fail(BSP_ERR_INVALID_ARG, "unknown mode");
    return BSP_OK;
}

extern "C" int bsp_decode_run(const bsp_plan_info *plan, const void *q, const void *k_pages, const void *v_pages,
                              const int32_t *kv_indices, int64_t num_pages, float sm_scale, void *o, float *lse,
                              void *workspace, bsp_stream_t stream) {
    clear_error();
    int rc = check_plan(plan, BSP_MODE_DECODE, workspace);
    if (rc != BSP_OK) return rc;
    if (!q || !k_pages || !v_pages || !o) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (num_pages < 0) return fail(BSP_ERR_INVALID_ARG, "num_pages must not be negative");
    if ((rc = check_aligned16(q, k_pages, v_pages, o, workspace)) != BSP_OK) return rc;
    // split outputs are merged inside the decode kernel (by the CTA that writes
    // an output's last partial state): one launch
    return launch_decode(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, o, lse, workspace, stream);
}

extern "C" int bsp_decode_run_fp8(const bsp_plan_info *plan, const void *q, const void *k_pages,
                                  const void *v_pages, const int32_t *kv_indices, int64_t num_pages, float sm_scale,
                                  float k_scale, float v_scale, void *o, float *lse, void *workspace,
                                  bsp_stream_t stream) {
    clear_error();
    int rc = check_plan(plan, BSP_MODE_DECODE, workspace);
    if (rc != BSP_OK) return rc;
    if (!q || !k_pages || !v_pages || !o) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if ((rc = check_aligned16(q, k_pages, v_pages, o, workspace)) != BSP_OK) return rc;
    return launch_decode_fp8(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, k_scale, v_scale, o, lse,
                             workspace, stream);
}

extern "C" int bsp_prefill_run(const bsp_plan_info *plan, const void *q, const void *k_pages, const void *v_pages,
                               const int32_t *kv_indices, int64_t num_pages, float sm_scale, void *o, float *lse,
                               void *workspace, bsp_stream_t stream) {
    clear_error();
    int rc = check_plan(plan, BSP_MODE_PREFILL, workspace);
    if (rc != BSP_OK) return rc;
    if (!q || !k_pages || !v_pages || !o) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (num_pages < 1) return fail(BSP_ERR_INVALID_ARG, "num_pages must be positive");
    if ((rc = check_aligned16(q, k_pages, v_pages, o, workspace)) != BSP_OK) return rc;
    rc = launch_prefill(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, o, lse, workspace, stream);
    if (rc != BSP_OK) return rc;
    return launch_reduce(plan, o, lse, workspace, stream);
}

namespace {

// Prefill over the 8-bit cache converts the plan's pages into a bf16 copy first where a
// cached token is read by 3 query tiles or more on average (pages of a power of two, 8 or
// more tokens: the kernel that converts inside takes the codes by TMA) or 1.5 (by cp.async),
// and a CTA has four 128-key tiles or more to work on. Measured (copy first / converted
// inside the kernel), 16-token pages: 16 x 8192 tokens, one tile per token 263 / 194 us, 2
// tiles 356 / 325, 3 tiles 475 / 475, 4 tiles 596 / 627; 24 tiles, 16 x 1536 343 / 411;
// 12-token pages: one tile 276 / 260, page size 1 310 / 326, 8 tiles 552 / 1060; under a
// wave of work, 2 x 150 tokens 19.5 / 16.4 us (a launch less).
constexpr int64_t kRegionReads2Tma = 6, kRegionReads2 = 3;  // twice the query tiles per cached token
constexpr int64_t kRegionTokens = 4 * 128;  // KV tokens of work per CTA
constexpr int64_t kRegionPageRows = 1 << 27;  // rows of a page, all heads: the copy counts a page's vectors in 32 bits

// Decode over it gathers the plan's exponents into table order first where pages have one
// token and a CTA has 2560 tokens or more to work on, or two and twice that. Measured (read
// by page / gathered first), 64/8 heads, one token: 32 requests x 4096 tokens 71.7 / 57.1 us,
// 64 x 4585 163 / 127, 48 x 1024 (2587 tokens per CTA) 31.2 / 29.8, about even at 40 x 1024
// (2156) 28.5 / 28.0; two: 32 x 4096 (6899) 62.0 / 56.0, 64 x 1024 (3449) 39.6 / 40.2; five:
// 32 x 4096 53.0 / 56.4.
constexpr int64_t kGatherTokens = 2560;

// A plan without queries and the NULL pointers of empty tensors: nothing to do.
bool no_queries(const bsp_plan_info *plan, int mode, const void *q, const void *o) {
    clear_error();
    return plan && plan->valid == 1 && plan->problem.mode == mode && plan->num_qo_tokens == 0 && !q && !o;
}

int check_fp8_block(const bsp_plan_info *plan, int mode, const void *q, const void *k_pages, const void *v_pages,
                    const int8_t *k_exp, const int8_t *v_exp, const int32_t *kv_indices, int64_t num_pages,
                    float sm_scale, const void *o, const void *workspace) {
    clear_error();
    int rc = check_plan(plan, mode, workspace);
    if (rc != BSP_OK) return rc;
    if (!std::isfinite(sm_scale)) return fail(BSP_ERR_INVALID_ARG, "sm_scale must be finite");
    if (!q || !k_pages || !v_pages || !k_exp || !v_exp || !o) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (num_pages < 1 || num_pages > INT32_MAX) return fail(BSP_ERR_INVALID_ARG, "num_pages must be in [1, 2^31 - 1]");
    if (num_pages * plan->problem.page_size >= UINT32_MAX)
        return fail(BSP_ERR_UNSUPPORTED, "the 8-bit cache takes at most 2^32 - 2 slots");
    if (!kv_indices && plan->num_table_pages > 0)
        return fail(BSP_ERR_INVALID_ARG, "kv_indices is NULL but the page table has pages");
    return check_aligned16(q, k_pages, v_pages, o, workspace);
}

// Table entries that a decode's region holds (its exponents), or an error.
int decode_region(const bsp_plan_info *plan, void *&region, size_t region_bytes, int64_t &entries) {
    entries = 0;
    if (!region) return BSP_OK;
    if (reinterpret_cast<uintptr_t>(region) % 16 != 0) return fail(BSP_ERR_INVALID_ARG, "the region is not 16-byte aligned");
    const size_t per_entry = 2 * (size_t)plan->problem.num_kv_heads;
    entries = (int64_t)std::min<size_t>(region_bytes / per_entry, INT32_MAX) / 16 * 16;
    if (entries < plan->num_table_pages) return fail(BSP_ERR_CAPACITY, "the region is too small for the plan's page table");
    if (entries == 0) region = nullptr;
    return BSP_OK;
}

// Pages that a prefill's region holds (its bf16 copy), or an error.
int prefill_region(const bsp_plan_info *plan, void *&region, size_t region_bytes, int64_t &pages) {
    pages = 0;
    if (!region) return BSP_OK;
    if (reinterpret_cast<uintptr_t>(region) % 32 != 0) return fail(BSP_ERR_INVALID_ARG, "the region is not 32-byte aligned");
    if ((int64_t)plan->problem.page_size * plan->problem.num_kv_heads > kRegionPageRows)
        return fail(BSP_ERR_UNSUPPORTED, "a copy takes pages of at most 2^27 rows over all heads: pass no region");
    const size_t per_page = (size_t)plan->problem.page_size * plan->problem.num_kv_heads * 512;  // bf16 K and V
    pages = (int64_t)std::min<size_t>(region_bytes / per_page, (size_t)(INT32_MAX / plan->problem.page_size));
    if (pages < plan->num_table_pages) return fail(BSP_ERR_CAPACITY, "the region is too small for the plan's page table");
    if (pages == 0) region = nullptr;
    return BSP_OK;
}

}  // namespace

extern "C" int bsp_decode_run_fp8_block(const bsp_plan_info *plan, const void *q, const void *k_pages,
                                        const void *v_pages, const int8_t *k_exp, const int8_t *v_exp,
                                        const int32_t *kv_indices, int64_t num_pages, float sm_scale, void *o,
                                        float *lse, void *region, size_t region_bytes, void *workspace,
                                        bsp_stream_t stream) {
    if (no_queries(plan, BSP_MODE_DECODE, q, o)) return BSP_OK;
    int rc = check_fp8_block(plan, BSP_MODE_DECODE, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o,
                             workspace);
    if (rc != BSP_OK) return rc;
    int64_t entries;
    if ((rc = decode_region(plan, region, region_bytes, entries)) != BSP_OK) return rc;
    return launch_decode_fp8_block(plan, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse,
                                   region, entries, workspace, stream);
}

extern "C" size_t bsp_decode_fp8_region_size(const bsp_plan_info *plan) {
    clear_error();
    if (!plan || plan->problem.mode != BSP_MODE_DECODE || plan->num_table_pages <= 0) return 0;
    if (plan->problem.page_size > 2 || plan->total_work < kGatherTokens * plan->problem.page_size * plan->capacity.num_ctas)
        return 0;
    return (((size_t)plan->num_table_pages + 15) & ~(size_t)15) * 2 * plan->problem.num_kv_heads;
}

extern "C" size_t bsp_prefill_fp8_region_size(const bsp_plan_info *plan) {
    clear_error();
    if (!plan || plan->problem.mode != BSP_MODE_PREFILL || plan->num_table_pages <= 0) return 0;
    const int64_t tokens = (int64_t)plan->num_table_pages * plan->problem.page_size;
    if (tokens > INT32_MAX || (int64_t)plan->problem.page_size * plan->problem.num_kv_heads > kRegionPageRows) return 0;
    const int32_t ps = plan->problem.page_size;
    const int64_t reads2 = ps >= 8 && (ps & (ps - 1)) == 0 ? kRegionReads2Tma : kRegionReads2;
    if (2 * plan->total_work < reads2 * tokens * plan->problem.num_kv_heads ||
        plan->total_work < kRegionTokens * plan->capacity.num_ctas)
        return 0;
    return (size_t)tokens * plan->problem.num_kv_heads * 512;
}

extern "C" int bsp_prefill_run_fp8_block(const bsp_plan_info *plan, const void *q, const void *k_pages,
                                         const void *v_pages, const int8_t *k_exp, const int8_t *v_exp,
                                         const int32_t *kv_indices, int64_t num_pages, float sm_scale, void *o,
                                         float *lse, void *region, size_t region_bytes, void *workspace,
                                         bsp_stream_t stream) {
    if (no_queries(plan, BSP_MODE_PREFILL, q, o)) return BSP_OK;
    int rc = check_fp8_block(plan, BSP_MODE_PREFILL, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o,
                             workspace);
    if (rc != BSP_OK) return rc;
    if (sm_scale <= 0.f) return fail(BSP_ERR_INVALID_ARG, "prefill needs a positive sm_scale");
    int64_t pages;
    if ((rc = prefill_region(plan, region, region_bytes, pages)) != BSP_OK) return rc;
    rc = launch_prefill_fp8_block(plan, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse,
                                  region, pages, workspace, stream);
    if (rc != BSP_OK) return rc;
    return launch_reduce(plan, o, lse, workspace, stream);
}

namespace {

// A differential run: a plan over pairs of maps, its arguments.
int check_diff(const bsp_plan_info *plan, int mode, const bsp_differential *diff, const void *q, const void *k_pages,
               const void *v_pages, const int8_t *k_exp, const int8_t *v_exp, const int32_t *kv_indices, int64_t num_pages,
               float sm_scale, const void *o, const float *lse, const void *workspace) {
    clear_error();
    int rc = check_plan(plan, mode, workspace);
    if (rc != BSP_OK) return rc;
    const bsp_problem &P = plan->problem;
    if (P.dtype != BSP_DTYPE_BF16 || P.head_dim != 128)
        return fail(BSP_ERR_UNSUPPORTED, "differential attention takes bf16 problems with head_dim 128 (halves of 64)");
    if (plan->group % 2 != 0)
        return fail(BSP_ERR_INVALID_ARG, "a differential plan has two of its query heads, the maps, per head: an even num_qo_heads / num_kv_heads");
    if (P.sink) return fail(BSP_ERR_UNSUPPORTED, "differential attention takes no sink");
    if (!diff || !diff->lambda) return fail(BSP_ERR_INVALID_ARG, "lambda is NULL");
    if (!std::isfinite(diff->out_scale) || !std::isfinite(diff->norm_eps) || diff->norm_eps < 0.f)
        return fail(BSP_ERR_INVALID_ARG, "out_scale and norm_eps must be finite, norm_eps >= 0");
    if (reinterpret_cast<uintptr_t>(diff->norm_weight) % 16 != 0) return fail(BSP_ERR_INVALID_ARG, "norm_weight is not 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(lse) % 8 != 0) return fail(BSP_ERR_INVALID_ARG, "lse is not 8-byte aligned");
    if (!std::isfinite(sm_scale) || (mode == BSP_MODE_PREFILL && sm_scale <= 0.f))
        return fail(BSP_ERR_INVALID_ARG, "sm_scale must be finite, and positive for prefill");
    if ((k_exp == nullptr) != (v_exp == nullptr)) return fail(BSP_ERR_INVALID_ARG, "k_exp and v_exp are given together");
    if (!q || !k_pages || !v_pages || !o) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (num_pages < 1 || num_pages > INT32_MAX) return fail(BSP_ERR_INVALID_ARG, "num_pages must be in [1, 2^31 - 1]");
    if (k_exp && num_pages * P.page_size >= UINT32_MAX)
        return fail(BSP_ERR_UNSUPPORTED, "the 8-bit cache takes at most 2^32 - 2 slots");
    if (!kv_indices && plan->num_table_pages > 0)
        return fail(BSP_ERR_INVALID_ARG, "kv_indices is NULL but the page table has pages");
    return check_aligned16(q, k_pages, v_pages, o, workspace);
}

}  // namespace

extern "C" int bsp_decode_run_diff(const bsp_plan_info *plan, const bsp_differential *diff, const void *q, const void *k_pages,
                                   const void *v_pages, const int8_t *k_exp, const int8_t *v_exp, const int32_t *kv_indices,
                                   int64_t num_pages, float sm_scale, void *o, float *lse, void *region, size_t region_bytes,
                                   void *workspace, bsp_stream_t stream) {
    if (no_queries(plan, BSP_MODE_DECODE, q, o)) return BSP_OK;
    int rc = check_diff(plan, BSP_MODE_DECODE, diff, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse, workspace);
    if (rc != BSP_OK) return rc;
    if (!k_exp) return launch_decode(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, o, lse, workspace, stream, diff);
    int64_t entries;
    if ((rc = decode_region(plan, region, region_bytes, entries)) != BSP_OK) return rc;
    return launch_decode_fp8_block(plan, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse, region,
                                   entries, workspace, stream, diff);
}

extern "C" size_t bsp_prefill_diff_region_size(const bsp_plan_info *plan) {
    clear_error();
    if (!plan || plan->problem.mode != BSP_MODE_PREFILL || plan->num_table_pages <= 0) return 0;
    return (size_t)plan->num_table_pages * plan->problem.page_size * plan->problem.num_kv_heads * 512;
}

extern "C" int bsp_prefill_run_diff(const bsp_plan_info *plan, const bsp_differential *diff, const void *q, const void *k_pages,
                                    const void *v_pages, const int8_t *k_exp, const int8_t *v_exp, const int32_t *kv_indices,
                                    int64_t num_pages, float sm_scale, void *o, float *lse, void *region, size_t region_bytes,
                                    void *workspace, bsp_stream_t stream) {
    if (no_queries(plan, BSP_MODE_PREFILL, q, o)) return BSP_OK;
    int rc = check_diff(plan, BSP_MODE_PREFILL, diff, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse, workspace);
    if (rc != BSP_OK) return rc;
    int64_t pages = 0;
    if (k_exp && (rc = prefill_region(plan, region, region_bytes, pages)) != BSP_OK) return rc;
    if (k_exp && !region && plan->num_table_pages > 0)
        return fail(BSP_ERR_INVALID_ARG, "a differential prefill over the 8-bit cache needs a region");
    if (k_exp && region)
        rc = launch_prefill_fp8_block(plan, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse, region,
                                      pages, workspace, stream, diff);
    else  // (an empty page table: no page is read)
        rc = launch_prefill(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, o, lse, workspace, stream, diff);
    if (rc != BSP_OK) return rc;
    return launch_reduce(plan, o, lse, workspace, stream, diff);
}

extern "C" int bsp_run_attention(const bsp_plan_info *plan, const void *q, const void *k_pages,
                                 const void *v_pages, const int32_t *kv_indices, int64_t num_pages,
                                 float sm_scale, void *o, float *lse, void *workspace, bsp_stream_t stream) {
    clear_error();
    if (!plan) return fail(BSP_ERR_INVALID_ARG, "plan is NULL");
    const int mode = plan->problem.mode;
    int rc = check_plan(plan, mode, workspace);
    if (rc != BSP_OK) return rc;
    if (!q || !k_pages || !v_pages || !o) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if ((rc = check_aligned16(q, k_pages, v_pages, o, workspace)) != BSP_OK) return rc;
    if (mode == BSP_MODE_DECODE) {
        if (num_pages < 0) return fail(BSP_ERR_INVALID_ARG, "num_pages must not be negative");
        return launch_decode(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, o, lse, workspace, stream);
    }
    if (num_pages < 1) return fail(BSP_ERR_INVALID_ARG, "num_pages must be positive");
    return launch_prefill(plan, q, k_pages, v_pages, kv_indices, num_pages, sm_scale, o, lse, workspace, stream);
}

extern "C" int bsp_run_merge_partials(const bsp_plan_info *plan, void *o, float *lse, void *workspace,
                                      bsp_stream_t stream) {
    clear_error();
    if (!plan) return fail(BSP_ERR_INVALID_ARG, "plan is NULL");
    int rc = check_plan(plan, plan->problem.mode, workspace);
    if (rc != BSP_OK) return rc;
    if (!o) return fail(BSP_ERR_INVALID_ARG, "o is NULL");
    return launch_reduce(plan, o, lse, workspace, stream);
}

extern "C" int bsp_check_bounded_wait(int64_t limit_cycles, int32_t *status, bsp_stream_t stream) {
    clear_error();
    if (!status) return fail(BSP_ERR_INVALID_ARG, "status is NULL");
    if (limit_cycles < 1 || limit_cycles > (int64_t{1} << 33))
        return fail(BSP_ERR_INVALID_ARG, "limit_cycles must be in [1, 2^33] (about 4 s)");
    return launch_wait_probe(limit_cycles, reinterpret_cast<int *>(status), stream);
}

extern "C" int bsp_merge_state(const void *o_a, const float *lse_a, const void *o_b, const float *lse_b, void *o_out,
                               float *lse_out, int64_t n_rows, int32_t num_heads, int32_t head_dim, int32_t dtype,
                               bsp_stream_t stream) {
    clear_error();
    if (n_rows < 0 || num_heads < 1 || head_dim < 1) return fail(BSP_ERR_INVALID_ARG, "bad merge_state sizes");
    if (dtype != BSP_DTYPE_BF16 && dtype != BSP_DTYPE_F32) return fail(BSP_ERR_INVALID_ARG, "bad dtype");
    if (n_rows > 0 && (!o_a || !lse_a || !o_b || !lse_b || !o_out || !lse_out))
        return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    return launch_merge_state(o_a, lse_a, o_b, lse_b, o_out, lse_out, n_rows, num_heads, head_dim, dtype, stream);
}

extern "C" int bsp_build_page_tables(int32_t batch, int32_t page_size, const int32_t *cached_lens,
                                     const int32_t *new_lens, const int32_t *free_pages, int64_t free_capacity,
                                     const int32_t *num_free, int32_t *block_table, int64_t block_table_stride,
                                     int32_t max_pages_per_request, int32_t *kv_indptr, int32_t *last_page_len,
                                     int32_t *kv_indices, int64_t max_table_pages, int32_t *qo_indptr,
                                     int64_t *slot_map, int32_t *positions, int64_t max_new_tokens, int32_t *counts,
                                     bsp_stream_t stream) {
    clear_error();
    if (batch < 0 || page_size < 1) return fail(BSP_ERR_INVALID_ARG, "batch must be >= 0 and page_size >= 1");
    if (free_capacity < 0 || max_table_pages < 0 || max_new_tokens < 0 || max_pages_per_request < 0)
        return fail(BSP_ERR_INVALID_ARG, "a capacity is negative");
    if (free_capacity > INT32_MAX || max_table_pages > INT32_MAX || max_new_tokens > INT32_MAX)
        return fail(BSP_ERR_INVALID_ARG, "a capacity exceeds 2^31 - 1");
    if (block_table_stride < max_pages_per_request)
        return fail(BSP_ERR_INVALID_ARG, "block_table_stride is below max_pages_per_request");
    if (!kv_indptr || !qo_indptr || !counts || !num_free) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (batch > 0 && (!cached_lens || !new_lens || !last_page_len || (max_pages_per_request > 0 && !block_table)))
        return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if ((free_capacity > 0 && !free_pages) || (max_table_pages > 0 && !kv_indices) ||
        (max_new_tokens > 0 && (!slot_map || !positions)))
        return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (reinterpret_cast<uintptr_t>(kv_indices) % 16 || reinterpret_cast<uintptr_t>(slot_map) % 16 ||
        reinterpret_cast<uintptr_t>(positions) % 16)
        return fail(BSP_ERR_INVALID_ARG, "kv_indices, slot_map and positions must be 16-byte aligned");
    return launch_page_tables(batch, page_size, cached_lens, new_lens, free_pages, free_capacity, num_free, block_table,
                              block_table_stride, max_pages_per_request, kv_indptr, last_page_len, kv_indices,
                              max_table_pages, qo_indptr, slot_map, positions, max_new_tokens, counts, stream);
}

extern "C" int bsp_append_kv_fp8(const void *k, const void *v, int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t v_token_stride, int64_t v_head_stride, int32_t dtype, int64_t n_tokens,
                                 const int64_t *slot_map, void *k_pages, void *v_pages, int8_t *k_exp, int8_t *v_exp,
                                 int64_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t head_dim,
                                 bsp_stream_t stream) {
    clear_error();
    if (dtype != BSP_DTYPE_BF16 && dtype != BSP_DTYPE_F32) return fail(BSP_ERR_INVALID_ARG, "bad dtype");
    if (head_dim != 128) return fail(BSP_ERR_UNSUPPORTED, "the e4m3 cache has head_dim 128");
    if (n_tokens < 0 || num_pages < 1 || num_pages > INT32_MAX || page_size < 1 || num_kv_heads < 1)
        return fail(BSP_ERR_INVALID_ARG, "bad append sizes");
    if (num_kv_heads > 32767 || n_tokens > INT32_MAX || num_pages * page_size >= UINT32_MAX)
        return fail(BSP_ERR_UNSUPPORTED, "append takes at most 32767 kv heads, 2^31 - 1 tokens and 2^32 - 2 slots");
    if (n_tokens == 0) return BSP_OK;
    if (!k || !v || !slot_map || !k_pages || !v_pages || !k_exp || !v_exp)
        return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    const int64_t elem = dtype == BSP_DTYPE_F32 ? 4 : 2;
    const int64_t st[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    for (int i = 0; i < 4; ++i)
        if (st[i] % (16 / elem) != 0)
            return fail(BSP_ERR_INVALID_ARG, "the strides of k and v must be multiples of 16 bytes");
    const void *ptr[4] = {k, v, k_pages, v_pages};
    for (int i = 0; i < 4; ++i)
        if (reinterpret_cast<uintptr_t>(ptr[i]) % 16 != 0)
            return fail(BSP_ERR_INVALID_ARG, "k, v and the page pools must be 16-byte aligned");
    return launch_append_kv(k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, dtype, n_tokens,
                            slot_map, k_pages, v_pages, k_exp, v_exp, num_pages, page_size, num_kv_heads, stream);
}

namespace {

// The page table and pool that the eviction calls share.
int check_table(int32_t batch, const int32_t *kv_indptr, const int32_t *kv_indices, int64_t max_table_pages,
                const int32_t *last_page_len, int64_t num_pages, int32_t page_size, int32_t num_kv_heads) {
    if (batch < 0 || batch > 65535) return fail(BSP_ERR_INVALID_ARG, "batch must be in [0, 65535]");
    if (page_size < 1 || num_kv_heads < 1 || num_pages < 1 || num_pages > INT32_MAX)
        return fail(BSP_ERR_INVALID_ARG, "page_size and num_kv_heads must be positive, num_pages in [1, 2^31 - 1]");
    if (max_table_pages < 0 || max_table_pages > INT32_MAX) return fail(BSP_ERR_INVALID_ARG, "max_table_pages must be in [0, 2^31 - 1]");
    if (num_kv_heads > 32767 || num_pages * page_size >= UINT32_MAX)
        return fail(BSP_ERR_UNSUPPORTED, "at most 32767 kv heads and 2^32 - 2 slots");
    if (max_table_pages * page_size / 64 * num_kv_heads >= INT32_MAX)
        return fail(BSP_ERR_UNSUPPORTED, "the page table is too large: tokens x kv heads must stay below 2^37");
    if (batch > 0 && (!kv_indptr || !last_page_len || (max_table_pages > 0 && !kv_indices)))
        return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    return BSP_OK;
}

// bsp_accumulate_weights, or with a stall_limit bsp_check_weights_wait.
int accumulate(const bsp_problem *problem, const void *q, const float *lse, int64_t n_tokens,
               const void *k_pages, const int8_t *k_exp, int64_t num_pages, float *weights,
               int32_t batch, const int32_t *qo_indptr, const int32_t *kv_indptr,
               const int32_t *kv_indices, int64_t max_table_pages, const int32_t *last_page_len,
               float sm_scale, float decay, const float *lambda, int64_t stall_limit, bsp_stream_t stream) {
    if (!problem) return fail(BSP_ERR_INVALID_ARG, "problem is NULL");
    bsp_problem P = *problem;
    P.mode = BSP_MODE_DECODE;  // (members that the call does not read, and their own limits)
    P.causal = 1;
    if (!check_problem(&P)) return last_code();
    int rc = check_table(batch, kv_indptr, kv_indices, max_table_pages, last_page_len, num_pages, P.page_size, P.num_kv_heads);
    if (rc != BSP_OK) return rc;
    const int D = P.head_dim, g = P.num_qo_heads / P.num_kv_heads;
    if (P.dtype == BSP_DTYPE_F32 ? (D != 32 && D != 64 && D != 128 && D != 256) : (D != 64 && D != 128))
        return fail(BSP_ERR_UNSUPPORTED, "weights take head_dim 64 and 128 (bf16) or 32, 64, 128, 256 (fp32)");
    if (k_exp && (P.dtype != BSP_DTYPE_BF16 || D != 128))
        return fail(BSP_ERR_UNSUPPORTED, "weights over the 8-bit cache take bf16 queries with head_dim 128");
    if (lambda && P.dtype != BSP_DTYPE_BF16) return fail(BSP_ERR_UNSUPPORTED, "differential weights are bf16 only");
    if (!std::isfinite(sm_scale) || !std::isfinite(decay) || decay < 0.f)
        return fail(BSP_ERR_INVALID_ARG, "sm_scale and decay must be finite, decay >= 0");
    if (n_tokens < 0 || (n_tokens > 0 && n_tokens > INT32_MAX / g))
        return fail(BSP_ERR_INVALID_ARG, "n_tokens must be >= 0, and n_tokens x group below 2^31");
    if (batch == 0 || max_table_pages == 0) return BSP_OK;
    if (!k_pages || !weights || (n_tokens > 0 && (!q || !lse))) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if ((rc = check_aligned16(q, k_pages, nullptr, nullptr, nullptr)) != BSP_OK) return rc;
    if (lambda && reinterpret_cast<uintptr_t>(lse) % 8 != 0) return fail(BSP_ERR_INVALID_ARG, "lse of two maps is not 8-byte aligned");
    return launch_accumulate_weights(&P, q, lse, n_tokens, k_pages, k_exp, num_pages, weights, batch, qo_indptr, kv_indptr,
                                     kv_indices, max_table_pages, last_page_len, sm_scale, decay, lambda, stall_limit, stream);
}

}  // namespace

extern "C" int bsp_accumulate_weights(const bsp_problem *problem, const void *q, const float *lse, int64_t n_tokens,
                                      const void *k_pages, const int8_t *k_exp, int64_t num_pages, float *weights,
                                      int32_t batch, const int32_t *qo_indptr, const int32_t *kv_indptr,
                                      const int32_t *kv_indices, int64_t max_table_pages, const int32_t *last_page_len,
                                      float sm_scale, float decay, const float *lambda, bsp_stream_t stream) {
    clear_error();
    return accumulate(problem, q, lse, n_tokens, k_pages, k_exp, num_pages, weights, batch, qo_indptr, kv_indptr, kv_indices,
                      max_table_pages, last_page_len, sm_scale, decay, lambda, 0, stream);
}

extern "C" int bsp_check_weights_wait(const bsp_problem *problem, const void *q, const float *lse, int64_t n_tokens,
                                      const void *k_pages, const int8_t *k_exp, int64_t num_pages, float *weights,
                                      int32_t batch, const int32_t *qo_indptr, const int32_t *kv_indptr,
                                      const int32_t *kv_indices, int64_t max_table_pages, const int32_t *last_page_len,
                                      float sm_scale, float decay, int64_t limit_cycles, bsp_stream_t stream) {
    clear_error();
    if (limit_cycles < 1 || limit_cycles > (int64_t{1} << 33))
        return fail(BSP_ERR_INVALID_ARG, "limit_cycles must be in [1, 2^33] (about 4 s)");
    if (problem && (problem->dtype != BSP_DTYPE_BF16 || problem->head_dim != 128 || problem->window_left > 0 || problem->logits_soft_cap != 0.f))
        return fail(BSP_ERR_UNSUPPORTED, "the self-test takes bf16 problems with head_dim 128, no window and no soft-cap");
    return accumulate(problem, q, lse, n_tokens, k_pages, k_exp, num_pages, weights, batch, qo_indptr, kv_indptr, kv_indices,
                      max_table_pages, last_page_len, sm_scale, decay, nullptr, limit_cycles, stream);
}

extern "C" int bsp_select_tokens(const float *weights, int64_t num_pages, int32_t page_size, int32_t num_kv_heads,
                                 int32_t batch, const int32_t *kv_indptr, const int32_t *kv_indices,
                                 int64_t max_table_pages, const int32_t *last_page_len, const int32_t *budget,
                                 int32_t max_keep, int32_t sinks, int32_t recent, int32_t *kept, int32_t *new_lens,
                                 bsp_stream_t stream) {
    clear_error();
    int rc = check_table(batch, kv_indptr, kv_indices, max_table_pages, last_page_len, num_pages, page_size, num_kv_heads);
    if (rc != BSP_OK) return rc;
    if (max_keep < 0 || sinks < 0 || recent < 0) return fail(BSP_ERR_INVALID_ARG, "max_keep, sinks and recent must be >= 0");
    if ((int64_t)batch * num_kv_heads > INT32_MAX / 8) return fail(BSP_ERR_UNSUPPORTED, "too many rows (requests x kv heads)");
    if (batch == 0) return BSP_OK;
    if (!weights || !budget || !new_lens || (max_keep > 0 && !kept)) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    return launch_select_tokens(weights, num_pages, page_size, num_kv_heads, batch, kv_indptr, kv_indices, max_table_pages,
                                last_page_len, budget, max_keep, sinks, recent, kept, new_lens, stream);
}

extern "C" int bsp_compact_cache(const int32_t *kept, const int32_t *new_lens, int32_t max_keep, int32_t batch,
                                 const int32_t *kv_indptr, const int32_t *kv_indices, int64_t max_table_pages,
                                 const int32_t *last_page_len, void *k_pages, void *v_pages, int8_t *k_exp, int8_t *v_exp,
                                 float *weights, int64_t num_pages, int32_t page_size, int32_t num_kv_heads,
                                 int32_t row_bytes, bsp_stream_t stream) {
    clear_error();
    int rc = check_table(batch, kv_indptr, kv_indices, max_table_pages, last_page_len, num_pages, page_size, num_kv_heads);
    if (rc != BSP_OK) return rc;
    if (max_keep < 0) return fail(BSP_ERR_INVALID_ARG, "max_keep must be >= 0");
    if (row_bytes < 16 || row_bytes % 16 != 0) return fail(BSP_ERR_INVALID_ARG, "row_bytes must be a positive multiple of 16");
    if ((k_exp == nullptr) != (v_exp == nullptr)) return fail(BSP_ERR_INVALID_ARG, "k_exp and v_exp are given together");
    if (k_exp && row_bytes != 128) return fail(BSP_ERR_UNSUPPORTED, "the e4m3 cache has head_dim 128");
    if (batch == 0 || max_keep == 0 || max_table_pages == 0) return BSP_OK;
    if (!kept || !new_lens || !k_pages || !v_pages) return fail(BSP_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if ((rc = check_aligned16(nullptr, k_pages, v_pages, nullptr, nullptr)) != BSP_OK) return rc;
    return launch_compact_cache(kept, new_lens, max_keep, batch, kv_indptr, kv_indices, max_table_pages, last_page_len,
                                k_pages, v_pages, k_exp, v_exp, weights, num_pages, page_size, num_kv_heads, row_bytes, stream);
}

extern "C" int bsp_check_device_error(const bsp_plan_info *plan, void *workspace, bsp_stream_t stream,
                                      int32_t *word_out) {
    clear_error();
    if (!word_out) return fail(BSP_ERR_INVALID_ARG, "word_out is NULL");
    *word_out = 0;
    if (!plan || plan->valid != 1 || !workspace) return fail(BSP_ERR_INVALID_ARG, "plan or workspace missing");
    uint8_t *status = static_cast<uint8_t *>(workspace) + plan->off_status;
    int32_t word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, status, sizeof(word), cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && word != 0) {
        e = cudaMemsetAsync(status, 0, sizeof(word), stream);
        // CTAs that gave up may have left partial counts in the reduction map's
        // arrival words; a later run of this plan would then fold too early
        if (e == cudaSuccess && plan->num_merges > 0)
            e = cudaMemset2DAsync(static_cast<uint8_t *>(workspace) + plan->off_merges +
                                      offsetof(bsp_merge_entry, arrived),
                                  sizeof(bsp_merge_entry), 0, sizeof(int32_t), (size_t)plan->num_merges, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    if (e != cudaSuccess) return fail(BSP_ERR_CUDA, std::string("status read: ") + cudaGetErrorString(e));
    *word_out = word;
    return BSP_OK;
}
