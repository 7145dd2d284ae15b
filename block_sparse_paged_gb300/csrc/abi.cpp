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
    int64_t entries = 0;
    if (region) {
        if (reinterpret_cast<uintptr_t>(region) % 16 != 0)
            return fail(BSP_ERR_INVALID_ARG, "the region is not 16-byte aligned");
        const size_t per_entry = 2 * (size_t)plan->problem.num_kv_heads;
        entries = (int64_t)std::min<size_t>(region_bytes / per_entry, INT32_MAX) / 16 * 16;
        if (entries < plan->num_table_pages) return fail(BSP_ERR_CAPACITY, "the region is too small for the plan's page table");
        if (entries == 0) region = nullptr;
    }
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
    int64_t pages = 0;
    if (region) {
        if (reinterpret_cast<uintptr_t>(region) % 32 != 0)
            return fail(BSP_ERR_INVALID_ARG, "the region is not 32-byte aligned");
        if ((int64_t)plan->problem.page_size * plan->problem.num_kv_heads > kRegionPageRows)
            return fail(BSP_ERR_UNSUPPORTED, "a copy takes pages of at most 2^27 rows over all heads: pass no region");
        const size_t per_page = (size_t)plan->problem.page_size * plan->problem.num_kv_heads * 512;  // bf16 K and V
        pages = (int64_t)std::min<size_t>(region_bytes / per_page, (size_t)(INT32_MAX / plan->problem.page_size));
        if (pages < plan->num_table_pages) return fail(BSP_ERR_CAPACITY, "the region is too small for the plan's page table");
        if (pages == 0) region = nullptr;
    }
    rc = launch_prefill_fp8_block(plan, q, k_pages, v_pages, k_exp, v_exp, kv_indices, num_pages, sm_scale, o, lse,
                                  region, pages, workspace, stream);
    if (rc != BSP_OK) return rc;
    return launch_reduce(plan, o, lse, workspace, stream);
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
