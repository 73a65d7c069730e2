// The C ABI of the paged-cache operators (include/qaff.h): argument checks, all on the host before
// any launch, and dispatch. Lengths, tables and slots live on the device and cannot be checked here:
// the kernels bound every index that they take from them.
#include "qaff.h"

#include "paged.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

namespace {

qaff_status fail(qaff_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    qaff::set_error(buf);
    return st;
}

qaff_status after_launch(const char* op, hipError_t e, hipStream_t stream) {
    static const bool sync = [] {
        const char* v = std::getenv("QAFF_DEBUG_SYNC");
        return v && v[0] && std::strcmp(v, "0") != 0;
    }();
    if (e == hipErrorInvalidConfiguration)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: more rows than one launch holds (2^32 threads)", op);
    if (e == hipSuccess && sync) e = hipStreamSynchronize(stream);
    if (e != hipSuccess) return fail(QAFF_ERR_DEVICE, "%s: %s", op, hipGetErrorString(e));
    return QAFF_OK;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A pointer that a non-empty size needs: set and aligned.
qaff_status check_ptr(const char* op, const char* name, const void* p, uintptr_t a) {
    if (!p) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: null %s", op, name);
    if (!aligned(p, a)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %s must be %d-byte aligned", op, name, (int)a);
    return QAFF_OK;
}

// log2 of a supported page size, or -1.
int page_shift_of(int32_t page_size) {
    for (int s = 3; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

qaff_status bad_page_size(const char* op, int32_t page_size) {
    return fail(QAFF_ERR_UNSUPPORTED, "%s: page size %d is not supported (8, 16, 32, 64, 128 or 256)", op, page_size);
}

constexpr int64_t k1G = 1LL << 30, k2G = 1LL << 31;

// The caches' sizes: every page holds kv_heads * page_size * head_dim elements, page_stride apart.
qaff_status check_cache(const char* op, int64_t pages, int64_t page_stride, int64_t kv_heads, int64_t head_dim,
                        int32_t page_size) {
    if (pages < 0 || page_stride < 0) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative cache size", op);
    if (pages >= k2G) return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^31 pages or more", op);
    if (kv_heads >= k2G) return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^31 cache heads or more", op);
    if (pages > 1 && page_stride < kv_heads * head_dim * page_size)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: pages %lld elements apart overlap", op, (long long)page_stride);
    return QAFF_OK;
}

}  // namespace

extern "C" {

qaff_status qaff_paged_plan(const int32_t* cached_lens, const int32_t* new_lens, int64_t requests,
                            const int32_t* free_pages, int64_t n_free, int32_t* block_tables, int64_t table_width,
                            int32_t page_size, int64_t tokens, int32_t* cu_new, int32_t* kv_lens, int32_t* positions,
                            int64_t* slots, int32_t* pages_used, hipStream_t stream) {
    const char* op = "qaff_paged_plan";
    qaff::set_error("");
    const int shift = page_shift_of(page_size);
    if (shift < 0) return bad_page_size(op, page_size);
    if (requests < 0 || n_free < 0 || table_width < 0 || tokens < 0)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (requests > qaff::kPlanMaxRequests)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: more than %lld requests", op, (long long)qaff::kPlanMaxRequests);
    if (tokens >= k2G) return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^31 tokens or more", op);
    qaff_status st = check_ptr(op, "cu_new", cu_new, 4);
    if (st == QAFF_OK) st = check_ptr(op, "pages_used", pages_used, 4);
    if (st == QAFF_OK && requests > 0) {
        st = check_ptr(op, "cached_lens", cached_lens, 4);
        if (st == QAFF_OK) st = check_ptr(op, "new_lens", new_lens, 4);
        if (st == QAFF_OK) st = check_ptr(op, "kv_lens", kv_lens, 4);
        if (st == QAFF_OK && n_free > 0) st = check_ptr(op, "free_pages", free_pages, 4);
        if (st == QAFF_OK && table_width > 0) st = check_ptr(op, "block_tables", block_tables, 4);
    }
    if (st == QAFF_OK && tokens > 0) {
        st = check_ptr(op, "positions", positions, 4);
        if (st == QAFF_OK) st = check_ptr(op, "slots", slots, 8);
    }
    if (st != QAFF_OK) return st;
    qaff::PlanArgs a{};
    a.cached = cached_lens;
    a.fresh = new_lens;
    a.free_pages = free_pages;
    a.tables = block_tables;
    a.cu_new = cu_new;
    a.kv_lens = kv_lens;
    a.positions = positions;
    a.slots = slots;
    a.pages_used = pages_used;
    a.n_free = n_free;
    a.table_width = table_width;
    a.tokens = tokens;
    a.requests = (int)requests;
    a.page_shift = shift;
    return after_launch(op, qaff::launch_paged_plan(a, stream), stream);
}

qaff_status qaff_rope_append(const void* q, const void* k, const void* v, qaff_dtype dtype, int64_t tokens,
                             int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t q_token_stride,
                             int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int32_t* positions, int32_t axes,
                             const int32_t* sections, int32_t interleaved, int32_t traditional, const float* inv_freq,
                             int64_t rot, const int64_t* slots, void* k_cache, void* v_cache, int64_t pages,
                             int64_t page_stride, int32_t page_size, void* q_out, hipStream_t stream) {
    const char* op = "qaff_rope_append";
    qaff::set_error("");
    if (dtype != QAFF_BF16 && dtype != QAFF_F16)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: dtype %d (bf16 or float16)", op, (int)dtype);
    const int shift = page_shift_of(page_size);
    if (shift < 0) return bad_page_size(op, page_size);
    if (tokens < 0 || heads < 0 || kv_heads < 0 || head_dim < 0 || rot < 0)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (q_token_stride < 0 || q_head_stride < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 ||
        v_head_stride < 0)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative stride", op);
    if (head_dim > 512) return fail(QAFF_ERR_UNSUPPORTED, "%s: head_dim %lld is above 512", op, (long long)head_dim);
    if (rot % 2 != 0 || rot > head_dim)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %lld turned values of %lld", op, (long long)rot, (long long)head_dim);
    if (tokens >= k2G || heads >= (1 << 20) || kv_heads >= (1 << 20))
        return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^31 tokens or 2^20 heads or more", op);
    if (axes < 1 || axes > 4) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %d axes (1 to 4)", op, axes);
    qaff::RopeArgs a{};
    const int half = (int)(rot / 2);
    if (!sections) {
        if (axes > 1) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %d axes need their sections", op, axes);
        a.sections[0] = half;
    } else {
        int64_t sum = 0;
        for (int i = 0; i < axes; ++i) {
            if (sections[i] < 0) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative section", op);
            a.sections[i] = sections[i];
            sum += sections[i];
            if (interleaved && i > 0 && sections[i] > 0 && (int64_t)(sections[i] - 1) * axes + i >= half)
                return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: section %d of %d pairs does not fit interleaved in %d", op, i,
                            sections[i], half);
        }
        if (sum != half)
            return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: sections add up to %lld of %d pairs", op, (long long)sum, half);
    }
    qaff_status st = check_cache(op, pages, page_stride, kv_heads, head_dim, page_size);
    if (st != QAFF_OK) return st;
    if (tokens == 0 || head_dim == 0 || heads + kv_heads == 0) return QAFF_OK;
    st = check_ptr(op, "positions", positions, 4);
    if (st == QAFF_OK && rot > 0) st = check_ptr(op, "inv_freq", inv_freq, 4);
    if (st == QAFF_OK && heads > 0) st = check_ptr(op, "q", q, 2);
    if (st == QAFF_OK && heads > 0) st = check_ptr(op, "q_out", q_out, 2);
    if (st == QAFF_OK && kv_heads > 0) {
        st = check_ptr(op, "k", k, 2);
        if (st == QAFF_OK) st = check_ptr(op, "v", v, 2);
        if (st == QAFF_OK) st = check_ptr(op, "slots", slots, 8);
        if (st == QAFF_OK && pages > 0) st = check_ptr(op, "k_cache", k_cache, 2);
        if (st == QAFF_OK && pages > 0) st = check_ptr(op, "v_cache", v_cache, 2);
    }
    if (st != QAFF_OK) return st;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.slots = slots;
    a.k_cache = static_cast<uint16_t*>(k_cache);
    a.v_cache = static_cast<uint16_t*>(v_cache);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.tokens = tokens;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.page_stride = page_stride;
    a.total_slots = pages << shift;
    a.heads = (int)heads;
    a.kv_heads = (int)kv_heads;
    a.dim = (int)head_dim;
    a.half = half;
    a.page_shift = shift;
    a.axes = axes;
    a.interleaved = interleaved != 0;
    return after_launch(op, qaff::launch_rope_append(a, dtype == QAFF_F16, traditional != 0, stream), stream);
}

size_t qaff_paged_attention_workspace_size(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                           int32_t page_size, int64_t table_width, int64_t requests,
                                           int64_t max_new) {
    if (tokens <= 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || head_dim <= 0 || head_dim > 256 ||
        requests <= 0 || requests > 65536 || table_width <= 0 || page_shift_of(page_size) < 0 ||
        tokens >= k2G / heads || table_width >= k1G / page_size)
        return 0;
    return qaff::paged_attention_workspace(tokens, heads, kv_heads, head_dim, table_width * page_size, requests, max_new);
}

qaff_status qaff_paged_attention(const void* q, qaff_dtype dtype, int64_t tokens, int64_t heads,
                                 int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
                                 const void* v_cache, int64_t pages, int64_t page_stride, int64_t kv_heads,
                                 int64_t head_dim, int32_t page_size, const int32_t* block_tables, int64_t table_width,
                                 const int32_t* cu_new, const int32_t* kv_lens, int64_t requests, int64_t max_new,
                                 float scale, int32_t causal, int64_t window, void* workspace, size_t workspace_bytes,
                                 void* out, float* lse, hipStream_t stream) {
    const char* op = "qaff_paged_attention";
    qaff::set_error("");
    if (dtype != QAFF_BF16 && dtype != QAFF_F16)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: dtype %d (bf16 or float16)", op, (int)dtype);
    const int shift = page_shift_of(page_size);
    if (shift < 0) return bad_page_size(op, page_size);
    if (tokens < 0 || heads < 0 || kv_heads < 0 || head_dim < 0 || requests < 0 || table_width < 0 || window < 0 ||
        max_new < 0)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (q_token_stride < 0 || q_head_stride < 0) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative stride", op);
    if (heads > 0 && (kv_heads == 0 || heads % kv_heads != 0))
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %lld heads over %lld cache heads", op, (long long)heads,
                    (long long)kv_heads);
    if (head_dim > 256) return fail(QAFF_ERR_UNSUPPORTED, "%s: head_dim %lld is above 256", op, (long long)head_dim);
    if (requests > 65536) return fail(QAFF_ERR_UNSUPPORTED, "%s: more than 65536 requests", op);
    if (heads > 0 && tokens >= k2G / heads)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: %lld tokens of %lld heads", op, (long long)tokens, (long long)heads);
    if (table_width >= k1G / page_size)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: a table of %lld pages is 2^30 tokens or more", op, (long long)table_width);
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: scale %g is not positive and finite", op, (double)scale);
    qaff_status st = check_cache(op, pages, page_stride, kv_heads, head_dim, page_size);
    if (st != QAFF_OK) return st;
    if (tokens == 0 || heads == 0 || head_dim == 0) return QAFF_OK;
    st = check_ptr(op, "q", q, 2);
    if (st == QAFF_OK) st = check_ptr(op, "out", out, 2);
    if (st == QAFF_OK) st = check_ptr(op, "cu_new", cu_new, 4);
    if (st == QAFF_OK && lse && !aligned(lse, 4))
        st = fail(QAFF_ERR_INVALID_ARGUMENT, "%s: lse must be 4-byte aligned", op);
    if (st == QAFF_OK && requests > 0) {
        st = check_ptr(op, "kv_lens", kv_lens, 4);
        if (st == QAFF_OK && table_width > 0) st = check_ptr(op, "block_tables", block_tables, 4);
        if (st == QAFF_OK && pages > 0) st = check_ptr(op, "k_cache", k_cache, 2);
        if (st == QAFF_OK && pages > 0) st = check_ptr(op, "v_cache", v_cache, 2);
    }
    if (st != QAFF_OK) return st;
    const size_t need = qaff_paged_attention_workspace_size(tokens, heads, kv_heads, head_dim, page_size, table_width,
                                                            requests, max_new);
    if (need > 0) {
        if (workspace_bytes < need)
            return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes, needs %zu", op, workspace_bytes, need);
        st = check_ptr(op, "workspace", workspace, 16);
        if (st != QAFF_OK) return st;
    }
    qaff::AttnArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k_cache = static_cast<const uint16_t*>(k_cache);
    a.v_cache = static_cast<const uint16_t*>(v_cache);
    a.tables = block_tables;
    a.cu = cu_new;
    a.kv_lens = kv_lens;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.partial = need > 0 ? static_cast<float*>(workspace) : nullptr;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.page_stride = page_stride;
    a.table_width = table_width;
    a.table_keys = (int)(table_width * page_size);
    a.pages = pages;
    a.window = window;
    a.tokens = (int)tokens;
    a.heads = (int)heads;
    a.kv_heads = (int)kv_heads;
    a.group = (int)(heads / kv_heads);
    a.dim = (int)head_dim;
    a.page_shift = shift;
    a.requests = (int)requests;
    a.causal = causal != 0;
    a.scale = scale;
    return after_launch(op, qaff::launch_paged_attention(a, dtype == QAFF_F16, max_new, stream), stream);
}

}  // extern "C"
