// Internal launchers of the paged-cache operators (C ABI: api_paged.cpp) and what their kernels
// share. Arguments are validated by api_paged.cpp; a launcher only enqueues work on `stream` and
// returns hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qaff {

// api.cpp: the calling thread's error text (qaff_last_error).
void set_error(const char* text) noexcept;
int device_cu_count();

// Whether `blocks` workgroups of `threads` fit one launch (fewer than 2^32 threads); a launcher whose
// grid does not returns hipErrorInvalidConfiguration before any launch.
inline bool grid_fits(int64_t blocks, int threads) { return blocks < (1LL << 32) / threads; }

constexpr int64_t kPlanMaxRequests = 16384;

struct PlanArgs {
    const int32_t* cached;
    const int32_t* fresh;  // new tokens of each request
    const int32_t* free_pages;
    int32_t* tables;
    int32_t* cu_new;
    int32_t* kv_lens;
    int32_t* positions;
    int64_t* slots;
    int32_t* pages_used;
    int64_t n_free, table_width, tokens;
    int requests;
    int page_shift;
};
hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t stream);

struct RopeArgs {
    const uint16_t *q, *k, *v;
    const int32_t* positions;  // [axes, tokens]
    const float* inv_freq;     // [half]
    const int64_t* slots;
    uint16_t *k_cache, *v_cache, *q_out;
    int64_t tokens, q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, page_stride, total_slots;
    int heads, kv_heads, dim, half, page_shift, axes, interleaved;
    int sections[4];
};
hipError_t launch_rope_append(const RopeArgs& a, bool f16, bool traditional, hipStream_t stream);

struct AttnArgs {
    const uint16_t *q, *k_cache, *v_cache;
    const int32_t *tables, *cu, *kv_lens;
    uint16_t* out;
    float* lse;      // may be null
    float* partial;  // workspace
    int64_t q_ts, q_hs, page_stride, table_width, pages, window;  // window 0: none
    int tokens, heads, kv_heads, group, dim, page_shift, requests, causal;
    int table_keys;  // table_width pages of keys
    float scale;
};
hipError_t launch_paged_attention(const AttnArgs& a, bool f16, int64_t max_new, hipStream_t stream);
size_t paged_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                 int64_t table_keys, int64_t requests, int64_t max_new);

}  // namespace qaff
