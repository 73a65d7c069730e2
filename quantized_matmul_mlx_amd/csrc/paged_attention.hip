// qaff_paged_attention: attention of a step's new tokens over the paged cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax: for a tile of scores s
// the new maximum m' scales what was summed by exp(m - m'), and o and l take the tile's exp(s - m').
// The result is o / l. Scores are kept in units of log2 (scale * log2(e) folded into one factor), so
// that the exponential is one v_exp_f32.
#include "mfma16.h"
#include "paged.h"

namespace qaff {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The request of row t, or -1 where no request holds it.
__device__ __forceinline__ int request_of(const AttnArgs& a, int t) {
    if (t < a.cu[0] || t >= a.cu[a.requests]) return -1;
    int lo = 0, hi = a.requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One wave per row (token, head), one key per lane, element loads: any head size and alignment.
template <bool F16>
__global__ __launch_bounds__(64) void attn_scalar_kernel(AttnArgs a) {
    __shared__ float q[256];
    __shared__ float prob[64];
    __shared__ int64_t place[64];
    const int lane = threadIdx.x;
    const int t = blockIdx.x / a.heads, h = blockIdx.x - t * a.heads;
    const int hk = h / a.group;
    const uint16_t* qr = a.q + t * a.q_ts + h * a.q_hs;
    for (int d = lane; d < a.dim; d += 64) q[d] = half_to_f32<F16>(qr[d]) * (a.scale * kLog2e);
    __syncthreads();
    const int b = a.requests > 0 ? request_of(a, t) : -1;
    int64_t lo = 0, hi = 0;  // keys that the row sees
    if (b >= 0) {
        const int64_t kv = a.kv_lens[b];
        const int64_t pos = kv - a.cu[b + 1] + t;
        hi = a.causal ? min(kv, pos + 1) : kv;
        lo = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
    }
    const int page_mask = (1 << a.page_shift) - 1;
    float m = -INFINITY, l = 0.f;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t j0 = lo; j0 < hi; j0 += 64) {
        const int64_t j = j0 + lane;
        float s = -INFINITY;
        int64_t at = -1;
        if (j < hi) {
            const int64_t e = j >> a.page_shift;
            const int64_t page = e < a.table_width ? a.tables[(int64_t)b * a.table_width + e] : -1;
            s = NAN;  // a page outside the pool
            if (page >= 0 && page < a.pages) {
                at = page * a.page_stride + (((int64_t)hk << a.page_shift) + (j & page_mask)) * a.dim;
                s = 0.f;
                for (int d = 0; d < a.dim; ++d) s += q[d] * half_to_f32<F16>(a.k_cache[at + d]);
            }
        }
        float top = s;
        for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float m_new = fmaxf(m, top);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float keep = exp2f(m - base);
        const float p = exp2f(s - base);
        float sum = p;
        for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
        l = l * keep + sum;
        m = m_new;
        __syncthreads();
        prob[lane] = p;
        place[lane] = at;
        __syncthreads();
        const int n = (int)min((int64_t)64, hi - j0);
        for (int i = 0; i < 4; ++i) {
            const int d = lane + 64 * i;
            if (d >= a.dim) break;
            float o = acc[i] * keep;
            for (int c = 0; c < n; ++c)
                o += place[c] < 0 ? prob[c] : prob[c] * half_to_f32<F16>(a.v_cache[place[c] + d]);
            acc[i] = o;
        }
    }
    // a row that sees no key: zeros and -infinity
    const bool empty = hi <= lo;
    uint16_t* o = a.out + ((int64_t)t * a.heads + h) * a.dim;
    for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        if (d < a.dim) o[d] = f32_to_half_bits<F16>(empty ? 0.f : acc[i] / l);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.heads + h] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

size_t paged_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_paged_attention(const AttnArgs& a, bool f16, int64_t, hipStream_t stream) {
    const unsigned grid = (unsigned)a.tokens * (unsigned)a.heads;
    if (f16) attn_scalar_kernel<true><<<grid, 64, 0, stream>>>(a);
    else attn_scalar_kernel<false><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace qaff
