// qaff_paged_attention: attention of a step's new tokens over the paged cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax: for a tile of scores s
// the new maximum m' scales what was summed by exp(m - m'), and o and l take the tile's exp(s - m').
// The result is o / l. Scores are kept in units of log2 (scale * log2(e) folded into one factor), so
// that the exponential is one v_exp_f32.
#include "mfma16.h"
#include "paged.h"
#include "paged_sched.h"
#include "wave.h"

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

// A wave takes one row (token t, head h) over keys [lo, hi) of request b, one key a lane, element
// loads: any head size and alignment, and nothing but the keys in the range enters. Leaves the running
// maximum (log2), the sum and o (lane + 64 i) of the range.
template <bool F16>
__device__ void scalar_row(const AttnArgs& a, int b, int t, int h, int64_t lo, int64_t hi, float& m, float& l,
                           float (&acc)[4]) {
    const int lane = threadIdx.x & 63;
    const int hk = h / a.group;
    const uint16_t* q = a.q + t * a.q_ts + h * a.q_hs;
    const int page_mask = (1 << a.page_shift) - 1;
    m = -INFINITY;
    l = 0.f;
    for (int i = 0; i < 4; ++i) acc[i] = 0.f;
#pragma unroll 1
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
                for (int d = 0; d < a.dim; ++d) s += half_to_f32<F16>(q[d]) * half_to_f32<F16>(a.k_cache[at + d]);
                s *= a.scale * kLog2e;
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
        for (int i = 0; i < 4; ++i) acc[i] *= keep;
        const int n = (int)min((int64_t)64, hi - j0);
        for (int c = 0; c < n; ++c) {
            const float w = __shfl(p, c);
            const int64_t from = __shfl(at, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = lane + 64 * i;
                if (d < a.dim) acc[i] += from < 0 ? w : w * half_to_f32<F16>(a.v_cache[from + d]);
            }
        }
    }
}

// The result of a row that sees no key is zeros and -infinity.
template <bool F16>
__device__ void store_scalar_row(const AttnArgs& a, int t, int h, bool empty, float m, float l, const float (&acc)[4]) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)t * a.heads + h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        if (d < a.dim) a.out[row * a.dim + d] = f32_to_half_bits<F16>(empty ? 0.f : acc[i] / l);
    }
    if (a.lse && lane == 0) a.lse[row] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <bool F16>
__global__ __launch_bounds__(64) void attn_scalar_kernel(AttnArgs a) {
    const int t = blockIdx.x / a.heads, h = blockIdx.x - t * a.heads;
    const int b = a.requests > 0 ? request_of(a, t) : -1;
    int64_t lo = 0, hi = 0;  // keys that the row sees
    if (b >= 0) {
        const int64_t kv = a.kv_lens[b];
        const int64_t pos = kv - a.cu[b + 1] + t;
        hi = a.causal ? min(kv, pos + 1) : kv;
        lo = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
        // keys past the table make the row NaN, and one of them is enough
        if (hi > a.table_keys + 1) {
            hi = a.table_keys + 1;
            lo = min(lo, (int64_t)a.table_keys);
        }
    }
    float m, l, acc[4];
    scalar_row<F16>(a, b, t, h, lo, hi, m, l, acc);
    store_scalar_row<F16>(a, t, h, hi <= lo, m, l, acc);
}

// ---- The matrix-core kernel ----
//
// A request's query heads that share a cache head are rows of one matrix: row r of the request is its
// token r / group with head r % group of the group, so every tile of keys is read once for all of
// them. A wave holds 32 rows and takes keys 32 at a time with v_mfma_f32_32x32x16:
//   S^T = K . Q^T   (A = 32 keys x 16 values from LDS, B = Q^T in registers)
//   O^T += V^T . P^T (A = V^T by transposing LDS reads, B = P^T)
// Transposed, a lane holds 16 scores of ONE row (lane % 32): its softmax needs one exchange between
// the wave's halves, and its rescaling factor is the lane's own. The lane's scores also are what B
// wants of P^T, if the 16 keys of a product are numbered as they lie: half h holds keys 4 h .. 4 h + 3
// and 8 + 4 h .. 8 + 4 h + 3 of each 16, and the reads of V^T take the same order.
//
// Two kernels share this. Chunks and prompts: 4 waves of 32 rows, K and V tiles of 64 keys staged once
// for the 128 rows. A few rows (decode): every wave of a workgroup takes all rows, at most 16, and other
// keys, with v_mfma_f32_16x16x32; the waves join in LDS. Where tiles are few, both cut a tile's keys
// into parts for several workgroups, and a second kernel joins those.
//
// LDS holds 16-byte pieces, piece c of row r at c ^ f(r), so that neither the row-wise reads of K nor
// the transposing reads of V (4 rows by 64 bytes, or 8 by 32, for half a wave) meet in a bank.

typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

struct Sched {
    int rows_lo, rows_hi;  // takes requests with rows_lo < rows <= rows_hi (rows = tokens * group)
    int parts;             // tiles of rows are cut along the keys into about so many parts in all; 0: not cut
    int min_part;          // key tiles that a part has at least
    float* part_o;         // [item, kv head, row of the tile, dim] sums of a part
    float2* part_ml;       // their running maximum (log2) and sum
};

// A workgroup's work: part `part` of `parts` of a tile of a request's rows.
struct Item {
    int tile, part, parts;
    int first;       // the item of part 0
    int row_end;     // rows of the request that the call has
    int start, end;  // its tokens, as cu gives them: the last is the one at position kv - 1
    int kv;
    int b;
};


// Item `want` (or the item of part 0 of tile `want`) of those that the schedule's requests make.
// Every wave scans the requests itself, 64 at a time: with up to 64 requests that is one load of
// each length and two scans, less than reading another kernel's schedule would cost. The scans of all
// workgroups together grow with the square of the requests: decoding over up to 500 keys a request, 256
// requests take 86 us, 1021 take 472 (38% more than four times as long), 4096 take 4.4 ms (three times
// sixteen times as long); over up to 4000 keys they do not show up to 1021 requests.
template <int ROWS, int KT>
__device__ __forceinline__ bool find_item(const AttnArgs& a, const Sched& s, int want, bool by_tile, Item& it) {
    const int lane = threadIdx.x & 63;
    const int count = a.requests;
    int start = 0, end = 0, kv = 0, tiles = 0, span = 0;
    auto load = [&](int b) {
        start = end = kv = tiles = span = 0;
        if (b < count) {
            start = a.cu[b];
            end = a.cu[b + 1];
            kv = a.kv_lens[b];
        }
        kv = max(kv, 0);
        // rows past the call's are not there, also of a request that begins before them
        if (start >= 0 && start < min(end, a.tokens)) {
            const int rows = (min(end, a.tokens) - start) * a.group;  // at most tokens * heads < 2^31
            tiles = tiles_of(rows, ROWS, s.rows_lo, s.rows_hi);
        }
        span = span_of(kv, a.window, a.table_keys, a.group, ROWS, KT);
    };
    load(lane);
    uint32_t len = 0x7fffffffu;  // key tiles of a part
    if (s.parts > 0) {
        // tiles times spans; where 32 bits might not hold the sum, nothing is cut
        const uint32_t cap = work_cap(count);
        bool past_cap = false;
        auto product = [&] {
            const uint64_t x = (uint64_t)(uint32_t)tiles * (uint32_t)span;
            past_cap |= x > cap;
            return (int)min(x, (uint64_t)cap);
        };
        int total = product();
        for (int b0 = 64; b0 < count; b0 += 64) {
            load(b0 + lane);
            total += product();
        }
        const uint32_t all = (uint32_t)lane_value(wave_scan(total), 63);
        if (!__any(past_cap)) len = part_length(all, s.parts, s.min_part);
        if (count > 64) load(lane);
    }
    int items_before = 0, tiles_before = 0;
    for (int b0 = 0;; b0 += 64) {
        const int parts = parts_of(span, len);
        const int items = tiles * parts;
        const int items_in = items_before + wave_scan(items), tiles_in = tiles_before + wave_scan(tiles);
        const uint64_t past = __ballot((by_tile ? tiles_in : items_in) > want);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int base = lane_value(items_in - items, at);
            const int n = lane_value(parts, at), t = lane_value(tiles, at);
            const int local = by_tile ? want - lane_value(tiles_in - tiles, at) : (int)((uint32_t)(want - base) / (uint32_t)n);
            it.first = base + local * n;
            it.part = by_tile ? 0 : want - it.first;
            it.parts = n;
            it.tile = t - 1 - local;  // a causal prompt's last rows see the most keys: they go first
            it.start = lane_value(start, at);
            it.end = lane_value(end, at);
            it.kv = lane_value(kv, at);
            it.row_end = (min(it.end, a.tokens) - it.start) * a.group;
            it.b = b0 + at;
            return true;
        }
        items_before = lane_value(items_in, 63);
        tiles_before = lane_value(tiles_in, 63);
        if (b0 + 64 >= count) break;
        load(b0 + 64 + lane);
    }
    // rows past the last request: one more request, without keys
    it.start = a.cu[count];
    it.end = a.tokens;
    it.row_end = it.start >= 0 && it.start < it.end ? (it.end - it.start) * a.group : 0;
    if (it.row_end <= s.rows_lo || it.row_end > s.rows_hi) return false;
    const int t = (int)(((uint32_t)it.row_end + ROWS - 1) / ROWS);
    const int local = want - (by_tile ? tiles_before : items_before);
    if (local >= t) return false;
    it.first = items_before + local;
    it.part = 0;
    it.parts = 1;
    it.tile = t - 1 - local;
    it.kv = 0;
    it.b = count;
    return true;
}

// Key tiles [begin, end) of an item's part, of n from tile t0 on: the first n % parts are one longer.
__device__ __forceinline__ void part_of(const Item& it, int t0, int n, int& begin, int& end) {
    const int each = (int)((uint32_t)n / (uint32_t)it.parts), more = n - each * it.parts;
    begin = t0 + it.part * each + min(it.part, more);
    end = begin + each + (it.part < more ? 1 : 0);
}

// The keys [lo, hi) that token i of the request sees. Keys past the table make the row NaN, and one
// of them is enough: a length beyond the table must not keep the loops busy.
__device__ __forceinline__ void seen_keys(const AttnArgs& a, const Item& it, int i, int& lo, int& hi) {
    const int pos = it.kv - (it.end - it.start) + i;
    hi = a.causal ? max(0, min(it.kv, pos + 1)) : it.kv;
    lo = a.window > 0 ? (int)max((int64_t)0, pos + 1 - a.window) : 0;
    if (hi > a.table_keys + 1) {
        hi = a.table_keys + 1;
        lo = min(lo, a.table_keys);
    }
}

// The maximum and the sum of v over the lanes that hold the same row: lane and lane ^ 32, and with 16
// rows a wave lane ^ 16 and lane ^ 48 too.
template <int R> __device__ __forceinline__ float max_of_row(float v) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    if (R == 16) {
        r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}
template <int R> __device__ __forceinline__ float sum_of_row(float v) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if (R == 16) {
        r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// Whether either 16-bit value of w is infinite or NaN.
template <bool F16>
__device__ __forceinline__ bool not_finite2(uint32_t w) {
    constexpr uint32_t E = F16 ? 0x7C00u : 0x7F80u;
    return (w & E) == E || ((w >> 16) & E) == E;
}
// Where piece c of row r of a tile lies: c ^ f(r). K is read a row a lane (16 lanes: 16 rows, one
// piece), V in half-waves of 4 rows by 4 pieces (R = 32) or 8 rows by 2 pieces (R = 16): each time the
// 256 bytes fall into all 64 banks.
template <int DP> __device__ __forceinline__ int swizzle_k(int row) { return DP == 64 ? (row >> 1) & 7 : row & 15; }
template <int DP, int R> __device__ __forceinline__ int swizzle_v(int row) {
    if (R == 16) return DP == 64 ? row & 6 : (row & 7) << 1;
    return DP == 64 ? (row & 2) << 1 : (row & 3) << 2;
}

// The two shapes of a wave's products, v_mfma_f32_32x32x16 (R = 32 rows) and 16x16x32 (R = 16).
template <int R> struct Shape;
template <> struct Shape<32> {
    typedef f32x16 acc;
    static constexpr int kVals = 16;
};
template <> struct Shape<16> {
    typedef f32x4 acc;
    static constexpr int kVals = 4;
};
template <bool F16> __device__ __forceinline__ f32x16 product(op8<F16> a, op8<F16> b, f32x16 c) {
    return mfma32x32x16<F16>(a, b, c);
}
template <bool F16> __device__ __forceinline__ f32x4 product(op8<F16> a, op8<F16> b, f32x4 c) {
    return mfma16x16x32<F16>(a, b, c);
}

// float16 probabilities carry a factor 2^7 (which the division by their sum takes out again): their
// smallest step is then 2^-31 of the largest, so long rows of small weights are not lost. With the
// slack of the running maximum below they stay under 2^15.
template <bool F16> constexpr float kLift = F16 ? 7.f : 0.f;
// The running maximum follows a row's true one only once that is 2^8 times larger: a stale maximum
// scales sums and probabilities alike, and most tiles then need no rescaling of the output sums.
constexpr float kSlack = 8.f;

// Keys outside [lo, hi) of the lane's row out of a tile's scores. Value i of block kb is key
// R kb + 8 (i / 4) + 4 part + i % 4 of the tile.
template <int R, int SB>
__device__ __forceinline__ void mask_scores(typename Shape<R>::acc (&sc)[SB], int key0, int part, int lo, int hi) {
    asm volatile("");  // keeps the caller's branch: few tiles need this, and selects would cost all of them
#pragma unroll
    for (int kb = 0; kb < SB; ++kb)
#pragma unroll
        for (int i = 0; i < Shape<R>::kVals; ++i) {
            const int key = key0 + kb * R + (i >> 2) * 8 + 4 * part + (i & 3);
            if (key < lo || key >= hi) sc[kb][i] = -INFINITY;
        }
}

// One tile of the running softmax: scores to probabilities (of the stale maximum), their sum into l,
// and the output sums to a new maximum where the old one is passed by more than the slack.
template <bool F16, int R, int SB, int OB>
__device__ __forceinline__ void softmax_tile(typename Shape<R>::acc (&sc)[SB], typename Shape<R>::acc (&acc)[OB],
                                             float factor, float& m, float& l) {
    float top = sc[0][0];
#pragma unroll
    for (int kb = 0; kb < SB; ++kb)
#pragma unroll
        for (int i = 0; i < Shape<R>::kVals; ++i) top = fmaxf(top, sc[kb][i]);
    top = max_of_row<R>(top) * factor;
    if (__any(top > m + kSlack)) {
        const float m_new = fmaxf(m, top);
        const float keep = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
        l *= keep;
#pragma unroll
        for (int n = 0; n < OB; ++n)
#pragma unroll
            for (int i = 0; i < Shape<R>::kVals; ++i) acc[n][i] *= keep;
        m = m_new;
    }
    const float base = m == -INFINITY ? 0.f : m - kLift<F16>;
#pragma unroll
    for (int kb = 0; kb < SB; ++kb)
#pragma unroll
        for (int i = 0; i < Shape<R>::kVals; ++i) {
            sc[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[kb][i], factor, -base));
            l += sc[kb][i];
        }
}

// Eight probabilities rounded to 16 bits, as the matrix instructions take them, for their product with V:
// half a step of the type each (2^-8 of it in bf16, 2^-11 in float16), while their sum l is taken before.
// The error of the output is 1.2 to 1.4 times what its own rounding at the end alone makes.
template <bool F16, typename V0, typename V1>
__device__ __forceinline__ op8<F16> pack8(V0 a, V1 b) {
    return __builtin_bit_cast(op8<F16>, u32x4a{pack_half2<F16>(a[0], a[1]), pack_half2<F16>(a[2], a[3]),
                                               pack_half2<F16>(b[0], b[1]), pack_half2<F16>(b[2], b[3])});
}

// Two transposing reads: 4 + 4 values of one column of V (see the layouts above) as an operand.
template <bool F16>
__device__ __forceinline__ op8<F16> read_column(uint16_t* p0, uint16_t* p1) {
    const u32x2 w0 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p0));
    const u32x2 w1 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p1));
    return __builtin_bit_cast(op8<F16>, u32x4a{w0.x, w0.y, w1.x, w1.y});
}

// Whether the lane's share of a tile of V in LDS holds an infinite or NaN value.
template <bool F16, int PIECES>
__device__ __forceinline__ bool tile_not_finite(const uint16_t* vl) {
    bool found = false;
#pragma unroll 1
    for (int x = threadIdx.x & 63; x < PIECES; x += 64) {
        const u32x4a w = *reinterpret_cast<const u32x4a*>(vl + x * 8);
        found |= not_finite2<F16>(w.x) || not_finite2<F16>(w.y) || not_finite2<F16>(w.z) || not_finite2<F16>(w.w);
    }
    return found;
}

// A weight of zero times an infinite or NaN value is NaN. Where a tile holds keys that some row does not
// see and such a value, the rows [x0, x1) of the item's tile are taken again, one by one, each over the
// keys that it sees alone. Rare, and kept out of the loops, whose registers it would cost.
template <bool F16, int ROWS>
__device__ void take_rows_again(const AttnArgs& a, const Sched& s, const Item& it, int item, int hk, int x0, int x1,
                                int step, int key_begin, int key_end) {
    const int lane = threadIdx.x & 63;
#pragma unroll 1
    for (int x = x0; x < x1; x += step) {
        const int r = it.tile * ROWS + x, i = r / a.group, h = hk * a.group + r - i * a.group;
        int from, to;
        seen_keys(a, it, i, from, to);
        float mx, lx, o[4];
        scalar_row<F16>(a, it.b, it.start + i, h, max(from, key_begin), min(to, key_end), mx, lx, o);
        if (it.parts == 1) {
            store_scalar_row<F16>(a, it.start + i, h, to <= from, mx, lx, o);
            continue;
        }
        const int64_t slot = ((int64_t)item * a.kv_heads + hk) * ROWS + x;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (lane + 64 * y < a.dim) s.part_o[slot * a.dim + lane + 64 * y] = o[y];
        if (lane == 0) s.part_ml[slot] = make_float2(mx, lx);
    }
}

// A few rows: NS waves, each with the tile's (at most 16) rows and every NS-th tile of 32 keys, no
// barrier in the loop. K is read from memory as the product wants it: 16 rows of 64 bytes an
// instruction, a lane's 2 rows the same for K and V, so a tile costs it 2 table lookups and 2
// addresses. A tile's keys are used before its values: their registers take the next tile's loads
// at once, so a wave has about a tile (16 KB at 128 values) in flight all the time. 64 decoding requests
// of up to 8192 keys take 203 us with the join, 5.34 TB/s: three quarters of what a plain read of 1 GiB
// reaches (7.1 TB/s); the counters show no busy unit, the waves wait for memory or to issue.
template <int DP, int NS> constexpr int kFewLds = NS * (32 * DP * 2 + kFewRows * 8);
template <bool F16, int DP, int NS, bool FULL>
__device__ __forceinline__ void few_rows(const AttnArgs& a, const Sched& s, int block, uint8_t* lds) {
    constexpr int KT = kFewKeys, R = kFewRows;
    constexpr int QF = DP / 32, OB = DP / 16;
    constexpr int BYTES = KT * DP * 2;  // of a wave: V's tile, then its rows' sums (16 rows of DP floats)
    float2* ml = reinterpret_cast<float2*>(lds + NS * BYTES);  // [wave][row]

    const int dim = FULL ? DP : a.dim;  // FULL: the head size is DP
    const int hk = block % a.kv_heads;
    const int item = block / a.kv_heads;
    Item it;
    if (!find_item<R, KT>(a, s, item, false, it)) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = lane >> 4, col = lane & 15;
    const int r0 = it.tile * R;
    const int rows = min(R, it.row_end - r0);
    const bool live = col < rows;
    const int token = (r0 + min(col, rows - 1)) / a.group;
    const int head = hk * a.group + (r0 + min(col, rows - 1)) - token * a.group;
    int lo, hi;
    seen_keys(a, it, token, lo, hi);
    int lo_all, hi_all, unused;
    seen_keys(a, it, r0 / a.group, lo_all, unused);
    seen_keys(a, it, (r0 + rows - 1) / a.group, unused, hi_all);
    const int kt0 = lo_all / KT;
    const int n_all = max(0, (hi_all + KT - 1) / KT - kt0);
    int kt_begin, kt_end;
    part_of(it, kt0, n_all, kt_begin, kt_end);
    // the first token sees the least far back keys, the last the farthest: between, no mask is needed
    int sure_lo, sure_hi;
    seen_keys(a, it, (r0 + rows - 1) / a.group, sure_lo, unused);
    seen_keys(a, it, r0 / a.group, unused, sure_hi);

    const int page_mask = (1 << a.page_shift) - 1;
    const int32_t* table = a.tables + (int64_t)it.b * a.table_width;
    const int64_t head_at = ((int64_t)hk << a.page_shift) * dim;
    const int last_entry = min(hi_all - 1, a.table_keys - 1) >> a.page_shift;
    // Loads need no condition: keys before lo_all and from hi_all on lie in pages that the item's keys
    // have, a page outside the pool is replaced by page 0, pieces past the head size by piece 0. What
    // such a load brings is put right before its use (fix).
    int page[2], bad = 0;
    u32x4a kreg[2][QF], vreg[2][QF];
    auto load_pages = [&](int kt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int entry = (kt * KT + 16 * i + col) >> a.page_shift;
            page[i] = table[min(entry, last_entry)];  // looked at only by load_tile: no wait for it here
        }
    };
    auto load_tile = [&](int kt) {
        bad = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool ok = (uint32_t)page[i] < (uint64_t)a.pages && min(kt * KT + 16 * i + col, hi_all - 1) < a.table_keys;
            if (!ok) bad |= 1 << i;
            const uint64_t at = (uint64_t)(uint32_t)(ok ? page[i] : 0) * (uint32_t)a.page_stride + head_at +
                                (uint32_t)(((kt * KT + 16 * i + col) & page_mask) * dim);
#pragma unroll
            for (int c = 0; c < QF; ++c) {
                const int d = 32 * c + 8 * part;
                kreg[i][c] = *reinterpret_cast<const u32x4a*>(a.k_cache + at + (d < dim ? d : 0));
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t at = (uint64_t)(uint32_t)(bad >> i & 1 ? 0 : page[i]) * (uint32_t)a.page_stride + head_at +
                                (uint32_t)(((kt * KT + 16 * i + col) & page_mask) * dim);
#pragma unroll
            for (int c = 0; c < QF; ++c) {
                const int d = 32 * c + 8 * part;
                vreg[i][c] = *reinterpret_cast<const u32x4a*>(a.v_cache + at + (d < dim ? d : 0));
            }
        }
    };
    auto fix_tile = [&](int kt) {
        asm volatile("");  // keeps the caller's branch
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = kt * KT + 16 * i + col;
            const bool in = key >= lo_all && key < hi_all, out_of_pool = bad >> i & 1;
#pragma unroll
            for (int c = 0; c < QF; ++c) {
                // NaN scores where the page is outside the pool: the rows that see the key are NaN
                if (out_of_pool) kreg[i][c] = u32x4a{0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};
                else if (32 * c + 8 * part >= dim) kreg[i][c] = u32x4a{0, 0, 0, 0};
                if (!in || out_of_pool) vreg[i][c] = u32x4a{0, 0, 0, 0};
            }
        }
    };

    int kt = kt_begin + wave;
    if (kt < kt_end) {
        load_pages(kt);
        load_tile(kt);
        load_pages(kt + NS);
    }
    // Q^T in registers: lane holds row `col`, values 32 c + 8 part ..
    op8<F16> q[QF];
    {
        const uint16_t* src = a.q + (int64_t)(it.start + token) * a.q_ts + (int64_t)head * a.q_hs;
#pragma unroll
        for (int c = 0; c < QF; ++c) {
            u32x4a v = {0, 0, 0, 0};
            if (live && 32 * c + 8 * part < dim) v = *reinterpret_cast<const u32x4a*>(src + 32 * c + 8 * part);
            q[c] = __builtin_bit_cast(op8<F16>, v);
        }
    }
    f32x4 acc[OB];
#pragma unroll
    for (int n = 0; n < OB; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    bool again = false;
    const float factor = a.scale * kLog2e;
    uint16_t* vl = reinterpret_cast<uint16_t*>(lds + wave * BYTES);
    // a lane's transposing reads: rows v_row and v_row + 16, pieces 2 n + v_piece, from value v_sub on
    const int v_row = 4 * part + (col >> 2), v_piece = (lane & 3) >> 1, v_sub = 4 * (lane & 1);

    for (; kt < kt_end; kt += NS) {
        if (dim < DP || kt * KT < lo_all || (kt + 1) * KT > hi_all || __any(bad)) fix_tile(kt);
        f32x4 sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < QF; ++c) sc[i] = product<F16>(__builtin_bit_cast(op8<F16>, kreg[i][c]), q[c], sc[i]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < QF; ++c) {
                const int row = 16 * i + col;
                *reinterpret_cast<u32x4a*>(vl + row * DP + (((4 * c + part) ^ swizzle_v<DP, R>(row)) * 8)) = vreg[i][c];
            }
        if (kt + NS < kt_end) {
            load_tile(kt + NS);
            load_pages(kt + 2 * NS);
        }
        const int key0 = kt * KT;
        if (key0 < sure_lo || key0 + KT > sure_hi) {
            mask_scores<R>(sc, key0, part, lo, hi);
            if (key0 < sure_lo || min(key0 + KT, hi_all) > sure_hi) again |= tile_not_finite<F16, KT * DP / 8>(vl);
        }
        op8<F16> vf[OB];  // all of them asked for before the softmax, whose time hides theirs
#pragma unroll
        for (int n = 0; n < OB; ++n) {
            uint16_t* src = vl + v_row * DP + ((v_piece + 2 * n) ^ swizzle_v<DP, R>(v_row)) * 8 + v_sub;
            vf[n] = read_column<F16>(src, src + 16 * DP);
        }
        __builtin_amdgcn_sched_barrier(0);
        softmax_tile<F16, R>(sc, acc, factor, m, l);
        const op8<F16> p = pack8<F16>(sc[0], sc[1]);
#pragma unroll
        for (int n = 0; n < OB; ++n) acc[n] = product<F16>(vf[n], p, acc[n]);
    }

    l = sum_of_row<R>(l);
    if (__syncthreads_or(again)) {
        take_rows_again<F16, R>(a, s, it, item, hk, wave, rows, NS, kt_begin * KT, kt_end * KT);
        return;
    }
    // Join the waves: sums as float4 pieces, piece d of row c at 16 d + (c ^ d % 16).
#pragma unroll
    for (int n = 0; n < OB; ++n) {
        const int d = 4 * n + part;
        *reinterpret_cast<f32x4*>(lds + wave * BYTES + (16 * d + (col ^ (d & 15))) * 16) = acc[n];
    }
    if (part == 0) ml[wave * R + col] = make_float2(m - kLift<F16>, l);
    __syncthreads();
    const int64_t slot0 = ((int64_t)item * a.kv_heads + hk) * R;
    for (int u = tid; u < rows * (DP / 4); u += 64 * NS) {
        const int row = u / (DP / 4), d = u % (DP / 4);
        float top = ml[row].x;
#pragma unroll
        for (int w = 1; w < NS; ++w) top = fmaxf(top, ml[w * R + row].x);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NS; ++w) {
            const float2 x = ml[w * R + row];
            const float k = __builtin_amdgcn_exp2f(x.x - base);
            sum += k * x.y;
            o += k * *reinterpret_cast<const f32x4*>(lds + w * BYTES + (16 * d + (row ^ (d & 15))) * 16);
        }
        if (4 * d >= dim) continue;
        if (it.parts > 1) {
            *reinterpret_cast<f32x4*>(s.part_o + (slot0 + row) * dim + 4 * d) = o;
            if (d == 0) s.part_ml[slot0 + row] = make_float2(top, sum);
            continue;
        }
        const int i = (r0 + row) / a.group, h = hk * a.group + (r0 + row) - i * a.group;
        int from, to;
        seen_keys(a, it, i, from, to);
        const bool empty = to <= from;
        const float inv = empty ? 0.f : 1.f / sum;
        const int64_t at = (int64_t)(it.start + i) * a.heads + h;
        *reinterpret_cast<uint2*>(a.out + at * dim + 4 * d) =
            make_uint2(pack_half2<F16>(o.x * inv, o.y * inv), pack_half2<F16>(o.z * inv, o.w * inv));
        if (a.lse && d == 0) a.lse[at] = empty ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
}

// Chunks and prompts: 4 waves of 32 rows. K and V tiles go through registers into LDS one tile ahead,
// one barrier a tile. A prompt of 8192 (32 heads of 128): 579 to 611 us, 900 to 949 TFLOP/s; the matrix
// cores are busy 46% of a CU's time and the vector units 52%, one after the other for the most part: the
// softmax, the tiles' addresses and LDS accesses take as many issue slots as the products take cycles.
// Interleaving the products with another tile's softmax within a wave, and loads straight into LDS, gave
// the same time.
constexpr int kManyWaves = kManyRows / 32;
template <int DP> constexpr int kManyKeys = many_keys(DP);
template <int DP> constexpr int kManyLds = 2 * 2 * kManyKeys<DP> * DP * 2;  // two buffers of K and V
template <bool F16, int DP, bool FULL>
__device__ __forceinline__ void many_rows(const AttnArgs& a, const Sched& s, int block, uint8_t* lds_bytes) {
    constexpr int R = 32, ROWS = kManyRows, NT = 64 * kManyWaves, KT = kManyKeys<DP>;
    constexpr int CH = DP / 8;               // 16-byte pieces of a row
    constexpr int PER = KT * CH / NT;        // pieces of a tile per thread, RSTEP rows apart
    constexpr int RSTEP = NT / CH;
    constexpr int TILE = KT * DP;            // elements
    constexpr int VALS = Shape<R>::kVals;    // a lane's values of a product
    constexpr int QF = DP / 16, SB = KT / R, OB = DP / R;
    typedef typename Shape<R>::acc acc_t;
    uint16_t* lds = reinterpret_cast<uint16_t*>(lds_bytes);

    const int dim = FULL ? DP : a.dim;
    const int hk = block % a.kv_heads;
    const int item = block / a.kv_heads;
    Item it;
    if (!find_item<ROWS, KT>(a, s, item, false, it)) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = lane / R, col = lane % R;  // this lane's share of its row
    const int r0 = it.tile * ROWS;
    const int rows = min(ROWS, it.row_end - r0);
    // this lane's row
    const int r = wave * R + col;
    const bool live = r < rows;
    const int token = (r0 + min(r, rows - 1)) / a.group;
    const int head = hk * a.group + (r0 + min(r, rows - 1)) - token * a.group;
    int lo, hi;
    seen_keys(a, it, token, lo, hi);
    // keys the workgroup reads: from the first that its first token sees to the last of its last
    int lo_all, hi_all, unused;
    seen_keys(a, it, r0 / a.group, lo_all, unused);
    seen_keys(a, it, (r0 + rows - 1) / a.group, unused, hi_all);
    const int kt0 = lo_all / KT;
    const int n_all = max(0, (hi_all + KT - 1) / KT - kt0);
    int kt_begin, kt_end;
    part_of(it, kt0, n_all, kt_begin, kt_end);
    // the wave's tiles below sure_hi and from sure_lo on need no mask; rows that are not there
    // need none either
    int sure_lo = live ? lo : 0, sure_hi = live ? hi : 0x7fffffff, any_hi = live ? hi : 0;
    for (int x = R / 2; x > 0; x >>= 1) {
        sure_lo = max(sure_lo, __shfl_xor(sure_lo, x));
        sure_hi = min(sure_hi, __shfl_xor(sure_hi, x));
        any_hi = max(any_hi, __shfl_xor(any_hi, x));
    }
    sure_lo = __builtin_amdgcn_readfirstlane(sure_lo);
    sure_hi = __builtin_amdgcn_readfirstlane(sure_hi);
    any_hi = __builtin_amdgcn_readfirstlane(any_hi);

    // Q^T in registers: lane holds row `col`, values 16 c + 8 part ..
    op8<F16> q[QF];
    {
        const uint16_t* src = a.q + (int64_t)(it.start + token) * a.q_ts + (int64_t)head * a.q_hs;
#pragma unroll
        for (int c = 0; c < QF; ++c) {
            const int d = 16 * c + 8 * part;
            u32x4a v = {0, 0, 0, 0};
            if (live && d < dim) v = *reinterpret_cast<const u32x4a*>(src + d);
            q[c] = __builtin_bit_cast(op8<F16>, v);
        }
    }

    // Staging: this thread's pieces are rows row0 + RSTEP i of a tile, piece `piece`. The rows that a
    // wave loads at once (2 to 8, from wave_row on) lie in one page, so the page and all but a fixed part
    // of the address are the wave's, in scalar registers.
    const int row0 = tid / CH, piece = tid % CH;
    const int wave_row = __builtin_amdgcn_readfirstlane(wave * (64 / CH));
    const int page_mask = (1 << a.page_shift) - 1;
    const int32_t* table = a.tables + (int64_t)it.b * a.table_width;
    const int last_entry = min(max(hi_all, 1) - 1, a.table_keys - 1) >> a.page_shift;
    const uint32_t lane_at = (uint32_t)((row0 - wave_row) * dim + (piece * 8 < dim ? piece * 8 : 0)) * 2;  // bytes
    // As in the other kernel, loads need no condition and are put right before their use. Lane i of
    // `pages` holds the page of row wave_row + RSTEP i of the tile that is loaded next.
    int pages;
    uint32_t bad = 0;
    u32x4a kreg[PER], vreg[PER];
    auto load_pages = [&](int kt) {
        const int key = kt * KT + wave_row + RSTEP * min(lane, PER - 1);
        pages = table[min(key >> a.page_shift, last_entry)];  // looked at only by load_tile: no wait for it here
    };
    auto load_tile = [&](int kt) {
        const int key = kt * KT + wave_row + RSTEP * min(lane, PER - 1);
        const bool ok = (uint32_t)pages < (uint64_t)a.pages && min(key, hi_all - 1) < a.table_keys;
        bad = (uint32_t)__ballot(!ok);
        // where that row lies in the caches, in bytes
        const uint64_t row_at = 2 * ((uint64_t)(uint32_t)(ok ? pages : 0) * (uint32_t)a.page_stride +
                                     (((uint64_t)hk << a.page_shift) + (key & page_mask)) * dim);
        const int at_lo = (int)(uint32_t)row_at, at_hi = (int)(row_at >> 32);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint64_t at = (uint64_t)(uint32_t)lane_value(at_hi, i) << 32 | (uint32_t)lane_value(at_lo, i);
            kreg[i] = *reinterpret_cast<const u32x4a*>(reinterpret_cast<const uint8_t*>(a.k_cache) + at + lane_at);
            vreg[i] = *reinterpret_cast<const u32x4a*>(reinterpret_cast<const uint8_t*>(a.v_cache) + at + lane_at);
        }
    };
    auto fix_tile = [&](int kt) {
        asm volatile("");  // keeps the caller's branch
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int key = kt * KT + row0 + RSTEP * i;
            const bool in = key >= lo_all && key < hi_all, out_of_pool = bad >> i & 1;
            // NaN scores where the page is outside the pool: the rows that see the key are NaN
            if (out_of_pool) kreg[i] = u32x4a{0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};
            else if (piece * 8 >= dim) kreg[i] = u32x4a{0, 0, 0, 0};
            if (!in || out_of_pool) vreg[i] = u32x4a{0, 0, 0, 0};
        }
    };

    acc_t acc[OB];
#pragma unroll
    for (int n = 0; n < OB; ++n)
#pragma unroll
        for (int i = 0; i < VALS; ++i) acc[n][i] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool again = false;
    const float factor = a.scale * kLog2e;

    // a lane's transposing reads: rows v_row + 16 f and + 8, pieces 4 n + v_piece, from value v_sub on
    const int v_row = 4 * part + ((lane & 15) >> 2);
    const int v_piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int v_sub = 4 * (lane & 1);

    if (kt_begin < kt_end) {
        load_pages(kt_begin);
        load_tile(kt_begin);
        load_pages(kt_begin + 1);
    }
    // Products and loads go before the other wave's softmax on the SIMD: both waves at their products would
    // wait for each other, while one at its products and one at its softmax do not (595 -> 583 us for a prompt
    // of 8192, 330 -> 313 us for 512 tokens over 32768).
    __builtin_amdgcn_s_setprio(1);
    for (int kt = kt_begin; kt < kt_end; ++kt) {
        if (dim < DP || kt * KT < lo_all || (kt + 1) * KT > hi_all || bad) fix_tile(kt);
        uint16_t* kl = lds + (kt & 1) * 2 * TILE;
        uint16_t* vl = kl + TILE;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int row = row0 + RSTEP * i;
            *reinterpret_cast<u32x4a*>(kl + row * DP + ((piece ^ swizzle_k<DP>(row)) * 8)) = kreg[i];
            *reinterpret_cast<u32x4a*>(vl + row * DP + ((piece ^ swizzle_v<DP, R>(row)) * 8)) = vreg[i];
        }
        if (kt + 1 < kt_end) {
            load_tile(kt + 1);
            load_pages(kt + 2);
        }
        // two buffers: the other one's readers are past the previous barrier
        __syncthreads();
        const int key0 = kt * KT;
        if (key0 >= any_hi) continue;  // keys past every row of this wave

        // Reads from LDS go out four products ahead of those that take them: left to itself, the compiler
        // reads an operand, waits and multiplies, and each wait is as long as four products. More ahead
        // would not fit the registers.
        constexpr int AHEAD = 4 / SB;  // depths of a stretch
        op8<F16> kf[QF][SB];
        auto read_keys = [&](int c0) {
#pragma unroll
            for (int c = c0; c < c0 + AHEAD; ++c)
#pragma unroll
                for (int kb = 0; kb < SB; ++kb) {
                    const int row = kb * R + col;
                    kf[c][kb] = *reinterpret_cast<const op8<F16>*>(
                        kl + row * DP + (((2 * c + part) ^ swizzle_k<DP>(row)) * 8));
                }
        };
        acc_t sc[SB];
#pragma unroll
        for (int kb = 0; kb < SB; ++kb)
#pragma unroll
            for (int i = 0; i < VALS; ++i) sc[kb][i] = 0.f;
        read_keys(0);
#pragma unroll
        for (int c0 = 0; c0 < QF; c0 += AHEAD) {
            if (c0 + AHEAD < QF) read_keys(c0 + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
            // blocks of keys inside: their products do not wait for each other
#pragma unroll
            for (int c = c0; c < c0 + AHEAD; ++c)
#pragma unroll
                for (int kb = 0; kb < SB; ++kb) sc[kb] = product<F16>(kf[c][kb], q[c], sc[kb]);
        }
        op8<F16> vf[2 * SB][OB];
        auto read_values = [&](int f) {
#pragma unroll
            for (int n = 0; n < OB; ++n) {
                uint16_t* src = vl + (v_row + 16 * f) * DP + ((v_piece + 4 * n) ^ swizzle_v<DP, R>(v_row)) * 8 + v_sub;
                vf[f][n] = read_column<F16>(src, src + 8 * DP);
            }
        };
        read_values(0);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(0);
        if (key0 < sure_lo || key0 + KT > sure_hi) mask_scores<R>(sc, key0, part, lo, hi);
        softmax_tile<F16, R>(sc, acc, factor, m, l);
        op8<F16> p[2 * SB];
#pragma unroll
        for (int f = 0; f < 2 * SB; ++f)
            p[f] = f % 2 ? pack8<F16>(__builtin_shufflevector(sc[f / 2], sc[f / 2], 8, 9, 10, 11),
                                      __builtin_shufflevector(sc[f / 2], sc[f / 2], 12, 13, 14, 15))
                         : pack8<F16>(__builtin_shufflevector(sc[f / 2], sc[f / 2], 0, 1, 2, 3),
                                      __builtin_shufflevector(sc[f / 2], sc[f / 2], 4, 5, 6, 7));
        if (key0 < sure_lo || min(key0 + KT, hi_all) > sure_hi) again |= tile_not_finite<F16, TILE / 8>(vl);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int f = 0; f < 2 * SB; ++f) {
            if (f + 1 < 2 * SB) read_values(f + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < OB; ++n) acc[n] = product<F16>(vf[f][n], p[f], acc[n]);
        }
    }

    if (__any(again)) {  // this wave's rows
        take_rows_again<F16, ROWS>(a, s, it, item, hk, wave * R, min(wave * R + R, rows), 1, kt_begin * KT, kt_end * KT);
        return;
    }
    l = sum_of_row<R>(l);
    if (!live) return;
    const float m_out = m - kLift<F16>;
    if (it.parts > 1) {
        const int64_t slot = ((int64_t)item * a.kv_heads + hk) * ROWS + r;
        float* o = s.part_o + slot * dim;
#pragma unroll
        for (int n = 0; n < OB; ++n)
#pragma unroll
            for (int i = 0; i < VALS / 4; ++i) {
                const int d = R * n + 8 * i + 4 * part;
                if (d < dim)
                    *reinterpret_cast<f32x4*>(o + d) =
                        f32x4{acc[n][4 * i], acc[n][4 * i + 1], acc[n][4 * i + 2], acc[n][4 * i + 3]};
            }
        if (part == 0) s.part_ml[slot] = make_float2(m_out, l);
        return;
    }
    const bool empty = hi <= lo;
    const float inv = empty ? 0.f : 1.f / l;
    const int64_t row = (int64_t)(it.start + token) * a.heads + head;
    uint16_t* o = a.out + row * dim;
#pragma unroll
    for (int n = 0; n < OB; ++n)
#pragma unroll
        for (int i = 0; i < VALS / 4; ++i) {
            const int d = R * n + 8 * i + 4 * part;
            if (d < dim)
                *reinterpret_cast<uint2*>(o + d) = make_uint2(pack_half2<F16>(acc[n][4 * i] * inv, acc[n][4 * i + 1] * inv),
                                                              pack_half2<F16>(acc[n][4 * i + 2] * inv, acc[n][4 * i + 3] * inv));
        }
    if (a.lse && part == 0) a.lse[row] = empty ? -INFINITY : (m_out + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool F16, int DP, int NS, bool FULL>
__global__ __launch_bounds__(64 * NS, DP > 128 ? 1 : 2) void attn_few_kernel(AttnArgs a, Sched s) {
    __shared__ __align__(16) uint8_t lds[kFewLds<DP, NS>];
    few_rows<F16, DP, NS, FULL>(a, s, blockIdx.x, lds);
}

template <bool F16, int DP, bool FULL>
__global__ __launch_bounds__(64 * kManyWaves, DP > 128 ? 1 : 2) void attn_many_kernel(AttnArgs a, Sched s) {
    __shared__ __align__(16) uint8_t lds[kManyLds<DP>];
    many_rows<F16, DP, FULL>(a, s, blockIdx.x, lds);
}

// Chunks or prompts beside decoding requests: both in one launch, the longer work first.
template <bool F16, int DP, bool FULL>
__global__ __launch_bounds__(64 * kManyWaves, DP > 128 ? 1 : 2) void attn_both_kernel(AttnArgs a, Sched many, Sched few,
                                                                                     int many_blocks) {
    __shared__ __align__(16) uint8_t lds[kManyLds<DP> > kFewLds<DP, kManyWaves> ? kManyLds<DP> : kFewLds<DP, kManyWaves>];
    if ((int)blockIdx.x < many_blocks) many_rows<F16, DP, FULL>(a, many, blockIdx.x, lds);
    else few_rows<F16, DP, kManyWaves, FULL>(a, few, (int)blockIdx.x - many_blocks, lds);
}

// Joins the parts of a tile's rows, in their order: o = sum_s w_s o_s / sum_s w_s l_s with
// w_s = 2^(m_s - max m). A workgroup holds RP rows, DP / 4 threads each; the threads left over take
// other parts of the same rows, up to kJoin parts at a time.
constexpr int kJoin = 512;
template <bool F16, int DP, int ROWS, int KT, int RP>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const Sched& s, int block, f32x4* so, float* weight) {
    constexpr int LANES = DP / 4, GROUPS = 256 / LANES / RP;
    static_assert(GROUPS >= 1 && (RP == 1 || GROUPS == 1), "");
    const int hk = block % a.kv_heads;
    Item it;
    if (!find_item<ROWS, KT>(a, s, block / a.kv_heads, true, it) || it.parts == 1) return;
    const int x = threadIdx.x % LANES, g = (threadIdx.x / LANES) % GROUPS, rp = threadIdx.x / (LANES * GROUPS);
    const int r0 = it.tile * ROWS, rows = min(ROWS, it.row_end - r0);
    const bool in = 4 * x < a.dim;
    const int lane_of_row = threadIdx.x % (LANES * GROUPS);
    for (int rb = blockIdx.y * RP; rb < rows; rb += gridDim.y * RP) {
        const int r = min(rb + rp, rows - 1);
        const int64_t slot0 = ((int64_t)it.first * a.kv_heads + hk) * ROWS + r;
        const int64_t step = (int64_t)a.kv_heads * ROWS;
        float m = -INFINITY, l = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (int p0 = 0; p0 < it.parts; p0 += kJoin / RP) {
            const int n = min(kJoin / RP, it.parts - p0);
            // this stretch's maximum and sum, by every wave for its own row
            float top = m;
            for (int p = threadIdx.x & (min(64, LANES * GROUPS) - 1); p < n; p += min(64, LANES * GROUPS))
                top = fmaxf(top, s.part_ml[slot0 + (p0 + p) * step].x);
            for (int y = min(64, LANES * GROUPS) / 2; y > 0; y >>= 1) top = fmaxf(top, __shfl_xor(top, y));
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            __syncthreads();
            for (int p = threadIdx.x & (min(64, LANES * GROUPS) - 1); p < n; p += min(64, LANES * GROUPS)) {
                const float2 ml = s.part_ml[slot0 + (p0 + p) * step];
                const float w = __builtin_amdgcn_exp2f(ml.x - base);
                sum += w * ml.y;
                if (lane_of_row < 64) weight[rp * (kJoin / RP) + p] = w;
            }
            for (int y = min(64, LANES * GROUPS) / 2; y > 0; y >>= 1) sum += __shfl_xor(sum, y);
            __syncthreads();
            const float keep = __builtin_amdgcn_exp2f(m - base);
            l = l * keep + sum;
            o *= keep;
            m = top;
            if (in) {
                const float* src = s.part_o + (slot0 + (int64_t)p0 * step) * a.dim + 4 * x;
#pragma unroll 8
                for (int p = g; p < n; p += GROUPS)
                    o += weight[rp * (kJoin / RP) + p] * *reinterpret_cast<const f32x4*>(src + p * step * a.dim);
            }
        }
        if (GROUPS > 1) {
            __syncthreads();
            so[g * LANES + x] = o;
            __syncthreads();
            if (g == 0)
                for (int p = 1; p < GROUPS; ++p) o += so[p * LANES + x];
        }
        if (g != 0 || rb + rp >= rows) continue;
        const int token = (r0 + r) / a.group, head = hk * a.group + (r0 + r) - token * a.group;
        int lo, hi;
        seen_keys(a, it, token, lo, hi);
        const bool empty = hi <= lo;
        const float inv = empty ? 0.f : 1.f / l;
        const int64_t row = (int64_t)(it.start + token) * a.heads + head;
        if (in)
            *reinterpret_cast<uint2*>(a.out + row * a.dim + 4 * x) =
                make_uint2(pack_half2<F16>(o.x * inv, o.y * inv), pack_half2<F16>(o.z * inv, o.w * inv));
        if (a.lse && x == 0) a.lse[row] = empty ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// The joins of both kernels' tiles: the many-rows kernel's (8 rows of 128 values a workgroup), then the
// few-rows kernel's (RP rows a workgroup).
template <bool F16, int DP, int RP>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, Sched many, Sched few, int many_blocks) {
    __shared__ f32x4 so[256];
    __shared__ float weight[kJoin];
    if ((int)blockIdx.x < many_blocks)
        join_rows<F16, DP, kManyRows, kManyKeys<DP>, 1024 / DP>(a, many, blockIdx.x, so, weight);
    else
        join_rows<F16, DP, kFewRows, kFewKeys, RP>(a, few, (int)blockIdx.x - many_blocks, so, weight);
}

template <bool F16, int DP, bool FULL>
hipError_t launch_tiles(const AttnArgs& a, const Launches& p, hipStream_t stream) {
    const size_t few_slots = p.few.slots(a.kv_heads), many_slots = p.many.slots(a.kv_heads);
    float* o = a.partial;
    float2* ml = reinterpret_cast<float2*>(o + (few_slots + many_slots) * a.dim);
    const Sched few{p.few.rows_lo, p.few.rows_hi, p.few.parts, p.few.min_part, o, ml};
    const Sched many{p.many.rows_lo, p.many.rows_hi, p.many.parts, p.many.min_part, o + few_slots * a.dim, ml + few_slots};
    const unsigned few_blocks = (unsigned)(p.few.items * a.kv_heads), many_blocks = (unsigned)(p.many.items * a.kv_heads);
    constexpr int kWide = DP > 128 ? 4 : 8;  // heads above 128 need more registers than 8 waves can have
    if (p.many.tiles && p.few.tiles)
        attn_both_kernel<F16, DP, FULL><<<many_blocks + few_blocks, 256, 0, stream>>>(a, many, few, (int)many_blocks);
    else if (p.many.tiles)
        attn_many_kernel<F16, DP, FULL><<<many_blocks, 256, 0, stream>>>(a, many);
    else if (p.few_waves == 8)
        attn_few_kernel<F16, DP, kWide, FULL><<<few_blocks, 64 * kWide, 0, stream>>>(a, few);
    else
        attn_few_kernel<F16, DP, 4, FULL><<<few_blocks, 256, 0, stream>>>(a, few);
    if (p.many.parts || p.few.parts) {
        const unsigned many_tiles = p.many.parts ? (unsigned)(p.many.tiles * a.kv_heads) : 0;
        const unsigned few_tiles = p.few.parts ? (unsigned)(p.few.tiles * a.kv_heads) : 0;
        // A row a workgroup, its parts spread over the threads, where a tile has many parts (two rows over
        // 120001 keys); several rows a workgroup, so fewer workgroups to look for their tile, otherwise (64
        // decoding requests: the two kernels 215 -> 209 us).
        const int few_rows = a.group < kFewRows ? a.group : kFewRows;
        constexpr int RP = 1024 / DP;
        if (p.few.parts >= 4 * p.few.tiles) {
            const dim3 grid(many_tiles + few_tiles, many_tiles ? kManyRows / RP : few_rows);
            join_kernel<F16, DP, 1><<<grid, 256, 0, stream>>>(a, many, few, (int)many_tiles);
        } else {
            const dim3 grid(many_tiles + few_tiles, many_tiles ? kManyRows / RP : (few_rows + RP - 1) / RP);
            join_kernel<F16, DP, RP><<<grid, 256, 0, stream>>>(a, many, few, (int)many_tiles);
        }
    }
    return hipGetLastError();
}

template <bool F16, int DP>
hipError_t launch_dim(const AttnArgs& a, const Launches& p, hipStream_t stream) {
    return a.dim == DP ? launch_tiles<F16, DP, true>(a, p, stream) : launch_tiles<F16, DP, false>(a, p, stream);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

size_t paged_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t table_keys,
                                 int64_t requests, int64_t max_new) {
    const Launches p = plan_launches(tokens, heads, kv_heads, head_dim, table_keys, requests, max_new,
                                     device_cu_count());
    return (p.few.slots(kv_heads) + p.many.slots(kv_heads)) * (size_t)(4 * head_dim + 8);
}

hipError_t launch_paged_attention(const AttnArgs& a, bool f16, int64_t max_new, hipStream_t stream) {
    // 16-byte loads of every row, and heads of whole 16-byte pieces (pages apart by a 32-bit count;
    // without any page there is nothing that a load could be pointed at instead)
    const bool pieces = a.dim % 8 == 0 && a.q_ts % 8 == 0 && a.q_hs % 8 == 0 && a.page_stride % 8 == 0 &&
                        a.page_stride < (1LL << 32) && a.pages > 0 && a.table_keys > 0 &&
                        aligned16(a.q) && aligned16(a.k_cache) && aligned16(a.v_cache) && aligned16(a.out);
    if (!pieces) {
        if (!grid_fits((int64_t)a.tokens * a.heads, 64)) return hipErrorInvalidConfiguration;
        const unsigned grid = (unsigned)a.tokens * (unsigned)a.heads;
        if (f16) attn_scalar_kernel<true><<<grid, 64, 0, stream>>>(a);
        else attn_scalar_kernel<false><<<grid, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    const Launches p = plan_launches(a.tokens, a.heads, a.kv_heads, a.dim, a.table_keys, a.requests, max_new,
                                     device_cu_count());
    if (!grid_fits((p.few.items + p.many.items) * a.kv_heads, 512) || !grid_fits((p.few.tiles + p.many.tiles) * a.kv_heads, 256))
        return hipErrorInvalidConfiguration;
    if (a.dim <= 64) return f16 ? launch_dim<true, 64>(a, p, stream) : launch_dim<false, 64>(a, p, stream);
    if (a.dim <= 128) return f16 ? launch_dim<true, 128>(a, p, stream) : launch_dim<false, 128>(a, p, stream);
    return f16 ? launch_dim<true, 256>(a, p, stream) : launch_dim<false, 256>(a, p, stream);
}

}  // namespace qaff
