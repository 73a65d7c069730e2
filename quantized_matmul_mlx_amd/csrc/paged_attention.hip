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
// NW waves make a workgroup of 32 NW rows: NW = 4 for chunks and prompts (keys staged once for 128
// rows), NW = 1 where a request has at most 32 rows (decode), there with the keys of a request split
// over as many workgroups as fill the chip.
//
// K and V tiles go through registers into LDS one tile ahead. LDS holds 16-byte pieces, piece c of
// row r at c ^ f(r), so that neither the row-wise reads of K nor the transposing reads of V (4 rows
// by 64 bytes for half a wave) meet in a bank.

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
    int row_end;     // rows of the request
    int start, end;  // its rows of q, as cu gives them
    int kv;
    int b;
};


// Item `want` (or the item of part 0 of tile `want`) of those that the schedule's requests make.
// Every wave scans the requests itself, 64 at a time: with up to 63 requests that is one load of
// each length and a few cross-lane sums, less than reading another kernel's schedule would cost.
// Rows past the last request are one more request without keys.
template <int ROWS, int KT>
__device__ bool find_item(const AttnArgs& a, const Sched& s, int want, bool by_tile, Item& it) {
    const int lane = threadIdx.x & 63;
    const int count = a.requests + 1;
    const int per_tile = ROWS / a.group + 2;  // tokens a tile may touch
    int start = 0, end = 0, kv = 0, tiles = 0, span = 0;
    auto load = [&](int b) {
        start = end = kv = tiles = span = 0;
        if (b < a.requests) {
            start = a.cu[b];
            end = a.cu[b + 1];
            kv = max(a.kv_lens[b], 0);
        } else if (b == a.requests) {
            start = a.cu[b];
            end = a.tokens;
        }
        if (start >= 0 && end > start && end <= a.tokens) {
            const int64_t rows = (int64_t)(end - start) * a.group;
            if (rows > s.rows_lo && rows <= s.rows_hi) tiles = (int)((rows + ROWS - 1) / ROWS);
        }
        int64_t keys = kv;
        if (a.window > 0) keys = min(keys, a.window + per_tile + KT);
        span = (int)((keys + KT - 1) / KT);
    };
    load(lane);
    int64_t len = 1LL << 40;  // key tiles a part has
    if (s.parts > 0) {
        int64_t total = (int64_t)tiles * span;
        for (int b0 = 64; b0 < count; b0 += 64) {
            load(b0 + lane);
            total += (int64_t)tiles * span;
        }
        for (int x = 32; x > 0; x >>= 1) total += __shfl_xor(total, x);
        len = max((int64_t)s.min_part, (total + s.parts - 1) / s.parts);
        if (count > 64) load(lane);
    }
    int items_before = 0, tiles_before = 0;
    for (int b0 = 0;; b0 += 64) {
        const int parts = max(1, (int)((span + len - 1) / len));
        const int items = tiles * parts;
        int items_in = items, tiles_in = tiles;
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(items_in, d), w = __shfl_up(tiles_in, d);
            if (lane >= d) items_in += u, tiles_in += w;
        }
        const int upto = by_tile ? tiles_before + tiles_in : items_before + items_in;
        const uint64_t past = __ballot(upto > want);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int base = __shfl(items_before + items_in - items, at);
            const int n = __shfl(parts, at), t = __shfl(tiles, at);
            const int local = by_tile ? want - __shfl(tiles_before + tiles_in - tiles, at) : (want - base) / n;
            it.first = base + local * n;
            it.part = by_tile ? 0 : want - it.first;
            it.parts = n;
            it.tile = t - 1 - local;  // a causal prompt's last rows see the most keys: they go first
            it.start = __shfl(start, at);
            it.end = __shfl(end, at);
            it.kv = __shfl(kv, at);
            it.row_end = (it.end - it.start) * a.group;
            it.b = b0 + at;
            return true;
        }
        items_before += __shfl(items_in, 63);
        tiles_before += __shfl(tiles_in, 63);
        if (b0 + 64 >= count) return false;
        load(b0 + 64 + lane);
    }
}

// The keys [lo, hi) that token i of the request sees.
__device__ __forceinline__ void seen_keys(const AttnArgs& a, const Item& it, int i, int& lo, int& hi) {
    const int pos = it.kv - (it.end - it.start) + i;
    hi = a.causal ? max(0, min(it.kv, pos + 1)) : it.kv;
    lo = a.window > 0 ? (int)max((int64_t)0, pos + 1 - a.window) : 0;
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
    static constexpr int kVals = 16, kDepth = 16;
};
template <> struct Shape<16> {
    typedef f32x4 acc;
    static constexpr int kVals = 4, kDepth = 32;
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

template <bool F16, int DP, int R, int NW, int KT>
__global__ __launch_bounds__(64 * NW, DP > 128 ? 1 : 2) void attn_kernel(AttnArgs a, Sched s) {
    constexpr int ROWS = R * NW, NT = 64 * NW;
    constexpr int CH = DP / 8;               // 16-byte pieces of a row
    constexpr int PER = KT * CH / NT;        // pieces of a tile per thread, RSTEP rows apart
    constexpr int RSTEP = NT / CH;
    constexpr int BUF = NW > 1 ? 2 : 1;
    constexpr int TILE = KT * DP;            // elements
    constexpr int VALS = Shape<R>::kVals;    // a lane's values of a product
    constexpr int QF = DP / Shape<R>::kDepth, SB = KT / R, PF = KT * R / 512, OB = DP / R;
    typedef typename Shape<R>::acc acc_t;
    __shared__ __align__(16) uint16_t lds[BUF][2][TILE];

    const int hk = blockIdx.x % a.kv_heads;
    const int item = blockIdx.x / a.kv_heads;
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
    const int kt_begin = kt0 + (int)((int64_t)n_all * it.part / it.parts);
    const int kt_end = kt0 + (int)((int64_t)n_all * (it.part + 1) / it.parts);
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

    // Q^T in registers: lane holds row `col`, values kDepth c + 8 part ..
    op8<F16> q[QF];
    {
        const uint16_t* src = a.q + (int64_t)(it.start + token) * a.q_ts + (int64_t)head * a.q_hs;
#pragma unroll
        for (int c = 0; c < QF; ++c) {
            const int d = Shape<R>::kDepth * c + 8 * part;
            u32x4a v = {0, 0, 0, 0};
            if (live && d < a.dim) v = *reinterpret_cast<const u32x4a*>(src + d);
            q[c] = __builtin_bit_cast(op8<F16>, v);
        }
    }

    // Staging: this thread's pieces are rows row0 + RSTEP i of a tile, piece `piece`. A key's offset in
    // its page is that of the tile's first key plus the row, or the row alone where pages are no longer
    // than tiles: (kt * KT & page_mask) + (row & page_mask), the second part fixed.
    const int row0 = tid / CH, piece = tid % CH;
    const int page_mask = (1 << a.page_shift) - 1;
    const int32_t* table = a.tables + (int64_t)it.b * a.table_width;
    const int64_t head_at = ((int64_t)hk << a.page_shift) * a.dim + piece * 8;
    const uint32_t stride = (uint32_t)a.page_stride;
    const bool whole = a.dim == DP;
    int page[PER];
    u32x4a kreg[PER], vreg[PER];
    auto load_pages = [&](int kt) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int entry = (kt * KT + row0 + RSTEP * i) >> a.page_shift;
            // the last key's entry stands for those past it
            page[i] = entry < a.table_width ? table[min(entry, (hi_all - 1) >> a.page_shift)] : -1;
        }
    };
    auto load_tile = [&](int kt) {
        const int64_t tile_at = head_at + (int64_t)((kt * KT) & page_mask) * a.dim;
        bool good = whole;
#pragma unroll
        for (int i = 0; i < PER; ++i) good &= (uint32_t)page[i] < (uint64_t)a.pages;
        if (kt * KT >= lo_all && (kt + 1) * KT <= hi_all && __all(good)) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint64_t at = (uint64_t)(uint32_t)page[i] * stride + tile_at +
                                    (uint32_t)(((row0 + RSTEP * i) & page_mask) * a.dim);
                kreg[i] = *reinterpret_cast<const u32x4a*>(a.k_cache + at);
                vreg[i] = *reinterpret_cast<const u32x4a*>(a.v_cache + at);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int row = row0 + RSTEP * i, key = kt * KT + row;
            u32x4a kv = {0, 0, 0, 0}, vv = {0, 0, 0, 0};
            if (key >= lo_all && key < hi_all) {
                if ((uint32_t)page[i] < (uint64_t)a.pages) {
                    if (piece * 8 < a.dim) {
                        const uint64_t at = (uint64_t)(uint32_t)page[i] * stride + tile_at +
                                            (uint32_t)((row & page_mask) * a.dim);
                        kv = *reinterpret_cast<const u32x4a*>(a.k_cache + at);
                        vv = *reinterpret_cast<const u32x4a*>(a.v_cache + at);
                    }
                } else {  // outside the pool: NaN scores, so the rows that see the key are NaN
                    kv = u32x4a{0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};
                }
            }
            kreg[i] = kv;
            vreg[i] = vv;
        }
    };

    acc_t acc[OB];
#pragma unroll
    for (int n = 0; n < OB; ++n)
#pragma unroll
        for (int i = 0; i < VALS; ++i) acc[n][i] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool redo = false;
    const float factor = a.scale * kLog2e;

    // A lane's reads of V: rows 32 f' + kRow e + v_row, pieces (R / 8) n + v_piece, from value v_sub on.
    const int v_row = 4 * part + ((lane & 15) >> 2);
    const int v_piece = (R == 32 ? 2 * ((lane >> 4) & 1) : 0) + ((lane & 3) >> 1);
    const int v_sub = 4 * (lane & 1);

    if (kt_begin < kt_end) {
        load_pages(kt_begin);
        load_tile(kt_begin);
        load_pages(kt_begin + 1);
    }
    for (int kt = kt_begin; kt < kt_end; ++kt) {
        uint16_t* kl = lds[BUF > 1 ? kt & 1 : 0][0];
        uint16_t* vl = lds[BUF > 1 ? kt & 1 : 0][1];
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
        if (NW > 1) __syncthreads();
        const int key0 = kt * KT;
        if (key0 >= any_hi) continue;  // keys past every row of this wave

        acc_t sc[SB];
#pragma unroll
        for (int kb = 0; kb < SB; ++kb) {
#pragma unroll
            for (int i = 0; i < VALS; ++i) sc[kb][i] = 0.f;
#pragma unroll
            for (int c = 0; c < QF; ++c) {
                const int row = kb * R + col;
                const op8<F16> kf = *reinterpret_cast<const op8<F16>*>(
                    kl + row * DP + ((((Shape<R>::kDepth / 8) * c + part) ^ swizzle_k<DP>(row)) * 8));
                sc[kb] = product<F16>(kf, q[c], sc[kb]);
            }
        }
        if (key0 < sure_lo || key0 + KT > sure_hi) {
#pragma unroll
            for (int kb = 0; kb < SB; ++kb)
#pragma unroll
                for (int i = 0; i < VALS; ++i) {
                    const int key = key0 + kb * R + (i >> 2) * 8 + 4 * part + (i & 3);
                    if (key < lo || key >= hi) sc[kb][i] = -INFINITY;
                }
        }
        float top = sc[0][0];
#pragma unroll
        for (int kb = 0; kb < SB; ++kb)
#pragma unroll
            for (int i = 0; i < VALS; ++i) top = fmaxf(top, sc[kb][i]);
        top = max_of_row<R>(top) * factor;
        if (__any(top > m + kSlack)) {
            const float m_new = fmaxf(m, top);
            const float keep = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
            l *= keep;
#pragma unroll
            for (int n = 0; n < OB; ++n)
#pragma unroll
                for (int i = 0; i < VALS; ++i) acc[n][i] *= keep;
            m = m_new;
        }
        const float base = m == -INFINITY ? 0.f : m - kLift<F16>;
#pragma unroll
        for (int kb = 0; kb < SB; ++kb)
#pragma unroll
            for (int i = 0; i < VALS; ++i) {
                sc[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[kb][i], factor, -base));
                l += sc[kb][i];
            }
        // rounded to 16 bits for the product with V; their sum l is taken before the rounding
        op8<F16> p[PF];
#pragma unroll
        for (int f = 0; f < PF; ++f) {
            float x[8];  // of one block of scores (two to a block), or of two blocks (R = 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = R == 32 ? sc[f / 2][8 * (f % 2) + i] : sc[2 * f + i / 4][i % 4];
            p[f] = __builtin_bit_cast(op8<F16>, u32x4a{pack_half2<F16>(x[0], x[1]), pack_half2<F16>(x[2], x[3]),
                                                       pack_half2<F16>(x[4], x[5]), pack_half2<F16>(x[6], x[7])});
        }
        // A weight of zero times an infinite or NaN value is NaN: where the tile holds keys that some
        // row does not see, look for such values.
        if (key0 < sure_lo || min(key0 + KT, hi_all) > sure_hi) {
#pragma unroll 1
            for (int x = lane; x < TILE / 8; x += 64) {
                const u32x4a w = *reinterpret_cast<const u32x4a*>(vl + x * 8);
                redo |= not_finite2<F16>(w.x) || not_finite2<F16>(w.y) || not_finite2<F16>(w.z) || not_finite2<F16>(w.w);
            }
        }
#pragma unroll
        for (int n = 0; n < OB; ++n) {
            const int at = ((v_piece + (R / 8) * n) ^ swizzle_v<DP, R>(v_row)) * 8 + v_sub;
#pragma unroll
            for (int f = 0; f < PF; ++f) {
                uint16_t* src = vl + (v_row + (R == 32 ? 16 : 32) * f) * DP + at;
                const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)src);
                const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + (R == 32 ? 8 : 16) * DP));
                const u32x2 w0 = __builtin_bit_cast(u32x2, v0), w1 = __builtin_bit_cast(u32x2, v1);
                acc[n] = product<F16>(__builtin_bit_cast(op8<F16>, u32x4a{w0.x, w0.y, w1.x, w1.y}), p[f], acc[n]);
            }
        }
    }

    if (__any(redo)) {  // this wave's rows again, one by one, each over the keys that it sees alone
#pragma unroll 1
        for (int x = wave * R; x < min(wave * R + R, rows); ++x) {
            const int i = (r0 + x) / a.group, h = hk * a.group + (r0 + x) - i * a.group;
            int from, to;
            seen_keys(a, it, i, from, to);
            float mx, lx, o[4];
            scalar_row<F16>(a, it.b, it.start + i, h, max(from, kt_begin * KT), min(to, kt_end * KT), mx, lx, o);
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
        return;
    }
    l = sum_of_row<R>(l);
    if (!live) return;
    const float m_out = m - kLift<F16>;
    if (it.parts > 1) {
        const int64_t slot = ((int64_t)item * a.kv_heads + hk) * ROWS + r;
        float* o = s.part_o + slot * a.dim;
#pragma unroll
        for (int n = 0; n < OB; ++n)
#pragma unroll
            for (int i = 0; i < VALS / 4; ++i) {
                const int d = R * n + 8 * i + 4 * part;
                if (d < a.dim)
                    *reinterpret_cast<f32x4*>(o + d) =
                        f32x4{acc[n][4 * i], acc[n][4 * i + 1], acc[n][4 * i + 2], acc[n][4 * i + 3]};
            }
        if (part == 0) s.part_ml[slot] = make_float2(m_out, l);
        return;
    }
    const bool empty = hi <= lo;
    const float inv = empty ? 0.f : 1.f / l;
    const int64_t row = (int64_t)(it.start + token) * a.heads + head;
    uint16_t* o = a.out + row * a.dim;
#pragma unroll
    for (int n = 0; n < OB; ++n)
#pragma unroll
        for (int i = 0; i < VALS / 4; ++i) {
            const int d = R * n + 8 * i + 4 * part;
            if (d < a.dim)
                *reinterpret_cast<uint2*>(o + d) = make_uint2(pack_half2<F16>(acc[n][4 * i] * inv, acc[n][4 * i + 1] * inv),
                                                              pack_half2<F16>(acc[n][4 * i + 2] * inv, acc[n][4 * i + 3] * inv));
        }
    if (a.lse && part == 0) a.lse[row] = empty ? -INFINITY : (m_out + __builtin_amdgcn_logf(l)) * kLn2;
}

// Joins the parts of a tile's rows, in their order: o = sum_s w_s o_s / sum_s w_s l_s with
// w_s = 2^(m_s - max m). A workgroup holds RP rows, DP / 4 threads each; the threads left over take
// other parts of the same rows, up to kJoin parts at a time.
constexpr int kJoin = 512;
template <bool F16, int DP, int ROWS, int KT, int RP>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, Sched s) {
    constexpr int LANES = DP / 4, GROUPS = 256 / LANES / RP;
    static_assert(GROUPS >= 1 && (RP == 1 || GROUPS == 1), "");
    __shared__ f32x4 so[GROUPS][LANES];
    __shared__ float weight[RP][kJoin / RP];
    const int hk = blockIdx.x % a.kv_heads;
    Item it;
    if (!find_item<ROWS, KT>(a, s, blockIdx.x / a.kv_heads, true, it) || it.parts == 1) return;
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
                if (lane_of_row < 64) weight[rp][p] = w;
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
                    o += weight[rp][p] * *reinterpret_cast<const f32x4*>(src + p * step * a.dim);
            }
        }
        if (GROUPS > 1) {
            __syncthreads();
            so[g][x] = o;
            __syncthreads();
            if (g == 0)
                for (int p = 1; p < GROUPS; ++p) o += so[p][x];
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

// How a call runs: the few-rows kernel (16-row tiles), the many-rows kernel (tiles of kManyRows) or
// both, and whether their tiles are cut along the keys.
constexpr int kManyWaves = 4, kManyRows = 32 * kManyWaves;
constexpr int kFewMax = 32;  // requests of more rows are the many-rows kernel's
constexpr int kFewPart = 2, kManyPart = 8;

struct Launches {
    struct One {
        int64_t tiles = 0;  // at most so many tiles (0: not launched)
        int rows = 0, rows_lo = 0, rows_hi = 0;
        int parts = 0;
        int64_t items() const { return tiles + parts; }
        size_t slots(int64_t kv_heads) const { return parts ? (size_t)(items() * kv_heads * rows) : 0; }
    } few, many;
};

Launches plan_launches(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t table_keys, int64_t requests,
                       int64_t max_new) {
    Launches p;
    const int64_t group = heads / kv_heads, rows = tokens * group, cus = device_cu_count();
    const int64_t holders = requests + 1 < tokens ? requests + 1 : tokens;  // requests with rows
    if (max_new <= kFewMax / group || rows <= kFewMax) {
        p.few.tiles = holders + rows / 16;
        p.few.rows_hi = 0x7fffffff;
    } else {
        if (requests > 1) {
            p.few.tiles = 2 * holders;
            p.few.rows_hi = kFewMax;
            p.many.rows_lo = kFewMax;
        }
        const int64_t large = rows / (kFewMax + 1) + 1;
        p.many.tiles = rows / kManyRows + (holders < large ? holders : large);
        p.many.rows_hi = 0x7fffffff;
    }
    p.few.rows = 16;
    p.many.rows = kManyRows;
    // Cut where whole tiles would leave workgroup slots empty: 8 waves of the few-rows kernel fit a
    // CU, 2 workgroups of the other. Twice as many parts, so that uneven ends are short.
    if (p.few.tiles && table_keys > 32 * kFewPart) p.few.parts = (int)((cus * 16 + kv_heads - 1) / kv_heads);
    const int64_t slots = (cus * 2 + kv_heads - 1) / kv_heads;
    if (p.many.tiles && p.many.tiles < slots && table_keys > 64 * kManyPart) p.many.parts = (int)(2 * slots);
    return p;
}

template <bool F16, int DP>
hipError_t launch_tiles(const AttnArgs& a, const Launches& p, hipStream_t stream) {
    constexpr int KT = DP > 128 ? 32 : 64;
    const size_t few_slots = p.few.slots(a.kv_heads), many_slots = p.many.slots(a.kv_heads);
    float* o = a.partial;
    float2* ml = reinterpret_cast<float2*>(o + (few_slots + many_slots) * a.dim);
    const Sched few{p.few.rows_lo, p.few.rows_hi, p.few.parts, kFewPart, o, ml};
    const Sched many{p.many.rows_lo, p.many.rows_hi, p.many.parts, kManyPart * 64 / KT, o + few_slots * a.dim,
                     ml + few_slots};
    if (p.many.tiles)
        attn_kernel<F16, DP, 32, kManyWaves, KT>
            <<<(unsigned)(p.many.items() * a.kv_heads), 64 * kManyWaves, 0, stream>>>(a, many);
    if (p.few.tiles) attn_kernel<F16, DP, 16, 1, 32><<<(unsigned)(p.few.items() * a.kv_heads), 64, 0, stream>>>(a, few);
    if (p.many.parts)
        join_kernel<F16, DP, kManyRows, KT, 1024 / DP>
            <<<dim3((unsigned)(p.many.tiles * a.kv_heads), kManyRows / (1024 / DP)), 256, 0, stream>>>(a, many);
    if (p.few.parts)
        join_kernel<F16, DP, 16, 32, 1>
            <<<dim3((unsigned)(p.few.tiles * a.kv_heads), a.group < 16 ? a.group : 16), 256, 0, stream>>>(a, few);
    return hipGetLastError();
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

size_t paged_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t table_keys,
                                 int64_t requests, int64_t max_new) {
    const Launches p = plan_launches(tokens, heads, kv_heads, table_keys, requests, max_new);
    return (p.few.slots(kv_heads) + p.many.slots(kv_heads)) * (size_t)(4 * head_dim + 8);
}

hipError_t launch_paged_attention(const AttnArgs& a, bool f16, int64_t max_new, hipStream_t stream) {
    // 16-byte loads of every row, and heads of whole 16-byte pieces (pages apart by a 32-bit count)
    const bool pieces = a.dim % 8 == 0 && a.q_ts % 8 == 0 && a.q_hs % 8 == 0 && a.page_stride % 8 == 0 &&
                        a.page_stride < (1LL << 32) &&
                        aligned16(a.q) && aligned16(a.k_cache) && aligned16(a.v_cache) && aligned16(a.out);
    if (!pieces) {
        const unsigned grid = (unsigned)a.tokens * (unsigned)a.heads;
        if (f16) attn_scalar_kernel<true><<<grid, 64, 0, stream>>>(a);
        else attn_scalar_kernel<false><<<grid, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    const Launches p = plan_launches(a.tokens, a.heads, a.kv_heads, a.table_width << a.page_shift, a.requests, max_new);
    if (a.dim <= 64) return f16 ? launch_tiles<true, 64>(a, p, stream) : launch_tiles<false, 64>(a, p, stream);
    if (a.dim <= 128) return f16 ? launch_tiles<true, 128>(a, p, stream) : launch_tiles<false, 128>(a, p, stream);
    return f16 ? launch_tiles<true, 256>(a, p, stream) : launch_tiles<false, 256>(a, p, stream);
}

}  // namespace qaff
