// How paged attention is cut into workgroups, as far as that is plain arithmetic: what a request comes
// to (the kernels' search for their work, paged_attention.hip) and how many workgroups a call launches
// (the host). Kept apart from the kernels so that the two can be checked against each other on the CPU.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qaff {

// Rows and keys of a tile: the few-rows kernel's, then the many-rows kernel's.
constexpr int kFewRows = 16, kFewKeys = 32;
constexpr int kManyRows = 128;
constexpr int many_keys(int head_dim) { return head_dim > 128 ? 32 : 64; }
constexpr int kFewMax = 32;  // requests of more rows are the many-rows kernel's where both run

// Tiles of a request's rows, for a kernel that takes requests with lo < rows <= hi.
__host__ __device__ inline int tiles_of(int rows, int tile_rows, int lo, int hi) {
    return rows > lo && rows <= hi ? (int)(((uint32_t)rows + (uint32_t)tile_rows - 1) / (uint32_t)tile_rows) : 0;
}

// Key tiles that a tile's rows see: all, or with a window that and the tokens a tile may touch.
__host__ __device__ inline int span_of(int kv, int64_t window, int table_keys, int group, int tile_rows, int tile_keys) {
    uint32_t keys = (uint32_t)kv;
    if (window > 0) {
        const uint32_t seen = (uint32_t)(window < 0x3fffffff ? window : 0x3fffffff) + (uint32_t)(tile_rows / group + 2 + tile_keys);
        keys = keys < seen ? keys : seen;
    }
    keys = keys < (uint32_t)table_keys ? keys : (uint32_t)table_keys;
    return (int)((keys + (uint32_t)tile_keys - 1) / (uint32_t)tile_keys);
}

// The most tiles times span of one of `count` requests: more, and 32 bits might not hold their sum.
__host__ __device__ inline uint32_t work_cap(int count) { return 0x7fffffffu / (uint32_t)(count > 1 ? count : 1); }

// Key tiles of a part, so that `work` (tiles times spans of all requests) makes about `parts` parts.
__host__ __device__ inline uint32_t part_length(uint32_t work, int parts, int min_part) {
    const uint32_t len = (work + (uint32_t)parts - 1) / (uint32_t)parts;
    return len > (uint32_t)min_part ? len : (uint32_t)min_part;
}

// Parts of a tile whose rows see `span` key tiles.
__host__ __device__ inline int parts_of(int span, uint32_t len) {
    const int parts = (int)(((uint32_t)span + len - 1) / len);
    return parts > 1 ? parts : 1;
}

// How a call runs: the few-rows kernel, the many-rows kernel or both, and whether their tiles are cut
// along the keys.
struct Launches {
    struct One {
        int64_t tiles = 0;  // at most so many tiles (0: not launched)
        int rows = 0, rows_lo = 0, rows_hi = 0;
        int parts = 0, min_part = 1;
        int64_t items = 0;
        size_t slots(int64_t kv_heads) const { return parts ? (size_t)(items * kv_heads * rows) : 0; }
        // Cut into about `want` parts of at least `least` tiles of `tile` keys.
        void cut(int64_t want, int least, int64_t table_keys, int tile) {
            min_part = least;
            const int64_t most = (table_keys + (int64_t)tile * least - 1) / ((int64_t)tile * least);  // parts of a tile
            if (tiles && most > 1 && want > 0) parts = (int)want;
            items = parts ? (tiles + parts < tiles * most ? tiles + parts : tiles * most) : tiles;
        }
    } few, many;
    int few_waves = 4;
};

inline Launches plan_launches(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t table_keys,
                              int64_t requests, int64_t max_new, int64_t cus) {
    Launches p;
    const int64_t group = heads / kv_heads, rows = tokens * group;
    const int64_t holders = requests + 1 < tokens ? requests + 1 : tokens;  // requests with rows
    if (max_new <= kFewMax / group || rows <= kFewMax) {
        p.few.tiles = holders + rows / kFewRows;
        p.few.rows_hi = 0x7fffffff;
    } else {
        // Of up to 4 requests with a chunk among them, the others may as well run with the chunks (one row
        // in a tile of 128, its keys cut into parts like theirs): looking for them in a kernel of their
        // own, and for their parts in a join, took 5 us where there were none.
        int64_t tails = holders;  // requests that may end inside a tile
        if (requests > 4) {
            p.few.tiles = kFewMax / kFewRows * holders;
            p.few.rows_hi = kFewMax;
            p.many.rows_lo = kFewMax;
            const int64_t large = rows / (kFewMax + 1) + 1;
            tails = holders < large ? holders : large;
        }
        p.many.tiles = rows / kManyRows + tails;
        p.many.rows_hi = 0x7fffffff;
    }
    p.few.rows = kFewRows;
    p.many.rows = kManyRows;
    // Few rows. A CU takes some 35 GB/s of keys and values whatever its waves (8 waves over 777 keys of 8
    // heads: 16 us), so only up to 256 keys (a tile a wave) does one workgroup of 8 waves take them all,
    // with nothing to join; beyond, 4 waves a workgroup and twice as many parts as workgroups fit the
    // chip, so that uneven ends are short (two rows over 120001 keys: 126 us, 152 with once as many).
    if (table_keys <= 256 && !p.many.tiles) p.few_waves = 8;
    // Beside the many-rows kernel's workgroups, which fill the chip, once is enough (two chunks and 31
    // decoding requests: 45.0 -> 42.4 us).
    const int64_t slots = (cus * 2 + kv_heads - 1) / kv_heads;  // workgroups that run at once, of a cache head
    // Many requests over long tables end unevenly: three times the slots (64 requests of up to 8192 keys: 209
    // -> 203 us, 128 of them 443 -> 439); over short tables the joins cost more (64 of up to 1500: 57 -> 60).
    const int64_t times = p.many.tiles ? 1 : p.few.tiles > slots / 2 && table_keys >= 4096 ? 3 : 2;
    p.few.cut(p.few_waves == 8 ? 0 : times * slots, 4, table_keys, kFewKeys);
    // Many rows: cut only where whole tiles would leave slots empty, into as many parts as there are slots:
    // twice as many cost more in partial sums (512 tokens over 32768: 38 MB) than even ends gain (322
    // against 309 us; over short caches 27.6 against 28.1).
    const int tile = many_keys((int)head_dim);
    p.many.cut(p.many.tiles < slots ? slots : 0, 512 / tile, table_keys, tile);
    return p;
}

}  // namespace qaff
