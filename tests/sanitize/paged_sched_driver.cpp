// The launch planning of paged attention (paged_sched.h) against the work that its kernels find: for
// calls of every kind, each request's rows belong to exactly one launched kernel, and the tiles and
// items launched are as many as the requests make, or more. Counted here request by request from the
// lengths; what a tile and a part are comes from the header, as it does in the kernels. And for prefix
// sums that are none (decreasing, overlapping, past the rows): the search stays within 32 bits, a tile
// within its request and a join within the parts that the launch has room for.
#include "paged_sched.h"

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

struct Request {
    int64_t fresh, kv;
};

struct Call {
    std::vector<Request> requests;
    int64_t padding;  // rows past the last request
    int group, kv_heads, dim, page;
    int64_t width, max_new, window;
};

static int failures = 0, calls = 0, cut_calls = 0, joins_made = 0;

// Tiles and items of one kernel's launch, as its workgroups count them.
static void count(const Call& c, const qaff::Launches::One& one, int tile_rows, int tile_keys, int64_t& tiles, int64_t& items) {
    const int table_keys = (int)(c.width * c.page);
    std::vector<int> t, span;
    uint64_t work = 0;
    bool past = false;
    for (const Request& r : c.requests) {
        t.push_back(qaff::tiles_of((int)r.fresh * c.group, tile_rows, one.rows_lo, one.rows_hi));
        span.push_back(qaff::span_of((int)r.kv, c.window, table_keys, c.group, tile_rows, tile_keys));
        const uint64_t x = (uint64_t)t.back() * (uint64_t)span.back();
        past |= x > qaff::work_cap((int)c.requests.size());
        work += x;
    }
    const bool cut = one.parts > 0 && !past;
    tiles = items = 0;
    for (size_t i = 0; i < t.size(); ++i) {
        tiles += t[i];
        items += (int64_t)t[i] * (cut ? qaff::parts_of(span[i], qaff::part_length((uint32_t)work, one.parts, one.min_part)) : 1);
    }
    const int rest = qaff::tiles_of((int)c.padding * c.group, tile_rows, one.rows_lo, one.rows_hi);
    tiles += rest;
    items += rest;
}

static void check(const Call& c) {
    int64_t tokens = c.padding;
    for (const Request& r : c.requests) tokens += r.fresh;
    if (tokens == 0) return;
    ++calls;
    const qaff::Launches p = qaff::plan_launches(tokens, (int64_t)c.group * c.kv_heads, c.kv_heads, c.dim, c.width * c.page,
                                                 (int64_t)c.requests.size(), c.max_new, 256);
    cut_calls += p.few.parts || p.many.parts;
    const char* why = nullptr;
    std::vector<Request> all = c.requests;
    all.push_back({c.padding, 0});
    for (const Request& r : all) {
        const int64_t rows = r.fresh * c.group;
        int takers = 0;
        for (const auto* one : {&p.few, &p.many}) takers += one->tiles > 0 && rows > one->rows_lo && rows <= one->rows_hi;
        if (rows > 0 && takers != 1) why = "a request that no kernel takes, or two do";
    }
    int64_t tiles = 0, items = 0;
    if (p.few.tiles) {
        count(c, p.few, qaff::kFewRows, qaff::kFewKeys, tiles, items);
        if (tiles > p.few.tiles || items > p.few.items) why = "few rows: work past the launch";
    }
    if (p.many.tiles && !why) {
        count(c, p.many, qaff::kManyRows, qaff::many_keys(c.dim), tiles, items);
        if (tiles > p.many.tiles || items > p.many.items) why = "many rows: work past the launch";
    }
    if (!why) return;
    if (++failures > 20) return;
    std::printf("%s: %lld tiles and %lld items; launched few %lld/%lld, many %lld/%lld; group %d, kv_heads %d, width %lld, "
                "max_new %lld, padding %lld, new",
                why, (long long)tiles, (long long)items, (long long)p.few.tiles, (long long)p.few.items,
                (long long)p.many.tiles, (long long)p.many.items, c.group, c.kv_heads, (long long)c.width,
                (long long)c.max_new, (long long)c.padding);
    for (const Request& r : c.requests) std::printf(" %lld", (long long)r.fresh);
    std::printf("\n");
}

static uint64_t state = 88172645463325252ull;
static int64_t random_to(int64_t n) {  // 0 .. n
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return (int64_t)(state % (uint64_t)(n + 1));
}

// A workgroup's search (find_item) for its item, or for the item of part 0 of its tile, over prefix sums
// of any kind, 64 requests at a time in 32-bit sums as the kernels take them.
static void search(const std::vector<int32_t>& cu, const std::vector<int32_t>& kv_lens, const Call& c, int tokens,
                   const qaff::Launches::One& one, int tile_rows, int tile_keys, bool by_tile, int want) {
    const int n = (int)kv_lens.size(), table_keys = (int)(c.width * c.page);
    std::vector<int> tiles(n), span(n), rows(n);
    uint32_t work = 0;
    bool past = false;
    for (int b = 0; b < n; ++b) {
        const int start = cu[b], end = cu[b + 1] < tokens ? cu[b + 1] : tokens, kv = kv_lens[b] > 0 ? kv_lens[b] : 0;
        if (start >= 0 && start < end) {
            rows[b] = (end - start) * c.group;
            tiles[b] = qaff::tiles_of(rows[b], tile_rows, one.rows_lo, one.rows_hi);
        }
        span[b] = qaff::span_of(kv, c.window, table_keys, c.group, tile_rows, tile_keys);
        const uint64_t x = (uint64_t)tiles[b] * (uint64_t)span[b], cap = qaff::work_cap(n);
        past |= x > cap;
        work += (uint32_t)(x < cap ? x : cap);
    }
    const uint32_t len = one.parts > 0 && !past ? qaff::part_length(work, one.parts, one.min_part) : 0x7fffffffu;
    int items_before = 0, tiles_before = 0;
    for (int b0 = 0; b0 < n; b0 += 64) {
        int items_in = items_before, tiles_in = tiles_before;  // the wave's sums, all of its lanes
        int at = -1, base = 0, tile_base = 0;
        for (int b = b0; b < n && b < b0 + 64; ++b) {
            const int items = tiles[b] * qaff::parts_of(span[b], len);
            if (at < 0 && (by_tile ? tiles_in + tiles[b] : items_in + items) > want) at = b, base = items_in, tile_base = tiles_in;
            items_in += items;
            tiles_in += tiles[b];
        }
        if (at >= 0) {
            const int parts = qaff::parts_of(span[at], len);
            const int local = by_tile ? want - tile_base : (want - base) / parts;
            const int first = base + local * parts, tile = tiles[at] - 1 - local;
            const bool in_rows = tile >= 0 && (int64_t)tile * tile_rows < rows[at];
            // What the join reads. However the requests overlap, the first `tiles` tiles have at most
            // tiles + work / len <= tiles + parts items, and the launch has room for those.
            const bool joins = by_tile && parts > 1;
            const bool in_room = !joins || (first >= 0 && (int64_t)first + parts <= one.items);
            joins_made += joins;
            if (!in_rows || !in_room) {
                if (++failures <= 20)
                    std::printf("search for %s %d: tile %d of %d, parts %d .. %d of %lld\n", by_tile ? "tile" : "item", want, tile,
                                tiles[at], first, first + parts, (long long)one.items);
            }
            return;
        }
        items_before = items_in;
        tiles_before = tiles_in;
    }
}

static void check_search(const std::vector<int32_t>& cu, const std::vector<int32_t>& kv_lens, const Call& c, int tokens) {
    const qaff::Launches p = qaff::plan_launches(tokens, (int64_t)c.group * c.kv_heads, c.kv_heads, c.dim, c.width * c.page,
                                                 (int64_t)kv_lens.size(), c.max_new, 256);
    auto all = [&](const qaff::Launches::One& one, int tile_rows, int tile_keys) {
        if (!one.tiles || one.items * c.kv_heads >= (1ll << 32) / 512) return;  // not launched
        for (int i = 0; i < 12; ++i) {
            search(cu, kv_lens, c, tokens, one, tile_rows, tile_keys, false, i ? (int)random_to(one.items - 1) : (int)one.items - 1);
            search(cu, kv_lens, c, tokens, one, tile_rows, tile_keys, true, i ? (int)random_to(one.tiles - 1) : (int)one.tiles - 1);
        }
    };
    all(p.few, qaff::kFewRows, qaff::kFewKeys);
    all(p.many, qaff::kManyRows, qaff::many_keys(c.dim));
}

int main() {
    // one token a request or a chunk beside them, exact and default max_new
    auto call = [](std::vector<int64_t> fresh, int64_t kv, int64_t padding, int heads, int kv_heads, bool exact, int64_t width) {
        Call c{{}, padding, heads / kv_heads, kv_heads, 128, 16, width, 0, 0};
        int64_t most = 0, sum = padding;
        for (int64_t n : fresh) {
            c.requests.push_back({n, kv > n ? kv : n});
            most = most > n ? most : n;
            sum += n;
        }
        c.max_new = exact ? most : sum;
        check(c);
    };
    for (int64_t width : {4, 125, 8192}) {
        for (int64_t kv : {1, 60, 2000, 100000}) {
            call({1, 1, 9}, kv, 0, 32, 8, true, width);
            call({1, 1, 1, 12}, kv, 0, 32, 8, true, width);
            call({1, 1, 5}, kv, 0, 64, 8, true, width);
            call({1, 1, 33}, kv, 0, 32, 32, true, width);
            call({4, 4, 4}, kv, 0, 32, 8, false, width);
            call({1, 1, 1}, kv, 0, 64, 4, false, width);
            call({1, 1, 1, 1}, kv, 0, 64, 4, false, width);
            call({1, 1, 1}, kv, 9, 32, 8, false, width);
            call({1, 9}, kv, 9, 32, 8, false, width);
        }
    }
    // every group, 1 to 8 requests and many, padding rows, short and long tables, all kinds of chunks
    const int dims[] = {64, 128, 256}, kv_heads[] = {1, 2, 8, 32}, pages[] = {8, 16, 256};
    const int64_t widths[] = {1, 3, 40, 1000, 16384};
    for (int i = 0; i < 200000; ++i) {
        Call c;
        const int64_t n = random_to(9) == 0 ? random_to(300) : random_to(8);
        const int64_t longest[] = {1, 4, 40, 300, 5000}, most = longest[random_to(4)];
        c.group = 1 + (int)random_to(39);
        c.kv_heads = kv_heads[random_to(3)];
        c.dim = dims[random_to(2)];
        c.page = pages[random_to(2)];
        c.width = widths[random_to(4)];
        c.window = random_to(3) ? 0 : 1 + random_to(4000);
        c.padding = random_to(2) ? 0 : random_to(200);
        int64_t exact = 0, sum = c.padding;
        for (int64_t b = 0; b < n; ++b) {
            const int64_t fresh = random_to(2) ? random_to(1) : random_to(most);
            const int64_t kv = random_to(20) == 0 ? 0x7fffffff : random_to(c.width * c.page);
            c.requests.push_back({fresh, kv});
            exact = exact > fresh ? exact : fresh;
            sum += fresh;
        }
        c.max_new = random_to(3) == 0 ? random_to(sum) : random_to(1) ? exact : sum;
        check(c);
    }
    // prefix sums that are none: requests that overlap, decrease, begin below 0 or end past the rows
    for (int i = 0; i < 20000; ++i) {
        Call c{{}, 0, 1 + (int)random_to(39), kv_heads[random_to(3)], dims[random_to(2)], pages[random_to(2)],
               widths[random_to(4)], 0, random_to(3) ? 0 : 1 + random_to(4000)};
        const int n = 1 + (int)(random_to(3) ? random_to(600) : random_to(5));
        const int64_t most = 0x7fffffff / ((int64_t)c.group * c.kv_heads);
        const int tokens = 1 + (int)(random_to(2) ? random_to(3000) : random_to(most - 1));
        c.max_new = random_to(1) ? random_to(tokens) : tokens;
        std::vector<int32_t> cu(n + 1), kv(n);
        for (int b = 0; b <= n; ++b)
            cu[b] = random_to(30) == 0 ? (int32_t)random_to(0xffffffffll) : b % 2 ? (int32_t)random_to(tokens) : (int32_t)random_to(tokens / 50);
        for (int b = 0; b < n; ++b)
            kv[b] = random_to(30) == 0 ? (int32_t)random_to(0xffffffffll) : (int32_t)random_to(random_to(2) ? 2000 : c.width * c.page);
        check_search(cu, kv, c, tokens);
    }
    std::printf("%d joins over prefix sums that are none\n", joins_made);
    if (joins_made < 5000) ++failures;
    std::printf("%d calls, %d of them cut along the keys, %d failures\n", calls, cut_calls, failures);
    if (failures || calls < 150000 || cut_calls < 50000) return 1;
    std::printf("all checks passed\n");
    return 0;
}
