// The paged cache's host code (host_pages.cpp) on the CPU: the driver's calls and the kernels are
// stood in for here, the "device" buffer is host memory.  Table edits are applied to it; an
// attention call's plan is walked with the kernels' own functions (pages_runs.cuh) instead of being run.
//
//   host_pages_main plan SEED N     plans of N random sessions cover every query's keys exactly once
//   host_pages_main mixed           plans of calls that mix few and many query rows
//   host_pages_main share           which groups read their common pages once
//   host_pages_main failures        calls that change the tables, with every allocation and launch failing in turn
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <new>
#include <random>
#include <string>

#include "host_pages.cpp"

using std::max;
using std::min;
#include "pages_runs.cuh"

// ---------------------------------------------------------------- stand-ins
static char g_error[512];

// Allocations of a library call and launches that succeed until one fails (-1: none fails), and the launches made.
static int g_good_allocations = -1, g_allocations = -1, g_good_launches = -1, g_made = 0;
struct Armed {                                            // allocations count while one of these lives
    Armed() { g_allocations = g_good_allocations; }
    ~Armed() {
        g_good_allocations = g_allocations;
        g_allocations = -1;
    }
};
__attribute__((noinline)) void *operator new(size_t n) {
    if (g_allocations >= 0 && g_allocations-- == 0) throw std::bad_alloc();
    void *p = std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
__attribute__((noinline)) void operator delete(void *p) noexcept { std::free(p); }
__attribute__((noinline)) void operator delete(void *p, size_t) noexcept { std::free(p); }
static cudaError_t launched() {
    if (g_good_launches >= 0 && g_good_launches-- == 0) return cudaErrorLaunchOutOfResources;
    ++g_made;
    return cudaSuccess;
}

#define REQUIRE(x, ...)                                                        \
    do {                                                                       \
        if (!(x)) {                                                            \
            std::printf("%s:%d: %s ", __FILE__, __LINE__, #x);                 \
            std::printf(" " __VA_ARGS__);                                      \
            std::printf("  [last error: %s]\n", g_error);              \
            std::exit(1);                                                      \
        }                                                                      \
    } while (0)

namespace sdv2 {
sdv2_status fail(sdv2_status st, const char *fmt, ...) {
    char text[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    std::snprintf(g_error, sizeof(g_error), "%s", text);
    return st;
}
sdv2_status cuda_fail(cudaError_t, const char *what) { return fail(SDV2_E_CUDA, "%s", what); }
sdv2_status check_device(int) { return SDV2_OK; }
void count_launch() {}
static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                       const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() { return encode; }
}  // namespace sdv2

static int g_sms = 148;
static bool g_idle = false;                               // nothing that a user's streams do is pending

extern "C" {
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { return *v = g_sms, cudaSuccess; }
cudaError_t cudaMemset(void *p, int value, size_t n) {
    REQUIRE(g_idle, "memory is cleared with work pending");
    if (value != 0) std::memset(p, value, n);            // (the buffer is fresh zeros)
    return cudaSuccess;
}
cudaError_t cudaMemcpy(void *to, const void *from, size_t n, cudaMemcpyKind) { return std::memcpy(to, from, n), cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return g_idle = true, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return "error"; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) {
    return *s = cudaStreamCaptureStatusNone, cudaSuccess;
}
}

// The launches of the last attention call.
enum class Kernel { tiles, rows };
struct Launch {
    Kernel kernel;
    PageWork work;
    bool beside;
};
static std::vector<Launch> g_launches;
static bool g_merged;
using SmallParams = PagesAttnParams<kSmallSections, kSmallMembers>;
using LargeParams = PagesAttnParams<kLargeSections, kLargeMembers>;
static SmallParams g_small;
static LargeParams g_large;
static bool g_is_small;
static void keep(const SmallParams &p) { g_small = p, g_is_small = true; }
static void keep(const LargeParams &p) { g_large = p, g_is_small = false; }

namespace sdv2 {
template <int kE, int kR>
cudaError_t launch_page_edits(const PageEdits<kE, kR> &e, bool, cudaStream_t) {
    const cudaError_t err = launched();
    if (err != cudaSuccess) return err;
    for (int c = 0; c < e.n_copies; ++c)
        std::copy(e.table + static_cast<int64_t>(e.copy[c][0]) * e.width,
                  e.table + static_cast<int64_t>(e.copy[c][0]) * e.width + e.copy[c][2],
                  e.table + static_cast<int64_t>(e.copy[c][1]) * e.width);
    for (int c = 0; c < e.n_clears; ++c) {
        int32_t *row = e.table + static_cast<int64_t>(e.clear[c][0]) * e.width;
        std::fill(row, row + e.clear[c][1], -1);
    }
    for (int i = 0; i < e.n_entries; ++i) e.table[e.entry_at[i]] = e.entry[i];
    for (int i = 0; i < e.n_lengths; ++i) e.lengths[e.length[i][0]] = e.length[i][1];
    *e.version = e.new_version;
    return cudaSuccess;
}
template <int kM>
cudaError_t launch_page_moves(const PageMoves<kM> &m, cudaStream_t) {
    const cudaError_t err = launched();
    if (err != cudaSuccess) return err;
    for (int i = 0; i < m.n; ++i)
        for (int j = m.first[i]; j < m.first[i + 1]; ++j)
            for (int side = 0; side < 2; ++side)
                for (int layer = 0; layer < m.layers; ++layer) {
                    uint8_t *base = m.base[side] + layer * m.layer_stride;
                    std::memcpy(base + m.dst[j] * m.page_bytes, base + m.src[i] * m.page_bytes, m.page_bytes);
                }
    return cudaSuccess;
}
cudaError_t launch_page_write(const PageWriteParams &, cudaStream_t) { return launched(); }
template <int kS, int kM>
cudaError_t launch_pages_tiles(const PagesAttnParams<kS, kM> &p, const PageWork &w, const CUtensorMap &,
                               const CUtensorMap &, bool, cudaStream_t) {
    keep(p);
    g_launches.push_back({Kernel::tiles, w, false});
    return cudaSuccess;
}
template <int kS, int kM>
cudaError_t launch_pages_rows(const PagesAttnParams<kS, kM> &p, const PageWork &w, bool, bool beside, int, cudaStream_t) {
    keep(p);
    g_launches.push_back({Kernel::rows, w, beside});
    return cudaSuccess;
}
template <int kS, int kM>
cudaError_t launch_pages_merge(const PagesAttnParams<kS, kM> &, int, bool, cudaStream_t) {
    g_merged = true;
    return cudaSuccess;
}
}  // namespace sdv2

// ---------------------------------------------------------------- a pool on host memory
struct Pool {
    sdv2_pages_config c{};
    sdv2_pages *h = nullptr;
    void *memory = nullptr;
    explicit Pool(const sdv2_pages_config &cfg) : c(cfg) {
        const size_t bytes = sdv2_pages_bytes(&c);
        REQUIRE(bytes > 0);
        memory = std::calloc(bytes + 256, 1);
        REQUIRE(memory);
        g_idle = false;
        void *base = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(memory) + 255) & ~uintptr_t(255));
        REQUIRE(sdv2_pages_create(&c, base, bytes, &h) == SDV2_OK);
    }
    ~Pool() {
        sdv2_pages_destroy(h);
        std::free(memory);
    }
    Pool(const Pool &) = delete;
    sdv2_status extend(const std::vector<int32_t> &counts) {
        Armed armed;
        return sdv2_pages_extend(h, counts.data(), nullptr);
    }
    sdv2_status fork(int32_t src, const std::vector<int32_t> &dst, bool deep = false) {
        Armed armed;
        return sdv2_pages_fork(h, src, dst.data(), static_cast<int32_t>(dst.size()), deep, nullptr);
    }
    sdv2_status free(const std::vector<int32_t> &s) {
        Armed armed;
        return sdv2_pages_free(h, s.data(), static_cast<int32_t>(s.size()), nullptr);
    }
    sdv2_status compact() {
        Armed armed;
        return sdv2_pages_compact(h, nullptr, nullptr);
    }
    sdv2_status attend(const std::vector<int32_t> &counts) {
        g_launches.clear();
        g_merged = false;
        static uint16_t io[8];
        void *aligned = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(io) + 15) & ~uintptr_t(15));
        return sdv2_pages_attention(h, 0, aligned, aligned, 0, 0, counts.data(), 0.125f, nullptr);
    }
    // The device's tables say what the host's books say, and those agree with one another.
    void check_books() const {
        const int32_t *table = reinterpret_cast<int32_t *>(h->base + h->r.table);
        const int32_t *lengths = reinterpret_cast<int32_t *>(h->base + h->r.length);
        REQUIRE(*reinterpret_cast<uint32_t *>(h->base + h->r.version) == h->version);
        std::vector<int32_t> users(c.pages, 0);
        int32_t used = 0;
        for (int32_t b = 0; b < c.streams; ++b) {
            REQUIRE(lengths[b] == h->tokens[b], "stream %d: %d on the device, %d here", b, lengths[b], h->tokens[b]);
            REQUIRE(h->n_pages[b] == h->pages_of(h->tokens[b]));
            for (int32_t i = 0; i < c.stream_pages; ++i) {
                const int32_t p = h->row(b)[i];
                REQUIRE(table[static_cast<int64_t>(b) * c.stream_pages + i] == p, "stream %d page %d", b, i);
                REQUIRE((p >= 0) == (i < h->n_pages[b]) && p < c.pages);
                if (p >= 0 && users[p]++ == 0) ++used;
            }
        }
        REQUIRE(users == h->users && used == h->used);
        for (int32_t p = 0; p < h->first_free; ++p) REQUIRE(users[p] > 0);
    }
};

// ---------------------------------------------------------------- a plan, walked
using Range = std::pair<int32_t, int32_t>;

// Every (query token, head) gets each key that it sees exactly once, over the parts that the
// launches leave and the merge reads; nothing is written twice; every bound holds.
template <typename P>
static void walk(const P &p, const Pool &pool, const std::vector<int32_t> &counts) {
    const sdv2_pages_config &c = pool.c;
    const int32_t rows_out = p.n_queries * p.heads;
    std::map<int64_t, Range> parts;                       // by partial row
    std::vector<Range> out(rows_out, {-1, -1});           // written whole
    for (const Launch &launch : g_launches) {
        const PageWork &w = launch.work;
        const bool rows_kernel = launch.kernel == Kernel::rows;
        REQUIRE(w.tile_log2 == (rows_kernel ? 4 : 7), "a plan in tiles of %d keys for the %s kernel", 1 << w.tile_log2,
                rows_kernel ? "row" : "tile");
        REQUIRE(w.places > 0 && w.workers > 0 && (static_cast<uint64_t>(w.places) + 1) * w.workers <= 0xffffffffull);
        REQUIRE(w.workers <= (rows_kernel ? g_sms * kRowWarps : g_sms));
        REQUIRE(w.tile_tokens * p.group <= (rows_kernel ? kRowsPerWorker : 128) && w.tile_tokens >= 1);
        REQUIRE(!rows_kernel || w.rows <= kRowsPerWorker);
        REQUIRE(w.cut_row + static_cast<int64_t>(w.workers) * w.cut_rows <= pool.h->r.rows);
        for (int worker = 0; worker < w.workers; ++worker) {
            int pos = static_cast<int>(first_place(w, worker));
            const int end = static_cast<int>(first_place(w, worker + 1));
            RunSpot spot;
            while (next_spot(p, w, &pos, end, &spot)) {
                const PagesRun r = run_at(p, w, worker, spot);
                const PageSection &s = p.section[r.sec];
                REQUIRE(r.sec >= w.begin && r.sec < w.end && r.head >= 0 && r.head < c.kv_heads);
                REQUIRE(r.n_rows > 0 && r.n_rows <= w.cut_rows && r.n_rows <= w.tile_tokens * p.group);
                REQUIRE(!rows_kernel || r.row_tile == 0);
                REQUIRE(r.begin >= 0 && r.n >= 0 && r.keys > 0);
                if (r.n > 0) REQUIRE(((r.begin + r.n - 1) << w.tile_log2) < r.keys, "tiles past the keys");
                for (int row = 0; row < r.n_rows; ++row) {
                    const int place = r.row_tile * w.tile_tokens + row / p.group;
                    REQUIRE(place < s.n_tokens);
                    const int token = query_token(p, s, place), head = r.head * p.group + row % p.group;
                    REQUIRE(token >= 0 && token < p.n_queries);
                    int seen = r.keys;
                    if (!r.common) seen = min(r.len, ((r.len - s.n_tokens + place) / p.block + 1) * p.block) - r.base;
                    const Range range(r.base + (r.begin << w.tile_log2),
                                      max(r.base + (r.begin << w.tile_log2), r.base + min((r.begin + r.n) << w.tile_log2, seen)));
                    if (r.whole && !r.common && s.common < 0) {
                        Range &o = out[token * p.heads + head];
                        REQUIRE(o.first < 0, "a row is written twice");
                        o = range;
                    } else {
                        const int64_t at = partial_row(p, w, r, worker, row, static_cast<int64_t>(token) * p.heads + head);
                        REQUIRE(at >= 0 && at < pool.h->r.rows);
                        REQUIRE(parts.emplace(at, range).second, "a partial row is written twice");
                    }
                }
            }
        }
    }
    // the streams' queries in order
    int32_t token = 0;
    size_t read = 0;
    for (int32_t b = 0; b < c.streams; ++b)
        for (int32_t i = 0; i < counts[b]; ++i, ++token) {
            const int32_t len = pool.h->tokens[b], at = len - counts[b] + i;
            const int32_t seen = min(len, (at / p.block + 1) * p.block);
            for (int32_t head = 0; head < c.heads; ++head) {
                const int32_t row = token * c.heads + head;
                std::vector<Range> got;
                if (out[row].first >= 0) got.push_back(out[row]);
                if (g_merged) {                           // (the merge kernel's way to its parts)
                    int own = p.n_common;
                    while (own + 1 < p.n_sections && p.section[own + 1].token0 <= token) ++own;
                    const int common = p.section[own].common;
                    std::vector<int64_t> from;
                    for (int k = 0; k < 2; ++k) {
                        if (k == 1 && common < 0) continue;
                        const PageWork &w = k ? p.common : p.own;
                        const PageSection &s = p.section[k ? common : own];
                        const int place = k ? p.section[own].common_token + token - p.section[own].token0 : token - s.token0;
                        const int rt = place / w.tile_tokens;
                        const uint32_t a = p.start[k ? common : own] +
                                           (rt * p.v.kv_heads + head / p.group) * (s.tiles + w.setup) + w.setup;
                        const int first = worker_of(w, a), n = worker_of(w, a + s.tiles - 1) - first + 1;
                        for (int piece = 0; piece < n; ++piece)
                            from.push_back(piece == 0 ? (k ? p.rows_common : 0) + static_cast<int64_t>(row)
                                                      : w.cut_row + static_cast<int64_t>(first + piece) * w.cut_rows +
                                                            (place - rt * w.tile_tokens) * p.group + head % p.group);
                    }
                    REQUIRE((out[row].first >= 0) == (from.size() == 1));
                    if (from.size() > 1)
                        for (int64_t x : from) {
                            const auto it = parts.find(x);
                            REQUIRE(it != parts.end(), "the merge reads a part that nobody writes");
                            got.push_back(it->second);
                            ++read;
                        }
                }
                std::sort(got.begin(), got.end());
                int32_t upto = 0;
                for (const Range &x : got) {
                    if (x.first == x.second) continue;
                    REQUIRE(x.first == upto, "stream %d token %d head %d: keys from %d on, had %d", b, at, head, x.first, upto);
                    upto = x.second;
                }
                REQUIRE(upto == seen, "stream %d token %d head %d: %d keys of %d", b, at, head, upto, seen);
            }
        }
    REQUIRE(read == parts.size(), "%zu parts written, %zu read", parts.size(), read);
}

static void check_plan(const Pool &pool, const std::vector<int32_t> &counts) {
    if (g_is_small)
        walk(g_small, pool, counts);
    else
        walk(g_large, pool, counts);
}

static sdv2_pages_config config(int32_t streams, int32_t heads, int32_t kv_heads, int32_t page, int32_t pages, int32_t queries,
                                int32_t block = 1) {
    sdv2_pages_config c{};
    c.streams = streams, c.layers = 1, c.heads = heads, c.kv_heads = kv_heads, c.head_dim = 64, c.page_tokens = page;
    c.pages = pages, c.stream_pages = pages, c.max_queries = queries, c.block_tokens = block;
    return c;
}

// ---------------------------------------------------------------- calls of few and many rows
static void mixed() {
    for (const int mode : {SDV2_SHARE_AUTO, SDV2_SHARE_ALWAYS})
        for (const int32_t alone : {0, 1, 17, 64, 300})                // queries of the stream outside the group
            for (const int32_t each : {1, 2, 3, 20})                   // of the group's members
                for (const int32_t prefix : {64, 4096, 9000}) {
                    sdv2_pages_config c = config(9, 12, 12, 64, 400, 1000);
                    c.head_dim = 128;
                    Pool pool(c);
                    REQUIRE(sdv2_pages_share(pool.h, mode) == SDV2_OK);
                    std::vector<int32_t> grow(9, 0);
                    grow[0] = prefix, grow[8] = 400;
                    REQUIRE(pool.extend(grow) == SDV2_OK);
                    REQUIRE(pool.fork(0, {1, 2, 3, 4, 5, 6, 7}) == SDV2_OK);
                    std::vector<int32_t> counts(9, each);
                    counts[8] = 0;
                    REQUIRE(pool.extend(counts) == SDV2_OK);
                    counts[8] = alone;
                    REQUIRE(pool.attend(counts) == SDV2_OK);
                    check_plan(pool, counts);
                    if (mode == SDV2_SHARE_ALWAYS) {                   // one query head to a key head
                        const bool few_own = max(each, alone) <= 16, few_common = 8 * each <= 16;
                        REQUIRE(g_merged && g_launches.size() == (few_own && !few_common ? 2u : 1u));
                        REQUIRE((g_launches[0].kernel == Kernel::rows) == (few_own && few_common) && !g_launches[0].beside);
                        REQUIRE((g_launches.back().kernel == Kernel::rows) == few_own);
                        REQUIRE(g_launches.size() == 1 || g_launches[1].beside);
                    }
                    REQUIRE(pool.extend(std::vector<int32_t>(9, 30)) == SDV2_OK);      // a replay after growth
                    check_plan(pool, counts);
                }
}

// ---------------------------------------------------------------- the sharing rule
// Whether `members` streams with `each` queries read their `pages` common pages of 16 KB (a layer's keys
// and values) once.  `idle` more members have no queries.
static bool shares(int mode, int32_t members, int32_t each, int32_t pages, int32_t idle = 0) {
    const int32_t n = members + idle;
    Pool pool(config(n, 4, 4, 16, pages + n * (each / 16 + 2), n * each));
    REQUIRE(sdv2_pages_share(pool.h, mode) == SDV2_OK);
    std::vector<int32_t> first(n, 0), counts(n, each), others;
    first[0] = pages * 16;
    for (int32_t b = 1; b < n; ++b) others.push_back(b);
    REQUIRE(pool.extend(first) == SDV2_OK && pool.fork(0, others) == SDV2_OK && pool.extend(counts) == SDV2_OK);
    std::fill(counts.begin() + members, counts.end(), 0);
    REQUIRE(pool.attend(counts) == SDV2_OK);
    REQUIRE(g_is_small && g_small.n_common <= 1);
    check_plan(pool, counts);
    if (g_small.n_common == 1) REQUIRE(g_small.section[0].keys == pages * 16);
    return g_small.n_common == 1;
}

static void share() {
    const int never = SDV2_SHARE_NEVER, automatic = SDV2_SHARE_AUTO, always = SDV2_SHARE_ALWAYS;
    REQUIRE(shares(always, 2, 1, 1) && shares(always, 2, 40, 1) && !shares(always, 1, 1, 5000, 3));
    REQUIRE(!shares(never, 8, 1, 5000) && !shares(never, 8, 40, 5000));
    // at most 16 rows: from five members on, where 24 MB are read less
    REQUIRE(shares(automatic, 5, 1, 384) && !shares(automatic, 5, 1, 383));
    REQUIRE(shares(automatic, 5, 3, 384) && !shares(automatic, 5, 3, 383));
    REQUIRE(shares(automatic, 16, 1, 103) && !shares(automatic, 16, 1, 102));
    REQUIRE(shares(automatic, 5, 1, 384, 7) && !shares(automatic, 5, 1, 383, 7));       // (idle members save nothing)
    // more rows: where 30 MB and 4 for every member are
    REQUIRE(shares(automatic, 5, 4, 800) && !shares(automatic, 5, 4, 799));
    REQUIRE(shares(automatic, 17, 1, 392) && !shares(automatic, 17, 1, 391));
    REQUIRE(shares(automatic, 2, 9, 2432) && !shares(automatic, 2, 9, 2431));
    // over 64 MB in any case
    REQUIRE(shares(automatic, 4, 1, 4097) && !shares(automatic, 4, 1, 4096));
    REQUIRE(shares(automatic, 2, 8, 4097) && !shares(automatic, 2, 8, 4096));
}

// ---------------------------------------------------------------- random sessions
static void sessions(uint64_t seed, int n) {
    std::mt19937_64 rng(seed);
    auto pick = [&](int64_t lo, int64_t hi) { return static_cast<int32_t>(lo + static_cast<int64_t>(rng() % (hi - lo + 1))); };
    const int32_t heads[][2] = {{1, 1}, {4, 2}, {6, 3}, {10, 2}, {8, 1}, {16, 2}, {12, 12}, {40, 8}, {128, 1}};
    for (int k = 0; k < n; ++k) {
        const int32_t *hh = heads[pick(0, 8)];
        const int32_t streams = pick(0, 4) == 0 ? pick(30, 80) : pick(1, 12), page = 16 << pick(0, 3);
        const int32_t pages = pick(0, 1) ? 3000 : 600;
        g_sms = pick(0, 3) == 0 ? pick(1, 160) : 148;
        Pool pool(config(streams, hh[0], hh[1], page, pages, 2000, pick(0, 2) ? 1 : pick(2, 200)));
        REQUIRE(sdv2_pages_share(pool.h, pick(0, 2)) == SDV2_OK);
        for (int step = 0; step < 12; ++step) {
            const int what = pick(0, 9);
            if (what < 4) {
                std::vector<int32_t> counts(streams, 0);
                for (int32_t &x : counts) x = pick(0, 2) ? 0 : (pick(0, 5) ? pick(1, 3 * page) : pick(1, page * pages / streams));
                const sdv2_status st = pool.extend(counts);
                REQUIRE(st == SDV2_OK || st == SDV2_E_STATE);
            } else if (what < 7 && streams > 1) {
                std::vector<int32_t> dst;
                const int32_t src = pick(0, streams - 1);
                for (int32_t b = 0; b < streams; ++b)
                    if (b != src && pool.h->tokens[b] == 0 && pick(0, 1)) dst.push_back(b);
                const sdv2_status st = pool.fork(src, dst, pick(0, 7) == 0);
                REQUIRE(st == SDV2_OK || st == SDV2_E_STATE);
            } else if (what < 8) {
                REQUIRE(pool.free({pick(0, streams - 1)}) == SDV2_OK);
            } else if (what < 9) {
                REQUIRE(pool.compact() == SDV2_OK);
            }
            pool.check_books();
            // queries of every stream alike, or different numbers, or few streams
            const int kind = pick(0, 3), most = pick(0, 2) == 0 ? 200 : (pick(0, 1) ? 20 : 3);
            std::vector<int32_t> counts(streams, 0);
            int32_t sum = 0;
            for (int32_t b = 0; b < streams; ++b) {
                const int32_t want = kind == 0 ? most : (kind == 1 ? pick(0, 1) : (pick(0, 3) ? pick(0, 2) : pick(1, most)));
                counts[b] = min(min(want, pool.h->tokens[b]), 2000 - sum);
                sum += counts[b];
            }
            if (sum == 0) continue;
            REQUIRE(pool.attend(counts) == SDV2_OK);
            check_plan(pool, counts);
            if (pick(0, 2) == 0) {                        // a replay after the streams have grown
                std::vector<int32_t> grow(streams, 0);
                for (int32_t &x : grow) x = pick(0, 40);
                if (pool.extend(grow) == SDV2_OK) check_plan(pool, counts);
            }
        }
    }
}

// ---------------------------------------------------------------- failures
// What a user of the pool can tell of it: tables, lengths, and the contents of the pages that streams have.
static std::string picture(const Pool &pool) {
    std::string out;
    const sdv2_pages_config &c = pool.c;
    const int64_t page_bytes = 2ll * c.kv_heads * c.page_tokens * c.head_dim;
    for (int32_t b = 0; b < c.streams; ++b) {
        int32_t tokens = 0, n = 0, shared = 0;
        REQUIRE(sdv2_pages_query(pool.h, b, &tokens, nullptr, 0, &n, &shared) == SDV2_OK);
        std::vector<int32_t> ids(n + 1);
        REQUIRE(sdv2_pages_query(pool.h, b, nullptr, ids.data(), n, nullptr, nullptr) == SDV2_OK);
        out += std::to_string(tokens) + "/" + std::to_string(shared) + ":";
        for (int32_t i = 0; i < n; ++i) {
            out += std::to_string(ids[i]) + " ";
            for (uint64_t side : {pool.h->r.k, pool.h->r.v})
                out.append(reinterpret_cast<char *>(pool.h->base + side) + ids[i] * page_bytes, page_bytes);
        }
    }
    return out + "|" + std::to_string(sdv2_pages_used(pool.h)) + "|" + std::to_string(pool.h->version);
}

static void fill_pages(const Pool &pool) {
    const int64_t page_bytes = 2ll * pool.c.kv_heads * pool.c.page_tokens * pool.c.head_dim;
    for (uint64_t side : {pool.h->r.k, pool.h->r.v})
        for (int64_t i = 0; i < pool.c.pages * page_bytes; ++i)
            pool.h->base[side + i] = static_cast<uint8_t>((i * 2654435761u >> 13) + i / page_bytes + (side ? 7 : 0));
}

// Does `call` on a fresh pool made by `start`, every allocation failing in turn, then every launch: a call
// that fails leaves the pool as it was, unless its table edits had begun.  `launches`: of a call that succeeds.
template <typename Start, typename Call>
static void every_failure(const sdv2_pages_config &c, Start start, Call call, int launches) {
    std::string before, after;
    int allocations = 0;
    {
        Pool pool(c);
        start(pool);
        fill_pages(pool);
        before = picture(pool);
        g_made = 0;
        g_good_allocations = 1 << 30;
        REQUIRE(call(pool) == SDV2_OK);
        allocations = (1 << 30) - g_good_allocations;
        g_good_allocations = -1;
        REQUIRE(g_made == launches && allocations > 0, "%d launches", g_made);
        pool.check_books();
        after = picture(pool);
        REQUIRE(before != after);
    }
    const int every = max(1, allocations / 5);            // (of thousands of like ones a few, and the last ones)
    for (int i = 0; i <= allocations; i = max(i + 1, min(i + every, allocations - 4))) {
        Pool pool(c);
        start(pool);
        fill_pages(pool);
        g_good_allocations = i;
        REQUIRE(call(pool) == (i == allocations ? SDV2_OK : SDV2_E_STATE));
        g_good_allocations = -1;
        pool.check_books();
        REQUIRE(picture(pool) == (i == allocations ? after : before), "allocation %d", i);
        if (i < allocations) {                            // and again, with memory
            REQUIRE(call(pool) == SDV2_OK);
            pool.check_books();
            REQUIRE(picture(pool) == after);
        }
    }
    for (int good = 0; good < launches; ++good) {
        Pool pool(c);
        start(pool);
        fill_pages(pool);
        g_good_launches = good;
        const uint32_t version = *reinterpret_cast<uint32_t *>(pool.h->base + pool.h->r.version);
        const std::vector<int32_t> lengths(reinterpret_cast<int32_t *>(pool.h->base + pool.h->r.length),
                                           reinterpret_cast<int32_t *>(pool.h->base + pool.h->r.length) + c.streams);
        REQUIRE(call(pool) == SDV2_E_CUDA);
        g_good_launches = -1;
        REQUIRE(picture(pool) == before, "launch %d", good);
        const bool begun = version != *reinterpret_cast<uint32_t *>(pool.h->base + pool.h->r.version) ||
                           !std::equal(lengths.begin(), lengths.end(),
                                       reinterpret_cast<int32_t *>(pool.h->base + pool.h->r.length));
        std::vector<int32_t> none(c.streams, 0), one(c.streams, 0);
        one[0] = 1;
        static uint16_t io[16];
        void *aligned = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(io) + 15) & ~uintptr_t(15));
        if (begun) {                                      // nothing that would read or change the tables
            REQUIRE(call(pool) == SDV2_E_STATE);
            REQUIRE(pool.extend(one) == SDV2_E_STATE && pool.attend(one) == SDV2_E_STATE);
            REQUIRE(pool.free({0}) == (pool.h->tokens[0] > 0 ? SDV2_E_STATE : SDV2_OK));    // (nothing to free)
            REQUIRE(sdv2_pages_write(pool.h, 0, aligned, aligned, 0, 0, one.data(), nullptr) == SDV2_E_STATE);
            REQUIRE(pool.compact() == SDV2_E_STATE);
            REQUIRE(g_launches.empty() && sdv2_pages_check(pool.h) == SDV2_OK && picture(pool) == before);
        } else {
            pool.check_books();
            REQUIRE(call(pool) == SDV2_OK);
            pool.check_books();
            REQUIRE(picture(pool) == after);
        }
    }
}

static void failures() {
    auto grown = [](Pool &p) { REQUIRE(p.extend({100, 0, 37, 0, 0}) == SDV2_OK); };
    auto forked = [&](Pool &p) {
        grown(p);
        REQUIRE(p.fork(0, {1, 3}) == SDV2_OK && p.extend({1, 30, 0, 2, 50}) == SDV2_OK);
    };
    auto holes = [&](Pool &p) {
        forked(p);
        REQUIRE(p.free({2}) == SDV2_OK);
    };
    const sdv2_pages_config small = config(5, 2, 1, 16, 60, 20);
    every_failure(small, grown, [](Pool &p) { return p.extend({3, 50, 0, 1, 0}); }, 1);
    every_failure(small, grown, [](Pool &p) { return p.fork(0, {1, 4}); }, 2);
    every_failure(small, grown, [](Pool &p) { return p.fork(2, {1, 4}, true); }, 2);
    every_failure(small, forked, [](Pool &p) { return p.free({0, 2}); }, 1);
    every_failure(small, holes, [](Pool &p) { return p.compact(); }, 2);
    // more entries and page copies than one launch holds
    const sdv2_pages_config large = config(5, 2, 1, 16, 12000, 20);
    auto none = [](Pool &) {};
    auto many = [](Pool &p) { REQUIRE(p.extend({16 * 2100, 16 * 2500, 0, 0, 5}) == SDV2_OK); };
    auto gone = [&](Pool &p) {
        many(p);
        REQUIRE(p.free({0}) == SDV2_OK);
    };
    every_failure(large, none, [](Pool &p) { return p.extend({16 * 2500, 16 * 2000, 0, 0, 5}); }, 3);
    every_failure(large, many, [](Pool &p) { return p.fork(0, {2, 3}, true); }, 6);
    every_failure(large, gone, [](Pool &p) { return p.compact(); }, 4);
}

int main(int argc, char **argv) {
    const std::string what = argc > 1 ? argv[1] : "";
    if (what == "mixed")
        mixed();
    else if (what == "share")
        share();
    else if (what == "failures")
        failures();
    else if (what == "plan" && argc == 4)
        sessions(std::strtoull(argv[2], nullptr, 10), std::atoi(argv[3]));
    else
        return 2;
    std::printf("ok\n");
    return 0;
}
