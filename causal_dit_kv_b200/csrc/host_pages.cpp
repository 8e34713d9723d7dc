// Host side of the paged cache: the streams' page lists and the users of every page,
// the plan of an attention call, and the launches.
#include <algorithm>
#include <cmath>
#include <memory>
#include <vector>

#include "host_common.h"
#include "token_ops.h"

using namespace sdv2;

namespace {

// What a run costs before and after its tiles, in tiles.  Measured on a batch of 192 units of one to
// eight tiles behind a common prefix: 120 us for 0 (runs cut by their tiles alone), 74 for 2, 64
// for 3, 57 for 4 and for 6; the row kernel's single-stream case 11.7, 10.5, 9.9, 10.2 and 10.6 us for
// 0, 2, 3, 4 and 6.
constexpr int kSetupTiles = 5, kSetupRows = 3;

struct Regions {
    uint64_t k, v, layer_stride, table, length, version, status, scratch, part_ml, part_o, end;
    int64_t rows;            // rows of the partial results
};

// Rows of the attention's partial results: one of the stream's own keys and one of the
// group's common keys per (query token, head), and for each of the call's two launches those
// of every worker's piece whose unit began with an earlier worker.
constexpr int32_t kCutRows = kPagesMaxCtas * 128;
static_assert(kCutRows == kPagesMaxCtas * kRowWarps * kRowsPerWorker, "the same for both kernels");
int64_t partial_rows(const sdv2_pages_config &c) { return 2ll * c.max_queries * c.heads + 2 * kCutRows; }

Regions regions(const sdv2_pages_config &c) {
    Regions r{};
    r.layer_stride = 2ull * c.pages * c.kv_heads * c.page_tokens * c.head_dim;
    r.k = 0;
    r.v = align_up(r.k + r.layer_stride * c.layers, 256);
    r.table = align_up(r.v + r.layer_stride * c.layers, 256);
    r.length = align_up(r.table + 4ull * c.streams * c.stream_pages, 256);
    r.version = align_up(r.length + 4ull * c.streams, 256);
    r.status = align_up(r.version + 4, 256);
    r.rows = partial_rows(c);
    r.scratch = r.part_ml = align_up(r.status + 4, 256);
    r.part_o = align_up(r.part_ml + 8ull * r.rows, 256);
    r.end = align_up(r.part_o + 4ull * c.head_dim * r.rows, 256);
    return r;
}

sdv2_status check_config(const sdv2_pages_config *c) {
    if (!c) return fail(SDV2_E_ARG, "config is NULL");
    if (c->streams < 1 || c->streams > kPagesMaxStreams)
        return fail(SDV2_E_SHAPE, "streams must be in 1..%d", kPagesMaxStreams);
    if (c->layers < 1 || c->layers > 1024) return fail(SDV2_E_SHAPE, "layers must be in 1..1024");
    if (c->heads < 1 || c->kv_heads < 1 || c->heads > 1024 || c->heads % c->kv_heads != 0 || c->heads / c->kv_heads > 128)
        return fail(SDV2_E_SHAPE, "heads must be a multiple of kv_heads (at most 128 times it), in 1..1024");
    if (c->head_dim != 64 && c->head_dim != 128) return fail(SDV2_E_SHAPE, "head_dim must be 64 or 128");
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return fail(SDV2_E_SHAPE, "page_tokens must be 16, 32, 64 or 128");
    if (c->pages < 1 || static_cast<int64_t>(c->pages) * c->kv_heads >= (1ll << 31))
        return fail(SDV2_E_SHAPE, "pages must be >= 1, pages x kv_heads < 2^31");
    if (c->stream_pages < 1 || static_cast<int64_t>(c->stream_pages) * c->page_tokens > (1ll << 25) ||
        static_cast<int64_t>(c->stream_pages) * c->streams >= (1ll << 31))
        return fail(SDV2_E_SHAPE, "stream_pages must be >= 1, x page_tokens <= 2^25, x streams < 2^31");
    if (c->max_queries < 1 || static_cast<int64_t>(c->max_queries) * c->heads >= (1ll << 29))
        return fail(SDV2_E_SHAPE, "max_queries must be >= 1, x heads < 2^29");
    if (c->block_tokens < 1) return fail(SDV2_E_SHAPE, "block_tokens must be >= 1");
    if (c->dtype != SDV2_DT_BF16 && c->dtype != SDV2_DT_FP16)
        return fail(SDV2_E_SHAPE, "dtype must be SDV2_DT_BF16 or SDV2_DT_FP16");
    return SDV2_OK;
}

}  // namespace

struct sdv2_pages {
    sdv2_pages_config cfg;
    Regions r;
    uint8_t *base;
    int device, sm_count;
    std::vector<CUtensorMap> tk, tv;      // [layers]
    std::vector<int32_t> table;           // [streams][stream_pages]
    std::vector<int32_t> n_pages, tokens; // [streams]
    std::vector<int32_t> users;           // [pages]
    int32_t used = 0;                     // pages with users
    int32_t first_free = 0;               // no page below it is free
    uint32_t version = 0;
    bool torn = false;                    // some of a call's table edits were launched, others failed
    // streams with the same first page, and the leading pages that all of them share
    // (kept until the next fork, free or compact: new pages are never shared ones)
    bool groups_known = false;
    int32_t share = 1;                    // SDV2_SHARE_AUTO
    std::vector<int32_t> group_of;        // [streams]: its group, -1 none
    std::vector<int32_t> group_pages;

    int32_t *row(int32_t b) { return table.data() + static_cast<size_t>(b) * cfg.stream_pages; }
    int32_t pages_of(int64_t n) const { return static_cast<int32_t>((n + cfg.page_tokens - 1) / cfg.page_tokens); }
    // The lowest free page from *at on (there is one), *at moved behind it: a call chooses its pages
    // with an *at of its own, that of first_free, and takes them when its launches have succeeded.
    int32_t next_free(int32_t *at) const {
        while (users[*at] != 0) ++*at;
        return (*at)++;
    }
    void take(int32_t p) {
        users[p] = 1;
        ++used;
    }
    void drop(int32_t p) {
        if (--users[p] == 0) {
            --used;
            first_free = std::min(first_free, p);
        }
    }
    PagesView view() const {
        PagesView w;
        w.table = reinterpret_cast<int32_t *>(base + r.table);
        w.lengths = reinterpret_cast<int32_t *>(base + r.length);
        w.version = reinterpret_cast<uint32_t *>(base + r.version);
        w.status = reinterpret_cast<uint32_t *>(base + r.status);
        w.expect = version;
        w.width = cfg.stream_pages;
        w.pages = cfg.pages;
        w.kv_heads = cfg.kv_heads;
        w.page_log2 = cfg.page_tokens == 16 ? 4 : (cfg.page_tokens == 32 ? 5 : (cfg.page_tokens == 64 ? 6 : 7));
        w.head_dim = cfg.head_dim;
        return w;
    }
};

namespace {

// A call that changes the tables first works out its edits and copies, then launches them, and
// only then changes the host's books: one that runs out of memory or whose launch fails changes nothing.

// Table edits of one call, launched in as few kernels as they fit into.
struct Edits {
    struct Copy { int32_t from, to, n; };
    std::vector<Copy> copies;
    std::vector<std::pair<int32_t, int32_t>> clears, lengths;
    std::vector<std::pair<uint32_t, int32_t>> entries;

    template <int kE, int kR>
    sdv2_status parts(sdv2_pages *h, uint32_t version, bool beside, cudaStream_t s) const {
        std::unique_ptr<PageEdits<kE, kR>> p(new PageEdits<kE, kR>);   // (one for all parts: a launch copies it)
        const PagesView w = h->view();
        p->table = w.table;
        p->lengths = w.lengths;
        p->version = w.version;
        p->new_version = version;
        p->width = w.width;
        size_t c = 0, x = 0, l = 0, e = 0;
        do {
            const bool first = c + x + l + e == 0;
            p->n_copies = p->n_clears = p->n_lengths = p->n_entries = 0;
            for (; c < copies.size() && p->n_copies < kR; ++c, ++p->n_copies) {
                p->copy[p->n_copies][0] = copies[c].from;
                p->copy[p->n_copies][1] = copies[c].to;
                p->copy[p->n_copies][2] = copies[c].n;
            }
            for (; x < clears.size() && p->n_clears < kR; ++x, ++p->n_clears) {
                p->clear[p->n_clears][0] = clears[x].first;
                p->clear[p->n_clears][1] = clears[x].second;
            }
            for (; l < lengths.size() && p->n_lengths < kR; ++l, ++p->n_lengths) {
                p->length[p->n_lengths][0] = lengths[l].first;
                p->length[p->n_lengths][1] = lengths[l].second;
            }
            for (; e < entries.size() && p->n_entries < kE; ++e, ++p->n_entries) {
                p->entry_at[p->n_entries] = entries[e].first;
                p->entry[p->n_entries] = entries[e].second;
            }
            const cudaError_t err = launch_page_edits(*p, beside && first, s);
            if (err != cudaSuccess) {
                h->torn = !first;
                return cuda_fail(err, "page table launch");
            }
            count_launch();
        } while (c < copies.size() || x < clears.size() || l < lengths.size() || e < entries.size());
        return SDV2_OK;
    }
    // version: the tables' new one; beside: the launch before it is the same call's page copies
    sdv2_status launch(sdv2_pages *h, uint32_t version, bool beside, cudaStream_t s) const {
        const bool small = copies.size() <= 32 && clears.size() <= 32 && lengths.size() <= 32 && entries.size() <= 64;
        return small ? parts<64, 32>(h, version, beside, s) : parts<2000, 256>(h, version, beside, s);
    }
};

// Page copies of one call: source src[i] to the pages dst[i].  (Those are free ones until the
// call's table edits are there.)
struct Moves {
    std::vector<int32_t> src;
    std::vector<std::vector<int32_t>> dst;

    template <int kM>
    sdv2_status parts(const sdv2_pages *h, cudaStream_t s) const {
        std::unique_ptr<PageMoves<kM>> p(new PageMoves<kM>);
        p->base[0] = h->base + h->r.k;
        p->base[1] = h->base + h->r.v;
        p->layer_stride = static_cast<int64_t>(h->r.layer_stride);
        p->page_bytes = 2ll * h->cfg.kv_heads * h->cfg.page_tokens * h->cfg.head_dim;
        p->layers = h->cfg.layers;
        p->first[0] = 0;
        for (size_t at = 0; at < src.size();) {
            p->n = 0;
            for (; at < src.size() && p->n < kM; ++at, ++p->n) {
                const std::vector<int32_t> &d = dst[at];
                int32_t f = p->first[p->n];
                if (f + static_cast<int32_t>(d.size()) > kM) break;     // (d.size() <= 255: the first one always fits)
                p->src[p->n] = src[at];
                for (int32_t x : d) p->dst[f++] = x;
                p->first[p->n + 1] = f;
            }
            const cudaError_t err = launch_page_moves(*p, s);
            if (err != cudaSuccess) return cuda_fail(err, "page copy launch");
            count_launch();
        }
        return SDV2_OK;
    }
    sdv2_status launch(const sdv2_pages *h, cudaStream_t s) const {
        size_t total = 0;
        for (const auto &d : dst) total += d.size();
        return total <= 64 ? parts<64>(h, s) : parts<2000>(h, s);
    }
};

sdv2_status check_whole(const sdv2_pages *h) {
    return h->torn ? fail(SDV2_E_STATE, "an earlier call's launches failed halfway: the device's page tables are lost")
                   : SDV2_OK;
}

// The checks of a call that changes the tables.
sdv2_status check_change(const sdv2_pages *h, cudaStream_t s) {
    sdv2_status st = check_whole(h);
    if (st == SDV2_OK) st = check_device(h->device);
    if (st != SDV2_OK) return st;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing(s, &cap);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(SDV2_E_STATE, "the stream cannot be used: %s", cudaGetErrorString(e));
    }
    if (cap != cudaStreamCaptureStatusNone)
        return fail(SDV2_E_STATE, "a call that changes the page tables cannot be captured");
    return SDV2_OK;
}

sdv2_status check_counts(const sdv2_pages *h, const int32_t *counts, int64_t *sum) {
    if (!counts) return fail(SDV2_E_ARG, "counts is NULL");
    *sum = 0;
    for (int32_t b = 0; b < h->cfg.streams; ++b) {
        if (counts[b] < 0) return fail(SDV2_E_ARG, "counts[%d] is negative", b);
        *sum += counts[b];
    }
    return SDV2_OK;
}

// Token stride: 0 becomes the contiguous one.
sdv2_status check_stride(int64_t *stride, int64_t row) {
    if (*stride == 0) *stride = row;
    if (*stride < row || *stride >= (1ll << 38))
        return fail(SDV2_E_SHAPE, "a token stride is shorter than a token's row, or too long");
    if (*stride % 8 != 0) return fail(SDV2_E_ALIGN, "token strides must be multiples of 8 elements");
    return SDV2_OK;
}

void know_groups(sdv2_pages *h) {
    if (h->groups_known) return;
    std::fill(h->group_of.begin(), h->group_of.end(), -1);
    h->group_pages.clear();
    for (int32_t b = 0; b < h->cfg.streams; ++b) {
        if (h->group_of[b] >= 0 || h->n_pages[b] == 0 || h->users[h->row(b)[0]] < 2) continue;
        const int32_t g = static_cast<int32_t>(h->group_pages.size());
        int32_t common = h->n_pages[b];
        h->group_of[b] = g;
        for (int32_t o = b + 1; o < h->cfg.streams; ++o) {
            if (h->n_pages[o] == 0 || h->row(o)[0] != h->row(b)[0]) continue;
            h->group_of[o] = g;
            const int32_t most = std::min(common, h->n_pages[o]);
            common = static_cast<int32_t>(std::mismatch(h->row(b), h->row(b) + most, h->row(o)).first - h->row(b));
        }
        h->group_pages.push_back(common);
    }
    h->groups_known = true;
}

void changed(sdv2_pages *h) {
    ++h->version;
    h->groups_known = false;
}

sdv2_status create(const sdv2_pages_config *cfg, void *dev_buf, size_t bytes, sdv2_pages **out) {
    if (!out) return fail(SDV2_E_ARG, "out is NULL");
    *out = nullptr;
    sdv2_status st = check_config(cfg);
    if (st != SDV2_OK) return st;
    if (!dev_buf) return fail(SDV2_E_ARG, "dev_buf is NULL");
    if ((reinterpret_cast<uintptr_t>(dev_buf) & 255u) != 0) return fail(SDV2_E_ALIGN, "dev_buf must be 256-byte aligned");
    const Regions r = regions(*cfg);
    if (bytes < r.end)
        return fail(SDV2_E_ALIGN, "buffer of %zu bytes is smaller than the %llu bytes required", bytes,
                    static_cast<unsigned long long>(r.end));
    PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode_fn();
    if (!encode) return fail(SDV2_E_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    std::unique_ptr<sdv2_pages> h(new sdv2_pages());
    const sdv2_pages_config &c = *cfg;
    h->cfg = c;
    // (a block longer than a stream can be masks nothing; keeps (i / b + 1) * b below 2^31)
    h->cfg.block_tokens = std::min(c.block_tokens, c.stream_pages * c.page_tokens);
    h->r = r;
    h->base = static_cast<uint8_t *>(dev_buf);
    h->table.assign(static_cast<size_t>(c.streams) * c.stream_pages, -1);
    h->n_pages.assign(c.streams, 0);
    h->tokens.assign(c.streams, 0);
    h->users.assign(c.pages, 0);
    h->group_of.assign(c.streams, -1);
    h->group_pages.reserve(c.streams);
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
    // (an allocator may have handed the memory out while work of a stream that this one does not wait for is on it)
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemset(dev_buf, 0, r.end);
    if (e == cudaSuccess) e = cudaMemset(h->base + r.table, 0xff, 4ull * c.streams * c.stream_pages);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "pages_create");
    // One map per layer and side: (d, n, P * Hkv), boxes of 64 channels x one page of one head,
    // 128-byte swizzle (the layout of the MMA's operand tiles, page after page).
    h->tk.resize(c.layers);
    h->tv.resize(c.layers);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_tokens),
                                static_cast<cuuint64_t>(c.pages) * c.kv_heads};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.head_dim) * 2,
                                   static_cast<cuuint64_t>(c.head_dim) * c.page_tokens * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(c.page_tokens), 1}, estr[3] = {1, 1, 1};
    for (int32_t l = 0; l < c.layers; ++l)
        for (int side = 0; side < 2; ++side) {
            const CUresult res =
                encode(side ? &h->tv[l] : &h->tk[l],
                       c.dtype == SDV2_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                       h->base + (side ? r.v : r.k) + r.layer_stride * l, dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
            if (res != CUDA_SUCCESS) return fail(SDV2_E_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(res));
        }
    *out = h.release();
    return SDV2_OK;
}

sdv2_status extend(sdv2_pages *h, const int32_t *counts, cudaStream_t s) {
    if (!h) return fail(SDV2_E_ARG, "pages is NULL");
    int64_t sum = 0;
    sdv2_status st = check_counts(h, counts, &sum);
    if (st != SDV2_OK) return st;
    int64_t need = 0;
    for (int32_t b = 0; b < h->cfg.streams; ++b) {
        const int64_t pages = (static_cast<int64_t>(h->tokens[b]) + counts[b] + h->cfg.page_tokens - 1) / h->cfg.page_tokens;
        if (pages > h->cfg.stream_pages) return fail(SDV2_E_STATE, "stream %d would need %lld pages", b, static_cast<long long>(pages));
        need += pages - h->n_pages[b];
    }
    if (need > h->cfg.pages - h->used)
        return fail(SDV2_E_STATE, "%lld pages needed, %d free", static_cast<long long>(need), h->cfg.pages - h->used);
    if (sum == 0) return SDV2_OK;
    if ((st = check_change(h, s)) != SDV2_OK) return st;
    Edits ed;
    ed.entries.reserve(static_cast<size_t>(need));
    ed.lengths.reserve(h->cfg.streams);
    int32_t free = h->first_free;
    for (int32_t b = 0; b < h->cfg.streams; ++b) {
        if (counts[b] == 0) continue;
        const int32_t n = h->pages_of(static_cast<int64_t>(h->tokens[b]) + counts[b]);
        for (int32_t i = h->n_pages[b]; i < n; ++i)
            ed.entries.emplace_back(static_cast<uint32_t>(static_cast<int64_t>(b) * h->cfg.stream_pages + i), h->next_free(&free));
        ed.lengths.emplace_back(b, h->tokens[b] + counts[b]);
    }
    if ((st = ed.launch(h, h->version, false, s)) != SDV2_OK) return st;
    for (const auto &x : ed.entries) {
        h->table[x.first] = x.second;
        h->take(x.second);
    }
    h->first_free = free;
    for (const auto &x : ed.lengths) {
        h->tokens[x.first] = x.second;
        h->n_pages[x.first] = h->pages_of(x.second);
    }
    return SDV2_OK;
}

sdv2_status write(sdv2_pages *h, int32_t layer, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                  const int32_t *counts, cudaStream_t s) {
    if (!h || !k || !v) return fail(SDV2_E_ARG, "NULL argument");
    if (layer < 0 || layer >= h->cfg.layers) return fail(SDV2_E_ARG, "layer %d out of range", layer);
    if (!aligned16(k) || !aligned16(v)) return fail(SDV2_E_ALIGN, "k and v must be 16-byte aligned");
    const int64_t row = static_cast<int64_t>(h->cfg.kv_heads) * h->cfg.head_dim;
    sdv2_status st = check_stride(&k_stride, row);
    if (st == SDV2_OK) st = check_stride(&v_stride, row);
    int64_t sum = 0;
    if (st == SDV2_OK) st = check_counts(h, counts, &sum);
    if (st != SDV2_OK) return st;
    if (sum >= (1ll << 30)) return fail(SDV2_E_SHAPE, "too many tokens");
    PageWriteParams p;
    p.n = 0;
    int32_t at = 0;
    for (int32_t b = 0; b < h->cfg.streams; ++b) {
        if (counts[b] == 0) continue;
        if (counts[b] > h->tokens[b]) return fail(SDV2_E_STATE, "stream %d has %d tokens", b, h->tokens[b]);
        for (int32_t i = (h->tokens[b] - counts[b]) / h->cfg.page_tokens; i < h->n_pages[b]; ++i)
            if (h->users[h->row(b)[i]] > 1)
                return fail(SDV2_E_STATE, "stream %d: the tokens lie in a page that it shares", b);
        p.stream[p.n] = b;
        p.first[p.n++] = at;
        at += counts[b];
    }
    p.first[p.n] = at;
    if (sum == 0) return SDV2_OK;
    if ((st = check_whole(h)) != SDV2_OK || (st = check_device(h->device)) != SDV2_OK) return st;
    p.v = h->view();
    p.in[0] = static_cast<const uint16_t *>(k);
    p.in[1] = static_cast<const uint16_t *>(v);
    p.out[0] = reinterpret_cast<uint16_t *>(h->base + h->r.k + h->r.layer_stride * layer);
    p.out[1] = reinterpret_cast<uint16_t *>(h->base + h->r.v + h->r.layer_stride * layer);
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    const cudaError_t e = launch_page_write(p, s);
    if (e != cudaSuccess) return cuda_fail(e, "page write launch");
    count_launch();
    return SDV2_OK;
}

// Whether a group reads its common pages once for all of its `members`, with `rows` query rows to a
// key head.  Apart, the members' reads meet in the L2, at 17 TB/s with few rows; once for all costs
// a launch of the tile kernel (over 16 rows) and a merge of every row.  Measured with 300 keys of
// each stream's own (us, apart / once): 64 streams of 32/8 heads x 128: 1024 common keys 30 / 31,
// 2048 47 / 33, 8192 138 / 45; 16 streams: 1024 15 / 17, 2048 18 / 17, 8192 41 / 25; 4 streams of
// 12 heads x 64, 16 tokens each: 2048 16 / 16, 8192 24 / 26.  16 rows or fewer: 16 streams of 12
// heads x 128: 256 11.7 / 11.1, 8192 58 / 20; 4 streams of 32/8: 8192 17.5 / 19.
// (Beside a stream of many rows the tile kernel takes these too: 16 streams of 12 heads x 128 beside 64
// queries of another, 4096 common keys 64 / 26, 8192 114 / 28.)
bool shared(const sdv2_pages *h, int64_t members, int64_t pages, int64_t rows) {
    if (h->share != SDV2_SHARE_AUTO) return h->share == SDV2_SHARE_ALWAYS;
    const int64_t mb = 1 << 20;
    const int64_t bytes = pages * h->cfg.page_tokens * h->cfg.kv_heads * h->cfg.head_dim * 4;
    if (bytes > 64 * mb) return true;                        // the L2 does not hold it from one member to the next
    const int64_t saved = (members - 1) * bytes;
    return rows <= kRowsPerWorker ? members > 4 && saved >= 24 * mb : saved >= (30 + 4 * members) * mb;
}

// Whether the launch leaves any unit in pieces: a worker border inside one.
template <typename P>
bool cuts_units(const P &p, const PageWork &w) {
    for (int worker = 1, i = w.begin; worker < w.workers; ++worker) {
        const int64_t pos = static_cast<int64_t>(worker) * w.places / w.workers;
        while (i + 1 < w.end && p.start[i + 1] <= pos) ++i;
        if ((pos - p.start[i]) % (p.section[i].tiles + w.setup) > w.setup) return true;
    }
    return false;
}

// The sections of one attention call and its launches.
template <int kS, int kM>
sdv2_status attend(sdv2_pages *h, int32_t layer, const void *q, void *out, int64_t q_stride, int64_t out_stride,
                   const int32_t *counts, int64_t sum, float scale, cudaStream_t s) {
    const sdv2_pages_config &c = h->cfg;
    std::unique_ptr<PagesAttnParams<kS, kM>> p(new PagesAttnParams<kS, kM>);
    p->v = h->view();
    p->q = static_cast<const uint16_t *>(q);
    p->out = static_cast<uint16_t *>(out);
    p->k_layer = reinterpret_cast<const uint16_t *>(h->base + h->r.k + h->r.layer_stride * layer);
    p->v_layer = reinterpret_cast<const uint16_t *>(h->base + h->r.v + h->r.layer_stride * layer);
    p->q_stride = q_stride;
    p->out_stride = out_stride;
    p->part_ml = reinterpret_cast<float2 *>(h->base + h->r.part_ml);
    p->part_o = reinterpret_cast<float *>(h->base + h->r.part_o);
    p->rows_common = c.max_queries * c.heads;
    p->heads = c.heads;
    p->group = c.heads / c.kv_heads;
    p->block = c.block_tokens;
    p->scale_log2 = scale * 1.4426950408889634f;
    p->n_queries = static_cast<int32_t>(sum);

    int32_t token_of[kPagesMaxStreams];   // first packed token of each stream
    int32_t at = 0, most_tokens = 0;
    for (int32_t b = 0; b < c.streams; ++b) {
        token_of[b] = at;
        at += counts[b];
        most_tokens = std::max(most_tokens, counts[b]);
    }
    // groups of active streams with common leading pages: every query sees all of those keys
    know_groups(h);
    const int n_groups = static_cast<int>(h->group_pages.size());
    int32_t section_of[kPagesMaxStreams];                    // of each group in this call (-1: none)
    int32_t place_of[kPagesMaxStreams];                      // first query's place of a stream among its section's
    p->n_members = 0;
    p->tokens_each = -1;
    int n = 0;
    int32_t member_at = 0, most_common = 0;
    for (int g = 0; g < n_groups; ++g) {
        section_of[g] = -1;
        int32_t members = 0, group_tokens = 0, first = -1;
        int32_t pages = h->group_pages[g];
        for (int32_t b = 0; b < c.streams; ++b) {
            if (h->group_of[b] != g || counts[b] == 0) continue;
            if (first < 0) first = b;
            ++members;
            group_tokens += counts[b];
            pages = std::min(pages, (h->tokens[b] - counts[b]) / c.page_tokens);
        }
        if (members < 2 || pages < 1 || !shared(h, members, pages, group_tokens * p->group)) continue;
        section_of[g] = n;
        PageSection &x = p->section[n++];
        x.stream = first;
        x.page0 = 0;
        x.keys = pages * c.page_tokens;
        x.token0 = member_at;
        x.n_tokens = group_tokens;
        x.common = -1;
        x.common_token = 0;
        most_common = std::max(most_common, group_tokens);
        int32_t place = 0;
        for (int32_t b = 0; b < c.streams; ++b) {
            if (h->group_of[b] != g || counts[b] == 0) continue;
            p->tokens_each = p->tokens_each < 0 || p->tokens_each == counts[b] ? counts[b] : 0;
            p->member_first[p->n_members] = member_at;
            p->member_token[p->n_members++] = token_of[b];
            place_of[b] = place;
            place += counts[b];
            member_at += counts[b];
        }
    }
    p->n_common = n;
    for (int32_t b = 0; b < c.streams; ++b) {
        if (counts[b] == 0) continue;
        const int32_t common = h->group_of[b] >= 0 ? section_of[h->group_of[b]] : -1;
        PageSection &x = p->section[n++];
        x.stream = b;
        x.page0 = common >= 0 ? p->section[common].keys / c.page_tokens : 0;
        x.keys = -1;
        x.token0 = token_of[b];
        x.n_tokens = counts[b];
        x.common = common;
        x.common_token = common >= 0 ? place_of[b] : 0;
    }
    p->n_sections = n;

    // Both parts' kernels: a warp per run where no unit has more than 16 rows.  A stream outside every
    // group may have more rows than the groups: one launch of the tile kernel takes both parts then.
    // (16 forks' next tokens on 8192 common keys beside 64 queries of another stream, 12 heads x 128: 27.9 us;
    // as two calls, each with its own kernel, 19.3 and 15.2.  40/8 heads: 28.3; 22.4 and 16.3.)
    const int32_t own_rows = most_tokens * p->group, common_rows = most_common * p->group;
    const bool few_own = own_rows <= kRowsPerWorker, few_common = few_own && common_rows <= kRowsPerWorker;
    auto work = [&](int begin, int end, bool few, int32_t rows, int32_t cut_row) {
        PageWork w{};
        w.begin = begin;
        w.end = end;
        w.tile_log2 = few ? kRowKeysLog2 : kTileKeysLog2;
        w.tile_tokens = (few ? kRowsPerWorker : 128) / p->group;
        w.cut_row = cut_row;
        w.cut_rows = few ? rows : 128;
        w.rows = rows;
        w.setup = few ? kSetupRows : kSetupTiles;
        int64_t places = 0, units = 0;
        for (int i = begin; i < end; ++i) {
            PageSection &x = p->section[i];
            const int64_t keys = x.keys >= 0 ? x.keys : h->tokens[x.stream] - static_cast<int64_t>(x.page0) * c.page_tokens;
            p->start[i] = static_cast<int32_t>(std::min<int64_t>(places, INT32_MAX));
            x.tiles = static_cast<int32_t>((keys + (1 << w.tile_log2) - 1) >> w.tile_log2);
            const int64_t n_units = static_cast<int64_t>((x.n_tokens + w.tile_tokens - 1) / w.tile_tokens) * c.kv_heads;
            units += n_units;
            places += n_units * (x.tiles + w.setup);
        }
        w.places = static_cast<uint32_t>(std::min<int64_t>(places, INT32_MAX));
        const int64_t ctas = std::min(h->sm_count, kPagesMaxCtas);
        const int64_t most = few ? std::min<int64_t>(ctas * kRowWarps, kCutRows / rows) : ctas;
        // A unit to a worker while there are workers; longer units are cut into runs of at least so many
        // places (two streams of 64 to 512 keys, 12 heads: 10.5 us with 7, 9.7 with 5, 7.3 with 3 or 2 in the
        // row kernel; 16 streams on 2048 common keys: 20.0, 16.7, 19.9 us with 7, 4, 2 in the tile kernel)
        const int64_t shortest = few ? 3 : 4;
        w.workers = static_cast<int32_t>(std::max<int64_t>(
            1, std::min<int64_t>({most, std::max(units, (places + shortest - 1) / shortest), 0xffffffffll / (static_cast<int64_t>(w.places) + 1)})));
        return w;
    };
    const int32_t cut = 2 * c.max_queries * c.heads;
    const bool together = p->n_common == 0 || few_common == few_own;
    p->own = work(together ? 0 : p->n_common, n, few_own, together ? std::max(own_rows, common_rows) : own_rows, cut);
    p->common = together ? p->own : work(0, p->n_common, few_common, common_rows, cut + kCutRows);
    if (p->own.places == INT32_MAX || p->common.places == INT32_MAX) return fail(SDV2_E_SHAPE, "too much work for one call");

    const bool half = c.dtype == SDV2_DT_FP16;
    cudaError_t e = cudaSuccess;
    if (!together) {
        e = launch_pages_tiles<kS, kM>(*p, p->common, h->tk[layer], h->tv[layer], half, s);
        if (e == cudaSuccess) count_launch();
    }
    if (e == cudaSuccess) {
        e = few_own ? launch_pages_rows<kS, kM>(*p, p->own, half, !together, h->sm_count, s)
                    : launch_pages_tiles<kS, kM>(*p, p->own, h->tk[layer], h->tv[layer], half, s);
        if (e == cudaSuccess) count_launch();
    }
    if (e == cudaSuccess && (p->n_common > 0 || cuts_units(*p, p->own))) {
        // most pieces of a unit, common and own together
        int64_t pieces = 0;
        for (int i = 0; i < n; ++i) {
            const PageWork &w = i < p->n_common ? p->common : p->own;
            const auto of = [&](int j, const PageWork &x) {
                return static_cast<int64_t>(p->section[j].tiles) * x.workers / x.places + 2;
            };
            const int32_t common = p->section[i].common;
            pieces = std::max(pieces, of(i, w) + (common >= 0 ? of(common, p->common) : 0));
        }
        const int64_t room = static_cast<int64_t>(h->sm_count) * 64 / (sum * c.heads);   // warps per row that run at once
        e = launch_pages_merge<kS, kM>(*p, pieces > 40 && room >= 8 ? 8 : (pieces > 10 && room >= 4 ? 4 : 1), half, s);
        if (e == cudaSuccess) count_launch();
    }
    return e == cudaSuccess ? SDV2_OK : cuda_fail(e, "pages_attention launch");
}

sdv2_status attention(sdv2_pages *h, int32_t layer, const void *q, void *out, int64_t q_stride, int64_t out_stride,
                      const int32_t *counts, float scale, cudaStream_t s) {
    if (!h || !q || !out) return fail(SDV2_E_ARG, "NULL argument");
    if (layer < 0 || layer >= h->cfg.layers) return fail(SDV2_E_ARG, "layer %d out of range", layer);
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(SDV2_E_ARG, "softmax_scale must be > 0");
    if (!aligned16(q) || !aligned16(out)) return fail(SDV2_E_ALIGN, "q and out must be 16-byte aligned");
    const int64_t row = static_cast<int64_t>(h->cfg.heads) * h->cfg.head_dim;
    sdv2_status st = check_stride(&q_stride, row);
    if (st == SDV2_OK) st = check_stride(&out_stride, row);
    int64_t sum = 0;
    if (st == SDV2_OK) st = check_counts(h, counts, &sum);
    if (st != SDV2_OK) return st;
    if (sum > h->cfg.max_queries)
        return fail(SDV2_E_SHAPE, "%lld query tokens, max_queries is %d", static_cast<long long>(sum), h->cfg.max_queries);
    int active = 0;
    for (int32_t b = 0; b < h->cfg.streams; ++b) {
        if (counts[b] > h->tokens[b]) return fail(SDV2_E_STATE, "stream %d has %d tokens", b, h->tokens[b]);
        active += counts[b] > 0;
    }
    if (sum == 0) return SDV2_OK;
    if ((st = check_whole(h)) != SDV2_OK || (st = check_device(h->device)) != SDV2_OK) return st;
    // (at most one group for every two active streams)
    return active + active / 2 <= kSmallSections && active <= kSmallMembers
               ? attend<kSmallSections, kSmallMembers>(h, layer, q, out, q_stride, out_stride, counts, sum, scale, s)
               : attend<kLargeSections, kLargeMembers>(h, layer, q, out, q_stride, out_stride, counts, sum, scale, s);
}

sdv2_status fork(sdv2_pages *h, int32_t src, const int32_t *dst, int32_t n, int32_t deep, cudaStream_t s) {
    if (!h || (n > 0 && !dst)) return fail(SDV2_E_ARG, "NULL argument");
    const sdv2_pages_config &c = h->cfg;
    if (src < 0 || src >= c.streams) return fail(SDV2_E_ARG, "stream %d out of range", src);
    if (n < 0 || n >= c.streams + (n == 0)) return fail(SDV2_E_ARG, "n must be in 0..streams - 1");
    bool seen[kPagesMaxStreams] = {};
    for (int32_t i = 0; i < n; ++i) {
        if (dst[i] < 0 || dst[i] >= c.streams) return fail(SDV2_E_ARG, "stream %d out of range", dst[i]);
        if (dst[i] == src || seen[dst[i]]) return fail(SDV2_E_ARG, "stream %d is given twice", dst[i]);
        seen[dst[i]] = true;
    }
    for (int32_t i = 0; i < n; ++i)
        if (h->tokens[dst[i]] != 0) return fail(SDV2_E_STATE, "stream %d is not empty", dst[i]);
    const int32_t full = deep ? 0 : h->tokens[src] / c.page_tokens;   // shared pages
    const int32_t copied = h->n_pages[src] - full;
    if (static_cast<int64_t>(copied) * n > c.pages - h->used)
        return fail(SDV2_E_STATE, "%lld pages needed, %d free", static_cast<long long>(copied) * n, c.pages - h->used);
    if (n == 0 || h->tokens[src] == 0) return SDV2_OK;
    sdv2_status st = check_change(h, s);
    if (st != SDV2_OK) return st;
    Edits ed;
    Moves mv;
    ed.copies.reserve(n);
    ed.lengths.reserve(n);
    ed.entries.reserve(static_cast<size_t>(copied) * n);
    mv.src.reserve(copied);
    mv.dst.resize(copied);
    for (int32_t i = 0; i < copied; ++i) {
        mv.src.push_back(h->row(src)[full + i]);
        mv.dst[i].reserve(n);
    }
    int32_t free = h->first_free;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t b = dst[i];
        for (int32_t j = full; j < full + copied; ++j) {
            const int32_t p = h->next_free(&free);
            mv.dst[j - full].push_back(p);
            ed.entries.emplace_back(static_cast<uint32_t>(static_cast<int64_t>(b) * c.stream_pages + j), p);
        }
        if (full > 0) ed.copies.push_back({src, b, full});
        ed.lengths.emplace_back(b, h->tokens[src]);
    }
    if (copied > 0 && (st = mv.launch(h, s)) != SDV2_OK) return st;
    if ((st = ed.launch(h, h->version + 1, copied > 0, s)) != SDV2_OK) return st;
    for (const auto &x : ed.entries) {
        h->table[x.first] = x.second;
        h->take(x.second);
    }
    h->first_free = free;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t b = dst[i];
        std::copy(h->row(src), h->row(src) + full, h->row(b));
        for (int32_t j = 0; j < full; ++j) ++h->users[h->row(src)[j]];
        h->n_pages[b] = h->n_pages[src];
        h->tokens[b] = h->tokens[src];
    }
    changed(h);
    return SDV2_OK;
}

sdv2_status free_streams(sdv2_pages *h, const int32_t *streams, int32_t n, cudaStream_t s) {
    if (!h || (n > 0 && !streams)) return fail(SDV2_E_ARG, "NULL argument");
    if (n < 0 || n > h->cfg.streams) return fail(SDV2_E_ARG, "n must be in 0..streams");
    bool seen[kPagesMaxStreams] = {};
    bool any = false;
    for (int32_t i = 0; i < n; ++i) {
        if (streams[i] < 0 || streams[i] >= h->cfg.streams) return fail(SDV2_E_ARG, "stream %d out of range", streams[i]);
        if (seen[streams[i]]) return fail(SDV2_E_ARG, "stream %d is given twice", streams[i]);
        seen[streams[i]] = true;
        any = any || h->tokens[streams[i]] > 0;
    }
    if (!any) return SDV2_OK;
    sdv2_status st = check_change(h, s);
    if (st != SDV2_OK) return st;
    Edits ed;
    ed.clears.reserve(n);
    ed.lengths.reserve(n);
    for (int32_t i = 0; i < n; ++i) {
        const int32_t b = streams[i];
        if (h->tokens[b] == 0) continue;
        ed.clears.emplace_back(b, h->n_pages[b]);
        ed.lengths.emplace_back(b, 0);
    }
    if ((st = ed.launch(h, h->version + 1, false, s)) != SDV2_OK) return st;
    for (const auto &x : ed.clears) {
        const int32_t b = x.first;
        for (int32_t j = 0; j < h->n_pages[b]; ++j) {
            h->drop(h->row(b)[j]);
            h->row(b)[j] = -1;
        }
        h->n_pages[b] = h->tokens[b] = 0;
    }
    changed(h);
    return SDV2_OK;
}

sdv2_status compact(sdv2_pages *h, int32_t *used, cudaStream_t s) {
    if (!h) return fail(SDV2_E_ARG, "pages is NULL");
    const sdv2_pages_config &c = h->cfg;
    if (used) *used = 0;
    bool any = false;
    for (int32_t p = h->used; p < c.pages && !any; ++p) any = h->users[p] > 0;
    if (!any) {
        if (used) *used = h->used;
        return check_whole(h);
    }
    sdv2_status st = check_change(h, s);
    if (st != SDV2_OK) return st;
    Edits ed;
    Moves mv;
    std::vector<int32_t> to(c.pages - h->used, -1);       // new place of page used + i
    for (int32_t p = h->used, hole = 0; p < c.pages; ++p) {
        if (h->users[p] == 0) continue;
        while (h->users[hole] != 0) ++hole;
        to[p - h->used] = hole++;
        mv.src.push_back(p);
        mv.dst.push_back({to[p - h->used]});
    }
    size_t entries = 0;
    for (int32_t p : mv.src) entries += h->users[p];
    ed.entries.reserve(entries);
    for (int32_t b = 0; b < c.streams; ++b)
        for (int32_t j = 0; j < h->n_pages[b]; ++j) {
            const int32_t p = h->row(b)[j];
            if (p >= h->used)
                ed.entries.emplace_back(static_cast<uint32_t>(static_cast<int64_t>(b) * c.stream_pages + j), to[p - h->used]);
        }
    if ((st = mv.launch(h, s)) != SDV2_OK || (st = ed.launch(h, h->version + 1, true, s)) != SDV2_OK) return st;
    for (const auto &x : ed.entries) h->table[x.first] = x.second;
    for (int32_t p : mv.src) {
        h->users[to[p - h->used]] = h->users[p];
        h->users[p] = 0;
    }
    h->first_free = h->used;
    changed(h);
    if (used) *used = h->used;
    return SDV2_OK;
}

template <typename F>
sdv2_status guarded(F f) {
    try {
        return f();
    } catch (...) {
        return fail(SDV2_E_STATE, "paged cache: out of host memory");
    }
}

void fill_layout(const sdv2_pages_config &c, sdv2_pages_layout *out) {
    const Regions r = regions(c);
    out->k_offset = r.k;
    out->v_offset = r.v;
    out->layer_stride = r.layer_stride;
    out->table_offset = r.table;
    out->length_offset = r.length;
    out->version_offset = r.version;
    out->status_offset = r.status;
    out->scratch_offset = r.scratch;
    out->scratch_bytes = r.end - r.scratch;
    out->total_bytes = r.end;
}

}  // namespace

extern "C" {

size_t sdv2_pages_bytes(const sdv2_pages_config *cfg) {
    return check_config(cfg) == SDV2_OK ? static_cast<size_t>(regions(*cfg).end) : 0;
}

sdv2_status sdv2_pages_layout_of(const sdv2_pages_config *cfg, sdv2_pages_layout *out) {
    if (!out) return fail(SDV2_E_ARG, "out is NULL");
    const sdv2_status st = check_config(cfg);
    if (st == SDV2_OK) fill_layout(*cfg, out);
    return st;
}

sdv2_status sdv2_pages_create(const sdv2_pages_config *cfg, void *dev_buf, size_t bytes, sdv2_pages **out) {
    return guarded([&] { return create(cfg, dev_buf, bytes, out); });
}

sdv2_status sdv2_pages_destroy(sdv2_pages *pages) {
    delete pages;
    return SDV2_OK;
}

sdv2_status sdv2_pages_extend(sdv2_pages *pages, const int32_t *counts, sdv2_stream stream) {
    return guarded([&] { return extend(pages, counts, reinterpret_cast<cudaStream_t>(stream)); });
}

sdv2_status sdv2_pages_write(sdv2_pages *pages, int32_t layer, const void *k, const void *v, int64_t k_stride,
                             int64_t v_stride, const int32_t *counts, sdv2_stream stream) {
    return guarded([&] {
        return write(pages, layer, k, v, k_stride, v_stride, counts, reinterpret_cast<cudaStream_t>(stream));
    });
}

sdv2_status sdv2_pages_attention(sdv2_pages *pages, int32_t layer, const void *q, void *out, int64_t q_stride,
                                 int64_t out_stride, const int32_t *counts, float softmax_scale, sdv2_stream stream) {
    return guarded([&] {
        return attention(pages, layer, q, out, q_stride, out_stride, counts, softmax_scale,
                         reinterpret_cast<cudaStream_t>(stream));
    });
}

sdv2_status sdv2_pages_fork(sdv2_pages *pages, int32_t src, const int32_t *dst, int32_t n, int32_t deep,
                            sdv2_stream stream) {
    return guarded([&] { return fork(pages, src, dst, n, deep, reinterpret_cast<cudaStream_t>(stream)); });
}

sdv2_status sdv2_pages_free(sdv2_pages *pages, const int32_t *streams, int32_t n, sdv2_stream stream) {
    return guarded([&] { return free_streams(pages, streams, n, reinterpret_cast<cudaStream_t>(stream)); });
}

sdv2_status sdv2_pages_compact(sdv2_pages *pages, int32_t *used, sdv2_stream stream) {
    return guarded([&] { return compact(pages, used, reinterpret_cast<cudaStream_t>(stream)); });
}

sdv2_status sdv2_pages_query(sdv2_pages *h, int32_t stream, int32_t *tokens, int32_t *page_ids, int32_t capacity,
                             int32_t *n_pages, int32_t *shared_pages) {
    if (!h) return fail(SDV2_E_ARG, "pages is NULL");
    if (stream < 0 || stream >= h->cfg.streams) return fail(SDV2_E_ARG, "stream %d out of range", stream);
    if (capacity < 0 || (capacity > 0 && !page_ids)) return fail(SDV2_E_ARG, "page_ids is NULL or capacity negative");
    return guarded([&] {
        know_groups(h);
        if (tokens) *tokens = h->tokens[stream];
        if (n_pages) *n_pages = h->n_pages[stream];
        if (shared_pages) *shared_pages = h->group_of[stream] >= 0 ? h->group_pages[h->group_of[stream]] : 0;
        if (page_ids) std::copy(h->row(stream), h->row(stream) + std::min(capacity, h->n_pages[stream]), page_ids);
        return SDV2_OK;
    });
}

sdv2_status sdv2_pages_share(sdv2_pages *pages, int32_t mode) {
    if (!pages) return fail(SDV2_E_ARG, "pages is NULL");
    if (mode != SDV2_SHARE_NEVER && mode != SDV2_SHARE_AUTO && mode != SDV2_SHARE_ALWAYS)
        return fail(SDV2_E_ARG, "mode must be SDV2_SHARE_NEVER, SDV2_SHARE_AUTO or SDV2_SHARE_ALWAYS");
    pages->share = mode;
    return SDV2_OK;
}

int32_t sdv2_pages_used(const sdv2_pages *pages) { return pages ? pages->used : -1; }

sdv2_status sdv2_pages_layout_get(const sdv2_pages *pages, sdv2_pages_layout *out) {
    if (!pages || !out) return fail(SDV2_E_ARG, "NULL argument");
    fill_layout(pages->cfg, out);
    return SDV2_OK;
}

sdv2_status sdv2_pages_check(sdv2_pages *h) {
    if (!h) return fail(SDV2_E_ARG, "pages is NULL");
    const sdv2_status st = check_device(h->device);
    if (st != SDV2_OK) return st;
    cudaError_t e = cudaDeviceSynchronize();
    uint32_t word = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&word, h->base + h->r.status, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && word != 0) e = cudaMemset(h->base + h->r.status, 0, 4);
    if (e == cudaSuccess && word != 0) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "pages_check");
    if (word & kStatusStale)
        return fail(SDV2_E_DEVICE, "device status 0x%x (a captured call was replayed after a fork, free or compact)", word);
    if (word != 0) return fail(SDV2_E_DEVICE, "device status 0x%x (a kernel gave up on a bounded wait)", word);
    return SDV2_OK;
}

}  // extern "C"
