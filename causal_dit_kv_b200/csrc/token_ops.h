// Internal declarations of the token-sequence operators: prompt attention (prompt.cu,
// host_prompt.cpp) and the paged cache (pages.cu, pages_attention.cu, host_pages.cpp).
// Nothing here is part of the public C ABI.
#pragma once

#include "sdv2_internal.h"

namespace sdv2 {

// ---------------------------------------------------------------- prompt attention
constexpr int kPromptMaxSeqs = 256;       // sequences of one launch (a call takes as many launches as it needs)
constexpr int kPromptSmallItems = 256;    // items of the small and of the large parameter block
constexpr int kPromptLargeItems = 6000;

// Work units (item, j), j < head_units.  pair_heads: unit j is query heads 2j and 2j + 1
// (one key head) on the item's 128 rows; otherwise head j on the item's 256 rows.
template <int kItems>
struct PromptParams {
    uint16_t *out;
    int64_t out_stride;                   // elements between tokens
    int32_t group, block, pair_heads, head_units, n_items, n_units;
    int32_t chunk_units;                  // head units whose items are done before the next ones'
    float scale_log2;                     // softmax_scale * log2(e)
    int32_t seq_first[kPromptMaxSeqs];    // first token and tokens of each sequence
    int32_t seq_len[kPromptMaxSeqs];
    uint32_t item[kItems];                // sequence << 24 | row tile, longest first
};

template <int kItems>
cudaError_t launch_prompt(const PromptParams<kItems> &p, const CUtensorMap &tq, const CUtensorMap &tk,
                          const CUtensorMap &tv, int head_dim, bool half, cudaStream_t s);
// Reads and clears the device word in which the prompt kernels record waits that ran out.
cudaError_t prompt_status(uint32_t *word);

// ---------------------------------------------------------------- paged cache
constexpr int kPagesMaxStreams = 256;
constexpr int kPagesMaxCtas = 160;        // attention CTAs of one launch, at most (scratch is sized for them)
constexpr int kRowWarps = 8;              // warps of an SM in the few-row kernel, each a worker of its own
constexpr int kRowsPerWorker = 16;        // query rows that one of them takes, at most
constexpr int kRowKeysLog2 = 4, kTileKeysLog2 = 7;   // keys of a tile of the few-row and of the tile kernel

// Status bits of the paged cache's word besides the waits of sdv2_internal.h.
constexpr uint32_t kStatusStale = 1u << 5;   // a replayed call whose tables have been forked, freed or compacted since

// Device state that every kernel of a handle takes.
struct PagesView {
    int32_t *table;                       // [streams][width], -1 behind a stream's pages
    int32_t *lengths;                     // [streams]
    uint32_t *version;                    // and the version that the call was made for
    uint32_t *status;
    uint32_t expect;
    int32_t width, pages, kv_heads, page_log2, head_dim;
};

// Edits of the tables: rows copied (entries 0 .. n - 1 of a stream's row to another's), row
// ends set to -1, entries and lengths set.  One launch's edits touch different entries.
template <int kEntries, int kRows>
struct PageEdits {
    int32_t *table, *lengths;
    uint32_t *version;
    uint32_t new_version;
    int32_t width, n_copies, n_clears, n_entries, n_lengths;
    int32_t copy[kRows][3];               // from, to, entries
    int32_t clear[kRows][2];              // stream, entries
    uint32_t entry_at[kEntries];
    int32_t entry[kEntries];
    int32_t length[kRows][2];             // stream, tokens
};

// Pages copied in every layer: source i goes to dst[first[i] .. first[i + 1] - 1].
template <int kMoves>
struct PageMoves {
    uint8_t *base[2];                     // keys and values
    int64_t layer_stride, page_bytes;
    int32_t layers, n;
    int32_t src[kMoves];
    int32_t first[kMoves + 1];
    int32_t dst[kMoves];
};

// New tokens' keys and values: token x of the call belongs to active stream i with
// first[i] <= x < first[i + 1].
struct PageWriteParams {
    PagesView v;
    const uint16_t *in[2];
    uint16_t *out[2];                     // this layer's keys and values
    int64_t stride[2];
    int32_t n;
    int32_t stream[kPagesMaxStreams];
    int32_t first[kPagesMaxStreams + 1];
};

// One part of the attention's work: the keys of a group's common pages with the queries of
// all its streams, or a stream's remaining keys with its own queries.  Units (row tile,
// key head) of `tiles` KV tiles each, numbered row tile first.
struct alignas(32) PageSection {
    int32_t tiles;
    int32_t stream;                       // whose table row names the pages
    int32_t page0;                        // first page of the keys
    int32_t keys;                         // common pages: their tokens; a stream's own: -1 (up to its length)
    int32_t token0, n_tokens;             // queries: packed tokens (own keys), or places in the groups' token order
    int32_t common, common_token;         // own keys: section of the common pages (-1: none), the first query's place there
};

// One launch's work: sections [begin, end).  Each unit takes `setup` places, for what a run costs
// before and after its tiles, then one place per tile of 1 << tile_log2 keys; the units' places,
// end to end, are cut evenly into `workers` runs (places x workers < 2^32).  A run that ends
// within a unit's setup places leaves the unit to the next worker.  A unit's later pieces leave
// their rows at partial row cut_row + worker * cut_rows.
struct PageWork {
    int32_t begin, end, workers, setup, tile_log2, tile_tokens, cut_row, cut_rows;
    uint32_t places;
    int32_t rows;                         // most query rows of a unit
};

template <int kSections, int kMembers>
struct PagesAttnParams {
    PagesView v;
    const uint16_t *q;
    uint16_t *out;
    const uint16_t *k_layer, *v_layer;
    int64_t q_stride, out_stride;
    float *part_o;                        // [rows][d] unnormalised partial outputs
    float2 *part_ml;                      // [rows] (row maximum in log2 units, row sum)
    int32_t rows_common;                  // first partial row of the common pages' pieces
    int32_t heads, group, block;
    int32_t n_sections, n_common, n_queries;
    float scale_log2;
    PageWork common, own;                 // the launches that take the common pages' sections and the streams'
    // groups' token order: member i is packed tokens member_token[i] .., at places member_first[i] ..
    int32_t n_members;
    int32_t tokens_each;                  // query tokens of every member, if they are all alike (0: they are not)
    int32_t member_first[kMembers];
    int32_t member_token[kMembers];
    // a section's first place among its launch's, apart from the rest: a search reads few lines of it
    int32_t start[kSections];
    PageSection section[kSections];       // the groups' common pages, then the streams by their packed tokens
};

constexpr int kSmallSections = 40, kSmallMembers = 40;
constexpr int kLargeSections = kPagesMaxStreams + kPagesMaxStreams / 2, kLargeMembers = kPagesMaxStreams;

template <int kEntries, int kRows>
cudaError_t launch_page_edits(const PageEdits<kEntries, kRows> &e, bool beside, cudaStream_t s);
template <int kMoves>
cudaError_t launch_page_moves(const PageMoves<kMoves> &m, cudaStream_t s);
cudaError_t launch_page_write(const PageWriteParams &p, cudaStream_t s);
// The work w of a call by 128-row tiles on the tensor cores' own kernel (tiles of 128 keys),
// or by at most kRowsPerWorker rows of one warp each (tiles of 16 keys); work cut for the other
// kernel is refused (cudaErrorInvalidValue).  `beside`: the launch
// before it in the stream is the same call's other one, which it need not wait for to begin.
template <int kSections, int kMembers>
cudaError_t launch_pages_tiles(const PagesAttnParams<kSections, kMembers> &p, const PageWork &w, const CUtensorMap &tk,
                               const CUtensorMap &tv, bool half, cudaStream_t s);
template <int kSections, int kMembers>
cudaError_t launch_pages_rows(const PagesAttnParams<kSections, kMembers> &p, const PageWork &w, bool half, bool beside,
                              int sm_count, cudaStream_t s);
template <int kSections, int kMembers>
cudaError_t launch_pages_merge(const PagesAttnParams<kSections, kMembers> &p, int warps_per_row, bool half,
                               cudaStream_t s);

}  // namespace sdv2
