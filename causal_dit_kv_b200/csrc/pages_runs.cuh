// How the paged attention's work is cut: the run of tiles that a worker (a CTA of the
// tile kernel, a warp of the row kernel) takes within one unit, and where partial results go.
// (Plain integer code: a test of the host's plans compiles it for the CPU.)
#pragma once

#include "token_ops.h"

namespace sdv2 {

struct PagesRun {
    int sec, row_tile, head;     // section, row tile, key head
    int n_rows;                  // query rows of the tile
    int begin, n;                // first KV tile of the run in the unit, tiles (0: nothing to read)
    int keys;                    // keys of the unit's page range (they end inside its last tile)
    int base;                    // place in the stream of its first key
    int len;                     // tokens of the stream (common keys: 0, not needed)
    int piece;                   // which piece of the unit this is (0: its first)
    int whole, common;           // the unit's only piece; keys of common pages
};

// First place of a worker's run, and the worker of a place: the last one whose run begins at or
// before it.
__device__ __forceinline__ uint32_t first_place(const PageWork &w, uint32_t worker) {
    return worker * w.places / w.workers;
}
__device__ __forceinline__ int worker_of(const PageWork &w, uint32_t place) {
    return static_cast<int>(((place + 1) * w.workers - 1) / w.places);
}

// Where a run lies, from the launch's parameters alone.
struct RunSpot {
    int sec, unit, at, taken, first;   // section, its unit, the run's first place in the unit, places, the unit's first place
};

// The next run of a worker from place *pos on, *pos moved behind it; false if there is none
// before `end`.
template <int kS, int kM>
__device__ __forceinline__ bool next_spot(const PagesAttnParams<kS, kM> &p, const PageWork &w, int *pos, int end, RunSpot *out) {
    while (*pos < end) {
        int lo = w.begin, hi = w.end;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.start[mid] <= *pos)
                lo = mid;
            else
                hi = mid;
        }
        const int span = p.section[lo].tiles + w.setup, in = *pos - p.start[lo];
        RunSpot s;
        s.sec = lo;
        s.unit = in / span;
        s.at = in - s.unit * span;
        s.taken = min(span - s.at, end - *pos);
        s.first = *pos - s.at;
        *pos += s.taken;
        if (s.at + s.taken <= w.setup) continue;         // the next worker's
        *out = s;
        return true;
    }
    return false;
}

// The run at a spot, with the stream's length as it is now (common keys: from the launch's parameters
// alone).
template <int kS, int kM>
__device__ __forceinline__ PagesRun run_at(const PagesAttnParams<kS, kM> &p, const PageWork &w, int worker, const RunSpot &o) {
    const PageSection &s = p.section[o.sec];
    PagesRun r;
    r.sec = o.sec;
    r.row_tile = o.unit / p.v.kv_heads;
    r.head = o.unit - r.row_tile * p.v.kv_heads;
    r.common = s.keys >= 0;
    r.base = s.page0 << p.v.page_log2;
    r.len = r.common ? 0 : p.v.lengths[s.stream];
    const int tokens = min(w.tile_tokens, s.n_tokens - r.row_tile * w.tile_tokens);
    r.n_rows = tokens * p.group;
    r.keys = r.common ? s.keys : r.len - r.base;
    // KV tiles that the tile's rows see: all of the common keys, or up to its last token's
    int seen = r.keys;
    if (!r.common) {
        const int last = r.len - s.n_tokens + r.row_tile * w.tile_tokens + tokens - 1;
        seen = min(r.len, (last / p.block + 1) * p.block) - r.base;
    }
    const int tiles = (seen + (1 << w.tile_log2) - 1) >> w.tile_log2;
    // (the unit's last piece takes what a longer stream has grown since the work was cut)
    const bool last_piece = o.at + o.taken == s.tiles + w.setup;
    r.begin = max(0, o.at - w.setup);
    r.n = max(0, (last_piece ? tiles : min(tiles, o.at + o.taken - w.setup)) - r.begin);
    r.piece = o.at <= w.setup ? 0 : worker - worker_of(w, o.first + w.setup);
    r.whole = r.piece == 0 && last_piece;
    return r;
}

// Packed token of the `place`-th query token of a section.
template <int kS, int kM>
__device__ __forceinline__ int query_token(const PagesAttnParams<kS, kM> &p, const PageSection &s, int place) {
    if (s.keys < 0) return s.token0 + place;
    const int x = s.token0 + place;
    if (p.tokens_each > 0) {
        const int i = x / p.tokens_each;
        return p.member_token[i] + x - i * p.tokens_each;
    }
    int lo = 0, hi = p.n_members;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.member_first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return p.member_token[lo] + x - p.member_first[lo];
}

// Partial row of the run's tile row `row`, whose output row is out_row.
template <int kS, int kM>
__device__ __forceinline__ int64_t partial_row(const PagesAttnParams<kS, kM> &p, const PageWork &w, const PagesRun &r,
                                               int worker, int row, int64_t out_row) {
    return r.piece > 0 ? w.cut_row + static_cast<int64_t>(worker) * w.cut_rows + row
                       : (r.common ? p.rows_common : 0) + out_row;
}

}  // namespace sdv2
