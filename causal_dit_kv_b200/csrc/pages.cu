// The paged cache's table edits, page copies and writes.
//
// Table edits: a few integers, carried in the launch's parameters, so that tables change
// in stream order without a host copy.  Bound by the launch; beside a call's page copies they
// cost nothing of their own (a fork into 16 streams of 65 pages: 37.8 us with both, 42 in a row).
//
// Page copies: every page is one contiguous block per layer and side (keys, values), all
// heads together; a block of threads takes 16 KB of it, reads that once and writes it to
// every destination, so a fork into n streams reads its source once.  Bound by HBM: 16 copies of one
// page of 30 layers (12 MB read, 189 written) 32 us; two calls that each move 32 such pages to the
// front (1510 MB) 234.5 us with the calls around them, 99 % of the measured copy rate.
//
// Writes: one warp per new token; it looks up the token's stream, page and place once
// and moves the token's keys and values, 16 bytes a lane.  Bound by HBM: 8192 tokens of 40 heads
// of 128 (336 MB moved) 56 to 57 us, 5.9 TB/s; for a step's few tokens by the call: 64 tokens of 8
// heads 8.7 to 9.2 us.
#include "ptx.cuh"
#include "token_ops.h"

namespace sdv2 {

template <int kEntries, int kRows>
__global__ void __launch_bounds__(256)
    page_edits_kernel(const __grid_constant__ PageEdits<kEntries, kRows> e, const bool beside) {
    // The launch before may be the same call's page copies, which had waited for everything before
    // them when they let this one start: only the end of this grid has to come after theirs.
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
    const int i0 = blockIdx.x * blockDim.x + threadIdx.x, n = gridDim.x * blockDim.x;
    for (int c = 0; c < e.n_copies; ++c) {
        const int32_t *from = e.table + static_cast<int64_t>(e.copy[c][0]) * e.width;
        int32_t *to = e.table + static_cast<int64_t>(e.copy[c][1]) * e.width;
        for (int i = i0; i < e.copy[c][2]; i += n) to[i] = from[i];
    }
    for (int c = 0; c < e.n_clears; ++c) {
        int32_t *row = e.table + static_cast<int64_t>(e.clear[c][0]) * e.width;
        for (int i = i0; i < e.clear[c][1]; i += n) row[i] = -1;
    }
    for (int i = i0; i < e.n_entries; i += n) e.table[e.entry_at[i]] = e.entry[i];
    for (int i = i0; i < e.n_lengths; i += n) e.lengths[e.length[i][0]] = e.length[i][1];
    if (i0 == 0) *e.version = e.new_version;
    if (beside) grid_dependency_wait();
}

template <int kEntries, int kRows>
cudaError_t launch_page_edits(const PageEdits<kEntries, kRows> &e, bool beside, cudaStream_t s) {
    const int blocks = e.n_copies > 16 ? 16 : 1;
    return launch_dependent(page_edits_kernel<kEntries, kRows>, dim3(blocks), dim3(256), 0, s, e, beside);
}

constexpr int kMoveChunk = 16384;         // bytes of a page that one block copies: 256 threads x 4 x 16

template <int kMoves>
__global__ void __launch_bounds__(256) page_moves_kernel(const __grid_constant__ PageMoves<kMoves> m, int chunks) {
    grid_dependency_wait();
    grid_launch_dependents();
    int b = blockIdx.x;
    const int chunk = b % chunks;
    b /= chunks;
    const int side = b & 1;
    b >>= 1;
    const int layer = b % m.layers, i = b / m.layers;
    uint8_t *base = m.base[side] + static_cast<int64_t>(layer) * m.layer_stride;
    const int64_t off = static_cast<int64_t>(chunk) * kMoveChunk + threadIdx.x * 16;
    const uint8_t *src = base + static_cast<int64_t>(m.src[i]) * m.page_bytes + off;
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (off + k * 4096 < m.page_bytes) x[k] = *reinterpret_cast<const uint4 *>(src + k * 4096);
    for (int j = m.first[i]; j < m.first[i + 1]; ++j) {
        uint8_t *dst = base + static_cast<int64_t>(m.dst[j]) * m.page_bytes + off;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (off + k * 4096 < m.page_bytes) *reinterpret_cast<uint4 *>(dst + k * 4096) = x[k];
    }
}

template <int kMoves>
cudaError_t launch_page_moves(const PageMoves<kMoves> &m, cudaStream_t s) {
    const int chunks = static_cast<int>((m.page_bytes + kMoveChunk - 1) / kMoveChunk);
    const int64_t blocks = static_cast<int64_t>(m.n) * m.layers * 2 * chunks;
    return launch_dependent(page_moves_kernel<kMoves>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, m, chunks);
}

__global__ void __launch_bounds__(128) page_write_kernel(const __grid_constant__ PageWriteParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int x = blockIdx.x * 4 + (threadIdx.x >> 5);     // token of the call
    if (x >= p.first[p.n]) return;
    if (*p.v.version != p.v.expect) {
        if (x == 0 && lane == 0) atomicOr(p.v.status, kStatusStale);
        return;
    }
    int lo = 0, hi = p.n;                                  // first[lo] <= x < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    const int stream = p.stream[lo];
    const int at = p.v.lengths[stream] - (p.first[lo + 1] - x);   // place in the stream
    const int idx = at >> p.v.page_log2;
    if (at < 0 || idx >= p.v.width) return;
    const int page = p.v.table[static_cast<int64_t>(stream) * p.v.width + idx];
    if (page < 0 || page >= p.v.pages) return;
    const int d8 = p.v.head_dim >> 3;                      // 16-byte vectors of a head
    const int shift = d8 == 16 ? 4 : 3;
    const int total = p.v.kv_heads * d8;
    const int64_t head_step = static_cast<int64_t>(d8) << p.v.page_log2;   // vectors between a page's heads
    const int64_t dst0 = static_cast<int64_t>(page) * p.v.kv_heads * head_step +
                         static_cast<int64_t>(at & ((1 << p.v.page_log2) - 1)) * d8;
    const uint4 *ks = reinterpret_cast<const uint4 *>(p.in[0] + static_cast<int64_t>(x) * p.stride[0]);
    const uint4 *vs = reinterpret_cast<const uint4 *>(p.in[1] + static_cast<int64_t>(x) * p.stride[1]);
    uint4 *kd = reinterpret_cast<uint4 *>(p.out[0]) + dst0, *vd = reinterpret_cast<uint4 *>(p.out[1]) + dst0;
    for (int i0 = lane; i0 < total; i0 += 128) {
        uint4 a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + 32 * k < total) {
                a[k] = ks[i0 + 32 * k];
                b[k] = vs[i0 + 32 * k];
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k;
            if (i < total) {
                const int64_t o = (i >> shift) * head_step + (i & (d8 - 1));
                kd[o] = a[k];
                vd[o] = b[k];
            }
        }
    }
}

cudaError_t launch_page_write(const PageWriteParams &p, cudaStream_t s) {
    return launch_dependent(page_write_kernel, dim3(static_cast<unsigned>((p.first[p.n] + 3) / 4)), dim3(128), 0, s, p);
}

template cudaError_t launch_page_edits<64, 32>(const PageEdits<64, 32> &, bool, cudaStream_t);
template cudaError_t launch_page_edits<2000, 256>(const PageEdits<2000, 256> &, bool, cudaStream_t);
template cudaError_t launch_page_moves<64>(const PageMoves<64> &, cudaStream_t);
template cudaError_t launch_page_moves<2000>(const PageMoves<2000> &, cudaStream_t);

}  // namespace sdv2
