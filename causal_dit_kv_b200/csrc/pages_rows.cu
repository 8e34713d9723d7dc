// Paged attention for at most 16 query rows per key head (single tokens and a few), and the
// merge of partial results.
//
// With so few rows the only cost that counts is reading K and V once, at HBM's rate.  Every
// warp is a worker of its own: it takes an equal run of 16-key tiles and needs no other
// warp, so eight runs per SM overlap their starts, ends and dependent chains (one CTA-wide
// pipeline paid about 8000 cycles at each change of unit).
//
// Tensor-core products of 16 x 8 x 16 (mma.sync: the tcgen05 kind's smallest tile has 64 rows,
// of which these calls fill 1 to 16), transposed so that keys and channels fill the 16 and the
// query rows the 8: S^T = K Q^T, O^T = V^T P^T.  The order of the channels inside q . k and of
// the rows of O^T is free, so each lane's operands are whole 16-byte pieces of K and V rows:
// lane (g, c) = (lane / 4, lane % 4) takes channels 32 j + 8 c .. + 7 of keys g and g + 8 for the
// scores, and channels 64 j + 8 g .. + 7 of keys 2c, 2c + 1, 2c + 8, 2c + 9 for the output.  P^T
// comes from S^T by transposing 8 x 8 blocks across the lanes.
// A tile's 16 keys are contiguous in their page; the warp copies them in 512-byte pieces (cp.async,
// kStages tiles ahead) to rows whose 16-byte pieces are permuted by the key, so that neither the
// copies nor both kinds of operand reads meet bank conflicts.  (Copies of just what each lane will
// use, which would need no permutation, ran at 4.5 TB/s: they touch twice the lines.)
// A row's running maximum is agreed on by all its lanes only when one of
// them sees a score over it by more than 2^8, so an ordinary tile has one vote and no reduction.
// Keys past the range are copied as zeros and their scores masked.
//
// 32 streams of 500 to 8000 keys, 32/8 heads of 128, bf16: 604 MB in 97 to 98.5 us with the merge, 6.1 TB/s;
// one stream of 1000 keys, 12 heads: 7.6 to 8.0 us, of which two launches and a run's chain of copies are
// nearly all.
#include <algorithm>
#include <atomic>

#include "attn_core.cuh"
#include "pages_runs.cuh"

namespace sdv2 {

template <int D>
struct RowsLayout {
    static constexpr int kCopies = D / 8;                 // 512-byte pieces of a tile: D / 16 of K, D / 16 of V
    static constexpr int kPerCopy = 256 / D;              // keys in each
    static constexpr int kTile = kCopies * 512;           // bytes of a tile
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kAlloc = kRowWarps / 2 * kStages * kTile;
    static_assert(2 * (kAlloc + 1024) <= 233472, "two CTAs to an SM");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
    return x;
}

// c += a (16 x 16) b (16 x 8), 16-bit operands, fp32 accumulators.
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 block of 16-bit values, row g and columns 2c, 2c + 1 in lane (g, c), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// N: blocks of 8 query rows (1 or 2).
template <int D, bool HALF, int N, int kS, int kM>
__global__ void __launch_bounds__(kRowWarps / 2 * 32, 2)
    pages_rows_kernel(const __grid_constant__ PagesAttnParams<kS, kM> p, const __grid_constant__ PageWork work,
                      const bool beside) {
    using L = RowsLayout<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int worker = blockIdx.x * (blockDim.x >> 5) + warp;
    int pos = 0, end = 0;
    if (worker < work.workers) {
        pos = static_cast<int>(first_place(work, worker));
        end = static_cast<int>(first_place(work, worker + 1));
    }
    RunSpot spot;
    bool more = next_spot(p, work, &pos, end, &spot);
    // The launch before is the same call's other half, which had waited for everything before it
    // when it let this one start: only the end of this grid has to come after its end.
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
    const bool stale = *p.v.version != p.v.expect;       // (looked at before anything is written)
    const int page_log2 = p.v.page_log2;
    // Piece x (16 bytes) of key y's row lies at place x ^ swizzle(y), swizzle(y) = (y & 6) ^ ((y & 1) << 2):
    // lanes of one access with keys 2i, 2i + 1 and four pieces each, or with two pieces of keys 2c,
    // take eight different places.
    const uint32_t stage0 = smem_addr(smem) + warp * (L::kStages * L::kTile);
    const int my_key = lane / (D / 8);                   // of a copy's kPerCopy keys
    const uint32_t my_piece = (lane & (D / 8 - 1)) ^ (my_key & 2) ^ ((my_key & 1) << 2);
    const uint32_t copy_to = stage0 + my_key * (D * 2);
    const uint32_t k_place = c ^ ((g & 6) ^ ((g & 1) << 2)), v_place = g ^ (2 * c);
    for (; more; more = next_spot(p, work, &pos, end, &spot)) {
        const PagesRun r = run_at(p, work, worker, spot);
        const PageSection &s = p.section[r.sec];

        // ---- copies: page ids of the run, 32 at a time, the next 32 in flight (not waiting for the
        // stream's length: entries behind its pages are -1)
        const int key0 = r.begin * 16;                   // first key of the run in the range
        int batch = key0 >> page_log2;
        const int32_t *row_ids = p.v.table + static_cast<int64_t>(s.stream) * p.v.width;
        const int last_id = p.v.width - 1 - s.page0;
        row_ids += s.page0;
        int ids = row_ids[min(batch + lane, last_id)];
        int ids_next = row_ids[min(batch + 32 + lane, last_id)];
        const int64_t page_elems = (static_cast<int64_t>(p.v.kv_heads) << page_log2) * D;
        const int64_t head_off = (static_cast<int64_t>(r.head) << page_log2) * D;
        const uint16_t *k_lane = p.k_layer + head_off + lane * 8, *v_lane = p.v_layer + head_off + lane * 8;
        uint32_t fill = 0;                               // offset of the stage that the next copies go to
        auto issue = [&](int tile) {                     // (tiles in order)
            if (tile < r.n) {
                const int key = key0 + tile * 16, index = key >> page_log2;
                if (index - batch >= 32) {
                    batch += 32;
                    ids = ids_next;
                    ids_next = row_ids[min(batch + 32 + lane, last_id)];
                }
                int id = __shfl_sync(0xffffffffu, ids, index - batch);
                id = min(max(id, 0), p.v.pages - 1);     // (the table lies in the caller's buffer)
                const int64_t off = id * page_elems + (key & ((1 << page_log2) - 1)) * D;
                const int there = r.keys - key;          // keys of the tile that there are
                const uint16_t *ks = k_lane + off, *vs = v_lane + off;
#pragma unroll
                for (int k = 0; k < L::kCopies / 2; ++k) {   // keys kPerCopy k + my_key, of K and of V
                    const uint32_t dst = copy_to + fill + k * 512 + ((my_piece ^ (L::kPerCopy * k & 6)) << 4);
                    const uint32_t bytes = L::kPerCopy * k + my_key < there ? 16u : 0u;
                    copy16(dst, ks + k * 256, bytes);
                    copy16(dst + L::kTile / 2, vs + k * 256, bytes);
                }
                fill = fill == (L::kStages - 1) * L::kTile ? 0 : fill + L::kTile;
            }
            copies_commit();
        };

        // ---- queries: row g of each block of 8 as the B operand of the scores
        uint4 q[N][D / 32];
#pragma unroll
        for (int b = 0; b < N; ++b) {
            const int row = 8 * b + g;
            const bool there = row < r.n_rows;
            const int place = there ? row / p.group : 0;
            const uint16_t *src = p.q + static_cast<int64_t>(query_token(p, s, place)) * p.q_stride +
                                  (r.head * p.group + (there ? row - place * p.group : 0)) * D + 8 * c;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                q[b][j] = there ? *reinterpret_cast<const uint4 *>(src + 32 * j) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < L::kStages - 1; ++i) issue(i);
        // keys that rows 8 b + 2 c + x see, from the range's first; all rows see those below `all`
        int seen[N][2];
        int all = r.keys;
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                seen[b][x] = r.keys;
                const int row = 8 * b + 2 * c + x;
                if (!r.common && row < r.n_rows) {
                    const int at = r.len - s.n_tokens + row / p.group;
                    seen[b][x] = min(r.len, (at / p.block + 1) * p.block) - r.base;
                }
            }
        if (!r.common) all = min(r.len, ((r.len - s.n_tokens) / p.block + 1) * p.block) - r.base;

        float m[N][2], l[N][2];                          // running maxima (in log2 units), sums of this lane's keys
        float o[N][D / 16][4];
#pragma unroll
        for (int b = 0; b < N; ++b) {
            m[b][0] = m[b][1] = -INFINITY;
            l[b][0] = l[b][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[b][j][i] = 0.0f;
        }
        uint32_t take = 0;                               // offset of the stage that holds tile `it`
        for (int it = 0; it < r.n; ++it) {
            copies_wait<L::kStages - 2>();
            __syncwarp();                                // the lanes' copies are all there; the stage before is read
            const uint32_t ks = stage0 + take + g * (D * 2), vs = stage0 + take + L::kTile / 2 + c * (4 * D);
            take = take == (L::kStages - 1) * L::kTile ? 0 : take + L::kTile;
            // S^T: keys g, g + 8 of rows 2c, 2c + 1; two chains, added at the end
            float sc[N][2][4];
#pragma unroll
            for (int b = 0; b < N; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[b][0][i] = sc[b][1][i] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint32_t at = ks + (j >> 1) * 128 + ((k_place ^ (4 * (j & 1))) << 4);
                const uint4 k0 = lds16(at), k1 = lds16(at + 8 * (D * 2));
#pragma unroll
                for (int b = 0; b < N; ++b) {
                    mma16816<HALF>(sc[b][0], k0.x, k1.x, k0.y, k1.y, q[b][j].x, q[b][j].y);
                    mma16816<HALF>(sc[b][1], k0.z, k1.z, k0.w, k1.w, q[b][j].z, q[b][j].w);
                }
            }
            uint32_t pt[N][2];                           // P^T: keys 2c, 2c + 1 (and + 8) of row g
#pragma unroll
            for (int b = 0; b < N; ++b) {
                float x[4];                              // [key g, g + 8][row 2c, 2c + 1]
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = (sc[b][0][i] + sc[b][1][i]) * p.scale_log2;
                if (key0 + it * 16 + 16 > all) {         // a key here is not every row's
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key0 + it * 16 + g + 8 * (i >> 1) >= seen[b][i & 1]) x[i] = -INFINITY;
                }
                const float m0 = fmaxf(x[0], x[2]), m1 = fmaxf(x[1], x[3]);
                if (__any_sync(0xffffffffu, m0 > m[b][0] + kCoreRescale || m1 > m[b][1] + kCoreRescale)) {
                    float t[2] = {m0, m1};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) t[i] = fmaxf(t[i], __shfl_xor_sync(0xffffffffu, t[i], d));
                        t[i] = fmaxf(t[i], m[b][i]);
                        const float alpha = m[b][i] == -INFINITY ? 0.0f : ex2_approx(m[b][i] - t[i]);
                        m[b][i] = t[i];
                        l[b][i] *= alpha;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[b][j][i] *= alpha;
                            o[b][j][2 + i] *= alpha;
                        }
                    }
                }
                const float r0 = m[b][0] == -INFINITY ? 0.0f : m[b][0], r1 = m[b][1] == -INFINITY ? 0.0f : m[b][1];
                const float p0 = ex2_approx(x[0] - r0), p1 = ex2_approx(x[1] - r1);
                const float p2 = ex2_approx(x[2] - r0), p3 = ex2_approx(x[3] - r1);
                l[b][0] += p0 + p2;
                l[b][1] += p1 + p3;
                pt[b][0] = transpose8(pack_16x2<HALF>(p0, p1));
                pt[b][1] = transpose8(pack_16x2<HALF>(p2, p3));
            }
            // O^T: V of keys 2c, 2c + 1 and 2c + 8, 2c + 9, pairs of keys packed per channel
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)             // keys 2c + (k & 1) + 8 (k / 2)
                    v[k] = lds16(vs + ((k & 1) + 8 * (k >> 1)) * (D * 2) + j * 128 + ((v_place ^ (4 * (k & 1))) << 4));
                const uint32_t *a = &v[0].x, *b = &v[1].x, *e = &v[2].x, *f = &v[3].x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = __byte_perm(a[i], b[i], 0x5410), a1 = __byte_perm(a[i], b[i], 0x7632);
                    const uint32_t a2 = __byte_perm(e[i], f[i], 0x5410), a3 = __byte_perm(e[i], f[i], 0x7632);
#pragma unroll
                    for (int n = 0; n < N; ++n) mma16816<HALF>(o[n][4 * j + i], a0, a1, a2, a3, pt[n][0], pt[n][1]);
                }
            }
            issue(it + L::kStages - 1);
        }
        copies_wait<0>();

        // ---- results: o[b][4 j + i][2 y + x] is channel 64 j + 8 g + 2 i + y of row 8 b + 2 c + x
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[b][x] += __shfl_xor_sync(0xffffffffu, l[b][x], d);
                const int row = 8 * b + 2 * c + x;
                if (row >= r.n_rows || stale) continue;
                const int place = row / p.group, head = r.head * p.group + row - place * p.group;
                const int token = query_token(p, s, place);
                if (r.whole && !r.common && s.common < 0) {
                    const float inv = 1.0f / l[b][x];
                    uint16_t *orow = p.out + static_cast<int64_t>(token) * p.out_stride + head * D + 8 * g;
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        uint32_t y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] = pack_16x2<HALF>(o[b][4 * j + i][x] * inv, o[b][4 * j + i][2 + x] * inv);
                        *reinterpret_cast<uint4 *>(orow + 64 * j) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                } else {
                    const int64_t part = partial_row(p, work, r, worker, row, static_cast<int64_t>(token) * p.heads + head);
                    if (r.n > 0) {
                        float *prow = p.part_o + part * D + 8 * g;
#pragma unroll
                        for (int j = 0; j < D / 64; ++j)
#pragma unroll
                            for (int i = 0; i < 4; i += 2)
                                *reinterpret_cast<float4 *>(prow + 64 * j + 2 * i) =
                                    make_float4(o[b][4 * j + i][x], o[b][4 * j + i][2 + x], o[b][4 * j + i + 1][x],
                                                o[b][4 * j + i + 1][2 + x]);
                    }
                    if (g == 0) p.part_ml[part] = make_float2(m[b][x], l[b][x]);
                }
            }
    }
    if (stale && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.v.status, kStatusStale);
    if (beside) grid_dependency_wait();
}

// Merge of the partial results.  A row's parts are the pieces of its unit of the stream's own keys
// and of its unit of the group's common keys; out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.
// kW warps take a row (token, head), each every kW-th part: the pieces' (m, l) are read by the lanes
// at once, then the parts' rows, four in flight; the warps' results meet in shared memory.  A
// long sequence of few heads is cut into a hundred pieces, which one warp took 17 us to read.
template <int D, bool HALF, int kW, int kS, int kM>
__global__ void __launch_bounds__(256) pages_merge_kernel(const __grid_constant__ PagesAttnParams<kS, kM> p) {
    // (what the launch's parameters say is worked out before the partial results are there)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kW;
    const uint32_t n_rows = static_cast<uint32_t>(p.n_queries) * p.heads;
    // (warps past the last row work on it too, and do not write)
    const uint32_t my_row = blockIdx.x * (8 / kW) + warp / kW, out_row = min(my_row, n_rows - 1);
    const int token = out_row / p.heads, head = out_row - token * p.heads;
    int lo = p.n_common, hi = p.n_sections;              // the section of the stream's own keys
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.section[mid].token0 <= token)
            lo = mid;
        else
            hi = mid;
    }
    // pieces of the row's unit in both sections: their number, the row of a later one
    int n[2] = {0, 0};
    int64_t cut[2] = {0, 0};
    const int own = lo, common = p.section[lo].common;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 1 && common < 0) continue;
        const PageWork &w = k ? p.common : p.own;
        const PageSection &s = p.section[k ? common : own];
        const int place = k ? p.section[own].common_token + token - p.section[own].token0 : token - s.token0;
        const int rt = place / w.tile_tokens;
        const uint32_t a = p.start[k ? common : own] + (rt * p.v.kv_heads + head / p.group) * (s.tiles + w.setup) + w.setup;
        const int first = worker_of(w, a);
        n[k] = worker_of(w, a + s.tiles - 1) - first + 1;
        cut[k] = w.cut_row + static_cast<int64_t>(first) * w.cut_rows + (place - rt * w.tile_tokens) * p.group + head % p.group;
    }
    const int total = n[0] + n[1];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t version = *p.v.version;
    auto part_row = [&](int i) -> int64_t {              // i-th part
        const bool k = i >= n[0];
        const int piece = k ? i - n[0] : i;
        if (piece == 0) return (k ? p.rows_common : 0) + static_cast<int64_t>(out_row);
        return k ? cut[1] + static_cast<int64_t>(piece) * p.common.cut_rows : cut[0] + static_cast<int64_t>(piece) * p.own.cut_rows;
    };
    float m = -INFINITY, l = 0.0f;
    float acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
    const int mine = (total - sub + kW - 1) / kW;        // this warp's parts: sub, sub + kW, ..
    // (a single part's row was written by the attention kernel)
    for (int i0 = 0; i0 < (total == 1 ? 0 : mine); i0 += 32) {
        const float2 ml = i0 + lane < mine ? p.part_ml[part_row(sub + (i0 + lane) * kW)] : make_float2(-INFINITY, 0.0f);
        float mb = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        mb = fmaxf(mb, m);
        const float c = m == -INFINITY ? 0.0f : exp2f(m - mb);
        l *= c;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= c;
        const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - mb);
        float lw = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
        l += lw;
        m = mb;
        const int nb = min(32, mine - i0);
        for (int j0 = 0; j0 < nb; j0 += 4) {
            float x[4][D / 32];
            float wj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                wj[j] = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                if (j0 + j >= nb) wj[j] = 0.0f;
                if (wj[j] != 0.0f) {                     // (a part without keys has no output row)
                    const float *src = p.part_o + part_row(sub + (i0 + j0 + j) * kW) * D + lane * (D / 32);
                    if constexpr (D == 128)
                        *reinterpret_cast<float4 *>(x[j]) = *reinterpret_cast<const float4 *>(src);
                    else
                        *reinterpret_cast<float2 *>(x[j]) = *reinterpret_cast<const float2 *>(src);
                } else {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) x[j][i] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < D / 32; ++i) acc[i] += wj[j] * x[j][i];
        }
    }
    if constexpr (kW > 1) {
        __shared__ float2 other_ml[8];
        __shared__ float other[8][D];
        if (lane == 0) other_ml[warp] = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) other[warp][lane * (D / 32) + i] = acc[i];
        __syncthreads();
        if (sub != 0) return;
        float top = m;
#pragma unroll
        for (int k = 1; k < kW; ++k) top = fmaxf(top, other_ml[warp + k].x);
        const float c = m == -INFINITY ? 0.0f : exp2f(m - top);
        l *= c;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= c;
#pragma unroll
        for (int k = 1; k < kW; ++k) {
            const float2 ml = other_ml[warp + k];
            const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
            l += w * ml.y;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] += w * other[warp + k][lane * (D / 32) + i];
        }
    }
    if (my_row >= n_rows || total == 1 || version != p.v.expect) return;
    const float inv = 1.0f / l;
    uint16_t *orow = p.out + static_cast<int64_t>(token) * p.out_stride + head * D + lane * (D / 32);
    if constexpr (D == 128)
        *reinterpret_cast<uint2 *>(orow) =
            make_uint2(pack_16x2<HALF>(acc[0] * inv, acc[1] * inv), pack_16x2<HALF>(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(orow) = pack_16x2<HALF>(acc[0] * inv, acc[1] * inv);
}

template <int D, bool HALF, int N, int kS, int kM>
static cudaError_t launch_rows_n(const PagesAttnParams<kS, kM> &p, const PageWork &w, bool beside, int sm_count,
                                 cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};          // (per device)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(pages_rows_kernel<D, HALF, N, kS, kM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 RowsLayout<D>::kAlloc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    // four warps to a CTA, two CTAs to an SM (a batch of 604 MB: 101 us, with 2 warps 121, with 8
    // 102); few workers are spread over all SMs
    const int warps = std::min(kRowWarps / 2, (w.workers + sm_count - 1) / sm_count);
    return launch_dependent(pages_rows_kernel<D, HALF, N, kS, kM>, dim3((w.workers + warps - 1) / warps), dim3(warps * 32),
                            static_cast<size_t>(warps * RowsLayout<D>::kStages * RowsLayout<D>::kTile), s, p, w, beside);
}

template <int D, bool HALF, int kS, int kM>
static cudaError_t launch_rows_d(const PagesAttnParams<kS, kM> &p, const PageWork &w, bool beside, int sm_count,
                                 cudaStream_t s) {
    return w.rows <= 8 ? launch_rows_n<D, HALF, 1>(p, w, beside, sm_count, s)
                       : launch_rows_n<D, HALF, 2>(p, w, beside, sm_count, s);
}

template <int kS, int kM>
cudaError_t launch_pages_rows(const PagesAttnParams<kS, kM> &p, const PageWork &w, bool half, bool beside,
                              int sm_count, cudaStream_t s) {
    if (w.tile_log2 != kRowKeysLog2 || w.rows > kRowsPerWorker) return cudaErrorInvalidValue;
    if (p.v.head_dim == 64)
        return half ? launch_rows_d<64, true>(p, w, beside, sm_count, s) : launch_rows_d<64, false>(p, w, beside, sm_count, s);
    return half ? launch_rows_d<128, true>(p, w, beside, sm_count, s) : launch_rows_d<128, false>(p, w, beside, sm_count, s);
}

template <int D, bool HALF, int kS, int kM>
static cudaError_t launch_merge_d(const PagesAttnParams<kS, kM> &p, int warps_per_row, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.n_queries) * p.heads;
    const dim3 grid(static_cast<unsigned>((rows * warps_per_row + 7) / 8));
    if (warps_per_row == 1) return launch_dependent(pages_merge_kernel<D, HALF, 1, kS, kM>, grid, dim3(256), 0, s, p);
    if (warps_per_row == 4) return launch_dependent(pages_merge_kernel<D, HALF, 4, kS, kM>, grid, dim3(256), 0, s, p);
    return launch_dependent(pages_merge_kernel<D, HALF, 8, kS, kM>, grid, dim3(256), 0, s, p);
}

template <int kS, int kM>
cudaError_t launch_pages_merge(const PagesAttnParams<kS, kM> &p, int warps_per_row, bool half, cudaStream_t s) {
    if (p.v.head_dim == 64)
        return half ? launch_merge_d<64, true>(p, warps_per_row, s) : launch_merge_d<64, false>(p, warps_per_row, s);
    return half ? launch_merge_d<128, true>(p, warps_per_row, s) : launch_merge_d<128, false>(p, warps_per_row, s);
}

using SmallParams = PagesAttnParams<kSmallSections, kSmallMembers>;
using LargeParams = PagesAttnParams<kLargeSections, kLargeMembers>;
template cudaError_t launch_pages_rows(const SmallParams &, const PageWork &, bool, bool, int, cudaStream_t);
template cudaError_t launch_pages_rows(const LargeParams &, const PageWork &, bool, bool, int, cudaStream_t);
template cudaError_t launch_pages_merge(const SmallParams &, int, bool, cudaStream_t);
template cudaError_t launch_pages_merge(const LargeParams &, int, bool, cudaStream_t);

}  // namespace sdv2
