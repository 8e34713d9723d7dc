// Paged attention for at most 16 query rows per key head (single tokens and a few), and the
// merge of partial results.
//
// With so few rows the only cost that counts is reading K and V once, at HBM's rate.  Every
// warp is a worker of its own: it takes an equal run of 16-key tiles and needs no other
// warp, so eight runs per SM overlap their starts, ends and dependent chains (one CTA-wide
// pipeline paid about 8000 cycles at each change of unit).
//
// Tensor-core products of 16 rows x 8 columns x 16 (mma.sync: the smallest tile of the
// tcgen05 kind has 64 rows, of which these calls fill 1 to 16).  The order of the channels inside
// q . k and of the columns of V is free, so each lane's operands are whole 16-byte pieces of
// K and V rows: lane (g, c) = (lane / 4, lane % 4) takes channels 32 j + 8 c .. + 7 of keys g and
// g + 8 for the scores, and channels 64 j + 8 g .. + 7 of keys 2c, 2c + 1, 2c + 8, 2c + 9 for the
// output.  A lane copies just what it will use itself into its own slots of shared memory
// (cp.async, no barrier, no bank conflicts), kStages tiles ahead.
// Keys past the range are copied as zeros and their scores masked.
#include <algorithm>
#include <atomic>

#include "attn_core.cuh"
#include "pages_runs.cuh"

namespace sdv2 {

template <int D>
struct RowsLayout {
    static constexpr int kCopies = D / 8;                 // 16-byte pieces per lane of a tile: D / 16 of K, D / 16 of V
    static constexpr int kTile = kCopies * 512;           // bytes of a tile
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kAlloc = kRowWarps * kStages * kTile;
    static_assert(kAlloc <= 232448, "shared memory of one CTA");
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

template <int D, bool HALF, int kS, int kM>
__global__ void __launch_bounds__(kRowWarps * 32, 1)
    pages_rows_kernel(const __grid_constant__ PagesAttnParams<kS, kM> p, const __grid_constant__ PageWork work,
                      const bool beside) {
    using L = RowsLayout<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    // The launch before is the same call's other half, which had waited for everything before it
    // when it let this one start: only the end of this grid has to come after its end.
    if (!beside) grid_dependency_wait();
    grid_launch_dependents();
    const int worker = blockIdx.x * (blockDim.x >> 5) + warp;
    int pos = 0, end = 0;
    if (worker < work.workers) {
        pos = static_cast<int>(static_cast<int64_t>(worker) * work.tiles / work.workers);
        end = static_cast<int>(static_cast<int64_t>(worker + 1) * work.tiles / work.workers);
    }
    if (*p.v.version != p.v.expect) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.v.status, kStatusStale);
        pos = end = 0;
    }
    const int page_log2 = p.v.page_log2;
    const uint32_t stage0 = smem_addr(smem) + warp * (L::kStages * L::kTile) + lane * 16;
    for (int taken; pos < end; pos += taken) {
        const PagesRun r = pages_run(p, work, worker, pos, end, &taken);
        const PageSection &s = p.section[r.sec];

        // ---- queries: rows g and g + 8 of the tile as A operands
        uint4 q[2][D / 32];
        int token[2], head[2], seen[2];
        bool valid[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = g + 8 * h;
            valid[h] = row < r.n_rows;
            const int place = valid[h] ? row / p.group : 0;
            head[h] = r.head * p.group + (valid[h] ? row - place * p.group : 0);
            token[h] = query_token(p, s, place);
            seen[h] = r.keys;                            // keys the row sees, from the range's first
            if (!r.common) seen[h] = min(r.len, ((r.len - s.n_tokens + place) / p.block + 1) * p.block) - r.base;
            const uint16_t *src = p.q + static_cast<int64_t>(token[h]) * p.q_stride + head[h] * D + 8 * c;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                q[h][j] = valid[h] ? *reinterpret_cast<const uint4 *>(src + 32 * j) : make_uint4(0, 0, 0, 0);
        }

        // ---- copies: page ids of the run, 32 at a time, the next 32 in flight
        const int32_t *row_ids = p.v.table + static_cast<int64_t>(s.stream) * p.v.width + s.page0;
        const int last_page = max(0, ((r.keys + (1 << page_log2) - 1) >> page_log2) - 1);
        const int key0 = r.begin * 16;                   // first key of the run in the range
        int batch = key0 >> page_log2;
        int ids = r.n > 0 ? row_ids[min(batch + lane, last_page)] : 0;
        int ids_next = r.n > 0 ? row_ids[min(batch + 32 + lane, last_page)] : 0;
        const int64_t head_off = (static_cast<int64_t>(r.head) << page_log2) * D;
        const int64_t page_elems = (static_cast<int64_t>(p.v.kv_heads) << page_log2) * D;
        auto issue = [&](int tile) {                     // (tiles in order)
            if (tile < r.n) {
                const int key = key0 + tile * 16, index = key >> page_log2;
                if (index - batch >= 32) {
                    batch += 32;
                    ids = ids_next;
                    ids_next = row_ids[min(batch + 32 + lane, last_page)];
                }
                int id = __shfl_sync(0xffffffffu, ids, index - batch);
                id = min(max(id, 0), p.v.pages - 1);     // (the table lies in the caller's buffer)
                const int64_t off = id * page_elems + head_off + static_cast<int64_t>(key & ((1 << page_log2) - 1)) * D;
                const int there = r.keys - key;          // keys of the tile that there are
                const uint32_t dst = stage0 + (tile % L::kStages) * L::kTile;
                const uint16_t *ks = p.k_layer + off + g * D + 8 * c, *vs = p.v_layer + off + 2 * c * D + 8 * g;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        copy16(dst + (t * (D / 32) + j) * 512, ks + t * 8 * D + 32 * j, g + 8 * t < there ? 16 : 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
                        copy16(dst + (D / 16 + k * (D / 64) + j) * 512, vs + ((k & 1) + (k >> 1) * 8) * D + 64 * j,
                               2 * c + (k & 1) + (k >> 1) * 8 < there ? 16 : 0);
            }
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < L::kStages - 1; ++i) issue(i);

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};   // rows g, g + 8 (l: this lane's columns)
        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
        for (int it = 0; it < r.n; ++it) {
            copies_wait<L::kStages - 2>();
            const uint32_t st = stage0 + (it % L::kStages) * L::kTile;
            // scores of keys 0..7 and 8..15
            float sc[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[t][i] = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const uint4 k = lds16(st + (t * (D / 32) + j) * 512);
                    mma16816<HALF>(sc[t], q[0][j].x, q[1][j].x, q[0][j].y, q[1][j].y, k.x, k.y);
                    mma16816<HALF>(sc[t], q[0][j].z, q[1][j].z, q[0][j].w, q[1][j].w, k.z, k.w);
                }
            }
            const int first = key0 + it * 16 + 2 * c;    // key of sc[0][0]
            uint32_t pk[2][2];                           // P, [keys 0..7, 8..15][row g, g + 8]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float &x = sc[t][2 * h + i];
                        x = first + 8 * t + i < seen[h] ? x * p.scale_log2 : -INFINITY;
                    }
                float mt = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
                // the running maximum moves only when a tile exceeds it by more than 2^8
                const bool up = mt > m[h] + kCoreRescale || m[h] == -INFINITY;
                if (__any_sync(0xffffffffu, up && it > 0)) {
                    const float alpha = !up ? 1.0f : (m[h] == -INFINITY ? 0.0f : ex2_approx(m[h] - mt));
                    l[h] *= alpha;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][2 * h] *= alpha;
                        o[j][2 * h + 1] *= alpha;
                    }
                }
                if (up) m[h] = mt;
                const float ref = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float p0 = ex2_approx(sc[t][2 * h] - ref), p1 = ex2_approx(sc[t][2 * h + 1] - ref);
                    l[h] += p0 + p1;
                    pk[t][h] = pack_16x2<HALF>(p0, p1);
                }
            }
            // output: V of keys 2c, 2c + 1 and 2c + 8, 2c + 9, pairs of keys packed per channel
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = lds16(st + (D / 16 + k * (D / 64) + j) * 512);
                const uint32_t *a = &v[0].x, *b = &v[1].x, *e = &v[2].x, *f = &v[3].x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma16816<HALF>(o[8 * j + 2 * i], pk[0][0], pk[0][1], pk[1][0], pk[1][1],
                                   __byte_perm(a[i], b[i], 0x5410), __byte_perm(e[i], f[i], 0x5410));
                    mma16816<HALF>(o[8 * j + 2 * i + 1], pk[0][0], pk[0][1], pk[1][0], pk[1][1],
                                   __byte_perm(a[i], b[i], 0x7632), __byte_perm(e[i], f[i], 0x7632));
                }
            }
            issue(it + L::kStages - 1);
        }
        copies_wait<0>();

        // ---- results: o[8 j + i][2 h + x] is channel 64 j + 16 c + 8 x + i of row g + 8 h
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (!valid[h]) continue;
            if (r.whole && !r.common && s.common < 0) {
                const float inv = 1.0f / l[h];
                uint16_t *orow = p.out + static_cast<int64_t>(token[h]) * p.out_stride + head[h] * D + 16 * c;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] = pack_16x2<HALF>(o[8 * j + 2 * i][2 * h + x] * inv, o[8 * j + 2 * i + 1][2 * h + x] * inv);
                        *reinterpret_cast<uint4 *>(orow + 64 * j + 8 * x) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
            } else {
                const int64_t part = partial_row(p, work, r, worker, g + 8 * h,
                                                 static_cast<int64_t>(token[h]) * p.heads + head[h]);
                if (r.n > 0) {
                    float *prow = p.part_o + part * D + 16 * c;
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int i = 0; i < 8; i += 4)
                                *reinterpret_cast<float4 *>(prow + 64 * j + 8 * x + i) =
                                    make_float4(o[8 * j + i][2 * h + x], o[8 * j + i + 1][2 * h + x],
                                                o[8 * j + i + 2][2 * h + x], o[8 * j + i + 3][2 * h + x]);
                }
                if (c == 0) p.part_ml[part] = make_float2(m[h], l[h]);
            }
        }
    }
    if (beside) grid_dependency_wait();
}

// Merge of the partial results: a warp per output row (token, head).  Its parts are the
// pieces of its unit of the stream's own keys and of its unit of the group's common keys;
// out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.  The pieces' (m, l) are read by the
// lanes at once, then the rows, four in flight.
template <int D, bool HALF, int kS, int kM>
__global__ void __launch_bounds__(256) pages_merge_kernel(const __grid_constant__ PagesAttnParams<kS, kM> p) {
    grid_dependency_wait();
    grid_launch_dependents();
    if (*p.v.version != p.v.expect) return;
    const int lane = threadIdx.x & 31;
    const int64_t out_row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (out_row >= static_cast<int64_t>(p.n_queries) * p.heads) return;
    const int token = static_cast<int>(out_row / p.heads), head = static_cast<int>(out_row - static_cast<int64_t>(token) * p.heads);
    int lo = p.n_common, hi = p.n_sections;              // the section of the stream's own keys
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.section[mid].token0 <= token)
            lo = mid;
        else
            hi = mid;
    }
    // pieces of the row's unit in both sections: the first worker, their number, the row of a later one
    int n[2] = {0, 0}, first[2] = {0, 0};
    int64_t cut[2] = {0, 0};
    const int own = lo, common = p.section[lo].common;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 1 && common < 0) continue;
        const PageWork &w = k ? p.common : p.own;
        const PageSection &s = p.section[k ? common : own];
        const int place = k ? p.section[own].common_token + token - p.section[own].token0 : token - s.token0;
        const int rt = place / w.tile_tokens;
        const int64_t a = s.start + (static_cast<int64_t>(rt) * p.v.kv_heads + head / p.group) * s.tiles;
        first[k] = worker_of(w, a);
        n[k] = worker_of(w, a + s.tiles - 1) - first[k] + 1;
        cut[k] = w.cut_row + static_cast<int64_t>(first[k]) * w.cut_rows + (place - rt * w.tile_tokens) * p.group + head % p.group;
    }
    const int total = n[0] + n[1];
    if (total == 1) return;                              // written by the attention kernel
    auto part_row = [&](int i) -> int64_t {              // i-th part
        const bool k = i >= n[0];
        const int piece = k ? i - n[0] : i;
        if (piece == 0) return (k ? p.rows_common : 0) + out_row;
        return k ? cut[1] + static_cast<int64_t>(piece) * p.common.cut_rows : cut[0] + static_cast<int64_t>(piece) * p.own.cut_rows;
    };
    float m = -INFINITY, l = 0.0f;
    float acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
    for (int i0 = 0; i0 < total; i0 += 32) {
        const float2 ml = i0 + lane < total ? p.part_ml[part_row(i0 + lane)] : make_float2(-INFINITY, 0.0f);
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
        const int nb = min(32, total - i0);
        for (int j0 = 0; j0 < nb; j0 += 4) {
            float x[4][D / 32];
            float wj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                wj[j] = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                if (j0 + j >= nb) wj[j] = 0.0f;
                if (wj[j] != 0.0f) {                     // (a part without keys has no output row)
                    const float *src = p.part_o + part_row(i0 + j0 + j) * D + lane * (D / 32);
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
    const float inv = 1.0f / l;
    uint16_t *orow = p.out + static_cast<int64_t>(token) * p.out_stride + head * D + lane * (D / 32);
    if constexpr (D == 128)
        *reinterpret_cast<uint2 *>(orow) =
            make_uint2(pack_16x2<HALF>(acc[0] * inv, acc[1] * inv), pack_16x2<HALF>(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(orow) = pack_16x2<HALF>(acc[0] * inv, acc[1] * inv);
}

template <int D, bool HALF, int kS, int kM>
static cudaError_t launch_rows_d(const PagesAttnParams<kS, kM> &p, const PageWork &w, bool beside, int sm_count,
                                 cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};          // (per device)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(pages_rows_kernel<D, HALF, kS, kM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 RowsLayout<D>::kAlloc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    // few workers: fewer warps to a CTA, over all the SMs
    const int warps = std::min(kRowWarps, (w.workers + sm_count - 1) / sm_count);
    return launch_dependent(pages_rows_kernel<D, HALF, kS, kM>, dim3((w.workers + warps - 1) / warps), dim3(warps * 32),
                            static_cast<size_t>(warps * RowsLayout<D>::kStages * RowsLayout<D>::kTile), s, p, w, beside);
}

template <int kS, int kM>
cudaError_t launch_pages_rows(const PagesAttnParams<kS, kM> &p, const PageWork &w, bool half, bool beside,
                              int sm_count, cudaStream_t s) {
    if (p.v.head_dim == 64)
        return half ? launch_rows_d<64, true>(p, w, beside, sm_count, s) : launch_rows_d<64, false>(p, w, beside, sm_count, s);
    return half ? launch_rows_d<128, true>(p, w, beside, sm_count, s) : launch_rows_d<128, false>(p, w, beside, sm_count, s);
}

template <int kS, int kM>
cudaError_t launch_pages_merge(const PagesAttnParams<kS, kM> &p, bool half, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.n_queries) * p.heads;
    const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
    if (p.v.head_dim == 64)
        return half ? launch_dependent(pages_merge_kernel<64, true, kS, kM>, grid, dim3(256), 0, s, p)
                    : launch_dependent(pages_merge_kernel<64, false, kS, kM>, grid, dim3(256), 0, s, p);
    return half ? launch_dependent(pages_merge_kernel<128, true, kS, kM>, grid, dim3(256), 0, s, p)
                : launch_dependent(pages_merge_kernel<128, false, kS, kM>, grid, dim3(256), 0, s, p);
}

using SmallParams = PagesAttnParams<kSmallSections, kSmallMembers>;
using LargeParams = PagesAttnParams<kLargeSections, kLargeMembers>;
template cudaError_t launch_pages_rows(const SmallParams &, const PageWork &, bool, bool, int, cudaStream_t);
template cudaError_t launch_pages_rows(const LargeParams &, const PageWork &, bool, bool, int, cudaStream_t);
template cudaError_t launch_pages_merge(const SmallParams &, bool, cudaStream_t);
template cudaError_t launch_pages_merge(const LargeParams &, bool, cudaStream_t);

}  // namespace sdv2
