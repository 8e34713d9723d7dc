// Attention of every stream's newest tokens over the pages of its keys, on the sm_100a
// tensor cores; streams that share leading pages have those read once for all of them.
//
// The softmax over a stream's keys splits into the keys of the group's common pages and the
// stream's own: each part gives an unnormalised output, a row maximum and a row sum, which
// merge as in the online softmax.  The common part's query tile holds the rows of all the
// group's streams, so its keys are read once per 128 rows.
//
// Few rows and many keys: the bound is HBM, so the work is cut evenly by keys.  All units
// (128-row tile, key head) are laid end to end in KV tiles of 128 keys and every CTA, one per
// SM, takes an equal run of tiles, crossing units as it goes; a unit cut by a border leaves
// one partial result per CTA.  Rings of three K and three V tiles (192 KB) of 128 channels, six and
// six of 64, keep loads in flight across units.
//   warp 0      looks up pages, one TMA box per page and 64 channels (a lane each)
//   warp 1      MMA issuer: tile i of a run goes to accumulator set i & 1
//   warp 2      zeroes the rows of a run's last V tile behind its keys
//   warp 3      works out the CTA's runs, one ahead of the others
//   warps 4..7  softmax of set 0, 8..11 of set 1 (thread = query row); both gather the
//               queries into shared memory (read from memory while the run before is written
//               out) and merge the two sets at the end
// A query tile holds the rows (token, head of the group); rows beyond them cost no
// exponentials.
//
// What bounds it with full tiles: the chain of a tile (scores, softmax, product) on two sets, and
// a run's start and end (about five tiles' time, counted when the work is cut).  16 streams of 64
// queries on 4000 common keys and up to 900 of their own, 12 heads of 64, fp16: 52.3 us, 35 MB read,
// tensor pipe 27 %; 64 streams of one query on 16384 common keys, 40/8 heads of 128: 62 to 64 us
// with the row kernel's part and the merge.
#include <atomic>

#include "attn_core.cuh"
#include "pages_runs.cuh"

namespace sdv2 {

template <int D>
struct PagesLayout {
    static constexpr int kTile = 128 * D * 2;
    static constexpr int kSub = 128 * 128;
    static constexpr int kStages = D == 128 ? 3 : 6;      // of K and of V
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kXm = kQ;                        // (max, sum) of both sets, once the queries are done with
    // 32 rows x 64 bytes of results for each softmax warp (at 128 channels the rings leave no room of
    // its own: the queries' second half)
    static constexpr int kOut = D == 128 ? kQ + kSub : kV + kStages * kTile;
    static constexpr int kBar = kV + kStages * kTile + (D == 128 ? 0 : 8 * 2048);
    static constexpr int kQReady = 0;
    static constexpr int kKFull = 1, kKEmpty = kKFull + kStages;
    static constexpr int kVFull = kKEmpty + kStages, kVEmpty = kVFull + kStages;
    static constexpr int kSFull = kVEmpty + kStages, kPFull = kSFull + 2, kOFull = kPFull + 2;
    static constexpr int kVAsk = kOFull + 2, kVFix = kVAsk + 1, kDrain = kVFix + 1;
    static constexpr int kRunFull = kDrain + 1, kRunEmpty = kRunFull + 2, kNumBars = kRunEmpty + 2;
    static constexpr int kRuns = kBar + kNumBars * 8;     // two slots for the CTA's next runs
    static constexpr int kMisc = kRuns + 2 * static_cast<int>(sizeof(PagesRun));
    static constexpr int kAlloc = kMisc + 16 + 1024;
    static_assert(kAlloc <= 232448, "shared memory of one CTA");
};

// Valid keys of the run's last tile if the range ends inside it (0: it does not).
__device__ __forceinline__ int tail_keys(const PagesRun &r) {
    const int left = r.keys - (r.begin + r.n - 1) * 128;
    return r.n > 0 && left < 128 ? left : 0;
}

// A role's view of the CTA's runs, published by warp 3 in two slots.  Every role's thread (or warp,
// converged) calls next().
struct RunFeed {
    uint64_t *full, *empty;
    const PagesRun *slot;
    int n = 0;
    // The next run; false at the end or when a wait ran out.  whole_warp: all lanes call it.
    __device__ __forceinline__ bool next(PagesRun *r, bool whole_warp, int lane, volatile uint32_t *abort, uint32_t *status) {
        const int x = n & 1, round = (n >> 1) & 1;
        ++n;
        bool ok = mbar_wait(&full[x], round, abort, status, kStatusTmaWait);
        if (whole_warp) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        *r = slot[x];
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(&empty[x]);
        return r->n >= 0;
    }
};
constexpr int kRunReaders = 11;           // producer, MMA issuer, warp 2, eight softmax warps

template <int D, bool HALF, int kS, int kM>
__global__ void __launch_bounds__(kAttnThreads, 1)
    pages_tiles_kernel(const __grid_constant__ PagesAttnParams<kS, kM> p, const __grid_constant__ PageWork work,
                       const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
    using L = PagesLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + L::kMisc + 4);
    uint32_t *status = p.v.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int b = 0; b < L::kNumBars; ++b)
            mbar_init(&bars[b], b == L::kQReady ? 256
                                : b == L::kPFull || b == L::kPFull + 1 ? 128
                                : b >= L::kRunEmpty ? kRunReaders : 1);
        *abort_flag = 0u;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (the first run's place, and the run itself if its keys are common ones, worked out by warp 3
    // before the launch's inputs are there)
    int pos = 0, end = 0;
    RunSpot spot;
    bool more = false, early = false;
    PagesRun run;
    if (warp == 3) {
        pos = static_cast<int>(first_place(work, blockIdx.x));
        end = static_cast<int>(first_place(work, blockIdx.x + 1));
        more = next_spot(p, work, &pos, end, &spot);
        early = more && p.section[spot.sec].keys >= 0;
        if (early) run = run_at(p, work, blockIdx.x, spot);
    }
    grid_dependency_wait();                     // queries, pages and tables may come from the kernels before
    grid_launch_dependents();

    RunFeed feed;
    feed.full = &bars[L::kRunFull];
    feed.empty = &bars[L::kRunEmpty];
    feed.slot = reinterpret_cast<const PagesRun *>(smem + L::kRuns);
    const int page_log2 = p.v.page_log2;

    if (warp < 4) {
        regs_dec<80>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (the whole warp)
            const int ppt_log2 = 7 - page_log2, ppt = 1 << ppt_log2;   // pages of a KV tile
            const int box = lane / (D / 64), kb = lane % (D / 64);     // this lane's page of the tile, 64 channels
            const uint32_t box_bytes = 128u << page_log2;
            int kc = 0, vc = 0;
            bool ok = true;
            for (PagesRun r; ok && feed.next(&r, true, lane, abort_flag, status);) {
                if (r.n == 0) continue;
                const PageSection &s = p.section[r.sec];
                const int32_t *row = p.v.table + static_cast<int64_t>(s.stream) * p.v.width + s.page0;
                const int n_pages = (r.keys + (1 << page_log2) - 1) >> page_log2;   // of the key range
                // page ids of the run, 32 at a time, the next 32 in flight
                int batch = r.begin << ppt_log2;                     // index of ids_now's first page
                const int last_page = n_pages - 1;
                int ids_now = row[min(batch + lane, last_page)];
                int ids_next = row[min(batch + 32 + lane, last_page)];
                int id_k[3];                                          // this lane's page of K tiles it + 2, it + 1, it
                auto page_of = [&](int tile) {                        // (tiles in order)
                    const int first = (r.begin + tile) << ppt_log2;
                    if (first - batch >= 32) {
                        batch += 32;
                        ids_now = ids_next;
                        ids_next = row[min(batch + 32 + lane, last_page)];
                    }
                    return __shfl_sync(0xffffffffu, ids_now, first - batch + min(box, ppt - 1));
                };
                auto load = [&](int tile, int id, const CUtensorMap *map, int base, int full, int empty, int &c) {
                    const int st = c % L::kStages;
                    if (!warp_wait_all(&bars[empty + st], ((c / L::kStages) & 1) ^ 1, abort_flag, status, kStatusTmaWait))
                        return false;
                    const int first = (r.begin + tile) << ppt_log2;
                    const int boxes = min(ppt, n_pages - first);      // pages that there are
                    if (lane == 0) mbar_arrive_expect_tx(&bars[full + st], boxes * (D / 64) * box_bytes);
                    __syncwarp();
                    if (box < boxes)
                        tma_load_3d(smem + base + st * L::kTile + kb * L::kSub + box * box_bytes, map, &bars[full + st],
                                    kb * 64, 0, id * p.v.kv_heads + r.head);
                    ++c;
                    return true;
                };
                // K runs two tiles ahead of V: scores of both sets come before the first product with V
                id_k[2] = page_of(0);
                ok = load(0, id_k[2], &tmap_k, L::kK, L::kKFull, L::kKEmpty, kc);
                id_k[1] = id_k[2];
                if (ok && r.n > 1) {
                    id_k[1] = page_of(1);
                    ok = load(1, id_k[1], &tmap_k, L::kK, L::kKFull, L::kKEmpty, kc);
                }
                for (int it = 0; ok && it < r.n; ++it) {
                    ok = load(it, id_k[2], &tmap_v, L::kV, L::kVFull, L::kVEmpty, vc);
                    id_k[0] = 0;
                    if (ok && it + 2 < r.n) {
                        id_k[0] = page_of(it + 2);
                        ok = load(it + 2, id_k[0], &tmap_k, L::kK, L::kKFull, L::kKEmpty, kc);
                    }
                    id_k[2] = id_k[1];
                    id_k[1] = id_k[0];
                }
            }
            if (!ok && lane == 0) {             // let every copy in flight land before the CTA leaves
                const uint64_t t0 = global_timer_ns();
                auto drain = [&](int c, int full) {
                    for (int i = max(0, c - L::kStages); i < c; ++i)
                        while (!mbar_try_wait(&bars[full + i % L::kStages], (i / L::kStages) & 1))
                            if (global_timer_ns() - t0 > kWaitLimitNs) break;
                };
                drain(kc, L::kKFull);
                drain(vc, L::kVFull);
            }
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc_qk = idesc_16_f32<HALF>(128, 128, 0, 0);
            constexpr uint32_t idesc_pv = idesc_16_f32<HALF>(128, D, 0, 1);
            const uint64_t dq = smem_desc_sw128(smem_addr(smem + L::kQ), 16, 1024);
            const uint64_t dk = smem_desc_sw128(smem_addr(smem + L::kK), 16, 1024);
            const uint64_t dv = smem_desc_sw128(smem_addr(smem + L::kV), L::kSub, 1024);
            int kc = 0, vc = 0, runs = 0, fixes = 0, pc[2] = {0, 0};
            bool ok = true;
            auto issue_qk = [&](int t) {        // the next K tile's scores into set t
                const int st = kc % L::kStages;
                if (!mbar_wait(&bars[L::kKFull + st], (kc / L::kStages) & 1, abort_flag, status, kStatusMmaWait))
                    return false;
                tc_fence_after();
                const uint64_t b0 = dk + static_cast<uint64_t>(st * (L::kTile >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = static_cast<uint64_t>(((kk >> 2) * L::kSub + (kk & 3) * 32) >> 4);
                    umma_ss(tmem + t * 128, dq + off, b0 + off, idesc_qk, kk > 0 ? 1u : 0u);
                }
                umma_commit(&bars[L::kSFull + t]);
                umma_commit(&bars[L::kKEmpty + st]);
                ++kc;
                return true;
            };
            for (PagesRun r; ok && feed.next(&r, false, lane, abort_flag, status);) {
                if (r.n == 0) continue;
                ok = mbar_wait(&bars[L::kQReady], runs & 1, abort_flag, status, kStatusMmaWait);
                ++runs;
                if (!ok) break;
                tc_fence_after();
                ok = issue_qk(0) && (r.n < 2 || issue_qk(1));
                const bool tail = tail_keys(r) > 0;
                for (int it = 0; ok && it < r.n; ++it) {
                    const int t = it & 1, st = vc % L::kStages;
                    ok = mbar_wait(&bars[L::kVFull + st], (vc / L::kStages) & 1, abort_flag, status, kStatusMmaWait);
                    if (ok && tail && it == r.n - 1) {
                        mbar_arrive(&bars[L::kVAsk]);
                        ok = mbar_wait(&bars[L::kVFix], fixes & 1, abort_flag, status, kStatusMmaWait);
                        ++fixes;
                    }
                    if (ok) ok = mbar_wait(&bars[L::kPFull + t], (t ? pc[1] : pc[0]) & 1, abort_flag, status, kStatusMmaWait);
                    ++(t ? pc[1] : pc[0]);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t b0 = dv + static_cast<uint64_t>(st * (L::kTile >> 4));
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8,
                                b0 + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv, (it >= 2 || kk > 0) ? 1u : 0u);
                    umma_commit(&bars[L::kVEmpty + st]);
                    ++vc;
                    if (it + 2 < r.n)
                        ok = issue_qk(t);
                    else
                        umma_commit(&bars[L::kOFull + t]);
                }
            }
            // every MMA issued so far has finished before TMEM is released
            umma_commit(&bars[L::kDrain]);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&bars[L::kDrain], 0)) {
                if (global_timer_ns() - t0 > kWaitLimitNs) {
                    atomicOr(status, kStatusMmaWait);
                    break;
                }
            }
        } else if (warp == 2) {
            // ------------------------------------------------ ends of key ranges in V
            int vc = 0, fixes = 0;
            for (PagesRun r; feed.next(&r, true, lane, abort_flag, status);) {
                vc += r.n;
                const int valid = tail_keys(r);
                if (valid == 0) continue;
                if (!warp_wait_all(&bars[L::kVAsk], fixes & 1, abort_flag, status, kStatusTmaWait)) break;
                ++fixes;
                zero_tail_rows<D>(smem + L::kV + (vc - 1) % L::kStages * L::kTile, valid, lane);
                if (lane == 0) mbar_arrive(&bars[L::kVFix]);
            }
        } else if (warp == 3 && lane == 0) {
            // ------------------------------------------------ the CTA's runs
            const uint32_t version = *p.v.version;
            if (more && !early) run = run_at(p, work, blockIdx.x, spot);   // (both loads at once)
            if (version != p.v.expect) {         // (none: the tables are not those of the call)
                if (blockIdx.x == 0) atomicOr(status, kStatusStale);
                more = false;
            }
            PagesRun *slot = reinterpret_cast<PagesRun *>(smem + L::kRuns);
            for (int i = 0;; ++i) {
                const int x = i & 1;
                if (!more) run.n = -1;
                if (!mbar_wait(&bars[L::kRunEmpty + x], ((i >> 1) & 1) ^ 1, abort_flag, status, kStatusTmaWait)) break;
                slot[x] = run;
                mbar_arrive(&bars[L::kRunFull + x]);
                if (!more) break;
                more = next_spot(p, work, &pos, end, &spot);
                if (more) run = run_at(p, work, blockIdx.x, spot);
            }
        }
    } else {
        // ------------------------------------------------ queries, softmax and epilogue
        regs_inc<208>();
        const int t = (warp - 4) >> 2;               // accumulator set
        const int row = ((warp & 3) << 5) + lane;    // query row (TMEM lane)
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) << 5) << 16;
        const uint32_t s_tmem = tmem + lane_base + t * 128, o_tmem = tmem + lane_base + 256 + t * 128;
        float2 *xm = reinterpret_cast<float2 *>(smem + L::kXm);
        int sc = 0, oc[2] = {0, 0};
        bool ok = true;
        // this thread's row of a run: the run's tiles, the keys it sees from the run's first on, where its
        // result goes (an element of out, or a partial row), and half of its queries (by set)
        constexpr int kC = D / 16;                                   // 16-byte chunks of half a row
        struct Row {
            int n, seen;
            bool there, valid, busy, direct;                         // busy: the warp has rows
            int64_t to;
            uint4 x[kC];
        };
        auto fetch = [&](Row &w) {
            PagesRun r;
            w.there = feed.next(&r, true, lane, abort_flag, status);
            if (!w.there) return;
            const PageSection &s = p.section[r.sec];
            w.n = r.n;
            w.valid = row < r.n_rows;
            w.busy = ((warp & 3) << 5) < r.n_rows;
            const int in_tile = w.valid ? row / p.group : 0;
            const int place = r.row_tile * work.tile_tokens + in_tile;
            const int head = r.head * p.group + (w.valid ? row - in_tile * p.group : 0);
            const int token = query_token(p, s, place);
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(token) * p.q_stride + head * D) + t * kC;
#pragma unroll
            for (int c = 0; c < kC; ++c) w.x[c] = w.valid ? src[c] : make_uint4(0, 0, 0, 0);
            w.seen = r.keys;
            if (!r.common) w.seen = min(r.len, ((r.len - s.n_tokens + place) / p.block + 1) * p.block) - r.base;
            w.seen -= r.begin * 128;
            w.direct = r.whole && !r.common && s.common < 0;
            w.to = w.direct ? static_cast<int64_t>(token) * p.out_stride + head * D
                            : partial_row(p, work, r, blockIdx.x, row, static_cast<int64_t>(token) * p.heads + head);
        };
        // All 256 threads go on to a run, and leave, together: at a barrier that carries whether each
        // of them has one (a warp whose wait ran out has none).
        Row now;
        fetch(now);
        bool go = named_bar_and(1, 256, now.there);
        while (go) {
            const int n = now.n, seen = now.seen;
            const bool valid = now.valid, busy = now.busy, direct = now.direct;
            const int64_t to = now.to;
            if (n > 0) {
                // the queries to their 128-byte-swizzled places (every score of the run before has been
                // read: its products with Q are done)
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const int cc = t * kC + c;                       // chunk of the whole row
                    *reinterpret_cast<uint4 *>(smem + L::kQ + (cc >> 3) * L::kSub + row * 128 +
                                               (((cc & 7) ^ (row & 7)) << 4)) = now.x[c];
                }
                fence_proxy_async_shared();
                tc_fence_before();
                mbar_arrive(&bars[L::kQReady]);
            }
            const int n_mine = (n + 1 - t) >> 1;
            float m_run = -INFINITY, l_run = 0.0f;
            for (int it = 0; it < n_mine; ++it, ++sc) {
                ok = warp_wait_all(&bars[L::kSFull + t], sc & 1, abort_flag, status, kStatusSoftmaxWait);
                if (!ok) break;
                if (busy) {
                    tc_fence_after();
                    ScoreRow x;
                    load_scores(s_tmem, x);
                    const int cols = seen - (2 * it + t) * 128;
                    if (__any_sync(0xffffffffu, cols < 128)) mask_scores(x, cols);
                    const float m_tile = max_score(x) * p.scale_log2;
                    bool rescale = false;
                    float alpha = 1.0f;
                    // (a row may see none of a tile's keys: its maximum stays -inf, its P is 0)
                    if (m_tile > m_run + kCoreRescale || m_run == -INFINITY) {
                        rescale = it > 0;
                        alpha = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m_tile);
                        l_run *= alpha;
                        m_run = m_tile;
                    }
                    l_run += exp_store<HALF>(x, p.scale_log2, m_run == -INFINITY ? 0.0f : -m_run, s_tmem);
                    if (__any_sync(0xffffffffu, rescale)) rescale_row<D>(o_tmem, alpha);
                    tmem_wait_st();
                    tc_fence_before();
                }
                mbar_arrive(&bars[L::kPFull + t]);
            }

            // ---- both sets merged: thread (t, row) takes columns [t D / 2, (t + 1) D / 2)
            // (a warp whose wait ran out comes to the barrier too: all 256 threads leave together)
            if (ok) fetch(now);                          // the next run's row, on its way meanwhile
            const bool has0 = n > 0, has1 = n > 1;
            if (ok && has0) ok = warp_wait_all(&bars[L::kOFull + 0], oc[0]++ & 1, abort_flag, status, kStatusSoftmaxWait);
            if (ok && has1) ok = warp_wait_all(&bars[L::kOFull + 1], oc[1]++ & 1, abort_flag, status, kStatusSoftmaxWait);
            xm[t * 128 + row] = make_float2(m_run, l_run);
            ok = named_bar_and(1, 256, ok);
            if (!ok) break;
            tc_fence_after();
            const float2 a0 = xm[row], a1 = xm[128 + row];
            const float m = fmaxf(a0.x, a1.x);
            const float w0 = a0.x == -INFINITY ? 0.0f : ex2_approx(a0.x - m);
            const float w1 = a1.x == -INFINITY ? 0.0f : ex2_approx(a1.x - m);
            const float l = w0 * a0.y + w1 * a1.y;
            const uint32_t o0 = tmem + lane_base + 256 + t * (D / 2);
            if (busy && has0) {
                const float inv = direct ? 1.0f / l : 1.0f;
                // 64 bytes a row at a time through shared memory, so that four lanes write them (a thread
                // writing its own row touched 32 lines with every store)
                uint8_t *out_tile = smem + L::kOut + (warp - 4) * 2048;
                uint64_t mine = 0;                           // where the thread's row goes, 0: nowhere
                if (valid)
                    mine = direct ? reinterpret_cast<uint64_t>(p.out + to + t * (D / 2))
                                  : reinterpret_cast<uint64_t>(p.part_o + to * D + t * (D / 2));
                uint64_t dst[4];                             // of rows 8 k + lane / 4
#pragma unroll
                for (int k = 0; k < 4; ++k) dst[k] = __shfl_sync(0xffffffffu, mine, 8 * k + (lane >> 2));
                auto put = [&](const uint32_t (&y)[16], int at) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(out_tile + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int rr = 8 * k + (lane >> 2), c = lane & 3;
                        const uint4 x = *reinterpret_cast<const uint4 *>(out_tile + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
                        if (dst[k] != 0) *reinterpret_cast<uint4 *>(dst[k] + at + c * 16) = x;
                    }
                    __syncwarp();
                };
#pragma unroll 1
                for (int cb = 0; cb < D / 64; ++cb) {
                    uint32_t v[32], v1[32];
                    tmem_ld32(o0 + cb * 32, v);
                    if (has1) tmem_ld32(o0 + 128 + cb * 32, v1);
                    tmem_wait_ld_bind(v);
                    if (has1) {
                        reg_bind(v1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __float_as_uint((w0 * __uint_as_float(v[i]) + w1 * __uint_as_float(v1[i])) * inv);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(w0 * __uint_as_float(v[i]) * inv);
                    }
                    uint32_t y[16];
                    if (direct) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            y[i] = pack_16x2<HALF>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        put(y, cb * 64);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = v[16 * h + i];
                            put(y, cb * 128 + h * 64);
                        }
                    }
                }
            }
            if (valid && !direct && t == 0) p.part_ml[to] = make_float2(m, l);
            tc_fence_before();
            go = named_bar_and(1, 256, now.there);       // (xm and both accumulators have been read)
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool HALF, int kS, int kM>
static cudaError_t launch_d(const PagesAttnParams<kS, kM> &p, const PageWork &w, const CUtensorMap &tk,
                            const CUtensorMap &tv, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};          // (per device)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(pages_tiles_kernel<D, HALF, kS, kM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PagesLayout<D>::kAlloc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return launch_dependent(pages_tiles_kernel<D, HALF, kS, kM>, dim3(w.workers), dim3(kAttnThreads),
                            static_cast<size_t>(PagesLayout<D>::kAlloc), s, p, w, tk, tv);
}

template <int kS, int kM>
cudaError_t launch_pages_tiles(const PagesAttnParams<kS, kM> &p, const PageWork &w, const CUtensorMap &tk,
                               const CUtensorMap &tv, bool half, cudaStream_t s) {
    if (w.tile_log2 != kTileKeysLog2) return cudaErrorInvalidValue;
    if (p.v.head_dim == 64) return half ? launch_d<64, true>(p, w, tk, tv, s) : launch_d<64, false>(p, w, tk, tv, s);
    return half ? launch_d<128, true>(p, w, tk, tv, s) : launch_d<128, false>(p, w, tk, tv, s);
}

template cudaError_t launch_pages_tiles(const PagesAttnParams<kSmallSections, kSmallMembers> &, const PageWork &,
                                        const CUtensorMap &, const CUtensorMap &, bool, cudaStream_t);
template cudaError_t launch_pages_tiles(const PagesAttnParams<kLargeSections, kLargeMembers> &, const PageWork &,
                                        const CUtensorMap &, const CUtensorMap &, bool, cudaStream_t);

}  // namespace sdv2
