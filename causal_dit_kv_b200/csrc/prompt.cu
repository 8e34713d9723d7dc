// Attention over whole packed prompts on the sm_100a tensor cores.
//
// out_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j of i's own sequence with
// floor(j / b) <= floor(i / b): causal token by token (b = 1) or by blocks of b tokens (the
// causal DiT's mask, b = tokens of a chunk).  Query head h reads key head h / group.
//
// One CTA = work units of two 128-row query tiles that share every K/V tile: the same
// rows of two heads of one key head (even groups), or 256 consecutive rows of one head.
// Sharing halves the K/V bytes from L2, which at 64 KB per tile pair and SM would
// otherwise reach the L2's rate.
//   warp 0      TMA producer: query tiles, K tiles (128 keys) and V tiles into rings
//   warp 1      MMA issuer (one thread): S_t = Q_t K^T, O_t += P_t V
//   warp 2      zeroes the rows of a sequence's last V tile that lie past its end
//   warps 4..7  softmax and epilogue of query tile 0 (a thread per row), 8..11 of tile 1
// TMEM: S_0 | S_1 | O_0 | O_1 (128 columns each); P_t, 16-bit, over the first half of S_t.
// While one tile is in the softmax the tensor core works on the other.
// Units are taken longest first, so the launch does not end on a long one.  The grid has one
// CTA per unit; each running CTA (one per SM) takes further units over from CTAs that have not
// started (clusterlaunchcontrol), so its set-up is paid once, the next unit's first tiles and
// scores are under way while the last one's results are written, and SMs that run faster take more.
// Every wait is bounded; a wait that runs out records itself in g_prompt_status.
//
// What bounds it: per 128 keys the two tiles' softmax (1930 cycles each, of which 1400 are the 128
// exponentials a thread) and the round trip to the tensor core between them (score wait, four
// products, 1500 cycles) overlap to 3400 cycles; tensor pipe 57 % and exponential unit 52 % busy.
// Prompts of 77 to 4096 tokens, 32/8 heads of 128, bf16: 191 us in a burst (1.00 PFLOP/s), 221 us
// (0.87) in a long run, which meets the 1000 W limit; 8192 tokens in blocks of 1024, 40 heads: 754 us
// in a long run (1.03 PFLOP/s); 6289 tokens, 16/2 heads of 64, fp16: 53 us, where the products take
// as long as with 128 channels for half the work; six prompts of 1 to 200 tokens, 12 heads: 10 us.
#include <atomic>

#include "attn_core.cuh"
#include "token_ops.h"

namespace sdv2 {

__device__ uint32_t g_prompt_status;

struct PromptUnit {
    int first, len;          // the sequence's tokens
    int row0[2], head[2];    // each query tile's first row in the sequence, and its head
    int n[2], n_max;         // KV tiles that each query tile sees (0: no such tile); n_max -1: no more units
    int kv_head;
};

template <int D>
struct PromptLayout {
    static constexpr int kTile = 128 * D * 2;             // bytes of a Q, K or V tile
    static constexpr int kSub = 128 * 128;                // its 64-column (128-byte) sub-tiles
    static constexpr int kKStages = D == 128 ? 2 : 4;
    static constexpr int kVStages = D == 128 ? 2 : 4;     // (a third V tile of 128 channels gained nothing)
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kKStages * kTile;
    static constexpr int kOut = kV + kVStages * kTile;    // 32 rows x 128 bytes of results for each softmax warp
    static constexpr int kBar = kOut + 8 * 4096;
    static constexpr int kQFull = 0, kQEmpty = 1;
    static constexpr int kKFull = 2, kKEmpty = kKFull + kKStages;
    static constexpr int kVFull = kKEmpty + kKStages, kVEmpty = kVFull + kVStages;
    static constexpr int kSFull = kVEmpty + kVStages, kPFull = kSFull + 2, kOFull = kPFull + 2;
    static constexpr int kVAsk = kOFull + 2, kVFix = kVAsk + 1, kDrain = kVFix + 1;
    // units: the current one is near its end, answer to a request landed, unit published in a slot,
    // slot read by every role
    static constexpr int kNear = kDrain + 1, kAnswer = kNear + 1, kUnitFull = kAnswer + 1, kUnitEmpty = kUnitFull + 2, kNumBars = kUnitEmpty + 2;
    static constexpr int kAnswerAt = kBar + ((kNumBars * 8 + 15) & ~15);   // 16 bytes
    static constexpr int kUnits = kAnswerAt + 16;         // two unit slots
    static constexpr int kMisc = kUnits + 2 * static_cast<int>(sizeof(PromptUnit));   // TMEM base, abort flag
    static constexpr int kAlloc = kMisc + 16 + 1024;      // room to align the base to 1024 bytes
    static_assert(kAlloc <= 232448, "shared memory of one CTA");
};

template <int kItems>
__device__ __forceinline__ PromptUnit prompt_unit(const PromptParams<kItems> &p, int u) {
    PromptUnit w;
    // chunks of head units one after another, so that what runs at a time shares keys that fit the L2
    const int chunk = u / (p.n_items * p.chunk_units), in = u - chunk * p.n_items * p.chunk_units;
    const int width = min(p.chunk_units, p.head_units - chunk * p.chunk_units);
    const int i = in / width, j = chunk * p.chunk_units + in - i * width;
    const uint32_t it = p.item[i];
    const int seq = it >> 24, tile = it & 0xffffffu;
    w.first = p.seq_first[seq];
    w.len = p.seq_len[seq];
    w.kv_head = (p.pair_heads ? 2 * j : j) / p.group;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        w.row0[t] = p.pair_heads ? tile * 128 : tile * 256 + t * 128;
        w.head[t] = p.pair_heads ? 2 * j + t : j;
        w.n[t] = 0;
        if (w.row0[t] < w.len) {
            const int last = min(w.row0[t] + 127, w.len - 1);
            w.n[t] = (min(w.len, (last / p.block + 1) * p.block) + 127) >> 7;
        }
    }
    w.n_max = max(w.n[0], w.n[1]);
    return w;
}

// Valid rows of the unit's last V tile, if that reaches past the sequence (0: it does not).
__device__ __forceinline__ int tail_rows(const PromptUnit &w) {
    const int left = w.len - (w.n_max - 1) * 128;
    return left < 128 ? left : 0;
}

// Ask for the next CTA that has not started; the 16-byte answer lands at `answer`, counted on `bar`.
__device__ __forceinline__ void request_cta(void *answer, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
}

// The CTA number in an answer, or -1 if none was left.
__device__ __forceinline__ int answered_cta(const void *answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_addr(answer))
        : "memory");
    return got ? static_cast<int>(x) : -1;
}

// A role's view of the CTA's units, in order, as warp 3 publishes them in two slots (worked out
// once: the divisions and the reads of the launch's lists took each role 2500 cycles a unit).
// Every role's thread (or warp, converged) calls next().
struct UnitFeed {
    uint64_t *full, *empty;
    const PromptUnit *slot;
    int n = 0;
    // The next unit; false at the end or when a wait ran out.  whole_warp: all lanes call it.
    __device__ __forceinline__ bool next(PromptUnit *w, bool whole_warp, int lane, volatile uint32_t *abort, uint32_t *status) {
        const int x = n & 1, round = (n >> 1) & 1;
        ++n;
        bool ok = mbar_wait(&full[x], round, abort, status, kStatusTmaWait);
        if (whole_warp) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        *w = slot[x];
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(&empty[x]);
        return w->n_max >= 0;
    }
};
constexpr int kUnitReaders = 11;          // producer, MMA issuer, warp 2, eight softmax warps

template <int D, bool HALF, int kItems>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prompt_attention_kernel(const __grid_constant__ PromptParams<kItems> p, const __grid_constant__ CUtensorMap tmap_q,
                            const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
    using L = PromptLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + L::kMisc + 4);
    uint32_t *status = &g_prompt_status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int b = 0; b < L::kNumBars; ++b)
            mbar_init(&bars[b], b == L::kPFull || b == L::kPFull + 1 ? 128 : (b >= L::kUnitEmpty ? kUnitReaders : 1));
        *abort_flag = 0u;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
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
    PromptUnit unit;                            // (warp 3's, worked out before the inputs are there)
    if (warp == 3) unit = prompt_unit(p, blockIdx.x);
    grid_dependency_wait();                     // the inputs may come from the kernel just before
    grid_launch_dependents();

    UnitFeed feed;
    feed.full = &bars[L::kUnitFull];
    feed.empty = &bars[L::kUnitEmpty];
    feed.slot = reinterpret_cast<const PromptUnit *>(smem + L::kUnits);

    if (warp < 4) {
        regs_dec<120>();                         // (104: 197 us for five ragged prompts, 80, where the issuer spills: 207; 120: 193)
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int kc = 0, vc = 0, uc = 0;         // K tiles, V tiles and units issued so far
            bool ok = true;
            for (PromptUnit w; ok && feed.next(&w, false, lane, abort_flag, status); ++uc) {
                ok = mbar_wait(&bars[L::kQEmpty], (uc & 1) ^ 1, abort_flag, status, kStatusTmaWait);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars[L::kQFull], ((w.n[0] > 0) + (w.n[1] > 0)) * L::kTile);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (w.n[t] > 0)
#pragma unroll
                        for (int kb = 0; kb < D / 64; ++kb)
                            tma_load_3d(smem + L::kQ + t * L::kTile + kb * L::kSub, &tmap_q, &bars[L::kQFull], kb * 64,
                                        w.head[t], w.first + w.row0[t]);
                auto load = [&](int it, const CUtensorMap *map, int base, int stages, int full, int empty, int &c) {
                    const int st = c % stages;
                    if (!mbar_wait(&bars[empty + st], ((c / stages) & 1) ^ 1, abort_flag, status, kStatusTmaWait))
                        return false;
                    mbar_arrive_expect_tx(&bars[full + st], L::kTile);
#pragma unroll
                    for (int kb = 0; kb < D / 64; ++kb)
                        tma_load_3d(smem + base + st * L::kTile + kb * L::kSub, map, &bars[full + st], kb * 64, w.kv_head,
                                    w.first + it * 128);
                    ++c;
                    return true;
                };
                // K tile it + 1 is needed half a step before V tile it
                ok = load(0, &tmap_k, L::kK, L::kKStages, L::kKFull, L::kKEmpty, kc);
                for (int it = 0; ok && it < w.n_max; ++it) {
                    if (it + 1 < w.n_max) ok = load(it + 1, &tmap_k, L::kK, L::kKStages, L::kKFull, L::kKEmpty, kc);
                    if (ok) ok = load(it, &tmap_v, L::kV, L::kVStages, L::kVFull, L::kVEmpty, vc);
                }
            }
            if (!ok) {                          // let every copy in flight land before the CTA leaves
                const uint64_t t0 = global_timer_ns();
                auto drain = [&](int c, int stages, int full) {
                    for (int i = max(0, c - stages); i < c; ++i)
                        while (!mbar_try_wait(&bars[full + i % stages], (i / stages) & 1))
                            if (global_timer_ns() - t0 > kWaitLimitNs) break;
                };
                drain(kc, L::kKStages, L::kKFull);
                drain(vc, L::kVStages, L::kVFull);
                // (the queries of unit uc, or uc - 1, were the last ones issued)
                for (int i = max(0, uc - 1); i <= uc; ++i)
                    for (int n = 0; n < 1000 && !mbar_try_wait(&bars[L::kQFull], i & 1); ++n) {}
            }
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc_qk = idesc_16_f32<HALF>(128, 128, 0, 0);
            constexpr uint32_t idesc_pv = idesc_16_f32<HALF>(128, D, 0, 1);
            const uint64_t dq = smem_desc_sw128(smem_addr(smem + L::kQ), 16, 1024);
            const uint64_t dk = smem_desc_sw128(smem_addr(smem + L::kK), 16, 1024);
            const uint64_t dv = smem_desc_sw128(smem_addr(smem + L::kV), L::kSub, 1024);
            auto issue_qk = [&](int t, int st) {
                const uint64_t a0 = dq + static_cast<uint64_t>(t * (L::kTile >> 4));
                const uint64_t b0 = dk + static_cast<uint64_t>(st * (L::kTile >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = static_cast<uint64_t>(((kk >> 2) * L::kSub + (kk & 3) * 32) >> 4);
                    umma_ss(tmem + t * 128, a0 + off, b0 + off, idesc_qk, kk > 0 ? 1u : 0u);
                }
                umma_commit(&bars[L::kSFull + t]);
            };
            auto issue_pv = [&](int t, int st, bool acc) {
                const uint64_t b0 = dv + static_cast<uint64_t>(st * (L::kTile >> 4));
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, b0 + static_cast<uint64_t>((kk * 2048) >> 4),
                            idesc_pv, (acc || kk > 0) ? 1u : 0u);
            };
            int kc = 0, vc = 0, uc = 0, fixes = 0, pc[2] = {0, 0};
            bool ok = true;
            for (PromptUnit w; ok && feed.next(&w, false, lane, abort_flag, status); ++uc) {
                ok = mbar_wait(&bars[L::kQFull], uc & 1, abort_flag, status, kStatusMmaWait) &&
                     mbar_wait(&bars[L::kKFull + kc % L::kKStages], (kc / L::kKStages) & 1, abort_flag, status,
                               kStatusMmaWait);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (w.n[t] > 0) issue_qk(t, kc % L::kKStages);
                umma_commit(&bars[L::kKEmpty + kc % L::kKStages]);
                ++kc;
                if (w.n_max == 1) umma_commit(&bars[L::kQEmpty]);
                const bool tail = tail_rows(w) > 0;
                for (int it = 0; ok && it < w.n_max; ++it) {
                    if (it == max(0, w.n_max - 3)) mbar_arrive(&bars[L::kNear]);
                    const int st = vc % L::kVStages;
                    ok = mbar_wait(&bars[L::kVFull + st], (vc / L::kVStages) & 1, abort_flag, status, kStatusMmaWait);
                    if (ok && tail && it == w.n_max - 1) {
                        mbar_arrive(&bars[L::kVAsk]);    // the tile has landed: warp 2 zeroes its tail
                        ok = mbar_wait(&bars[L::kVFix], fixes & 1, abort_flag, status, kStatusMmaWait);
                        ++fixes;
                    }
                    if (!ok) break;
                    const bool next_k = it + 1 < w.n_max;   // (waited for here, not between the products)
                    if (next_k)
                        ok = mbar_wait(&bars[L::kKFull + kc % L::kKStages], (kc / L::kKStages) & 1, abort_flag, status,
                                       kStatusMmaWait);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok || it >= w.n[t]) continue;
                        ok = mbar_wait(&bars[L::kPFull + t], pc[t] & 1, abort_flag, status, kStatusMmaWait);
                        ++pc[t];
                        if (!ok) continue;
                        tc_fence_after();
                        issue_pv(t, st, it > 0);
                        if (it + 1 < w.n[t]) {
                            issue_qk(t, kc % L::kKStages);
                        } else {
                            umma_commit(&bars[L::kOFull + t]);
                        }
                    }
                    if (!ok) break;
                    umma_commit(&bars[L::kVEmpty + st]);
                    ++vc;
                    if (next_k) {
                        umma_commit(&bars[L::kKEmpty + kc % L::kKStages]);
                        ++kc;
                    }
                    if (it + 2 == w.n_max) umma_commit(&bars[L::kQEmpty]);
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
            // ------------------------------------------------ ends of sequences in V
            // (asked by the MMA issuer: a parity wait on the ring itself could be passed by)
            int vc = 0, fixes = 0;
            for (PromptUnit w; feed.next(&w, true, lane, abort_flag, status);) {
                vc += w.n_max;
                const int valid = tail_rows(w);
                if (valid == 0) continue;
                if (!warp_wait_all(&bars[L::kVAsk], fixes & 1, abort_flag, status, kStatusTmaWait)) break;
                ++fixes;
                zero_tail_rows<D>(smem + L::kV + (vc - 1) % L::kVStages * L::kTile, valid, lane);
                if (lane == 0) mbar_arrive(&bars[L::kVFix]);
            }
        } else if (warp == 3 && lane == 0) {
            // ------------------------------------------------ the CTA's units
            // (its own, then one request at a time, when the current unit is near its end: asked for
            // earlier, long units would pile up on the CTAs that began with long ones; none after the
            // first that finds no CTA left)
            PromptUnit *slot = reinterpret_cast<PromptUnit *>(smem + L::kUnits);
            for (int i = 0;; ++i) {
                const int x = i & 1;
                if (!mbar_wait(&bars[L::kUnitEmpty + x], ((i >> 1) & 1) ^ 1, abort_flag, status, kStatusTmaWait)) break;
                slot[x] = unit;
                mbar_arrive(&bars[L::kUnitFull + x]);
                if (unit.n_max < 0 || !mbar_wait(&bars[L::kNear], i & 1, abort_flag, status, kStatusTmaWait)) break;
                mbar_arrive_expect_tx(&bars[L::kAnswer], 16);
                request_cta(smem + L::kAnswerAt, &bars[L::kAnswer]);
                const int u = mbar_wait(&bars[L::kAnswer], i & 1, abort_flag, status, kStatusTmaWait)
                                  ? answered_cta(smem + L::kAnswerAt)
                                  : -1;
                fence_proxy_async_shared();      // the answer has been read before the next one is written
                if (u >= 0)
                    unit = prompt_unit(p, u);
                else
                    unit.n_max = -1;
            }
        }
    } else {
        // ------------------------------------------------ softmax and epilogue
        regs_inc<192>();
        const int t = (warp - 4) >> 2;
        const int row = ((warp & 3) << 5) + lane;    // TMEM lane == row of the query tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) << 5) << 16;
        const uint32_t s_tmem = tmem + lane_base + t * 128, o_tmem = tmem + lane_base + 256 + t * 128;
        int sc = 0, oc = 0;                          // score tiles and accumulators seen so far
        bool ok = true;
        for (PromptUnit w; ok && feed.next(&w, true, lane, abort_flag, status);) {
            const int n = t ? w.n[1] : w.n[0];
            if (n == 0) continue;
            const int i = (t ? w.row0[1] : w.row0[0]) + row;   // the row's place in its sequence
            const int seen = min(w.len, (min(i, w.len - 1) / p.block + 1) * p.block);   // keys it sees
            float m_run = 0.0f, l_run = 0.0f;        // running max of scale log2(e) s, running sum
            for (int it = 0; it < n; ++it, ++sc) {
                ok = warp_wait_all(&bars[L::kSFull + t], sc & 1, abort_flag, status, kStatusSoftmaxWait);
                if (!ok) break;
                tc_fence_after();
                ScoreRow r;
                load_scores(s_tmem, r);
                const int valid = seen - it * 128;
                if (__any_sync(0xffffffffu, valid < 128)) mask_scores(r, valid);
                const float m_tile = max_score(r) * p.scale_log2;
                bool rescale = false;
                float alpha = 1.0f;
                if (it == 0) {                       // (every row sees its sequence's first key)
                    m_run = m_tile;
                } else if (m_tile > m_run + kCoreRescale) {
                    rescale = true;
                    alpha = ex2_approx(m_run - m_tile);
                    l_run *= alpha;
                    m_run = m_tile;
                }
                l_run += exp_store<HALF>(r, p.scale_log2, -m_run, s_tmem);
                // O_t is idle: PV(t, it - 1) completed before S(t, it) was signalled, and
                // PV(t, it) waits for this thread's arrival below
                if (__any_sync(0xffffffffu, rescale)) rescale_row<D>(o_tmem, alpha);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars[L::kPFull + t]);
            }
            if (!ok) break;
            ok = warp_wait_all(&bars[L::kOFull + t], oc & 1, abort_flag, status, kStatusSoftmaxWait);
            ++oc;
            if (!ok) break;
            tc_fence_after();
            const float inv = 1.0f / l_run;
            // 64 columns at a time through shared memory, so that eight lanes write 128 bytes of a row (a
            // thread writing its own row touched 32 lines with every store: 4000 cycles a unit)
            uint8_t *out_tile = smem + L::kOut + (warp - 4) * 4096;
            const int row_first = (t ? w.row0[1] : w.row0[0]) + ((warp & 3) << 5);   // of the warp's rows
            uint16_t *out = p.out + (t ? w.head[1] : w.head[0]) * D + (lane & 7) * 8;
#pragma unroll 1
            for (int h = 0; h < D / 64; ++h) {
#pragma unroll
                for (int cb = 0; cb < 2; ++cb) {
                    uint32_t r[32];
                    tmem_ld32(o_tmem + h * 64 + cb * 32, r);
                    tmem_wait_ld_bind(r);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint4 x;
                        x.x = pack_16x2<HALF>(__uint_as_float(r[8 * v + 0]) * inv, __uint_as_float(r[8 * v + 1]) * inv);
                        x.y = pack_16x2<HALF>(__uint_as_float(r[8 * v + 2]) * inv, __uint_as_float(r[8 * v + 3]) * inv);
                        x.z = pack_16x2<HALF>(__uint_as_float(r[8 * v + 4]) * inv, __uint_as_float(r[8 * v + 5]) * inv);
                        x.w = pack_16x2<HALF>(__uint_as_float(r[8 * v + 6]) * inv, __uint_as_float(r[8 * v + 7]) * inv);
                        *reinterpret_cast<uint4 *>(out_tile + lane * 128 + (((cb * 4 + v) ^ (lane & 7)) << 4)) = x;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int rr = 4 * k + (lane >> 3);
                    const uint4 x = *reinterpret_cast<const uint4 *>(out_tile + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                    if (row_first + rr < w.len)
                        *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(w.first + row_first + rr) * p.out_stride + h * 64) = x;
                }
                __syncwarp();
            }
            tc_fence_before();                       // (the next unit's first PV follows this thread's next arrival)
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

template <int D, bool HALF, int kItems>
static cudaError_t launch_prompt_d(const PromptParams<kItems> &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                   const CUtensorMap &tv, cudaStream_t s) {
    // (an attribute of the current device's copy of the kernel: set once per device)
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(prompt_attention_kernel<D, HALF, kItems>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PromptLayout<D>::kAlloc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return launch_dependent(prompt_attention_kernel<D, HALF, kItems>, dim3(p.n_units), dim3(kAttnThreads),
                            static_cast<size_t>(PromptLayout<D>::kAlloc), s, p, tq, tk, tv);
}

template <int kItems>
cudaError_t launch_prompt(const PromptParams<kItems> &p, const CUtensorMap &tq, const CUtensorMap &tk,
                          const CUtensorMap &tv, int head_dim, bool half, cudaStream_t s) {
    if (head_dim == 64)
        return half ? launch_prompt_d<64, true>(p, tq, tk, tv, s)
                    : launch_prompt_d<64, false>(p, tq, tk, tv, s);
    return half ? launch_prompt_d<128, true>(p, tq, tk, tv, s)
                : launch_prompt_d<128, false>(p, tq, tk, tv, s);
}

template cudaError_t launch_prompt<kPromptSmallItems>(const PromptParams<kPromptSmallItems> &, const CUtensorMap &,
                                                      const CUtensorMap &, const CUtensorMap &, int, bool, cudaStream_t);
template cudaError_t launch_prompt<kPromptLargeItems>(const PromptParams<kPromptLargeItems> &, const CUtensorMap &,
                                                      const CUtensorMap &, const CUtensorMap &, int, bool, cudaStream_t);

cudaError_t prompt_status(uint32_t *word) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_prompt_status, sizeof(uint32_t));
    if (e == cudaSuccess && *word != 0) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_prompt_status, &zero, sizeof(uint32_t));
    }
    return e;
}

}  // namespace sdv2
