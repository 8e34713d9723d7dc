// Host side of sdv2_prompt_attention: argument checks, the order of the work units, TMA
// descriptors and launches.
#include <algorithm>
#include <cmath>
#include <memory>
#include <vector>

#include "host_common.h"
#include "token_ops.h"

using namespace sdv2;

namespace {

// Tensor map of a packed 16-bit tensor (d, heads, tokens) in boxes of 64 channels x 1 head
// x 128 tokens, 128-byte swizzle (the layout of the MMA's operand tiles).
bool map_tokens(CUtensorMap *m, const void *ptr, bool half, int64_t d, int64_t heads, int64_t tokens, int64_t stride) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, 128}, estr[3] = {1, 1, 1};
    return get_encode_fn()(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Item {
    uint32_t code;      // sequence << 24 | row tile
    int32_t tiles;      // KV tiles it sees
};

// Row tiles of the launch's sequences, longest first: a counting sort by their KV tiles, so
// that equal ones keep their order and the cost stays linear.
void order_items(const int32_t *len, int n_seqs, int rows, int64_t block, std::vector<uint32_t> *out) {
    std::vector<Item> items;
    int32_t most = 0;
    for (int s = 0; s < n_seqs; ++s)
        for (int32_t r = 0; r < len[s]; r += rows) {
            const int64_t last = std::min(r + rows, len[s]) - 1;
            const int64_t seen = std::min<int64_t>(len[s], (last / block + 1) * block);
            const int32_t tiles = static_cast<int32_t>((seen + 127) / 128);
            items.push_back({static_cast<uint32_t>(s) << 24 | static_cast<uint32_t>(r / rows), tiles});
            most = std::max(most, tiles);
        }
    std::vector<int32_t> at(static_cast<size_t>(most) + 2, 0);
    for (const Item &i : items) ++at[most - i.tiles + 1];
    for (int32_t i = 1; i <= most; ++i) at[i] += at[i - 1];
    out->resize(items.size());
    for (const Item &i : items) (*out)[at[most - i.tiles]++] = i.code;
}

template <int kItems>
sdv2_status launch_items(const sdv2_prompt_config &c, void *out, int64_t out_stride, float scale, const int32_t *first,
                         const int32_t *len, int n_seqs, const uint32_t *items, int n_items, bool pair,
                         const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    // (every field and entry that the kernel reads is set below)
    std::unique_ptr<PromptParams<kItems>> p(new PromptParams<kItems>);
    p->out = static_cast<uint16_t *>(out);
    p->out_stride = out_stride;
    p->group = c.heads / c.kv_heads;
    p->block = c.block_tokens;
    p->pair_heads = pair ? 1 : 0;
    p->head_units = pair ? c.heads / 2 : c.heads;
    p->n_items = n_items;
    p->n_units = n_items * p->head_units;
    // Head units in as many chunks as keep a chunk's keys and values within 48 MB of the L2, so that
    // they come from memory once (8192 tokens, 40 heads x 128, 168 MB: 271 MB read instead of 930,
    // 766 us under the power limit instead of 810; 64, 32 and 20 MB: 769, 770 and 770).
    int64_t keys = 0;
    for (int i = 0; i < n_seqs; ++i) keys += len[i];
    const int64_t kv_bytes = keys * c.kv_heads * c.head_dim * 4, chunk_bytes = 48ll << 20;
    const int64_t chunks = std::min<int64_t>(p->head_units, (kv_bytes + chunk_bytes - 1) / chunk_bytes);
    p->chunk_units = static_cast<int32_t>((p->head_units + chunks - 1) / chunks);
    p->scale_log2 = scale * 1.4426950408889634f;
    std::copy(first, first + n_seqs, p->seq_first);
    std::copy(len, len + n_seqs, p->seq_len);
    std::copy(items, items + n_items, p->item);
    cudaError_t e = launch_prompt<kItems>(*p, tq, tk, tv, c.head_dim, c.dtype == SDV2_DT_FP16, s);
    if (e != cudaSuccess) return cuda_fail(e, "prompt_attention launch");
    count_launch();
    return SDV2_OK;
}

sdv2_status prompt_attention(const sdv2_prompt_config *cfg, const void *q, const void *k, const void *v, void *out,
                             const int64_t *offsets, int32_t n_seqs, float scale, cudaStream_t s) {
    if (!cfg || !q || !k || !v || !out || !offsets) return fail(SDV2_E_ARG, "NULL argument");
    sdv2_prompt_config c = *cfg;
    if (c.head_dim != 64 && c.head_dim != 128) return fail(SDV2_E_SHAPE, "head_dim must be 64 or 128");
    if (c.heads < 1 || c.kv_heads < 1 || c.heads % c.kv_heads != 0 || c.heads > 1024)
        return fail(SDV2_E_SHAPE, "heads must be a multiple of kv_heads, in 1..1024");
    if (c.block_tokens < 1) return fail(SDV2_E_SHAPE, "block_tokens must be >= 1");
    if (c.dtype != SDV2_DT_BF16 && c.dtype != SDV2_DT_FP16)
        return fail(SDV2_E_SHAPE, "dtype must be SDV2_DT_BF16 or SDV2_DT_FP16");
    if (n_seqs < 0) return fail(SDV2_E_ARG, "n_seqs must be >= 0");
    if (c.tokens < 0 || c.tokens >= (1ll << 30)) return fail(SDV2_E_SHAPE, "tokens must be in 0..2^30 - 1");
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(SDV2_E_ARG, "softmax_scale must be > 0");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return fail(SDV2_E_ALIGN, "q, k, v and out must be 16-byte aligned");
    int64_t *strides[4] = {&c.q_stride, &c.k_stride, &c.v_stride, &c.out_stride};
    for (int i = 0; i < 4; ++i) {
        const int64_t row = static_cast<int64_t>(i == 0 || i == 3 ? c.heads : c.kv_heads) * c.head_dim;
        if (*strides[i] == 0) *strides[i] = row;
        if (*strides[i] < row || *strides[i] >= (1ll << 38))
            return fail(SDV2_E_SHAPE, "a token stride is shorter than a token's row, or too long");
        if (*strides[i] % 8 != 0) return fail(SDV2_E_ALIGN, "token strides must be multiples of 8 elements");
    }
    if (n_seqs > 0 && (offsets[0] < 0 || offsets[n_seqs] > c.tokens))
        return fail(SDV2_E_ARG, "offsets must lie in 0..tokens");
    for (int32_t i = 0; i < n_seqs; ++i) {
        if (offsets[i + 1] < offsets[i]) return fail(SDV2_E_ARG, "offsets must not decrease");
        // (a CTA's work on one query tile stays well below the bound of its waits)
        if (offsets[i + 1] - offsets[i] > (1 << 25)) return fail(SDV2_E_SHAPE, "a sequence has more than 2^25 tokens");
    }
    if (n_seqs == 0 || offsets[n_seqs] == offsets[0]) return SDV2_OK;
    // a block longer than every sequence is the same mask as one that long (keeps the
    // kernel's (i / block + 1) * block below 2^31)
    c.block_tokens = static_cast<int32_t>(std::min<int64_t>(c.block_tokens, c.tokens));

    if (!get_encode_fn()) return fail(SDV2_E_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const bool half = c.dtype == SDV2_DT_FP16;
    CUtensorMap tq, tk, tv;
    if (!map_tokens(&tq, q, half, c.head_dim, c.heads, c.tokens, c.q_stride) ||
        !map_tokens(&tk, k, half, c.head_dim, c.kv_heads, c.tokens, c.k_stride) ||
        !map_tokens(&tv, v, half, c.head_dim, c.kv_heads, c.tokens, c.v_stride))
        return fail(SDV2_E_CUDA, "cuTensorMapEncodeTiled failed");
    // Even groups: a unit is two heads of one key head on the same 128 rows (finer units,
    // both tiles see the same keys); otherwise 256 consecutive rows of one head.
    const bool pair = (c.heads / c.kv_heads) % 2 == 0;
    std::vector<uint32_t> items;
    int32_t first[kPromptMaxSeqs], len[kPromptMaxSeqs];
    for (int32_t s0 = 0; s0 < n_seqs;) {
        int n = 0;
        for (; s0 < n_seqs && n < kPromptMaxSeqs; ++s0) {
            if (offsets[s0 + 1] == offsets[s0]) continue;
            first[n] = static_cast<int32_t>(offsets[s0]);
            len[n++] = static_cast<int32_t>(offsets[s0 + 1] - offsets[s0]);
        }
        order_items(len, n, pair ? 128 : 256, c.block_tokens, &items);
        for (size_t i = 0; i < items.size(); i += kPromptLargeItems) {
            const int m = static_cast<int>(std::min<size_t>(items.size() - i, kPromptLargeItems));
            const sdv2_status st =
                m <= kPromptSmallItems
                    ? launch_items<kPromptSmallItems>(c, out, c.out_stride, scale, first, len, n, items.data() + i, m,
                                                      pair, tq, tk, tv, s)
                    : launch_items<kPromptLargeItems>(c, out, c.out_stride, scale, first, len, n, items.data() + i, m,
                                                      pair, tq, tk, tv, s);
            if (st != SDV2_OK) return st;
        }
    }
    return SDV2_OK;
}

}  // namespace

extern "C" {

sdv2_status sdv2_prompt_attention(const sdv2_prompt_config *cfg, const void *q, const void *k, const void *v, void *out,
                                  const int64_t *offsets, int32_t n_seqs, float softmax_scale, sdv2_stream stream) {
    try {
        return prompt_attention(cfg, q, k, v, out, offsets, n_seqs, softmax_scale,
                                reinterpret_cast<cudaStream_t>(stream));
    } catch (...) {
        return fail(SDV2_E_STATE, "prompt_attention: out of host memory");
    }
}

sdv2_status sdv2_prompt_check(void) {
    cudaError_t e = cudaDeviceSynchronize();
    uint32_t word = 0;
    if (e == cudaSuccess) e = prompt_status(&word);
    if (e != cudaSuccess) return cuda_fail(e, "prompt_check");
    if (word != 0) return fail(SDV2_E_DEVICE, "device status 0x%x (a kernel gave up on a bounded wait)", word);
    return SDV2_OK;
}

}  // extern "C"
