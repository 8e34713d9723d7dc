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

// Work units u = item * head_units + j.  pair_heads: unit j is query heads 2j and 2j + 1
// (one key head) on the item's 128 rows; otherwise head j on the item's 256 rows.
template <int kItems>
struct PromptParams {
    uint16_t *out;
    int64_t out_stride;                   // elements between tokens
    int32_t group, block, pair_heads, head_units, n_units;
    float scale_log2;                     // softmax_scale * log2(e)
    int32_t seq_first[kPromptMaxSeqs];    // first token and tokens of each sequence
    int32_t seq_len[kPromptMaxSeqs];
    uint32_t item[kItems];                // sequence << 24 | row tile, longest first
};

template <int kItems>
cudaError_t launch_prompt(const PromptParams<kItems> &p, const CUtensorMap &tq, const CUtensorMap &tk,
                          const CUtensorMap &tv, int head_dim, bool half, int sm_count, cudaStream_t s);
// Reads and clears the device word in which the prompt kernels record waits that ran out.
cudaError_t prompt_status(uint32_t *word);

}  // namespace sdv2
