// moe_balance_fwd for a caller that keeps the counts for the backward and hands them out too.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// counts_again: where the counts are written once more, or NULL.
moe_status balance_forward(int64_t T, int64_t n_ids, int32_t K, int64_t num_seqs, int32_t mask_ndim, int32_t dtype,
                           const void* logits, const int32_t* topk_idx, const uint8_t* x_active_mask,
                           const int32_t* seq_offsets, float* loss, float* z_loss, int32_t* counts,
                           int32_t* counts_again, int32_t* seq_tokens, void* workspace, size_t ws_bytes, void* stream);

}  // namespace moe
