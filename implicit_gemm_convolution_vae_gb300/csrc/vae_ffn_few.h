// The gated feed-forward block on few tokens (see vae_ffn_few.cu).
#pragma once

#include "vae_common.cuh"

namespace vae {

constexpr int kFewTokens = 32;  // at most

// Both products of the block; gate and up may be NULL. Arguments as vae_gated_ffn's, checked before; `rest` [m][f] holds
// what the rounding of hidden left.
int ffn_few(const vae_gated_ffn_desc& a, const void* x, const void* wg, const void* wu, const void* wd, const float* residual, void* y,
            void* gate, void* up, void* hidden, void* rest, cudaStream_t stream);

}  // namespace vae
