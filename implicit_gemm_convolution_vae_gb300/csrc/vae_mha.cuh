// Multi-head attention on latent tokens: what the forward and the gradient
// kernels share. Which keys a row sees, argument checks, sizes.
#pragma once

#include "vae_types.cuh"

namespace vae {

struct MhaShape {
    int b, sq, sk, hq, hkv, g, d, block;
    const int *q_len, *k_len;
};

// The valid length of batch entry `e`: lens[e] clamped to [0, n], or n.
__device__ __forceinline__ int mha_len(const int* lens, int e, int n) {
    if (lens == nullptr) return n;
    const int v = __ldg(lens + e);
    return v < 0 ? 0 : (v > n ? n : v);
}

// Query i sees the keys [0, limit): the whole valid length, or up to the end of
// the block that its position i + kl - ql lies in.
__device__ __forceinline__ int mha_key_limit(int i, int ql, int kl, int block) {
    if (block <= 0) return kl;
    const int at = i + kl - ql;
    if (at < 0) return 0;
    const long long end = (static_cast<long long>(at) / block + 1) * block;
    return end < kl ? static_cast<int>(end) : kl;
}

// Checks the desc (backward: the gradients' strides too); fills `s`.
int mha_check(const vae_attention_desc* d, bool backward, MhaShape* s);

}  // namespace vae
