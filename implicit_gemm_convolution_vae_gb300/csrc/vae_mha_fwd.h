// Internal interface of the attention forward kernel.
#pragma once

#include <mutex>

#include "vae_mha.cuh"

namespace vae {

size_t mha_fwd_bytes(const MhaShape& s);
int mha_fwd_run(const vae_attention_desc* a, const MhaShape& s, const void* q, const void* k, const void* v, void* o,
                float* lse, void* ws, cudaStream_t st);

}  // namespace vae
