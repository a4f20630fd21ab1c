// Internal interface of the attention gradient.
#pragma once

#include "vae_mha.cuh"

namespace vae {

size_t mha_bwd_bytes(const MhaShape& s);
int mha_bwd_run(const vae_attention_desc* a, const MhaShape& s, const void* dout, const void* q, const void* k,
                const void* v, const void* o, const float* lse, void* dq, void* dk, void* dv, void* ws,
                cudaStream_t st);

}  // namespace vae
