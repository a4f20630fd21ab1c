// Multi-head attention on latent tokens: the public entry points, their
// argument checks and the tensor maps that the kernels share.
#include <cmath>

#include "vae_mha_bwd.h"
#include "vae_mha_fwd.h"
#include "vae_overlap.h"

namespace vae {

namespace {

// A tensor of a call, for the check that what is written shares no memory with anything else.
struct MhaPart {
    const char* name;
    Extent at;
    bool written;
};
int mha_apart(const MhaPart* t, int count) {
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < i; ++j)
            if ((t[i].written || t[j].written) && extents_meet(t[i].at, t[j].at))
                return set_error(VAE_ERR_ARG, "attention: %s may not overlap %s", t[i].name, t[j].name);
    return VAE_OK;
}
Extent lens_extent(const int* lens, int b) { return extent_dense(lens, lens != nullptr ? static_cast<size_t>(b) * sizeof(int) : 0); }

}  // namespace

int mha_check(const vae_attention_desc* a, bool backward, MhaShape* s) {
    if (a == nullptr) return set_error(VAE_ERR_ARG, "attention: NULL desc");
    if (a->type != VAE_F16 && a->type != VAE_BF16)
        return set_error(VAE_ERR_ARG, "attention: f16 and bf16 tensors are taken");
    if (a->b < 1 || a->sq < 1 || a->sk < 1 || a->hq < 1 || a->hkv < 1)
        return set_error(VAE_ERR_SHAPE, "attention: b, sq, sk, hq, hkv >= 1 are needed");
    if (a->hq % a->hkv != 0)
        return set_error(VAE_ERR_SHAPE, "attention: %d query heads do not share %d key heads", a->hq, a->hkv);
    if (a->d < 8 || a->d > 128 || a->d % 8 != 0)
        return set_error(VAE_ERR_SHAPE, "attention: d must be a multiple of 8 from 8 to 128, got %d", a->d);
    if (!(a->scale > 0.f) || !std::isfinite(a->scale))
        return set_error(VAE_ERR_ARG, "attention: scale must be > 0 and finite");
    if (a->block < 0) return set_error(VAE_ERR_ARG, "attention: block must be >= 0");
    if (static_cast<long long>(a->b) * a->hq * a->sq > 0x7fffff00LL ||
        static_cast<long long>(a->b) * a->hkv * a->sk > 0x7fffff00LL)
        return set_error(VAE_ERR_SHAPE, "attention: over 2^31 - 256 rows");
    const struct {
        const char* name;
        const long long* st;
        int n, h;
    } t[8] = {{"q", a->q_stride, a->sq, a->hq},   {"k", a->k_stride, a->sk, a->hkv},  {"v", a->v_stride, a->sk, a->hkv},
              {"o", a->o_stride, a->sq, a->hq},   {"do", a->do_stride, a->sq, a->hq}, {"dq", a->dq_stride, a->sq, a->hq},
              {"dk", a->dk_stride, a->sk, a->hkv}, {"dv", a->dv_stride, a->sk, a->hkv}};
    for (int i = 0; i < (backward ? 8 : 4); ++i) {
        const int dim[3] = {a->b, t[i].n, t[i].h};
        const bool written = i == 3 || i > 4;  // rows of o, dq, dk, dv must not lie in one another
        for (int k = 0; k < 3; ++k)
            if (dim[k] > 1 && (t[i].st[k] < (written ? a->d : 8) || t[i].st[k] % 8 != 0 || t[i].st[k] >= (1LL << 38)))
                return set_error(VAE_ERR_SHAPE, "attention: %s's strides must be positive multiples of 8, and d at least where it is written "
                                 "(stride %d: %lld)", t[i].name, k, t[i].st[k]);
        if (written && extent_folds(extent_tokens(nullptr, t[i].st, a->b, t[i].n, t[i].h, a->d, 2)))
            return set_error(VAE_ERR_SHAPE, "attention: rows of %s lie in one another", t[i].name);
    }
    s->b = a->b;
    s->sq = a->sq;
    s->sk = a->sk;
    s->hq = a->hq;
    s->hkv = a->hkv;
    s->g = a->hq / a->hkv;
    s->d = a->d;
    s->block = a->block;
    s->fill = a->fill != 0;
    // gp: the largest power of two in g, half a tile's rows at most
    s->gp_log2 = 0;
    while (s->gp_log2 < 6 && s->g % (2 << s->gp_log2) == 0) ++s->gp_log2;
    s->nsub = s->g >> s->gp_log2;
    const long long rows = static_cast<long long>(a->sq) << s->gp_log2;
    s->ntile = static_cast<int>((rows + kMhaTile - 1) / kMhaTile);
    s->nkb = (a->sk - 1) / kMhaTile + 1;
    s->q_len = a->q_len_dev;
    s->k_len = a->k_len_dev;
    return VAE_OK;
}

int mha_map(CUtensorMap* map, const vae_attention_desc* a, const void* p, const long long* stride, int n, int h,
            int heads, int tokens) {
    const uint64_t dims[4] = {static_cast<uint64_t>(a->d), static_cast<uint64_t>(h), static_cast<uint64_t>(n),
                              static_cast<uint64_t>(a->b)};
    // (the stride of a dimension of one is never used: any valid value)
    const uint64_t st[3] = {h > 1 ? static_cast<uint64_t>(stride[2]) * 2 : 16,
                            n > 1 ? static_cast<uint64_t>(stride[1]) * 2 : 16,
                            a->b > 1 ? static_cast<uint64_t>(stride[0]) * 2 : 16};
    const uint32_t box[4] = {64, static_cast<uint32_t>(heads), static_cast<uint32_t>(tokens), 1};
    return encode_tiled(map, a->type == VAE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace vae

using namespace vae;

extern "C" {

size_t vae_attention_workspace_bytes(const vae_attention_desc* desc) {
    clear_error();
    MhaShape s;
    return mha_check(desc, false, &s) == VAE_OK ? mha_fwd_bytes(s) : 0;
}

int vae_attention(const vae_attention_desc* desc, const void* q_dev, const void* k_dev, const void* v_dev, void* o_dev,
                  float* lse_dev, void* workspace_dev, size_t workspace_bytes, vae_stream_t stream) {
    clear_error();
    MhaShape s;
    int rc = mha_check(desc, false, &s);
    if (rc != VAE_OK) return rc;
    if (q_dev == nullptr || k_dev == nullptr || v_dev == nullptr || o_dev == nullptr || lse_dev == nullptr)
        return set_error(VAE_ERR_ARG, "attention: NULL tensor");
    if (!aligned16(q_dev) || !aligned16(k_dev) || !aligned16(v_dev) || !aligned16(o_dev) || !aligned16(lse_dev) ||
        !aligned16(workspace_dev))
        return set_error(VAE_ERR_ALIGN, "attention: pointers must be 16-byte aligned");
    if (o_dev == q_dev || o_dev == k_dev || o_dev == v_dev)
        return set_error(VAE_ERR_ARG, "attention: o may not be q, k or v");
    const size_t need = mha_fwd_bytes(s);
    if (need > 0 && (workspace_dev == nullptr || workspace_bytes < need))
        return set_error(VAE_ERR_NOMEM, "attention: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    const auto tokens = [&](const void* p, const long long* st, int n, int h) { return extent_tokens(p, st, s.b, n, h, s.d, 2); };
    const MhaPart parts[] = {{"q", tokens(q_dev, desc->q_stride, s.sq, s.hq), false},
                             {"k", tokens(k_dev, desc->k_stride, s.sk, s.hkv), false},
                             {"v", tokens(v_dev, desc->v_stride, s.sk, s.hkv), false},
                             {"q_len", lens_extent(s.q_len, s.b), false},
                             {"k_len", lens_extent(s.k_len, s.b), false},
                             {"o", tokens(o_dev, desc->o_stride, s.sq, s.hq), true},
                             {"lse", extent_dense(lse_dev, static_cast<size_t>(s.b) * s.hq * s.sq * sizeof(float)), true},
                             {"the workspace", extent_dense(workspace_dev, need), need > 0}};
    if ((rc = mha_apart(parts, need > 0 ? 8 : 7)) != VAE_OK) return rc;
    if ((rc = check_device()) != VAE_OK) return rc;
    return mha_fwd_run(desc, s, q_dev, k_dev, v_dev, o_dev, lse_dev, workspace_dev,
                       reinterpret_cast<cudaStream_t>(stream));
}

size_t vae_attention_backward_workspace_bytes(const vae_attention_desc* desc) {
    clear_error();
    MhaShape s;
    return mha_check(desc, true, &s) == VAE_OK ? mha_bwd_bytes(s) : 0;
}

int vae_attention_backward(const vae_attention_desc* desc, const void* do_dev, const void* q_dev, const void* k_dev,
                           const void* v_dev, const void* o_dev, const float* lse_dev, void* dq_dev, void* dk_dev,
                           void* dv_dev, void* workspace_dev, size_t workspace_bytes, vae_stream_t stream) {
    clear_error();
    MhaShape s;
    int rc = mha_check(desc, true, &s);
    if (rc != VAE_OK) return rc;
    const void* all[10] = {do_dev, q_dev, k_dev, v_dev, o_dev, lse_dev, dq_dev, dk_dev, dv_dev, workspace_dev};
    for (const void* p : all)
        if (p == nullptr) return set_error(VAE_ERR_ARG, "attention: NULL tensor or workspace");
    for (const void* p : all)
        if (!aligned16(p)) return set_error(VAE_ERR_ALIGN, "attention: pointers must be 16-byte aligned");
    const void* in[5] = {do_dev, q_dev, k_dev, v_dev, o_dev};
    for (const void* p : in)
        if (p == dq_dev || p == dk_dev || p == dv_dev)
            return set_error(VAE_ERR_ARG, "attention: a gradient may not be written over an input");
    if (dq_dev == dk_dev || dq_dev == dv_dev || dk_dev == dv_dev)
        return set_error(VAE_ERR_ARG, "attention: dq, dk and dv must be tensors of their own");
    const size_t need = mha_bwd_bytes(s);
    if (workspace_bytes < need)
        return set_error(VAE_ERR_NOMEM, "attention: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    const auto tokens = [&](const void* p, const long long* st, int n, int h) { return extent_tokens(p, st, s.b, n, h, s.d, 2); };
    const MhaPart parts[] = {{"do", tokens(do_dev, desc->do_stride, s.sq, s.hq), false},
                             {"q", tokens(q_dev, desc->q_stride, s.sq, s.hq), false},
                             {"k", tokens(k_dev, desc->k_stride, s.sk, s.hkv), false},
                             {"v", tokens(v_dev, desc->v_stride, s.sk, s.hkv), false},
                             {"o", tokens(o_dev, desc->o_stride, s.sq, s.hq), false},
                             {"lse", extent_dense(lse_dev, static_cast<size_t>(s.b) * s.hq * s.sq * sizeof(float)), false},
                             {"q_len", lens_extent(s.q_len, s.b), false},
                             {"k_len", lens_extent(s.k_len, s.b), false},
                             {"dq", tokens(dq_dev, desc->dq_stride, s.sq, s.hq), true},
                             {"dk", tokens(dk_dev, desc->dk_stride, s.sk, s.hkv), true},
                             {"dv", tokens(dv_dev, desc->dv_stride, s.sk, s.hkv), true},
                             {"the workspace", extent_dense(workspace_dev, need), true}};
    if ((rc = mha_apart(parts, 12)) != VAE_OK) return rc;
    if ((rc = check_device()) != VAE_OK) return rc;
    return mha_bwd_run(desc, s, do_dev, q_dev, k_dev, v_dev, o_dev, lse_dev, dq_dev, dk_dev, dv_dev, workspace_dev,
                       reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
