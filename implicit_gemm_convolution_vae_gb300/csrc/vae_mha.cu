// Multi-head attention on latent tokens and its gradient (public entry points
// at the end).
//
// The gradient: four threads share a row and hold a quarter of its channels
// each in registers; the other side's rows pass through shared memory in tiles
// of 32, converted to f32. It runs twice over the pairs: once per query row for dq, once per
// key row (over the queries and the heads that share the key) for dk and dv;
// the probabilities are recomputed from lse in both, and nothing is added
// across threads in an order that could change.
#include <cmath>

#include "vae_mha_fwd.h"

namespace vae {

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
        for (int k = 0; k < 3; ++k)
            if (dim[k] > 1 && (t[i].st[k] < 8 || t[i].st[k] % 8 != 0 || t[i].st[k] >= (1LL << 38)))
                return set_error(VAE_ERR_SHAPE, "attention: %s's strides must be positive multiples of 8 (stride %d: %lld)",
                                 t[i].name, k, t[i].st[k]);
    }
    s->b = a->b;
    s->sq = a->sq;
    s->sk = a->sk;
    s->hq = a->hq;
    s->hkv = a->hkv;
    s->g = a->hq / a->hkv;
    s->d = a->d;
    s->block = a->block;
    // gp: the largest power of two in g, a tile's rows at most
    s->gp_log2 = 0;
    while (s->gp_log2 < 7 && s->g % (2 << s->gp_log2) == 0) ++s->gp_log2;
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

namespace {

constexpr int kTile = 32;     // rows of the other side in shared memory
constexpr int kRows = 64;     // rows per block
constexpr int kThreads = 256;  // four per row
constexpr int kQuarter = 32;  // channels per thread, at most
constexpr int kPitch = 132;   // floats of a shared row

struct Strides {
    long long b, s, h;
};
inline Strides strides(const long long* st) { return {st[0], st[1], st[2]}; }

template <int T>
__device__ __forceinline__ void load_row_q(const void* p, long long off, int d, int part, bool live, float (&v)[kQuarter]) {
    const typename Elem<T>::type* x = static_cast<const typename Elem<T>::type*>(p) + off;
#pragma unroll
    for (int e = 0; e < kQuarter; e += 8) {
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        // eights part, part + 4, ... of the row
        const int at = (e / 8 * 4 + part) * 8;
        if (live && at < d) load8<T>(x + at, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[e + k] = t[k];
    }
}

// Rows [r0, r0 + kTile) of x into shared memory as f32; 0 behind n or d.
template <int T>
__device__ __forceinline__ void load_tile(const void* p, long long off, long long stride, int r0, int n, int d,
                                          float (*s)[kPitch]) {
    const typename Elem<T>::type* x = static_cast<const typename Elem<T>::type*>(p) + off;
    for (int i = threadIdx.x; i < kTile * 16; i += kThreads) {
        const int r = i / 16, c = i % 16 * 8;
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r0 + r < n && c < d) load8<T>(x + (r0 + r) * stride + c, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[r][c + k] = t[k];
    }
}
__device__ __forceinline__ float part_dot(const float (&a)[kQuarter], const float* s, int part) {
    float r = 0.f;
#pragma unroll
    for (int e = 0; e < kQuarter; ++e) r += a[e] * s[(e / 8 * 4 + part) * 8 + e % 8];
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    return r + __shfl_xor_sync(0xffffffffu, r, 2);
}
__device__ __forceinline__ void part_axpy(float (&a)[kQuarter], float w, const float* s, int part) {
#pragma unroll
    for (int e = 0; e < kQuarter; ++e) a[e] += w * s[(e / 8 * 4 + part) * 8 + e % 8];
}
template <int T>
__device__ __forceinline__ void store_row_q(void* p, long long off, int d, int part, const float (&v)[kQuarter], float w) {
    typename Elem<T>::type* x = static_cast<typename Elem<T>::type*>(p) + off;
#pragma unroll
    for (int e = 0; e < kQuarter; e += 8) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = v[e + k] * w;
        const int at = (e / 8 * 4 + part) * 8;
        if (at < d) store8<T>(x + at, t);
    }
}

// D = sum(do * o) of each row.
template <int T>
__global__ void __launch_bounds__(kThreads) mha_delta_kernel(MhaShape s, const void* dout, Strides ds, const void* o,
                                                             Strides os, float* delta) {
    pdl_wait();
    const int e = blockIdx.z, h = blockIdx.y, part = threadIdx.x & 3;
    const int i = blockIdx.x * kRows + threadIdx.x / 4;
    const bool live = i < mha_len(s.q_len, e, s.sq);
    float a[kQuarter], b[kQuarter];
    load_row_q<T>(dout, e * ds.b + static_cast<long long>(i) * ds.s + h * ds.h, s.d, part, live, a);
    load_row_q<T>(o, e * os.b + static_cast<long long>(i) * os.s + h * os.h, s.d, part, live, b);
    float r = 0.f;
#pragma unroll
    for (int c = 0; c < kQuarter; ++c) r += a[c] * b[c];
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    r += __shfl_xor_sync(0xffffffffu, r, 2);
    if (live && part == 0) delta[(static_cast<long long>(e) * s.hq + h) * s.sq + i] = r;
}

template <int T>
__global__ void __launch_bounds__(kThreads)
    mha_dq_kernel(MhaShape s, float scale, const void* dout, Strides ds, const void* q, Strides qs, const void* k, Strides ks,
                  const void* v, Strides vs, const float* lse, const float* delta, void* dq, Strides dqs) {
    __shared__ float kt[kTile][kPitch], vt[kTile][kPitch];
    pdl_wait();
    const int e = blockIdx.z, h = blockIdx.y, hk = h / s.g, part = threadIdx.x & 3;
    const int i = blockIdx.x * kRows + threadIdx.x / 4;
    const int ql = mha_len(s.q_len, e, s.sq), kl = mha_len(s.k_len, e, s.sk);
    const int lim = i < ql ? mha_key_limit(i, ql, kl, s.block) : 0;
    const int i1 = min(ql, static_cast<int>(blockIdx.x + 1) * kRows) - 1;
    const int blim = i1 >= static_cast<int>(blockIdx.x) * kRows ? mha_key_limit(i1, ql, kl, s.block) : 0;
    float a[kQuarter], g[kQuarter], acc[kQuarter];
    load_row_q<T>(q, e * qs.b + static_cast<long long>(i) * qs.s + h * qs.h, s.d, part, i < ql, a);
    load_row_q<T>(dout, e * ds.b + static_cast<long long>(i) * ds.s + h * ds.h, s.d, part, i < ql, g);
#pragma unroll
    for (int c = 0; c < kQuarter; ++c) acc[c] = 0.f;
    const long long row = (static_cast<long long>(e) * s.hq + h) * s.sq + i;
    const float L = i < ql ? lse[row] : 0.f, D = i < ql ? delta[row] : 0.f;
    for (int j0 = 0; j0 < blim; j0 += kTile) {
        __syncthreads();
        load_tile<T>(k, e * ks.b + hk * ks.h, ks.s, j0, kl, s.d, kt);
        load_tile<T>(v, e * vs.b + hk * vs.h, vs.s, j0, kl, s.d, vt);
        __syncthreads();
        for (int j = 0; j < kTile; ++j) {
            const float x = part_dot(a, kt[j], part) * scale, dp = part_dot(g, vt[j], part);
            if (j0 + j < lim) part_axpy(acc, expf(x - L) * (dp - D), kt[j], part);
        }
    }
    if (i < ql) store_row_q<T>(dq, e * dqs.b + static_cast<long long>(i) * dqs.s + h * dqs.h, s.d, part, acc, scale);
}

template <int T>
__global__ void __launch_bounds__(kThreads)
    mha_dkv_kernel(MhaShape s, float scale, const void* dout, Strides ds, const void* q, Strides qs, const void* k, Strides ks,
                   const void* v, Strides vs, const float* lse, const float* delta, void* dk, Strides dks, void* dv,
                   Strides dvs) {
    __shared__ float qt[kTile][kPitch], gt[kTile][kPitch];
    __shared__ float lt[kTile], dt[kTile];
    pdl_wait();
    const int e = blockIdx.z, hk = blockIdx.y, part = threadIdx.x & 3;
    const int j = blockIdx.x * kRows + threadIdx.x / 4;
    const int ql = mha_len(s.q_len, e, s.sq), kl = mha_len(s.k_len, e, s.sk);
    float a[kQuarter], b[kQuarter], ak[kQuarter], av[kQuarter];
    load_row_q<T>(k, e * ks.b + static_cast<long long>(j) * ks.s + hk * ks.h, s.d, part, j < kl, a);
    load_row_q<T>(v, e * vs.b + static_cast<long long>(j) * vs.s + hk * vs.h, s.d, part, j < kl, b);
#pragma unroll
    for (int c = 0; c < kQuarter; ++c) ak[c] = av[c] = 0.f;
    if (static_cast<int>(blockIdx.x) * kRows >= kl) return;
    for (int h = hk * s.g; h < (hk + 1) * s.g; ++h)
        for (int i0 = 0; i0 < ql; i0 += kTile) {
            __syncthreads();
            load_tile<T>(q, e * qs.b + h * qs.h, qs.s, i0, ql, s.d, qt);
            load_tile<T>(dout, e * ds.b + h * ds.h, ds.s, i0, ql, s.d, gt);
            if (threadIdx.x < kTile && i0 + static_cast<int>(threadIdx.x) < ql) {
                const long long row = (static_cast<long long>(e) * s.hq + h) * s.sq + i0 + threadIdx.x;
                lt[threadIdx.x] = lse[row];
                dt[threadIdx.x] = delta[row];
            }
            __syncthreads();
            for (int i = 0; i < kTile && i0 + i < ql; ++i) {
                const float x = part_dot(a, qt[i], part) * scale, dp = part_dot(b, gt[i], part);
                if (j >= mha_key_limit(i0 + i, ql, kl, s.block)) continue;
                const float p = expf(x - lt[i]);
                part_axpy(av, p, gt[i], part);
                part_axpy(ak, p * (dp - dt[i]), qt[i], part);
            }
        }
    if (j >= kl) return;
    store_row_q<T>(dk, e * dks.b + static_cast<long long>(j) * dks.s + hk * dks.h, s.d, part, ak, scale);
    store_row_q<T>(dv, e * dvs.b + static_cast<long long>(j) * dvs.s + hk * dvs.h, s.d, part, av, 1.f);
}

size_t bwd_bytes(const MhaShape& s) {
    return (static_cast<size_t>(s.b) * s.hq * s.sq * sizeof(float) + 15) / 16 * 16;
}

template <int T>
cudaError_t bwd_launch(const vae_attention_desc* a, const MhaShape& s, const void* dout, const void* q, const void* k,
                       const void* v, const void* o, const float* lse, void* dq, void* dk, void* dv, float* delta,
                       cudaStream_t st) {
    const dim3 gq((s.sq + kRows - 1) / kRows, s.hq, s.b), gk((s.sk + kRows - 1) / kRows, s.hkv, s.b);
    cudaError_t e = launch_kernel(mha_delta_kernel<T>, gq, dim3(kThreads), 0, st, s, dout, strides(a->do_stride), o,
                                  strides(a->o_stride), delta);
    if (e != cudaSuccess) return e;
    e = launch_kernel(mha_dq_kernel<T>, gq, dim3(kThreads), 0, st, s, a->scale, dout, strides(a->do_stride), q,
                      strides(a->q_stride), k, strides(a->k_stride), v, strides(a->v_stride), lse,
                      static_cast<const float*>(delta), dq, strides(a->dq_stride));
    if (e != cudaSuccess) return e;
    return launch_kernel(mha_dkv_kernel<T>, gk, dim3(kThreads), 0, st, s, a->scale, dout, strides(a->do_stride), q,
                         strides(a->q_stride), k, strides(a->k_stride), v, strides(a->v_stride), lse,
                         static_cast<const float*>(delta), dk, strides(a->dk_stride), dv, strides(a->dv_stride));
}

}  // namespace
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
    const size_t need = mha_fwd_bytes(s);
    if (need > 0 && (workspace_dev == nullptr || workspace_bytes < need))
        return set_error(VAE_ERR_NOMEM, "attention: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((rc = check_device()) != VAE_OK) return rc;
    return mha_fwd_run(desc, s, q_dev, k_dev, v_dev, o_dev, lse_dev, workspace_dev,
                       reinterpret_cast<cudaStream_t>(stream));
}

size_t vae_attention_backward_workspace_bytes(const vae_attention_desc* desc) {
    clear_error();
    MhaShape s;
    return mha_check(desc, true, &s) == VAE_OK ? bwd_bytes(s) : 0;
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
    if (workspace_bytes < bwd_bytes(s))
        return set_error(VAE_ERR_NOMEM, "attention: workspace of %zu bytes, %zu needed", workspace_bytes, bwd_bytes(s));
    if ((rc = check_device()) != VAE_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float* delta = static_cast<float*>(workspace_dev);
    VAE_CUDA_CHECK(desc->type == VAE_F16
                       ? bwd_launch<VAE_F16>(desc, s, do_dev, q_dev, k_dev, v_dev, o_dev, lse_dev, dq_dev, dk_dev,
                                             dv_dev, delta, st)
                       : bwd_launch<VAE_BF16>(desc, s, do_dev, q_dev, k_dev, v_dev, o_dev, lse_dev, dq_dev, dk_dev,
                                              dv_dev, delta, st));
    return VAE_OK;
}

}  // extern "C"
