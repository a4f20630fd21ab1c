// Layer norm of rows and its gradient (public entry points at the end).
//
// A row is read once into registers, so the two-pass statistics (mean, then
// the mean square around it) and everything after them cost no further memory
// traffic: both directions are bound by reading their inputs and writing their
// output once. Rows of up to 1280 channels belong to one warp (shuffles only);
// wider ones to a block. Rows whose length is a multiple of eight move in
// 16-byte vectors, others element by element in the same registers.
//
// The gradients of gamma and beta are column sums over all rows: every thread
// keeps the same columns on every row it meets, so it sums them in registers,
// the warps of a block add up in shared memory one after another, each block
// writes one partial row, and a second kernel adds the blocks' rows. Every
// order is fixed, so the sums do not change from call to call.
#include <algorithm>
#include <cmath>

#include "vae_types.cuh"

namespace vae {

namespace {

constexpr int kLnMaxC = 16384;
constexpr int kLnWarpVec = 5;   // eights of a row per lane, at most, in the one-warp form
constexpr int kLnFwdWarps = 4;  // rows (warps) per block of the forward's one-warp form
constexpr int kLnBwdWarps = 8;  // rows in flight per block of the gradient's one-warp form
constexpr int kLnBwdBlocks = 304;  // blocks of the gradient, at most: two per SM

// The row's elements of this thread: eights tid, tid + T, ... (kV8) or single
// elements tid, tid + T, ... (8 * NV of them); 0 behind the row's end.
template <int T, int NV, bool kV8>
__device__ __forceinline__ void load_row_t(const void* base, size_t off, int c, int tid, int nt, float (&v)[NV][8]) {
    using E = typename Elem<T>::type;
    const E* p = static_cast<const E*>(base) + off;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (kV8) {
            const int i = (tid + k * nt) * 8;
            if (i < c) {
                load8<T>(p + i, v[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[k][e] = 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = tid + (k * 8 + e) * nt;
                v[k][e] = i < c ? to_f32<T>(p[i]) : 0.f;
            }
        }
    }
}
template <int NV, bool kV8>
__device__ __forceinline__ void load_row(const void* base, int type, size_t off, int c, int tid, int nt,
                                         float (&v)[NV][8]) {
    if (type == VAE_F32) load_row_t<VAE_F32, NV, kV8>(base, off, c, tid, nt, v);
    else if (type == VAE_F16) load_row_t<VAE_F16, NV, kV8>(base, off, c, tid, nt, v);
    else load_row_t<VAE_BF16, NV, kV8>(base, off, c, tid, nt, v);
}
template <int T, int NV, bool kV8>
__device__ __forceinline__ void store_row_t(void* base, size_t off, int c, int tid, int nt, const float (&v)[NV][8]) {
    using E = typename Elem<T>::type;
    E* p = static_cast<E*>(base) + off;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if constexpr (kV8) {
            const int i = (tid + k * nt) * 8;
            if (i < c) store8<T>(p + i, v[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = tid + (k * 8 + e) * nt;
                if (i < c) p[i] = from_f32<T>(v[k][e]);
            }
        }
    }
}
template <int NV, bool kV8>
__device__ __forceinline__ void store_row(void* base, int type, size_t off, int c, int tid, int nt,
                                          const float (&v)[NV][8]) {
    if (type == VAE_F32) store_row_t<VAE_F32, NV, kV8>(base, off, c, tid, nt, v);
    else if (type == VAE_F16) store_row_t<VAE_F16, NV, kV8>(base, off, c, tid, nt, v);
    else store_row_t<VAE_BF16, NV, kV8>(base, off, c, tid, nt, v);
}

// Whether element (k, e) of this thread lies in the row.
template <bool kV8>
__device__ __forceinline__ int elem_at(int k, int e, int tid, int nt) {
    return kV8 ? (tid + k * nt) * 8 + e : tid + (k * 8 + e) * nt;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum of `v` over the row's threads (a warp, or the block), the same bits
// in every thread. `red`: 32 floats of the block's, free again at the next call
// but one (callers alternate two of them).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if constexpr (!kWarp) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        const int nw = blockDim.x >> 5;
        v = warp_sum(static_cast<int>(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f);
    }
    return v;
}

// mean and 1 / sqrt(var + eps) of the row; x is left centred (0 behind the end).
template <int NV, bool kV8, bool kWarp>
__device__ __forceinline__ float centre_row(float (&x)[NV][8], int c, int tid, int nt, float eps, float* red0,
                                            float* red1) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[k][e];
    const float mean = row_sum<kWarp>(s, red0) / static_cast<float>(c);
    s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = elem_at<kV8>(k, e, tid, nt) < c ? x[k][e] - mean : 0.f;
            x[k][e] = d;
            s += d * d;
        }
    return 1.f / sqrtf(row_sum<kWarp>(s, red1) / static_cast<float>(c) + eps);
}

template <int NV, bool kV8, bool kWarp>
__global__ void __launch_bounds__(kWarp ? kLnFwdWarps * 32 : 512)
    ln_fwd_kernel(const void* __restrict__ x, int xt, int m, int c, const float* __restrict__ gamma,
                  const float* __restrict__ beta, float eps, void* y, int yt) {
    __shared__ float red[2][32];
    pdl_wait();
    const int nt = kWarp ? 32 : blockDim.x;
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x;
    const long long row = kWarp ? static_cast<long long>(blockIdx.x) * kLnFwdWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= m) return;  // (a whole warp of the one-warp form: no block barrier follows there)
    const size_t off = static_cast<size_t>(row) * c;
    float v[NV][8];
    load_row<NV, kV8>(x, xt, off, c, tid, nt, v);
    const float rstd = centre_row<NV, kV8, kWarp>(v, c, tid, nt, eps, red[0], red[1]);
    float w[NV][8];
    if (gamma != nullptr) load_row_t<VAE_F32, NV, kV8>(gamma, 0, c, tid, nt, w);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] *= gamma != nullptr ? rstd * w[k][e] : rstd;
    if (beta != nullptr) {
        load_row_t<VAE_F32, NV, kV8>(beta, 0, c, tid, nt, w);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] += w[k][e];
    }
    store_row<NV, kV8>(y, yt, off, c, tid, nt, v);
}

// Rows blockIdx, blockIdx + grid, ... (one-warp form: of each of the block's
// warps). part: [grid][2][c] partial sums of dy * n and dy, or NULL.
template <int NV, bool kV8, bool kWarp>
__global__ void __launch_bounds__(kWarp ? kLnBwdWarps * 32 : 512)
    ln_bwd_kernel(const void* __restrict__ dy, int dyt, const void* x, int xt, int m, int c,
                  const float* __restrict__ gamma, float eps, void* dx, float* __restrict__ part) {
    __shared__ float red[4][32];
    extern __shared__ float cols[];  // (one-warp form) the warps' column sums, [2][c]
    pdl_wait();
    const int nt = kWarp ? 32 : blockDim.x;
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x;
    const int warp = threadIdx.x >> 5;
    const long long step = kWarp ? static_cast<long long>(gridDim.x) * kLnBwdWarps : gridDim.x;
    const float inv_c = 1.f / static_cast<float>(c);
    float dg[NV][8], db[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[k][e] = db[k][e] = 0.f;
    for (long long row = kWarp ? static_cast<long long>(blockIdx.x) * kLnBwdWarps + warp : blockIdx.x; row < m;
         row += step) {
        const size_t off = static_cast<size_t>(row) * c;
        float v[NV][8], g[NV][8];
        load_row<NV, kV8>(x, xt, off, c, tid, nt, v);
        load_row<NV, kV8>(dy, dyt, off, c, tid, nt, g);
        const float rstd = centre_row<NV, kV8, kWarp>(v, c, tid, nt, eps, red[0], red[1]);
        float w[NV][8];
        if (gamma != nullptr) load_row_t<VAE_F32, NV, kV8>(gamma, 0, c, tid, nt, w);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[k][e] *= rstd;  // n
                dg[k][e] += g[k][e] * v[k][e];
                db[k][e] += g[k][e];
                if (gamma != nullptr) g[k][e] *= w[k][e];
                s1 += g[k][e];
                s2 += g[k][e] * v[k][e];
            }
        s1 = row_sum<kWarp>(s1, red[2]) * inv_c;
        s2 = row_sum<kWarp>(s2, red[3]) * inv_c;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = rstd * (g[k][e] - s1 - v[k][e] * s2);
        store_row<NV, kV8>(dx, xt, off, c, tid, nt, v);
    }
    if (part == nullptr) return;
    float* out = part + static_cast<size_t>(blockIdx.x) * 2 * c;
    if constexpr (kWarp) {
        for (int u = 0; u < kLnBwdWarps; ++u) {
            if (warp == u) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = elem_at<kV8>(k, e, tid, nt);
                        if (i < c) {
                            cols[i] = u == 0 ? dg[k][e] : cols[i] + dg[k][e];
                            cols[c + i] = u == 0 ? db[k][e] : cols[c + i] + db[k][e];
                        }
                    }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < 2 * c; i += blockDim.x) out[i] = cols[i];
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = elem_at<kV8>(k, e, tid, nt);
                if (i < c) {
                    out[i] = dg[k][e];
                    out[c + i] = db[k][e];
                }
            }
    }
}

// out[0 .. c) = sum over the blocks' partial rows, dgamma then dbeta: 32
// columns x 8 slices of blocks per thread block, the slices joined in order.
__global__ void __launch_bounds__(256) ln_cols_kernel(const float* __restrict__ part, int nblk, int c,
                                                      float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float s[8][32];
    pdl_wait();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (col < 2 * c)
        for (int b = slice; b < nblk; b += 8) a += part[static_cast<size_t>(b) * 2 * c + col];
    s[slice][lane] = a;
    __syncthreads();
    if (slice == 0 && col < 2 * c) {
        for (int i = 1; i < 8; ++i) a += s[i][lane];
        (col < c ? dgamma : dbeta - c)[col] = a;
    }
}

// How a row is held: warp form or the block's threads, and eights per thread.
struct LnPlan {
    bool v8, warp;
    int nv, threads;
};
LnPlan ln_plan(int c) {
    LnPlan p;
    p.v8 = c % 8 == 0;
    const int nvec = (c + 7) / 8;
    p.warp = nvec <= 32 * kLnWarpVec;
    if (p.warp) {
        p.nv = (nvec + 31) / 32;
        p.threads = 32;
    } else {
        p.nv = nvec <= 512 ? 2 : 4;
        p.threads = std::min(512, ((nvec + p.nv - 1) / p.nv + 31) / 32 * 32);
    }
    return p;
}
int ln_bwd_grid(int m, int c) {
    const LnPlan p = ln_plan(c);
    const int rows = p.warp ? (m - 1) / kLnBwdWarps + 1 : m;
    return std::min(rows, p.warp ? kLnBwdBlocks : 2 * kLnBwdBlocks);
}

// Calls f(NV, kV8, kWarp) as compile-time constants of the plan.
template <typename F>
cudaError_t ln_dispatch(const LnPlan& p, F&& f) {
#define VAE_LN_CASE(W, N)                                                                            \
    if (p.warp == W && p.nv == N)                                                                    \
        return p.v8 ? f(std::integral_constant<int, N>{}, std::true_type{}, std::bool_constant<W>{}) \
                    : f(std::integral_constant<int, N>{}, std::false_type{}, std::bool_constant<W>{});
    VAE_LN_CASE(true, 1)
    VAE_LN_CASE(true, 2)
    VAE_LN_CASE(true, 3)
    VAE_LN_CASE(true, 4)
    VAE_LN_CASE(true, 5)
    VAE_LN_CASE(false, 2)
    VAE_LN_CASE(false, 4)
#undef VAE_LN_CASE
    return cudaErrorInvalidValue;
}

int ln_check(const void* x, int xt, int m, int c, float eps, const void* y, int yt) {
    if (x == nullptr || y == nullptr) return set_error(VAE_ERR_ARG, "layer norm: NULL tensor");
    if (!type_ok(xt) || !type_ok(yt)) return set_error(VAE_ERR_ARG, "layer norm: unknown element type");
    if (m < 1 || c < 1 || c > kLnMaxC)
        return set_error(VAE_ERR_SHAPE, "layer norm: m >= 1 and 1 <= c <= %d are needed, got m %d, c %d", kLnMaxC, m, c);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return set_error(VAE_ERR_ARG, "layer norm: eps must be >= 0 and finite");
    return VAE_OK;
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" {

int vae_layernorm(const void* x_dev, int x_type, int m, int c, const float* gamma_dev, const float* beta_dev,
                  float eps, void* y_dev, int y_type, vae_stream_t stream) {
    clear_error();
    int rc = ln_check(x_dev, x_type, m, c, eps, y_dev, y_type);
    if (rc != VAE_OK) return rc;
    if (x_dev == y_dev && x_type != y_type)
        return set_error(VAE_ERR_ARG, "layer norm: in place needs x and y of one type");
    if (!aligned16(x_dev) || !aligned16(y_dev) || !aligned16(gamma_dev) || !aligned16(beta_dev))
        return set_error(VAE_ERR_ALIGN, "layer norm: pointers must be 16-byte aligned");
    if ((rc = check_device()) != VAE_OK) return rc;
    const LnPlan p = ln_plan(c);
    const unsigned grid = p.warp ? (static_cast<unsigned>(m) - 1u) / kLnFwdWarps + 1u : static_cast<unsigned>(m);
    VAE_CUDA_CHECK(ln_dispatch(p, [&](auto nv, auto v8, auto warp) {
        return launch_kernel(ln_fwd_kernel<nv.value, v8.value, warp.value>, dim3(grid),
                             dim3(warp.value ? kLnFwdWarps * 32 : p.threads), 0, reinterpret_cast<cudaStream_t>(stream),
                             x_dev, x_type, m, c, gamma_dev, beta_dev, eps, y_dev, y_type);
    }));
    return VAE_OK;
}

size_t vae_layernorm_backward_workspace_bytes(int m, int c) {
    if (m < 1 || c < 1 || c > kLnMaxC) return 0;
    return (static_cast<size_t>(ln_bwd_grid(m, c)) * 2 * c * sizeof(float) + 15) / 16 * 16;
}

int vae_layernorm_backward(const void* dy_dev, int dy_type, const void* x_dev, int x_type, int m, int c,
                           const float* gamma_dev, float eps, void* dx_dev, float* dgamma_dev, float* dbeta_dev,
                           void* workspace_dev, size_t workspace_bytes, vae_stream_t stream) {
    clear_error();
    int rc = ln_check(x_dev, x_type, m, c, eps, dx_dev, x_type);
    if (rc != VAE_OK) return rc;
    if (dy_dev == nullptr) return set_error(VAE_ERR_ARG, "layer norm: NULL tensor");
    if (!type_ok(dy_type)) return set_error(VAE_ERR_ARG, "layer norm: unknown element type");
    if ((dgamma_dev == nullptr) != (dbeta_dev == nullptr))
        return set_error(VAE_ERR_ARG, "layer norm: dgamma and dbeta come together");
    if (dx_dev == dy_dev && dy_type != x_type)
        return set_error(VAE_ERR_ARG, "layer norm: dx over dy needs one type");
    const bool sums = dgamma_dev != nullptr;
    if (sums && workspace_dev == nullptr) return set_error(VAE_ERR_ARG, "layer norm: NULL workspace");
    if (!aligned16(x_dev) || !aligned16(dy_dev) || !aligned16(dx_dev) || !aligned16(gamma_dev) ||
        !aligned16(dgamma_dev) || !aligned16(dbeta_dev) || !aligned16(workspace_dev))
        return set_error(VAE_ERR_ALIGN, "layer norm: pointers must be 16-byte aligned");
    if (sums && workspace_bytes < vae_layernorm_backward_workspace_bytes(m, c))
        return set_error(VAE_ERR_NOMEM, "layer norm: workspace of %zu bytes, %zu needed", workspace_bytes,
                         vae_layernorm_backward_workspace_bytes(m, c));
    if ((rc = check_device()) != VAE_OK) return rc;
    const LnPlan p = ln_plan(c);
    const int grid = ln_bwd_grid(m, c);
    float* part = sums ? static_cast<float*>(workspace_dev) : nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    VAE_CUDA_CHECK(ln_dispatch(p, [&](auto nv, auto v8, auto warp) {
        return launch_kernel(ln_bwd_kernel<nv.value, v8.value, warp.value>, dim3(static_cast<unsigned>(grid)),
                             dim3(warp.value ? kLnBwdWarps * 32 : p.threads),
                             warp.value && sums ? 2 * static_cast<size_t>(c) * sizeof(float) : 0, s, dy_dev, dy_type,
                             x_dev, x_type, m, c, gamma_dev, eps, dx_dev, part);
    }));
    if (sums)
        VAE_CUDA_CHECK(launch_kernel(ln_cols_kernel, dim3((2u * static_cast<unsigned>(c) + 31u) / 32u), dim3(256), 0, s,
                                     static_cast<const float*>(part), grid, c, dgamma_dev, dbeta_dev));
    return VAE_OK;
}

}  // extern "C"
