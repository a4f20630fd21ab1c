// The gated feed-forward block on few tokens (the C entry point is in vae_ffn.cu).
//
// A few tokens read every weight once and do next to nothing with it: the call takes as
// long as the weights' way from memory (1152 x 4608 in 16 bits: 32 MB, 4.7 us). So the
// rows of a weight are the M index of 16 x 8 x 16 matrix instructions on registers, the tokens
// their N index, and each lane brings its part of a row straight from memory in 16-byte
// loads, eight consecutive elements: the contraction index of one instruction may be any
// sixteen of them as long as weights and tokens agree, so lane t of four takes the
// elements 8 t .. 8 t + 7 of 32 for two instructions, and nothing passes through
// shared memory on the way in.
//
// A block takes 16 rows (of Wg and of the same rows of Wu, so that act(gate) * up stays with
// it), its eight warps every eighth piece of 32 of the contraction; where there are too
// few rows to give every SM two blocks, a cluster of blocks shares the contraction. The
// warps' sums join in shared memory, the blocks' in the first one's, in order. The second
// product's blocks are launched while the first's run and have their first weights on
// their way before they wait for hidden.
//
// hidden goes on as two values of the type, the rounded one and what the rounding left
// (in f16 times 2^11, which keeps it off the subnormal numbers): the second product takes both with the
// weights that it has anyway, and y carries its own rounding alone.
#include <algorithm>
#include <cfloat>

#include "vae_ffn.cuh"
#include "vae_ffn_few.h"

namespace vae {

namespace {

constexpr int kSums = 8;    // warps whose sums lie in shared memory
// Pieces of the contraction that a warp has on their way: as many as leave two blocks an SM their registers.
constexpr int ahead(int kn) { return kn == 1 ? 3 : 2; }
constexpr int kRows = 16;
constexpr int kMaxSplits = 8;

struct FewParams {
    const void *w0, *w1;     // weights [rows][k] (w1: of up)
    const void* x;           // [m][k]
    int m, rows, k;
    void* out;               // [m][rows]
    void* rest;              // gated: [m][rows], what the rounding of `out` left; else that of x
    void *gate, *up;         // or NULL
    int out_f32;
    const float* residual;
    const void* next;        // the weights of the product behind this one, and their bytes: asked for by this one, into L2
    long long next_bytes;
};

template <int T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (T == VAE_F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_weights(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int T>
constexpr float kRest = T == VAE_F16 ? 2048.f : 1.f;

// kN: tokens in eights; kWarps: 8 (two blocks an SM) or 16 (one).
template <int T, bool kGated, int kN, int kAct, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 2 : 1) few_kernel(const FewParams p) {
    constexpr int kMats = kGated ? 2 : 1, kAhead = ahead(kN);  // matrices
    constexpr int kOut = kMats * kN * 8 * kRows;  // sums of a block: [matrix][token][row]
    __shared__ float sums[kSums][kOut];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int splits = static_cast<int>(gridDim.y), split = static_cast<int>(blockIdx.y);
    const int row0 = static_cast<int>(blockIdx.x) * kRows;
    const int pieces = (p.k + 31) / 32;
    const int first = static_cast<int>(static_cast<long long>(pieces) * split / splits) + warp;
    const int last = static_cast<int>(static_cast<long long>(pieces) * (split + 1) / splits);
    const uint16_t* w[kMats];
    w[0] = static_cast<const uint16_t*>(p.w0);
    if constexpr (kGated) w[1] = static_cast<const uint16_t*>(p.w1);
    const long long r0 = static_cast<long long>(row0 + g) * p.k, r1 = r0 + 8LL * p.k;
    const bool has0 = row0 + g < p.rows, has1 = row0 + g + 8 < p.rows;

    uint4 a[kAhead][kMats][2];
    auto fetch = [&](int slot, int piece) {
        const int k = piece * 32 + t * 8;
        const bool in = piece < last && k < p.k;
#pragma unroll
        for (int i = 0; i < kMats; ++i) {
            a[slot][i][0] = in && has0 ? load_weights(w[i] + r0 + k) : make_uint4(0u, 0u, 0u, 0u);
            a[slot][i][1] = in && has1 ? load_weights(w[i] + r1 + k) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    if constexpr (kGated) {
        pdl_wait();
        pdl_launch_dependents();  // the second product's blocks may come as this one's leave room
    }
    // The weights are no result of the kernel before: the second product's are asked for ahead of the wait for hidden.
#pragma unroll
    for (int s = 0; s < kAhead; ++s) fetch(s, first + s * kWarps);
    if constexpr (!kGated) pdl_wait();
    if (kGated && threadIdx.x == 0) {
        const long long blocks = static_cast<long long>(gridDim.x) * splits, b = static_cast<long long>(blockIdx.x) * splits + split;
        const long long from = p.next_bytes / 16 * b / blocks * 16, to = p.next_bytes / 16 * (b + 1) / blocks * 16;
        const long long most = 1 << 16;  // (few blocks: the first part of their share)
        if (to > from) prefetch_l2_bulk(static_cast<const char*>(p.next) + from, static_cast<uint32_t>(to - from < most ? to - from : most));
    }

    float d[2][kN][4] = {};  // of gate and up, or of hidden and its rest
    const uint16_t *x = static_cast<const uint16_t*>(p.x), *y = static_cast<const uint16_t*>(p.rest);
    for (int piece = first; piece < last; piece += kAhead * kWarps) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
            const int k = (piece + s * kWarps) * 32 + t * 8;
            uint4 b[kN], c[kGated ? 1 : kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const int token = n * 8 + g;
                const bool in = token < p.m && k < p.k && piece + s * kWarps < last;
                const long long at = static_cast<long long>(token) * p.k + k;
                b[n] = in ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (!kGated) c[n] = in ? *reinterpret_cast<const uint4*>(y + at) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 u = a[s][i % kMats][0], v = a[s][i % kMats][1];
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const uint4 e = kGated || i == 0 ? b[n] : c[kGated ? 0 : n];
                    mma16816<T>(d[i][n], u.x, v.x, u.y, v.y, e.x, e.y);
                    mma16816<T>(d[i][n], u.z, v.z, u.w, v.w, e.z, e.w);
                }
            }
            fetch(s, piece + (s + kAhead) * kWarps);
        }
    }
    if constexpr (!kGated) {
        // (a sum that is infinite or NaN without the rest stays so: an infinite weight times a rest of 0, or of the other sign,
        // would make a NaN of it)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (fabsf(d[0][n][e]) <= FLT_MAX) d[0][n][e] = fmaf(d[1][n][e], 1.f / kRest<T>, d[0][n][e]);
    }
    // d: rows g, g + 8; tokens 2 t, 2 t + 1. Sixteen warps: the upper ones' first, which the lower ones add to theirs.
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kMats; ++i)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f(sums[warp % kSums][(i * kN * 8 + n * 8 + 2 * t + (e & 1)) * kRows + g + (e >> 1) * 8], d[i][n][e]);
    };
    if constexpr (kWarps > kSums) {
        if (warp >= kSums) each([](float& at, float v) { at = v; });
        __syncthreads();
    }
    if (warp < kSums) each([](float& at, float v) { at = kWarps > kSums ? v + at : v; });
    __syncthreads();
    for (int o = threadIdx.x; o < kOut; o += kWarps * 32) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kSums; ++k) v += sums[k][o];
        sums[0][o] = v;
    }
    if (splits > 1) cluster_sync();
    else __syncthreads();
    if (split == 0) {
        for (int o = threadIdx.x; o < kN * 8 * kRows; o += kWarps * 32) {
            const int token = o / kRows, row = row0 + o % kRows;
            float v[kMats];
#pragma unroll
            for (int i = 0; i < kMats; ++i) {
                const int at = i * kN * 8 * kRows + o;
                v[i] = sums[0][at];
                for (int k = 1; k < splits; ++k) {
                    float r;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(mapa_shared(smem_u32(&sums[0][at]), static_cast<uint32_t>(k))) : "memory");
                    v[i] += r;
                }
            }
            if (token >= p.m || row >= p.rows) continue;
            const long long at = static_cast<long long>(token) * p.rows + row;
            using E = typename Elem<T>::type;
            if constexpr (kGated) {
                const float h = act_value<kAct>(v[0]) * v[1];
                const E near = from_f32<T>(h);
                const float rest = (h - to_f32<T>(near)) * kRest<T>;
                static_cast<E*>(p.out)[at] = near;
                static_cast<E*>(p.rest)[at] = from_f32<T>(rest - rest == 0.f ? rest : 0.f);  // (of what is not finite: 0)
                if (p.gate != nullptr) {
                    static_cast<E*>(p.gate)[at] = from_f32<T>(v[0]);
                    static_cast<E*>(p.up)[at] = from_f32<T>(v[1]);
                }
            } else if (p.out_f32) {
                static_cast<float*>(p.out)[at] = p.residual != nullptr ? v[0] + p.residual[at] : v[0];
            } else {
                static_cast<E*>(p.out)[at] = from_f32<T>(v[0]);
            }
        }
    }
    if (splits > 1) cluster_sync();  // the other blocks' sums have been read
}

template <int T, bool kGated, int kN, int kAct, int kWarps>
int launch_warps(const FewParams& p, int splits, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.rows + kRows - 1) / kRows, splits);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = !kGated || pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    VAE_CUDA_CHECK(cudaLaunchKernelEx(&cfg, few_kernel<T, kGated, kN, kAct, kWarps>, p));
    return VAE_OK;
}

template <int T, bool kGated, int kN, int kAct>
int launch_n(const FewParams& p, cudaStream_t stream) {
    // One wave of blocks, sixteen warps an SM: a second wave costs more than it brings (1152 x 4608: 288 blocks of the
    // first product 6.6 us, 576 10.1). Where the rows give at most one block an SM, it has all sixteen warps (512 x
    // 2048: 6.4 us a call, with eight and twice the clusters 9.5); clusters share the contraction as long as they find
    // SMs and every warp a piece.
    const int groups = (p.rows + kRows - 1) / kRows, pieces = (p.k + 31) / 32;
    if (groups > 152) return launch_warps<T, kGated, kN, kAct, 8>(p, 1, stream);
    int splits = 1;
    while (splits < kMaxSplits && groups * splits * 2 <= 152 && pieces >= 2 * splits * 16) splits *= 2;
    return launch_warps<T, kGated, kN, kAct, 16>(p, splits, stream);
}

template <int T, bool kGated, int kAct>
int launch_tokens(const FewParams& p, cudaStream_t stream) {
    if (p.m <= 8) return launch_n<T, kGated, 1, kAct>(p, stream);
    return p.m <= 16 ? launch_n<T, kGated, 2, kAct>(p, stream) : launch_n<T, kGated, 4, kAct>(p, stream);
}

template <int T>
int few_type(const vae_gated_ffn_desc& a, const void* x, const void* wg, const void* wu, const void* wd, const float* residual, void* y,
             void* gate, void* up, void* hidden, void* rest, cudaStream_t stream) {
    FewParams p{};
    p.w0 = wg;
    p.w1 = wu;
    p.x = x;
    p.m = a.m;
    p.rows = a.f;
    p.k = a.c;
    p.out = hidden;
    p.rest = rest;
    p.gate = gate;
    p.up = up;
    p.next = wd;
    p.next_bytes = 2LL * a.c * a.f;
    const int rc = a.activation == VAE_ACT_SILU   ? launch_tokens<T, true, VAE_ACT_SILU>(p, stream)
                   : a.activation == VAE_ACT_GELU ? launch_tokens<T, true, VAE_ACT_GELU>(p, stream)
                                                  : launch_tokens<T, true, VAE_ACT_GELU_TANH>(p, stream);
    if (rc != VAE_OK) return rc;
    p = FewParams{};
    p.w0 = wd;
    p.x = hidden;
    p.rest = rest;
    p.m = a.m;
    p.rows = a.c;
    p.k = a.f;
    p.out = y;
    p.out_f32 = a.y_type == VAE_F32;
    p.residual = residual;
    return launch_tokens<T, false, VAE_ACT_SILU>(p, stream);
}

}  // namespace

int ffn_few(const vae_gated_ffn_desc& a, const void* x, const void* wg, const void* wu, const void* wd, const float* residual, void* y,
            void* gate, void* up, void* hidden, void* rest, cudaStream_t stream) {
    return a.type == VAE_F16 ? few_type<VAE_F16>(a, x, wg, wu, wd, residual, y, gate, up, hidden, rest, stream)
                             : few_type<VAE_BF16>(a, x, wg, wu, wd, residual, y, gate, up, hidden, rest, stream);
}

}  // namespace vae
