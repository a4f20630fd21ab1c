// Layer norm of rows and its gradient (public entry points at the end).
//
// A row is read once into registers, so the two-pass statistics (mean, then
// the mean square around it) and everything after them cost no further memory
// traffic: both directions are bound by reading their inputs and writing their
// output once.
//
// Ring form (many rows of up to 5120 channels; forward: of a multiple of eight):
// one block per SM stays; rows belong to groups of one to eight warps, whose next
// rows are already on the way into shared memory by bulk copies while they work
// on the last ones. Registers hold those only and the loads never pause.
// Plain form (few rows, or longer ones): rows of up to 1280 channels belong to
// one warp, wider ones to a block, loaded straight into registers, in 16-byte
// vectors where the length is a multiple of eight, else element by element.
// Measured on GB300: 16384x1152 f32 to f16 (113 MB) 20.4 us in the ring form, 24.9
// in the plain one; its gradient over 65536 rows (755 MB) 123 us (6.1 TB/s) and 192.
// Rows of 8192, 4096 of them in f32 and f16 (plain form, a block a row): 51 us (floor
// 30), the gradient 149 us (floor 49).
//
// The gradients of gamma and beta are column sums over all rows: every thread
// keeps the same columns on every row it meets, so it sums them in registers,
// the warps of a block join in shared memory in a fixed order, each block writes
// one partial row, and a second kernel adds the blocks' rows. Every
// order is fixed, so the sums do not change from call to call.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "vae_overlap.h"
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
    extern __shared__ float cols[];  // (one-warp form) the warps' column sums, [warps][2][c]
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
        // the warps' sums side by side, then joined in order
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = elem_at<kV8>(k, e, tid, nt);
                if (i < c) {
                    cols[warp * 2 * c + i] = dg[k][e];
                    cols[warp * 2 * c + c + i] = db[k][e];
                }
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * c; i += blockDim.x) {
            float a = cols[i];
#pragma unroll
            for (int u = 1; u < kLnBwdWarps; ++u) a += cols[u * 2 * c + i];
            out[i] = a;
        }
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
    pdl_launch_dependents();
}

// ───────────────────────────── ring form ─────────────────────────────

constexpr int kRingBlocks = 152;  // one per SM
constexpr int kRingStages = 4;    // chunks of a group in flight, at most
constexpr size_t kRingSmem = 220 * 1024;

// Rows that a group takes together (a chunk: they lie side by side in memory),
// as many as its registers hold: the sums of a chunk's rows cross the warp
// together, and gamma and beta are read once for them.
__host__ __device__ constexpr int ring_rows(int nq) { return nq <= 2 ? 4 : 2; }
// Warps per block, at most: what leaves each thread its registers.
__host__ __device__ constexpr int ring_warps(int nq, bool backward) { return backward || nq > 5 ? 12 : 16; }

struct LnRing {
    int m, c, xt, yt, dyt;
    int nq, wide, warps;  // fours per thread, warps per row (a group), warps per block
    int stages;
    unsigned row_x, row_dy;         // bytes of a row of x and dy
    unsigned second, stage;         // offset of dy in a stage, bytes of a stage
    unsigned consts, bars;          // offsets of gamma and beta, and of the barriers
    float eps;
    const void *x, *dy;
    const float *gamma, *beta;
    void* out;            // y or dx
    float* part;
    DevStatus* status;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ void ln_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Four elements, as two pairs. (Fours of neighbouring lanes touch every bank of
// shared memory once; eights of f32 would meet in half of them.)
struct Four {
    float2 a, b;
};
template <int T>
__device__ __forceinline__ Four four_in(const uint8_t* p, int i) {
    if constexpr (T == VAE_F32) {
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
    } else {
        const uint2 v = reinterpret_cast<const uint2*>(p)[i];
        return {unpack2<T>(v.x), unpack2<T>(v.y)};
    }
}
template <int T>
__device__ __forceinline__ void four_out(uint8_t* p, int i, Four v) {
    if constexpr (T == VAE_F32) reinterpret_cast<float4*>(p)[i] = make_float4(v.a.x, v.a.y, v.b.x, v.b.y);
    else reinterpret_cast<uint2*>(p)[i] = make_uint2(pack2<T>(v.a.x, v.a.y), pack2<T>(v.b.x, v.b.y));
}
// A thread's four number k of a row of n fours: four tid + k nt, or in rows whose
// length is no multiple of eight (kOdd, n elements) the single elements
// tid + (4 k + e) nt; `other` behind the row's end.
__device__ __forceinline__ int odd_at(int k, int e, int tid, int nt) { return tid + (4 * k + e) * nt; }
template <int T, bool kOdd>
__device__ __forceinline__ Four get4(const uint8_t* p, int n, int k, int tid, int nt, float other) {
    if constexpr (!kOdd) {
        const int i = tid + k * nt;
        return i < n ? four_in<T>(p, i) : Four{make_float2(other, other), make_float2(other, other)};
    } else {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = odd_at(k, e, tid, nt);
            v[e] = i < n ? to_f32<T>(reinterpret_cast<const typename Elem<T>::type*>(p)[i]) : other;
        }
        return {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
    }
}
template <int T, bool kOdd>
__device__ __forceinline__ void put4(uint8_t* p, int n, int k, int tid, int nt, Four v) {
    if constexpr (!kOdd) {
        const int i = tid + k * nt;
        if (i < n) four_out<T>(p, i, v);
    } else {
        const float f[4] = {v.a.x, v.a.y, v.b.x, v.b.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = odd_at(k, e, tid, nt);
            if (i < n) reinterpret_cast<typename Elem<T>::type*>(p)[i] = from_f32<T>(f[e]);
        }
    }
}
template <int T, int NQ, bool kOdd>
__device__ __forceinline__ void row_in_t(const uint8_t* p, int n, int tid, int nt, Four (&v)[NQ]) {
#pragma unroll
    for (int k = 0; k < NQ; ++k) v[k] = get4<T, kOdd>(p, n, k, tid, nt, 0.f);
}
template <int NQ, bool kOdd>
__device__ __forceinline__ void row_in(const uint8_t* p, int type, int n, int tid, int nt, Four (&v)[NQ]) {
    if (type == VAE_F32) row_in_t<VAE_F32, NQ, kOdd>(p, n, tid, nt, v);
    else if (type == VAE_F16) row_in_t<VAE_F16, NQ, kOdd>(p, n, tid, nt, v);
    else row_in_t<VAE_BF16, NQ, kOdd>(p, n, tid, nt, v);
}
template <int T, int NQ, bool kOdd>
__device__ __forceinline__ void row_out_t(uint8_t* p, int n, int tid, int nt, const Four (&v)[NQ]) {
#pragma unroll
    for (int k = 0; k < NQ; ++k) put4<T, kOdd>(p, n, k, tid, nt, v[k]);
}
template <int NQ, bool kOdd>
__device__ __forceinline__ void row_out(uint8_t* p, int type, int n, int tid, int nt, const Four (&v)[NQ]) {
    if (type == VAE_F32) row_out_t<VAE_F32, NQ, kOdd>(p, n, tid, nt, v);
    else if (type == VAE_F16) row_out_t<VAE_F16, NQ, kOdd>(p, n, tid, nt, v);
    else row_out_t<VAE_BF16, NQ, kOdd>(p, n, tid, nt, v);
}

// A run of `bytes` at base + at into dst by a bulk copy, which takes whole
// 16-byte units: from the unit that it starts in to the one that it ends in,
// but not past `end`, the tensor's; what a last, partial unit holds comes by
// hand (before the arrival on the barrier, which the readers acquire). The run
// starts at dst + at % 16. Returns the bytes that the copy brings.
template <bool kOdd>
__device__ __forceinline__ uint32_t run_bytes(size_t at, size_t bytes, size_t end) {
    if constexpr (!kOdd) return static_cast<uint32_t>(bytes);
    const size_t from = at & ~size_t(15), to = (at + bytes + 15) & ~size_t(15);
    return static_cast<uint32_t>((to <= end ? to : end & ~size_t(15)) - from);
}
template <bool kOdd>
__device__ __forceinline__ void run_tail(uint8_t* dst, const void* base, size_t at, size_t bytes, size_t end) {
    if constexpr (kOdd) {
        const size_t from = at & ~size_t(15), to = (at + bytes + 15) & ~size_t(15);
        if (to <= end) return;
        for (size_t b = end & ~size_t(15); b < end; b += 2)
            *reinterpret_cast<uint16_t*>(dst + (b - from)) = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(base) + b);
    }
}

// The warps of a group meet (a barrier of the group's own).
__device__ __forceinline__ void group_sync(int group, int wide) {
    if (wide == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(wide * 32) : "memory");
}
// N sums over the group's threads, the same bits in each; `red`: [wide][N] floats of this group and call site.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float* red, int group, int wide, int part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (wide > 1) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[part * N + i] = v[i];
        group_sync(group, wide);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = red[i];
        for (int k = 1; k < wide; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += red[k * N + i];
    }
}

// Chunks g, g + G, ... of all groups g < G of the grid. kBwd: the gradient.
template <int NQ, bool kBwd, bool kOdd>
__global__ void __launch_bounds__(ring_warps(NQ, kBwd) * 32, 1) ln_ring_kernel(const LnRing p) {
    constexpr int R = ring_rows(NQ);
    constexpr int kMaxWarps = ring_warps(NQ, kBwd);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[3][kMaxWarps * 2 * R];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wide = p.wide, group = warp / wide, part = warp % wide, groups = p.warps / wide;
    const int nt = wide * 32, tid = part * 32 + lane, c = p.c;
    const int nr = kOdd ? c : c / 4;  // of a row: elements, or fours
    uint8_t* ring = smem + static_cast<size_t>(group) * p.stages * p.stage;
    const uint8_t* gam = smem + p.consts;
    const uint8_t* bet = gam + static_cast<size_t>(c) * 4;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.bars) + group * kRingStages;
    const int all = static_cast<int>(gridDim.x) * groups, first = static_cast<int>(blockIdx.x) * groups + group;
    const int chunks = (p.m - 1) / R + 1;
    const int n = first < chunks ? (chunks - 1 - first) / all + 1 : 0;  // this group's chunks
    auto fetch = [&](int k, int st) {  // one lane of the group: the group's chunk k into stage st = k % stages
        const size_t row = (static_cast<size_t>(first) + static_cast<size_t>(k) * all) * R;
        const unsigned rows = p.m - row < static_cast<size_t>(R) ? static_cast<unsigned>(p.m - row) : R;
        const uint32_t bar = smem_u32(&full[st]);
        uint8_t* dst = ring + static_cast<size_t>(st) * p.stage;
        const size_t ax = row * p.row_x, nx = static_cast<size_t>(rows) * p.row_x, ex = static_cast<size_t>(p.m) * p.row_x;
        const size_t ay = row * p.row_dy, ny = static_cast<size_t>(rows) * p.row_dy, ey = static_cast<size_t>(p.m) * p.row_dy;
        const uint32_t bx = run_bytes<kOdd>(ax, nx, ex), by = kBwd ? run_bytes<kOdd>(ay, ny, ey) : 0u;
        run_tail<kOdd>(dst, p.x, ax, nx, ex);
        if (kBwd) run_tail<kOdd>(dst + p.second, p.dy, ay, ny, ey);
        mbar_arrive_expect_tx(bar, bx + by);
        if (bx > 0) ln_bulk(smem_u32(dst), static_cast<const uint8_t*>(p.x) + (kOdd ? ax & ~size_t(15) : ax), bx, bar);
        if (by > 0) ln_bulk(smem_u32(dst + p.second), static_cast<const uint8_t*>(p.dy) + (kOdd ? ay & ~size_t(15) : ay), by, bar);
    };
    if (threadIdx.x == 0) abort_flag = 0;
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&full[i]), 1u);
        fence_mbar_init();
    }
    pdl_wait();
    if (tid == 0)
        for (int k = 0; k < n && k < p.stages; ++k) fetch(k, k);
    const bool has_g = p.gamma != nullptr, has_b = !kBwd && p.beta != nullptr;
    using Const = std::conditional_t<kOdd, float, float4>;
    if (has_g || has_b)
        for (int i = threadIdx.x; i < nr; i += blockDim.x) {
            if (has_g) reinterpret_cast<Const*>(smem + p.consts)[i] = reinterpret_cast<const Const*>(p.gamma)[i];
            if (has_b) reinterpret_cast<Const*>(smem + p.consts)[nr + i] = reinterpret_cast<const Const*>(p.beta)[i];
        }
    __syncthreads();
    const Four zero{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    Four dg[kBwd ? NQ : 1], db[kBwd ? NQ : 1];
    if constexpr (kBwd) {
#pragma unroll
        for (int k = 0; k < NQ; ++k) dg[k] = db[k] = zero;
    }
    const float inv_c = 1.f / static_cast<float>(c);
    bool ok = true;
    int st = 0, late = 0;
    uint32_t ph = 0;
    for (int k = 0; k < n; ++k) {
        // (a group whose wait ran out goes on through its barriers, but stores nothing)
        if (ok && !warp_all(mbar_wait(smem_u32(&full[st]), ph, &abort_flag, p.timeout_ns, p.status, kWhereNorm))) {
            ok = false;
            late = k;
        }
        const size_t row0 = (static_cast<size_t>(first) + static_cast<size_t>(k) * all) * R;
        const int rows = p.m - row0 < static_cast<size_t>(R) ? static_cast<int>(p.m - row0) : R;
        const uint8_t* src = ring + static_cast<size_t>(st) * p.stage;
        Four v[R][NQ], g[kBwd ? R : 1][NQ];
        float s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            row_in<NQ, kOdd>(src + (kOdd ? row0 * p.row_x & 15 : 0) + r * p.row_x, p.xt, r < rows ? nr : 0, tid, nt, v[r]);
            if constexpr (kBwd)
                row_in<NQ, kOdd>(src + p.second + (kOdd ? row0 * p.row_dy & 15 : 0) + r * p.row_dy, p.dyt, r < rows ? nr : 0, tid,
                                 nt, g[r]);
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NQ; ++i) t = add2(t, add2(v[r][i].a, v[r][i].b));
            s[r] = t.x + t.y;
        }
        group_sums<R>(s, &red[0][group * wide * R], group, wide, part);
        // every thread of the group has its part of the chunk in registers (wide > 1: the barrier in the sums)
        if (wide == 1) __syncwarp();
        if (tid == 0 && ok && k + p.stages < n) fetch(k + p.stages, st);
        if (++st == p.stages) {
            st = 0;
            ph ^= 1u;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 mm = make_float2(-s[r] * inv_c, -s[r] * inv_c);
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                if constexpr (!kOdd) {
                    v[r][i] = tid + i * nt < nr ? Four{add2(v[r][i].a, mm), add2(v[r][i].b, mm)} : zero;
                } else {
                    v[r][i] = {add2(v[r][i].a, mm), add2(v[r][i].b, mm)};
                    if (odd_at(i, 0, tid, nt) >= nr) v[r][i].a.x = 0.f;
                    if (odd_at(i, 1, tid, nt) >= nr) v[r][i].a.y = 0.f;
                    if (odd_at(i, 2, tid, nt) >= nr) v[r][i].b.x = 0.f;
                    if (odd_at(i, 3, tid, nt) >= nr) v[r][i].b.y = 0.f;
                }
                t = fma2(v[r][i].a, v[r][i].a, fma2(v[r][i].b, v[r][i].b, t));
            }
            s[r] = t.x + t.y;
        }
        group_sums<R>(s, &red[1][group * wide * R], group, wide, part);
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = 1.f / sqrtf(s[r] * inv_c + p.eps);
        if (rows < R)  // (0 for the rows that the last chunk lacks: with eps 0 theirs would be infinite)
#pragma unroll
            for (int r = 1; r < R; ++r)
                if (r >= rows) s[r] = 0.f;
        uint8_t* out = static_cast<uint8_t*>(p.out) + row0 * c * (((kBwd ? p.xt : p.yt) == VAE_F32) ? 4 : 2);
        const size_t out_row = static_cast<size_t>(c) * (((kBwd ? p.xt : p.yt) == VAE_F32) ? 4 : 2);
        if constexpr (!kBwd) {
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const Four w = get4<VAE_F32, kOdd>(gam, has_g ? nr : 0, i, tid, nt, 1.f);
                const Four b = get4<VAE_F32, kOdd>(bet, has_b ? nr : 0, i, tid, nt, 0.f);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 q = make_float2(s[r], s[r]);
                    v[r][i] = {fma2(mul2(v[r][i].a, q), w.a, b.a), fma2(mul2(v[r][i].b, q), w.b, b.b)};
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (ok && r < rows) row_out<NQ, kOdd>(out + r * out_row, p.yt, nr, tid, nt, v[r]);
        } else {
            float2 s1[R], s2[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s1[r] = s2[r] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const Four w = get4<VAE_F32, kOdd>(gam, has_g ? nr : 0, i, tid, nt, 1.f);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 q = make_float2(s[r], s[r]);
                    Four& y = g[r][i];
                    const Four& d = v[r][i];
                    dg[i] = {fma2(mul2(y.a, q), d.a, dg[i].a), fma2(mul2(y.b, q), d.b, dg[i].b)};
                    db[i] = {add2(db[i].a, y.a), add2(db[i].b, y.b)};
                    y = {mul2(y.a, w.a), mul2(y.b, w.b)};
                    s1[r] = add2(s1[r], add2(y.a, y.b));
                    s2[r] = fma2(y.a, d.a, fma2(y.b, d.b, s2[r]));
                }
            }
            float sums[2 * R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                sums[r] = s1[r].x + s1[r].y;
                sums[R + r] = s2[r].x + s2[r].y;
            }
            group_sums<2 * R>(sums, &red[2][group * wide * 2 * R], group, wide, part);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // dx = rstd (g - mean(g) - n mean(g n)), n = rstd v; rstd^3 by itself would leave f32 for rows far from
                // one (from about 2^42 and 2^-42 on), rstd times the sum over g v first stays near the size of g
                const float rstd = s[r], k1 = -rstd * sums[r] * inv_c, k2 = -rstd * (rstd * (rstd * sums[R + r] * inv_c));
                const float2 q = make_float2(rstd, rstd), q1 = make_float2(k1, k1), q2 = make_float2(k2, k2);
#pragma unroll
                for (int i = 0; i < NQ; ++i)
                    v[r][i] = {fma2(g[r][i].a, q, fma2(v[r][i].a, q2, q1)), fma2(g[r][i].b, q, fma2(v[r][i].b, q2, q1))};
                if (ok && r < rows) row_out<NQ, kOdd>(out + r * out_row, p.xt, nr, tid, nt, v[r]);
            }
        }
    }
    // Every copy lands before the block may exit (after a time-out: the chunks that were fetched and not met).
    if (!ok && tid == 0) {
        int never = 0;
        for (int k = late; k < n && k < late + p.stages; ++k)
            (void)mbar_wait(smem_u32(&full[k % p.stages]), static_cast<uint32_t>(k / p.stages) & 1u, &never, p.timeout_ns,
                            p.status, kWhereDrain);
    }
    if constexpr (kBwd) {
        if (p.part == nullptr) return;
        // the groups' column sums side by side over the ring (8 c bytes a group: less than its two stages), then joined in order
        float* cols = reinterpret_cast<float*>(smem);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            uint8_t* w = reinterpret_cast<uint8_t*>(cols + static_cast<size_t>(group) * 2 * c);
            put4<VAE_F32, kOdd>(w, nr, i, tid, nt, dg[i]);
            put4<VAE_F32, kOdd>(w + static_cast<size_t>(c) * 4, nr, i, tid, nt, db[i]);
        }
        __syncthreads();
        float* out = p.part + static_cast<size_t>(blockIdx.x) * 2 * c;
        for (int i = threadIdx.x; i < 2 * c; i += blockDim.x) {
            float a = cols[i];
            for (int u = 1; u < groups; ++u) a += cols[static_cast<size_t>(u) * 2 * c + i];
            out[i] = a;
        }
        pdl_launch_dependents();
    }
}

// out[0 .. c) = sum over the blocks' partial rows, dgamma then dbeta: 32
// columns x 32 slices of blocks per thread block, each slice's loads in flight
// together, the slices joined in order.
constexpr int kColSlices = 32;
__global__ void __launch_bounds__(kColSlices * 32) ln_cols_kernel(const float* __restrict__ part, int nblk, int c,
                                                                  float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float s[kColSlices][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    constexpr int kMost = (2 * kLnBwdBlocks + kColSlices - 1) / kColSlices;
    float a = 0.f;
    if (col < 2 * c) {
        float v[kMost];
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int b = slice + k * kColSlices;
            v[k] = b < nblk ? part[static_cast<size_t>(b) * 2 * c + col] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kMost; ++k) a += v[k];
    }
    s[slice][lane] = a;
    __syncthreads();
    // warp w joins column w's slices
    a = warp_sum(s[lane][slice]);
    const int out = blockIdx.x * 32 + slice;
    if (lane == 0 && out < 2 * c) (out < c ? dgamma : dbeta - c)[out] = a;
}

// How a row is held: warp form or the block's threads, and eights per thread.
struct LnPlan {
    bool v8, warp;
    int nv, threads;
};
LnPlan ln_plan(int c, bool backward) {
    LnPlan p;
    p.v8 = c % 8 == 0;
    const int nvec = (c + 7) / 8;
    // (the gradient element by element: over 512 channels a warp's registers would leave one block an SM)
    p.warp = nvec <= (backward && !p.v8 ? 64 : 32 * kLnWarpVec);
    if (p.warp) {
        p.nv = (nvec + 31) / 32;
        p.threads = 32;
    } else {
        p.nv = nvec <= 512 ? 2 : 4;
        p.threads = std::min(512, ((nvec + p.nv - 1) / p.nv + 31) / 32 * 32);
    }
    return p;
}
// The ring form's plan for rows of x (and dy: backward); false where the plain
// form is used: rows over 5120 channels, so few of them that a group would not
// have two chunks, tensors off the 16-byte boundaries that the copies need, and
// forward rows of a length that is no multiple of eight (16384x1155, f32 to f16:
// 39 us in the ring against 27 in the plain form; their gradient, f32 and f16, 66
// against 107).
bool ln_ring_plan(int m, int c, int xt, int dyt, bool backward, bool aligned, LnRing* r) {
    const bool odd = c % 8 != 0;
    if (c > 5120 || c < 8 || !aligned || (odd && !backward)) return false;
    const int most = backward ? 640 : 1280;  // channels of one warp's share of a row
    r->wide = c <= most ? 1 : (c <= 2 * most ? 2 : (c <= 4 * most ? 4 : 8));
    r->nq = ((c + 3) / 4 + r->wide * 32 - 1) / (r->wide * 32);
    const int rows = ring_rows(r->nq);
    r->row_x = static_cast<unsigned>(c * type_size(xt));
    r->row_dy = backward ? static_cast<unsigned>(c * type_size(dyt)) : 0u;
    // (odd lengths: up to two partial units more)
    r->second = odd ? (rows * r->row_x + 32 + 15) / 16 * 16 : rows * r->row_x;
    r->stage = r->second + (backward ? (odd ? (rows * r->row_dy + 32 + 15) / 16 * 16 : rows * r->row_dy) : 0);
    const int max_warps = ring_warps(r->nq, backward);
    const size_t consts = (static_cast<size_t>(c) * (backward ? 4 : 8) + 15) / 16 * 16;
    const size_t bars = static_cast<size_t>(max_warps) * kRingStages * 8;
    const size_t left = kRingSmem - consts - bars;
    // As many groups as fit with two stages each (the gradient: three, where that leaves one; 65536x1152 in f32 and f16
    // 125 us against 136), then as many stages as fit.
    if (left < 2 * static_cast<size_t>(r->stage)) return false;
    const size_t fit = std::max<size_t>(1, left / ((backward ? 3 : 2) * static_cast<size_t>(r->stage)));
    const int groups = static_cast<int>(std::min<size_t>(fit, max_warps / r->wide));
    if (groups < 1 || m < 2 * kRingBlocks * groups * rows) return false;
    r->warps = groups * r->wide;
    r->stages = static_cast<int>(std::min<size_t>(kRingStages, left / (static_cast<size_t>(groups) * r->stage)));
    r->consts = static_cast<unsigned>(static_cast<size_t>(groups) * r->stages * r->stage);
    r->bars = static_cast<unsigned>(r->consts + consts);
    r->m = m;
    r->c = c;
    r->xt = xt;
    r->dyt = dyt;
    return true;
}
size_t ln_ring_smem(const LnRing& r) { return r.bars + static_cast<size_t>(r.warps) * kRingStages * 8; }

template <int NQ, bool kBwd, bool kOdd>
int ln_ring_launch_as(const LnRing& r, cudaStream_t st) {
    static CtxOnce once;
    static std::mutex mu;
    {
        int dev;
        VAE_CUDA_CHECK(cudaGetDevice(&dev));
        std::lock_guard<std::mutex> lk(mu);
        if (!once.done(dev)) {
            VAE_CUDA_CHECK(cudaFuncSetAttribute(ln_ring_kernel<NQ, kBwd, kOdd>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                static_cast<int>(kRingSmem)));
            once.mark(dev);
        }
    }
    VAE_CUDA_CHECK(launch_kernel(ln_ring_kernel<NQ, kBwd, kOdd>, dim3(kRingBlocks), dim3(r.warps * 32), ln_ring_smem(r), st, r));
    return VAE_OK;
}
template <int NQ, bool kBwd>
int ln_ring_launch(const LnRing& r, cudaStream_t st) {
    if constexpr (kBwd)
        if (r.c % 8 != 0) return ln_ring_launch_as<NQ, kBwd, true>(r, st);
    return ln_ring_launch_as<NQ, kBwd, false>(r, st);
}
template <bool kBwd>
int ln_ring_run(LnRing& r, cudaStream_t st) {
    r.status = device_status_ptr();
    r.timeout_ns = wait_timeout_ns();
    if (r.status == nullptr) return VAE_ERR_CUDA;
    switch (r.nq) {
        case 1: return ln_ring_launch<1, kBwd>(r, st);
        case 2: return ln_ring_launch<2, kBwd>(r, st);
        case 3: return ln_ring_launch<3, kBwd>(r, st);
        case 4: return ln_ring_launch<4, kBwd>(r, st);
        case 5: return ln_ring_launch<5, kBwd>(r, st);
        default: break;
    }
    if constexpr (!kBwd) switch (r.nq) {
            case 6: return ln_ring_launch<6, kBwd>(r, st);
            case 7: return ln_ring_launch<7, kBwd>(r, st);
            case 8: return ln_ring_launch<8, kBwd>(r, st);
            case 9: return ln_ring_launch<9, kBwd>(r, st);
            default: return ln_ring_launch<10, kBwd>(r, st);
        }
    return set_error(VAE_ERR_SHAPE, "layer norm: no ring form for %d channels", r.c);
}

int ln_bwd_grid(int m, int c) {
    const LnPlan p = ln_plan(c, true);
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

// Rows of a multiple of eight channels move in 16-byte vectors; others by the element.
bool ln_aligned(const void* p, size_t element, int c) {
    return reinterpret_cast<uintptr_t>(p) % (c % 8 == 0 ? 16 : element) == 0;
}

int ln_check(const void* x, int xt, int m, int c, float eps, const void* y, int yt) {
    if (x == nullptr || y == nullptr) return set_error(VAE_ERR_ARG, "layer norm: NULL tensor");
    if (!type_ok(xt) || !type_ok(yt)) return set_error(VAE_ERR_ARG, "layer norm: unknown element type");
    if (m < 1 || c < 1 || c > kLnMaxC)
        return set_error(VAE_ERR_SHAPE, "layer norm: m >= 1 and 1 <= c <= %d are needed, got m %d, c %d", kLnMaxC, m, c);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return set_error(VAE_ERR_ARG, "layer norm: eps must be >= 0 and finite");
    return VAE_OK;
}

// `what` is written over none of the rest.
struct LnPart {
    const char* name;
    const void* p;
    size_t bytes;
};
int ln_apart(const LnPart& what, std::initializer_list<LnPart> rest) {
    if (what.p == nullptr) return VAE_OK;
    for (const LnPart& r : rest)
        if (r.p != nullptr && extents_meet(extent_dense(what.p, what.bytes), extent_dense(r.p, r.bytes)))
            return set_error(VAE_ERR_ARG, "layer norm: %s may not overlap %s", what.name, r.name);
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
    if (!ln_aligned(x_dev, type_size(x_type), c) || !ln_aligned(y_dev, type_size(y_type), c) ||
        !ln_aligned(gamma_dev, 4, c) || !ln_aligned(beta_dev, 4, c))
        return set_error(VAE_ERR_ALIGN, "layer norm: pointers must be 16-byte aligned (to their elements where c %% 8 != 0)");
    const size_t n = static_cast<size_t>(m) * c, row = static_cast<size_t>(c) * sizeof(float);
    if ((rc = ln_apart({"y", y_dev, n * type_size(y_type)}, {{"x", x_dev == y_dev ? nullptr : x_dev, n * type_size(x_type)},
                                                             {"gamma", gamma_dev, row}, {"beta", beta_dev, row}})) != VAE_OK)
        return rc;
    if ((rc = check_device()) != VAE_OK) return rc;
    LnRing r{};
    if (ln_ring_plan(m, c, x_type, x_type, false, aligned16(x_dev), &r)) {
        r.x = x_dev;
        r.gamma = gamma_dev;
        r.beta = beta_dev;
        r.eps = eps;
        r.out = y_dev;
        r.yt = y_type;
        return ln_ring_run<false>(r, reinterpret_cast<cudaStream_t>(stream));
    }
    const LnPlan p = ln_plan(c, false);
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
    if (!ln_aligned(x_dev, type_size(x_type), c) || !ln_aligned(dy_dev, type_size(dy_type), c) ||
        !ln_aligned(dx_dev, type_size(x_type), c) || !ln_aligned(gamma_dev, 4, c) || !ln_aligned(dgamma_dev, 4, c) ||
        !ln_aligned(dbeta_dev, 4, c) || !aligned16(workspace_dev))
        return set_error(VAE_ERR_ALIGN, "layer norm: pointers must be 16-byte aligned (to their elements where c %% 8 != 0)");
    if (sums && workspace_bytes < vae_layernorm_backward_workspace_bytes(m, c))
        return set_error(VAE_ERR_NOMEM, "layer norm: workspace of %zu bytes, %zu needed", workspace_bytes,
                         vae_layernorm_backward_workspace_bytes(m, c));
    const size_t n = static_cast<size_t>(m) * c, row = static_cast<size_t>(c) * sizeof(float);
    const LnPart x{"x", x_dev, n * type_size(x_type)}, dy{"dy", dy_dev, n * type_size(dy_type)}, dx{"dx", dx_dev, x.bytes};
    const LnPart gamma{"gamma", gamma_dev, row}, dgamma{"dgamma", dgamma_dev, row}, dbeta{"dbeta", dbeta_dev, row};
    const LnPart none{"", nullptr, 0};
    // (dgamma and dbeta are written once x, dy and gamma have been read)
    if ((rc = ln_apart(dx, {dx_dev == x_dev ? none : x, dx_dev == dy_dev ? none : dy, gamma, dgamma, dbeta})) != VAE_OK ||
        (rc = ln_apart(dgamma, {dbeta})) != VAE_OK ||
        (sums && (rc = ln_apart({"the workspace", workspace_dev, vae_layernorm_backward_workspace_bytes(m, c)},
                                {x, dy, dx, gamma, dgamma, dbeta})) != VAE_OK))
        return rc;
    if ((rc = check_device()) != VAE_OK) return rc;
    const LnPlan p = ln_plan(c, true);
    int grid = ln_bwd_grid(m, c);
    float* part = sums ? static_cast<float*>(workspace_dev) : nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LnRing r{};
    if (ln_ring_plan(m, c, x_type, dy_type, true, aligned16(x_dev) && aligned16(dy_dev), &r)) {
        r.x = x_dev;
        r.dy = dy_dev;
        r.gamma = gamma_dev;
        r.eps = eps;
        r.out = dx_dev;
        r.part = part;
        grid = kRingBlocks;
        if ((rc = ln_ring_run<true>(r, s)) != VAE_OK) return rc;
    } else {
        VAE_CUDA_CHECK(ln_dispatch(p, [&](auto nv, auto v8, auto warp) {
            const auto kernel = ln_bwd_kernel<nv.value, v8.value, warp.value>;
            const size_t cols = warp.value && sums ? kLnBwdWarps * 2 * static_cast<size_t>(c) * sizeof(float) : 0;
            if (cols > 48 * 1024) {
                const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           static_cast<int>(cols));
                if (e != cudaSuccess) return e;
            }
            return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(warp.value ? kLnBwdWarps * 32 : p.threads),
                                 cols, s, dy_dev, dy_type, x_dev, x_type, m, c, gamma_dev, eps, dx_dev, part);
        }));
    }
    if (sums)
        VAE_CUDA_CHECK(launch_next(ln_cols_kernel, dim3((2u * static_cast<unsigned>(c) + 31u) / 32u),
                                     dim3(kColSlices * 32), 0, s,
                                     static_cast<const float*>(part), grid, c, dgamma_dev, dbeta_dev));
    return VAE_OK;
}

}  // extern "C"
