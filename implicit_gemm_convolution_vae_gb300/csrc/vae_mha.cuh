// Multi-head attention on latent tokens: what the forward and the gradient
// kernels share. Which keys a row sees, how rows are tiled, argument checks,
// and the tcgen05 pieces that the mid attention does not use: operands stored
// with the contraction index outside (MN-major) and left operands in TMEM.
//
// Rows. The query heads that share a key head stand side by side as rows: with
// gp the largest power of two that divides g = hq / hkv (64 at most), row
// r = token * gp + head of the group, so that one 128-row tile of q (a TMA box
// of 128/gp tokens x gp heads) meets each key tile once for all of them. What
// is left of g (sub = g / gp) are tiles of their own.
#pragma once

#include "vae_types.cuh"

namespace vae {

struct MhaShape {
    int b, sq, sk, hq, hkv, g, d, block;
    int fill;           // rows behind the lengths are written as 0
    int gp_log2, nsub;  // gp = 1 << gp_log2, nsub = g / gp
    int ntile;          // 128-row tiles of sq * gp rows
    int nkb;            // 128-key tiles of sk
    const int *q_len, *k_len;
};

constexpr int kMhaTile = 128;          // rows of q and keys per tile
constexpr int kMhaChunkBytes = 16384;  // 128 rows x 64 channels of 16 bits, 128-byte swizzle

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
    const int at = i - ql + kl;  // (in this order no sum passes 31 bits)
    if (at < 0) return 0;
    const long long end = (static_cast<long long>(at) / block + 1) * block;
    return end < kl ? static_cast<int>(end) : kl;
}

// Checks the desc (backward: the gradients' strides too); fills `s`.
int mha_check(const vae_attention_desc* d, bool backward, MhaShape* s);

struct MhaStrides {
    long long b, s, h;
};
inline MhaStrides mha_strides(const long long* st) { return {st[0], st[1], st[2]}; }

// Tensor map of a [b][n][h][d] tensor of 16-bit elements: boxes of 64 channels
// x `heads` heads x `tokens` tokens; what lies behind d or n reads as 0.
int mha_map(CUtensorMap* map, const vae_attention_desc* a, const void* p, const long long* stride, int n, int h,
            int heads, int tokens);

// ───────────────────────────── tcgen05 pieces ─────────────────────────────

// Instruction descriptor of kind::f16 with f32 accumulators: A K-major (or in
// TMEM), B K-major, or MN-major when trans_b.
__host__ __device__ constexpr uint32_t mha_idesc(int type, int M, int N, bool trans_b) {
    return (1u << 4) | ((type == VAE_BF16 ? 1u : 0u) << 7) | ((type == VAE_BF16 ? 1u : 0u) << 10) |
           ((trans_b ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of an MN-major operand tile as TMA leaves a [rows][64 channels]
// box with the 128-byte swizzle, read with the rows as the contraction index:
// 8-row groups 1024 bytes apart (stride offset), the next 64 channels a chunk
// further (leading offset). Sixteen rows on: 2048 bytes.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kMhaChunkBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// D(tmem) (+)= A(tmem: 16-bit pairs per column, a row per lane) * B(smem desc).
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp, always the same. The MMA warps run their loops
// with all lanes and issue under this predicate: a loop that only one lane
// entered cannot keep the descriptors in uniform registers, and each M = 128,
// N = 128 MMA (64 cycles of tensor work) then took about 114 cycles to issue.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

// D = A B^T of two K-major tiles in shared memory, kSteps x 16 channels.
template <int kSteps>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const uint32_t off = static_cast<uint32_t>((k >> 2) * (kMhaChunkBytes >> 4) + (k & 3) * 2);
        umma_f16(d_tmem, a + off, b + off, id, k != 0 ? 1u : 0u);
    }
}
// D (+)= A B with 128 columns of A as 16-bit pairs in TMEM: two halves kHalf
// columns apart, 32 columns each; B MN-major.
template <int kHalf>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        umma_f16_ts(d_tmem, a_tmem + static_cast<uint32_t>((k >> 2) * kHalf + (k & 3) * 8), b + (2048u >> 4) * k, id,
                    k != 0 ? 1u : acc);
}

// D = A B^T with A's rows in TMEM (16 channels in eight columns), B K-major.
template <int kSteps>
__device__ __forceinline__ void mma_ts_k(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        umma_f16_ts(d_tmem, a_tmem + 8u * k, b + static_cast<uint32_t>((k >> 2) * (kMhaChunkBytes >> 4) + (k & 3) * 2), id,
                    k != 0 ? 1u : 0u);
}

// What packing a and b to 16 bits leaves of them, packed. Where a tile has room
// for its rows twice, the second copies take this part of P and dS: the products
// with the two are added. One rounding of P or dS is as large as the result's
// own. Over many rows and keys both add up to 1.4 times the latter's error, but
// over few they may fall together (2.2 times in bf16 for one row over 16 keys).
template <int T>
__device__ __forceinline__ uint32_t pack2_rest(float a, float b) {
    const float2 h = unpack2<T>(pack2<T>(a, b));
    return pack2<T>(a - h.x, b - h.y);
}

// 2^x, approximate (relative error near 2^-22); under 2^-126 it is 0.
__device__ __forceinline__ float mha_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Writes 0 to the rows of a 128-row query tile of key head hk that lie behind
// ql (and -infinity to their lse, where there is one), or to the rows from kl
// on of a key tile; every thread of the block.
__device__ __forceinline__ void mha_fill_row(void* x, long long off, int d, int part) {
    for (int c = part * 8; c < d; c += 32)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x) + off + c) = make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void mha_fill_queries(const MhaShape& s, int e, int hk, int sub, int tile, int ql, void* x,
                                                 long long sb, long long ss, long long sh, float* lse) {
    const int gp = 1 << s.gp_log2;
    if (ql == s.sq || tile >= s.ntile || ((tile + 1) * static_cast<long long>(kMhaTile) - 1) >> s.gp_log2 < ql) return;
    for (int k = threadIdx.x; k < kMhaTile * 4; k += blockDim.x) {
        const int r = tile * kMhaTile + k / 4, i = r >> s.gp_log2, h = hk * s.g + sub * gp + (r & (gp - 1));
        if (i < ql || i >= s.sq) continue;
        mha_fill_row(x, e * sb + i * ss + h * sh, s.d, k & 3);
        if (lse != nullptr && (k & 3) == 0) lse[(static_cast<long long>(e) * s.hq + h) * s.sq + i] = -INFINITY;
    }
}
__device__ __forceinline__ void mha_fill_keys(const MhaShape& s, int e, int hk, int kb, int kl, void* x, long long sb,
                                              long long ss, long long sh) {
    for (int k = threadIdx.x; k < kMhaTile * 4; k += blockDim.x) {
        const int j = kb * kMhaTile + k / 4;
        if (j >= kl && j < s.sk) mha_fill_row(x, e * sb + j * ss + hk * sh, s.d, k & 3);
    }
}

// Zeroes rows [from, 128) of a tile of `chunks` chunks in shared memory; the
// whole warp. The caller fences towards the async proxy.
__device__ __forceinline__ void mha_zero_rows(uint8_t* tile, int from, int to, int chunks, int lane) {
    for (int c = 0; c < chunks; ++c)
        for (int i = from * 8 + lane; i < to * 8; i += 32)
            *reinterpret_cast<uint4*>(tile + c * kMhaChunkBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace vae
