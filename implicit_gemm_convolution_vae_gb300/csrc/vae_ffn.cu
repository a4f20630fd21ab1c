// The gated feed-forward block and its gradient (public entry points at the end).
//
//   gate = x Wg^T, up = x Wu^T, hidden = act(gate) o up, y = hidden Wd^T;
//   dhidden = dy Wd, dup = dhidden o act(gate), dgate = dhidden o up o act'(gate),
//   dx = dgate Wg + dup Wu, dWg = dgate^T x, dWu = dup^T x, dWd = dy^T hidden.
//
// One product kernel, on pairs of CTAs (tcgen05 cta_group::2), with an epilogue for
// each: D = A B^T of 256 x 256 tiles, 128 rows of A and half of B's rows in each CTA's
// shared memory, f32 accumulators in TMEM, two of them, so that the epilogue of a tile
// runs under the products of the next. An operand whose contraction index is not its
// inner one (Wd and Wg, Wu backward, all operands of the weights' gradients) is read
// as it lies in memory, MN-major: nothing is transposed. The tile of the first product
// holds 128 gate and 128 up columns of the same hidden channels (the even CTA loads
// rows of Wg, the odd one of Wu), so act(gate) o up never leaves the registers.
#include <algorithm>
#include <mutex>

#include "vae_overlap.h"
#include "vae_types.cuh"

namespace vae {

namespace {

constexpr int kTile = 128;              // rows of A, and of B, per CTA
constexpr int kBk = 64;                 // contraction per stage: one 128-byte swizzle row
constexpr int kOperand = kTile * kBk * 2;  // bytes
constexpr int kStage = 2 * kOperand;
constexpr int kStages = 7;
constexpr int kEpiWarps = 8, kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kSmem = 1024 + kStages * kStage + 512;
static_assert(kSmem <= 232448, "shared memory over 227 KB");
constexpr uint32_t kTmemCols = 512;     // two accumulators of 256 columns
constexpr int kGroup = 8;               // row tiles that share their column tiles in L2

// The products. A and B stand as [rows][contraction] (K-major) or [contraction][rows].
enum : int {
    kGate,      // x, (Wg, Wu) -> hidden (gate, up)
    kDown,      // hidden, Wd -> y
    kBackGate,  // dy, Wd^T -> dgate, dup
    kDx,        // (dgate, dup), (Wg, Wu)^T -> dx
    kDw,        // dgate^T, x^T -> dWg; dup^T, x^T -> dWu; dy^T, hidden^T -> dWd
};
__host__ __device__ constexpr bool a_mn(int kind) { return kind == kDw; }
__host__ __device__ constexpr bool b_mn(int kind) { return kind >= kBackGate; }

struct Maps {
    CUtensorMap a[3], b[3];
};

struct Params {
    int rows[3], cols[3];      // of D, per problem
    int tiles_n[3];
    int first[4];              // a problem's first tile
    int nk, segments;          // stages of a tile (per segment: products that add up)
    int activation;
    void* out[3];              // kGate: hidden, gate, up; kBackGate: dgate, dup; others: D of each problem
    int out_f32;
    const float* residual;
    const void *gate, *up;     // kBackGate
    const unsigned* amax;      // f16 gradients: the largest |dy|'s bits
    int wide;                  // rows of D on 32 bytes
    DevStatus* status;
    unsigned long long timeout_ns;
};

struct Smem {
    uint8_t* ring;
    uint64_t *full, *empty, *accf, *acce, *drain;
    uint32_t* tmem_slot;
    int* abort_flag;
};
__device__ __forceinline__ Smem carve(uint8_t* raw) {
    Smem s;
    s.ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t* b = reinterpret_cast<uint64_t*>(s.ring + kStages * kStage);
    s.full = b;
    s.empty = b + kStages;
    s.accf = b + 2 * kStages;
    s.acce = s.accf + 2;
    s.drain = s.acce + 2;
    s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
    s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
    return s;
}

struct Tile {
    int z, m0, n0;  // problem, first row of the pair, first column
};
// Row tiles in groups of kGroup, their column tiles side by side: the pairs at work share rows of A and of B.
template <int kKind>
__device__ __forceinline__ Tile tile_at(const Params& p, int t) {
    Tile r;
    r.z = 0;
    if constexpr (kKind == kDw) r.z = t >= p.first[2] ? 2 : t >= p.first[1] ? 1 : 0;
    t -= p.first[r.z];
    const int nn = p.tiles_n[r.z], nm = (p.rows[r.z] + 2 * kTile - 1) / (2 * kTile);
    const int g = t / (kGroup * nn), in = t - g * kGroup * nn;
    const int tall = nm - g * kGroup < kGroup ? nm - g * kGroup : kGroup;
    r.m0 = (g * kGroup + in % tall) * 2 * kTile;
    r.n0 = in / tall * (kKind == kGate ? kTile : 2 * kTile);
    return r;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}

// One operand of a stage: 128 rows from `row` on, 64 of the contraction from `k` on.
template <bool kMn>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int row, int k) {
    if constexpr (kMn) {  // two boxes of 64 rows each, as they lie
        tma_load_2d_pair(smem_u32(dst), map, bar, row, k);
        tma_load_2d_pair(smem_u32(dst + kOperand / 2), map, bar, row + 64, k);
    } else {
        tma_load_2d_pair(smem_u32(dst), map, bar, k, row);
    }
}

// Descriptor of an MN-major operand: rows of 64 along M or N (128 bytes, swizzled), eight
// contraction rows 1024 bytes apart, the next 64 along M or N 8 KB further. Sixteen of the
// contraction on: 2048 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kOperand / 2) >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

template <int kKind>
__device__ void role_producer(const Params& p, const Smem& s, const Maps& maps, int rank) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, arm_par = 0;
    bool ok = true;
    const int tiles = p.first[3], step = static_cast<int>(gridDim.x >> 1);
    for (int t = static_cast<int>(blockIdx.x >> 1); ok && t < tiles; t += step) {
        const Tile ti = tile_at<kKind>(p, t);
        const int row = ti.m0 + rank * kTile, col = kKind == kGate ? ti.n0 : ti.n0 + rank * kTile;
        for (int seg = 0; ok && seg < p.segments; ++seg) {
            const CUtensorMap* ma = &maps.a[kKind == kDx ? seg : ti.z];
            const CUtensorMap* mb = &maps.b[kKind == kDx ? seg : kKind == kGate ? rank : ti.z];
            for (int k = 0; k < p.nk; ++k) {
                ok = mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, s.abort_flag, p.timeout_ns, p.status, kWhereProducerEmpty);
                if (!ok) break;
                const uint32_t fb = smem_u32(&s.full[stage]);
                if (rank == 0) mbar_arrive_expect_tx(fb, 2u * kStage);
                const uint32_t fb0 = mapa_shared(fb, 0u);
                uint8_t* a = s.ring + stage * kStage;
                load_operand<a_mn(kKind)>(a, ma, fb0, row, k * kBk);
                load_operand<b_mn(kKind)>(a + kOperand, mb, fb0, col, k * kBk);
                armed |= 1u << stage;
                arm_par = (arm_par & ~(1u << stage)) | (phase << stage);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    }
    // Every copy lands before the CTA can exit: the even CTA sees them on its full barriers, the odd one
    // on its empty barriers (the products that read a slot complete after its copies).
    int never = 0;
    for (int st = 0; st < kStages; ++st)
        if (armed & (1u << st))
            (void)mbar_wait(smem_u32(rank == 0 ? &s.full[st] : &s.empty[st]), (arm_par >> st) & 1u, &never, p.timeout_ns,
                            p.status, kWhereDrain);
}

// The whole warp runs the loop and one lane issues: descriptors stay in uniform registers.
template <int T, int kKind>
__device__ void role_mma(const Params& p, const Smem& s, uint32_t tmem) {
    constexpr uint32_t ab = T == VAE_BF16 ? 1u : 0u;
    constexpr uint32_t idesc = (1u << 4) | (ab << 7) | (ab << 10) | ((a_mn(kKind) ? 1u : 0u) << 15) |
                               ((b_mn(kKind) ? 1u : 0u) << 16) | ((2u * kTile >> 3) << 17) | ((2u * kTile >> 4) << 24);
    constexpr uint32_t astep = a_mn(kKind) ? 2048 >> 4 : 2, bstep = b_mn(kKind) ? 2048 >> 4 : 2;
    const uint32_t ring = smem_u32(s.ring);
    const uint64_t ad = a_mn(kKind) ? mn_desc(ring) : sw128_kmajor_desc(ring);
    const uint64_t bd = b_mn(kKind) ? mn_desc(ring + kOperand) : sw128_kmajor_desc(ring + kOperand);
    int stage = 0, buf = 0;
    uint32_t phase = 0, accphase = 0;
    bool ok = true;
    const int tiles = p.first[3], step = static_cast<int>(gridDim.x >> 1), nk = p.nk * p.segments;
    for (int t = static_cast<int>(blockIdx.x >> 1); ok && t < tiles; t += step) {
        ok = warp_all(mbar_wait_cluster(smem_u32(&s.acce[buf]), accphase ^ 1u, s.abort_flag, p.timeout_ns, p.status, kWhereMmaAccEmpty));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * 2 * kTile);
        for (int k = 0; k < nk; ++k) {
            ok = warp_all(mbar_wait(smem_u32(&s.full[stage]), phase, s.abort_flag, p.timeout_ns, p.status, kWhereMmaFull));
            if (!ok) break;
            tc_fence_after();
            const uint32_t off = static_cast<uint32_t>(stage) * (kStage >> 4);
            if (elect_one()) {
#pragma unroll
                for (uint32_t i = 0; i < kBk / 16; ++i)
                    umma_f16_pair(d, ad + (off + i * astep), bd + (off + i * bstep), idesc, i != 0 || k != 0 ? 1u : 0u);
                umma_commit_pair(smem_u32(&s.empty[stage]));
                if (k + 1 == nk) umma_commit_pair(smem_u32(&s.accf[buf]));
            }
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        buf ^= 1;
        if (buf == 0) accphase ^= 1u;
    }
    if (elect_one()) {
        umma_commit_pair(smem_u32(s.drain));
        int never = 0;
        (void)mbar_wait(smem_u32(s.drain), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
    }
    __syncwarp();
}

// ───────────────────────────── activations ─────────────────────────────

// act(g), and its derivative.
__device__ __forceinline__ float act_value(int kind, float g) {
    if (kind == VAE_ACT_GELU) return 0.5f * g * (1.f + erff(g * 0.70710678118654752440f));
    const float z = kind == VAE_ACT_SILU ? g : 1.59576912160573071176f * (g + 0.044715f * g * g * g);
    return g * __fdividef(1.f, 1.f + __expf(-z));  // (1 + tanh(z / 2)) / 2 is the logistic function of z
}
__device__ __forceinline__ float2 act_both(int kind, float g) {
    if (kind == VAE_ACT_GELU) {
        const float cdf = 0.5f * (1.f + erff(g * 0.70710678118654752440f));
        return make_float2(g * cdf, cdf + g * 0.39894228040143267794f * __expf(-0.5f * g * g));
    }
    const bool silu = kind == VAE_ACT_SILU;
    const float z = silu ? g : 1.59576912160573071176f * (g + 0.044715f * g * g * g);
    const float dz = silu ? 1.f : 1.59576912160573071176f * (1.f + 0.134145f * g * g);
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return make_float2(g * s, s * (1.f + g * dz * (1.f - s)));
}

// The power of two that brings the largest |dy| to 4..8 (1 where there is none, or it is not finite).
__device__ __forceinline__ float dy_scale(const unsigned* amax) {
    if (amax == nullptr) return 1.f;
    const unsigned bits = *amax;
    const int e = static_cast<int>(bits >> 23) - 127;
    return bits == 0u || bits >= 0x7f800000u ? 1.f : __uint_as_float(static_cast<unsigned>(2 - e + 127) << 23);
}

// ───────────────────────────── epilogue ─────────────────────────────

struct B32 {
    uint32_t r[8];
};
// Sixteen 16-bit elements of a row (eight where `left` is less): whole 32-byte sectors where rows lie on them.
__device__ __forceinline__ void store16(void* at, const B32& v, int left, bool wide) {
    if (wide && left >= 16) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v.r[0]), "r"(v.r[1]), "r"(v.r[2]),
                     "r"(v.r[3]), "r"(v.r[4]), "r"(v.r[5]), "r"(v.r[6]), "r"(v.r[7])
                     : "memory");
        return;
    }
    *static_cast<uint4*>(at) = make_uint4(v.r[0], v.r[1], v.r[2], v.r[3]);
    if (left >= 16) *(static_cast<uint4*>(at) + 1) = make_uint4(v.r[4], v.r[5], v.r[6], v.r[7]);
}
__device__ __forceinline__ B32 load16(const void* at, int left) {
    const uint4 a = __ldg(static_cast<const uint4*>(at));
    const uint4 b = left >= 16 ? __ldg(static_cast<const uint4*>(at) + 1) : make_uint4(0u, 0u, 0u, 0u);
    return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
template <int T>
__device__ __forceinline__ B32 pack16(const float (&v)[16]) {
    B32 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.r[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    return r;
}

// Warp w: lane quadrant w % 4 of TMEM (a row per lane), half w / 4 of the columns.
template <int T, int kKind>
__device__ void role_epilogue(const Params& p, const Smem& s, uint32_t tmem, int warp, int lane, int rank) {
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    int buf = 0;
    uint32_t phase = 0;
    const int tiles = p.first[3], step = static_cast<int>(gridDim.x >> 1);
    for (int t = static_cast<int>(blockIdx.x >> 1); t < tiles; t += step) {
        const Tile ti = tile_at<kKind>(p, t);
        const int row = ti.m0 + rank * kTile + quad * 32 + lane, cols = p.cols[ti.z];
        const bool live = row < p.rows[ti.z];
        const long long at0 = static_cast<long long>(row) * cols;
        constexpr int kCols = kKind == kGate ? 64 : 128;  // of this warp
        const int n0 = ti.n0 + half * kCols;
        B32 g, u;
        if constexpr (kKind == kBackGate) {
            if (live && n0 < cols) {
                g = load16(static_cast<const uint16_t*>(p.gate) + at0 + n0, cols - n0);
                u = load16(static_cast<const uint16_t*>(p.up) + at0 + n0, cols - n0);
            }
        }
        if (!warp_all(mbar_wait_cluster(smem_u32(&s.accf[buf]), phase, s.abort_flag, p.timeout_ns, p.status, kWhereEpiAccFull))) break;
        tc_fence_after();
        const uint32_t acc = tmem + lanes + static_cast<uint32_t>(buf * 2 * kTile + half * kCols);
        float scale = 1.f;
        if constexpr (kKind == kBackGate) scale = dy_scale(p.amax);
        if constexpr (kKind == kDx || kKind == kDw) scale = ti.z < 2 ? 1.f / dy_scale(p.amax) : 1.f;
        for (int c = 0; c < kCols; c += 16) {
            const int n = n0 + c, left = cols - n;
            if (left <= 0) break;  // (the same for the whole warp)
            uint32_t x[16];
            float v[16];
            __syncwarp();
            if constexpr (kKind == kGate) {
                uint32_t y[16];
                tmem_ld16(acc + static_cast<uint32_t>(c), x);
                tmem_ld16(acc + static_cast<uint32_t>(kTile + c), y);
                tmem_ld_wait_regs(x);
                tmem_ld_wait_regs(y);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = act_value(p.activation, __uint_as_float(x[i])) * __uint_as_float(y[i]);
                if (live) {
                    store16(static_cast<uint16_t*>(p.out[0]) + at0 + n, pack16<T>(v), left, p.wide);
                    if (p.out[1] != nullptr) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[i]);
                        store16(static_cast<uint16_t*>(p.out[1]) + at0 + n, pack16<T>(v), left, p.wide);
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(y[i]);
                        store16(static_cast<uint16_t*>(p.out[2]) + at0 + n, pack16<T>(v), left, p.wide);
                    }
                }
            } else if constexpr (kKind == kBackGate) {
                tmem_ld16(acc + static_cast<uint32_t>(c), x);
                const B32 gg = g, uu = u;
                if (live && c + 16 < kCols && left > 16) {  // the next ones are on their way meanwhile
                    g = load16(static_cast<const uint16_t*>(p.gate) + at0 + n + 16, left - 16);
                    u = load16(static_cast<const uint16_t*>(p.up) + at0 + n + 16, left - 16);
                }
                tmem_ld_wait_regs(x);
                float w[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 g2 = unpack2<T>(gg.r[i]), u2 = unpack2<T>(uu.r[i]);
                    const float2 a0 = act_both(p.activation, g2.x), a1 = act_both(p.activation, g2.y);
                    const float d0 = __uint_as_float(x[2 * i]) * scale, d1 = __uint_as_float(x[2 * i + 1]) * scale;
                    v[2 * i] = d0 * u2.x * a0.y;
                    v[2 * i + 1] = d1 * u2.y * a1.y;
                    w[2 * i] = d0 * a0.x;
                    w[2 * i + 1] = d1 * a1.x;
                }
                if (live) {
                    store16(static_cast<uint16_t*>(p.out[0]) + at0 + n, pack16<T>(v), left, p.wide);
                    store16(static_cast<uint16_t*>(p.out[1]) + at0 + n, pack16<T>(w), left, p.wide);
                }
            } else {
                tmem_ld16(acc + static_cast<uint32_t>(c), x);
                tmem_ld_wait_regs(x);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(x[i]) * scale;
                if (!live) continue;
                void* out = p.out[ti.z];
                if (p.out_f32) {
                    float* y = static_cast<float*>(out) + at0 + n;
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        if (i >= left) continue;
                        float4 r = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        if (p.residual != nullptr) {
                            const float4 o = *reinterpret_cast<const float4*>(p.residual + at0 + n + i);
                            r = make_float4(r.x + o.x, r.y + o.y, r.z + o.z, r.w + o.w);
                        }
                        *reinterpret_cast<float4*>(y + i) = r;
                    }
                } else {
                    store16(static_cast<uint16_t*>(out) + at0 + n, pack16<T>(v), left, p.wide);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.acce[buf]), 0u));
        buf ^= 1;
        if (buf == 0) phase ^= 1u;
    }
}

template <int T, int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const Smem s = carve(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_ctarank());
    if (threadIdx.x == 0) {
        *s.abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1u);  // the even producer's arrive; both CTAs' bytes as transactions
            mbar_init(smem_u32(&s.empty[i]), 1u);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.accf[i]), 1u);
            mbar_init(smem_u32(&s.acce[i]), 2u * kEpiWarps);
        }
        mbar_init(smem_u32(s.drain), 1u);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(smem_u32(s.tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&maps.a[0]);
        tma_prefetch_desc(&maps.b[0]);
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM exist before any remote arrive or pair product
    tc_fence_after();
    const uint32_t tmem = *s.tmem_slot;
    if (warp < kEpiWarps) {
        role_epilogue<T, kKind>(p, s, tmem, warp, lane, rank);
    } else if (warp == kTmaWarp) {
        if (lane == 0) role_producer<kKind>(p, s, maps, rank);
        __syncwarp();
    } else if (rank == 0) {
        role_mma<T, kKind>(p, s, tmem);
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (rank != 0 && warp == kMmaWarp) {  // the drain's commit reaches this CTA's barrier too, before it may exit
        int never = 0;
        (void)mbar_wait(smem_u32(s.drain), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
        __syncwarp();
    }
    cluster_sync();  // the even CTA's products into both TMEMs are done; no remote arrives remain
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// The largest |x| of f16 values, as the bits of an f32 (an atomic maximum has no order); *amax is 0 before.
__global__ void __launch_bounds__(256) amax_kernel(const uint4* x, long long n8, unsigned* amax) {
    pdl_wait();
    unsigned top = 0u;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<long long>(gridDim.x) * 256) {
        const uint4 v = __ldg(x + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<VAE_F16>(u[k] & 0x7fff7fffu);
            top = max(top, max(__float_as_uint(f.x), __float_as_uint(f.y)));
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0 && top != 0u) atomicMax(amax, top);
    pdl_launch_dependents();
}

// ───────────────────────────── host ─────────────────────────────

// A matrix [rows][inner] as the boxes that a stage takes of it: 64 of the inner index, `box_rows` of the other.
int ffn_map(CUtensorMap* map, int type, const void* p, int rows, int inner, int box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(inner), static_cast<uint64_t>(rows)};
    const uint64_t st[1] = {static_cast<uint64_t>(inner) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
    return encode_tiled(map, type == VAE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, st,
                        box, CU_TENSOR_MAP_SWIZZLE_128B);
}

std::mutex g_mu;

template <int T, int kKind>
int ffn_setup() {
    static CtxOnce once;
    int dev = 0;
    VAE_CUDA_CHECK(cudaGetDevice(&dev));
    std::lock_guard<std::mutex> lk(g_mu);
    if (!once.done(dev)) {
        VAE_CUDA_CHECK(cudaFuncSetAttribute(ffn_kernel<T, kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
        once.mark(dev);
    }
    return VAE_OK;
}

template <int T, int kKind>
int ffn_launch(const Maps& maps, Params& p, bool ahead, cudaStream_t stream) {
    int rc = ffn_setup<T, kKind>();
    if (rc != VAE_OK) return rc;
    p.status = device_status_ptr();
    if (p.status == nullptr) return VAE_ERR_CUDA;
    p.timeout_ns = wait_timeout_ns();
    p.first[0] = 0;
    for (int z = 0; z < 3; ++z) {
        p.tiles_n[z] = 1;
        p.first[z + 1] = p.first[z];
        if (z > 0 && kKind != kDw) continue;
        const int wide = kKind == kGate ? kTile : 2 * kTile;
        p.tiles_n[z] = (p.cols[z] + wide - 1) / wide;
        p.first[z + 1] += (p.rows[z] + 2 * kTile - 1) / (2 * kTile) * p.tiles_n[z];
    }
    const int pairs = std::min(p.first[3], sm_count() / 2);
    VAE_CUDA_CHECK(launch_kernel_as(ahead || pdl_enabled(), ffn_kernel<T, kKind>, dim3(2 * pairs), dim3(kThreads), kSmem, stream, maps, p));
    return VAE_OK;
}

struct FfnTensor {
    const char* name;
    const void* p;
    size_t bytes;
    bool written;
};
int ffn_apart(const FfnTensor* t, int count) {
    for (int i = 0; i < count; ++i) {
        if (t[i].p == nullptr) continue;
        if (!aligned16(t[i].p)) return set_error(VAE_ERR_ALIGN, "gated ffn: %s must be 16-byte aligned", t[i].name);
        for (int j = 0; j < i; ++j)
            if (t[j].p != nullptr && (t[i].written || t[j].written) &&
                extents_meet(extent_dense(t[i].p, t[i].bytes), extent_dense(t[j].p, t[j].bytes)))
                return set_error(VAE_ERR_ARG, "gated ffn: %s may not overlap %s", t[i].name, t[j].name);
    }
    return VAE_OK;
}

int ffn_check(const vae_gated_ffn_desc* a, bool backward) {
    if (a == nullptr) return set_error(VAE_ERR_ARG, "gated ffn: NULL desc");
    if (a->type != VAE_F16 && a->type != VAE_BF16) return set_error(VAE_ERR_ARG, "gated ffn: f16 and bf16 tensors are taken");
    if (a->m < 1 || a->m > (1 << 24)) return set_error(VAE_ERR_SHAPE, "gated ffn: 1 to 2^24 tokens, got %d", a->m);
    if (a->c < 8 || a->c > 16384 || a->c % 8 != 0)
        return set_error(VAE_ERR_SHAPE, "gated ffn: c must be a multiple of 8 from 8 to 16384, got %d", a->c);
    if (a->f < 8 || a->f > 65536 || a->f % 8 != 0)
        return set_error(VAE_ERR_SHAPE, "gated ffn: f must be a multiple of 8 from 8 to 65536, got %d", a->f);
    if (a->activation < VAE_ACT_SILU || a->activation > VAE_ACT_GELU_TANH) return set_error(VAE_ERR_ARG, "gated ffn: unknown activation");
    const int out = backward ? a->dw_type : a->y_type;
    if (out != a->type && out != VAE_F32)
        return set_error(VAE_ERR_ARG, "gated ffn: %s of the tensors' type or f32 are taken", backward ? "weight gradients" : "outputs");
    return VAE_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
size_t mc_bytes(const vae_gated_ffn_desc& a) { return static_cast<size_t>(a.m) * a.c * 2; }
size_t mf_bytes(const vae_gated_ffn_desc& a) { return static_cast<size_t>(a.m) * a.f * 2; }
size_t cf_bytes(const vae_gated_ffn_desc& a) { return static_cast<size_t>(a.c) * a.f * 2; }

#define VAE_TRY(expr)               \
    do {                            \
        const int rc_ = (expr);     \
        if (rc_ != VAE_OK) return rc_; \
    } while (0)

template <int T>
int ffn_forward(const vae_gated_ffn_desc& a, const void* x, const void* wg, const void* wu, const void* wd, const float* residual,
                void* y, void* gate, void* up, void* hidden, cudaStream_t stream) {
    Maps maps;
    Params p{};
    VAE_TRY(ffn_map(&maps.a[0], T, x, a.m, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wg, a.f, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[1], T, wu, a.f, a.c, kTile));
    p.rows[0] = a.m;
    p.cols[0] = a.f;
    p.nk = (a.c + kBk - 1) / kBk;
    p.segments = 1;
    p.activation = a.activation;
    p.out[0] = hidden;
    p.out[1] = gate;
    p.out[2] = up;
    const auto on32 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 32 == 0; };
    p.wide = a.f % 16 == 0 && on32(hidden) && on32(gate) && on32(up);
    VAE_TRY((ffn_launch<T, kGate>(maps, p, false, stream)));
    p = Params{};
    VAE_TRY(ffn_map(&maps.a[0], T, hidden, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wd, a.c, a.f, kTile));
    p.rows[0] = a.m;
    p.cols[0] = a.c;
    p.nk = (a.f + kBk - 1) / kBk;
    p.segments = 1;
    p.out[0] = y;
    p.out_f32 = a.y_type == VAE_F32;
    p.residual = residual;
    p.wide = a.c % 16 == 0 && on32(y);
    return ffn_launch<T, kDown>(maps, p, true, stream);
}

template <int T>
int ffn_backward(const vae_gated_ffn_desc& a, const void* dy, const void* x, const void* wg, const void* wu, const void* wd,
                 const void* gate, const void* up, const void* hidden, void* dx, void* dwg, void* dwu, void* dwd, char* ws,
                 cudaStream_t stream) {
    unsigned* amax = nullptr;
    void *dgate = ws + 256, *dup = ws + 256 + up256(mf_bytes(a));
    bool ahead = false;
    if (T == VAE_F16) {
        amax = reinterpret_cast<unsigned*>(ws);
        VAE_CUDA_CHECK(cudaMemsetAsync(amax, 0, sizeof(unsigned), stream));
        const long long n8 = static_cast<long long>(a.m) * a.c / 8;
        const unsigned grid = static_cast<unsigned>(std::min<long long>((n8 + 255) / 256, 152 * 8));
        VAE_CUDA_CHECK(launch_kernel(amax_kernel, dim3(grid), dim3(256), 0, stream, static_cast<const uint4*>(dy), n8, amax));
        ahead = true;
    }
    const auto on32 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 32 == 0; };
    Maps maps;
    Params p{};
    VAE_TRY(ffn_map(&maps.a[0], T, dy, a.m, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wd, a.c, a.f, kBk));
    p.rows[0] = a.m;
    p.cols[0] = a.f;
    p.nk = (a.c + kBk - 1) / kBk;
    p.segments = 1;
    p.activation = a.activation;
    p.gate = gate;
    p.up = up;
    p.out[0] = dgate;
    p.out[1] = dup;
    p.amax = amax;
    p.wide = a.f % 16 == 0;
    VAE_TRY((ffn_launch<T, kBackGate>(maps, p, ahead, stream)));
    p = Params{};
    VAE_TRY(ffn_map(&maps.a[0], T, dgate, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.a[1], T, dup, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wg, a.f, a.c, kBk));
    VAE_TRY(ffn_map(&maps.b[1], T, wu, a.f, a.c, kBk));
    p.rows[0] = a.m;
    p.cols[0] = a.c;
    p.nk = (a.f + kBk - 1) / kBk;
    p.segments = 2;
    p.out[0] = dx;
    p.amax = amax;
    p.wide = a.c % 16 == 0 && on32(dx);
    VAE_TRY((ffn_launch<T, kDx>(maps, p, true, stream)));
    if (dwg == nullptr) return VAE_OK;
    p = Params{};
    VAE_TRY(ffn_map(&maps.a[0], T, dgate, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.a[1], T, dup, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.a[2], T, dy, a.m, a.c, kBk));
    VAE_TRY(ffn_map(&maps.b[0], T, x, a.m, a.c, kBk));
    maps.b[1] = maps.b[0];
    VAE_TRY(ffn_map(&maps.b[2], T, hidden, a.m, a.f, kBk));
    p.rows[0] = p.rows[1] = p.cols[2] = a.f;
    p.cols[0] = p.cols[1] = p.rows[2] = a.c;
    p.nk = (a.m + kBk - 1) / kBk;
    p.segments = 1;
    p.out[0] = dwg;
    p.out[1] = dwu;
    p.out[2] = dwd;
    p.out_f32 = a.dw_type == VAE_F32;
    p.amax = amax;
    p.wide = a.c % 16 == 0 && a.f % 16 == 0 && on32(dwg) && on32(dwu) && on32(dwd);
    return ffn_launch<T, kDw>(maps, p, true, stream);
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" {

size_t vae_gated_ffn_workspace_bytes(const vae_gated_ffn_desc* desc) {
    clear_error();
    if (ffn_check(desc, false) != VAE_OK) return 0;
    return desc->save ? 0 : up256(mf_bytes(*desc));  // hidden, where it is not saved
}

int vae_gated_ffn(const vae_gated_ffn_desc* desc, const void* x_dev, const void* w_gate_dev, const void* w_up_dev,
                  const void* w_down_dev, const float* residual_dev, void* y_dev, void* gate_dev, void* up_dev,
                  void* hidden_dev, void* workspace_dev, size_t workspace_bytes, vae_stream_t stream) {
    clear_error();
    VAE_TRY(ffn_check(desc, false));
    const vae_gated_ffn_desc& a = *desc;
    if (x_dev == nullptr || w_gate_dev == nullptr || w_up_dev == nullptr || w_down_dev == nullptr || y_dev == nullptr)
        return set_error(VAE_ERR_ARG, "gated ffn: NULL tensor");
    const bool save = a.save != 0;
    if ((gate_dev != nullptr) != save || (up_dev != nullptr) != save || (hidden_dev != nullptr) != save)
        return set_error(VAE_ERR_ARG, "gated ffn: gate, up and hidden are given where they are saved, and only there");
    if (residual_dev != nullptr && a.y_type != VAE_F32) return set_error(VAE_ERR_ARG, "gated ffn: a residual needs an f32 output");
    const size_t need = vae_gated_ffn_workspace_bytes(desc), yb = mc_bytes(a) * (a.y_type == VAE_F32 ? 2 : 1);
    if (need != 0 && workspace_dev == nullptr) return set_error(VAE_ERR_ARG, "gated ffn: NULL workspace");
    if (workspace_bytes < need)
        return set_error(VAE_ERR_NOMEM, "gated ffn: workspace of %zu bytes, %zu are needed", workspace_bytes, need);
    const FfnTensor t[] = {{"x", x_dev, mc_bytes(a), false},
                           {"w_gate", w_gate_dev, cf_bytes(a), false},
                           {"w_up", w_up_dev, cf_bytes(a), false},
                           {"w_down", w_down_dev, cf_bytes(a), false},
                           {"y", y_dev, yb, true},
                           {"gate", gate_dev, mf_bytes(a), true},
                           {"up", up_dev, mf_bytes(a), true},
                           {"hidden", hidden_dev, mf_bytes(a), true},
                           {"the workspace", need != 0 ? workspace_dev : nullptr, need, true},
                           {"the residual", y_dev == residual_dev ? nullptr : residual_dev, yb, false}};
    VAE_TRY(ffn_apart(t, 10));
    VAE_TRY(check_device());
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    void* hidden = save ? hidden_dev : workspace_dev;
    return a.type == VAE_F16
               ? ffn_forward<VAE_F16>(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, st)
               : ffn_forward<VAE_BF16>(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, st);
}

size_t vae_gated_ffn_backward_workspace_bytes(const vae_gated_ffn_desc* desc) {
    clear_error();
    if (ffn_check(desc, true) != VAE_OK) return 0;
    return 256 + 2 * up256(mf_bytes(*desc));  // the largest |dy|, dgate, dup
}

int vae_gated_ffn_backward(const vae_gated_ffn_desc* desc, const void* dy_dev, const void* x_dev, const void* w_gate_dev,
                           const void* w_up_dev, const void* w_down_dev, const void* gate_dev, const void* up_dev,
                           const void* hidden_dev, void* dx_dev, void* dw_gate_dev, void* dw_up_dev, void* dw_down_dev,
                           void* workspace_dev, size_t workspace_bytes, vae_stream_t stream) {
    clear_error();
    VAE_TRY(ffn_check(desc, true));
    const vae_gated_ffn_desc& a = *desc;
    if (dy_dev == nullptr || x_dev == nullptr || w_gate_dev == nullptr || w_up_dev == nullptr || w_down_dev == nullptr ||
        gate_dev == nullptr || up_dev == nullptr || hidden_dev == nullptr || dx_dev == nullptr || workspace_dev == nullptr)
        return set_error(VAE_ERR_ARG, "gated ffn: NULL tensor or workspace");
    if ((dw_gate_dev == nullptr) != (dw_down_dev == nullptr) || (dw_up_dev == nullptr) != (dw_down_dev == nullptr))
        return set_error(VAE_ERR_ARG, "gated ffn: the weights' gradients come together");
    const size_t need = vae_gated_ffn_backward_workspace_bytes(desc), wb = cf_bytes(a) * (a.dw_type == VAE_F32 ? 2 : 1);
    if (workspace_bytes < need)
        return set_error(VAE_ERR_NOMEM, "gated ffn: workspace of %zu bytes, %zu are needed", workspace_bytes, need);
    const FfnTensor t[] = {{"dy", dy_dev, mc_bytes(a), false},         {"x", x_dev, mc_bytes(a), false},
                           {"w_gate", w_gate_dev, cf_bytes(a), false}, {"w_up", w_up_dev, cf_bytes(a), false},
                           {"w_down", w_down_dev, cf_bytes(a), false}, {"gate", gate_dev, mf_bytes(a), false},
                           {"up", up_dev, mf_bytes(a), false},         {"hidden", hidden_dev, mf_bytes(a), false},
                           {"dx", dx_dev, mc_bytes(a), true},          {"dw_gate", dw_gate_dev, wb, true},
                           {"dw_up", dw_up_dev, wb, true},             {"dw_down", dw_down_dev, wb, true},
                           {"the workspace", workspace_dev, need, true}};
    VAE_TRY(ffn_apart(t, 13));
    VAE_TRY(check_device());
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace_dev);
    return a.type == VAE_F16 ? ffn_backward<VAE_F16>(a, dy_dev, x_dev, w_gate_dev, w_up_dev, w_down_dev, gate_dev, up_dev,
                                                     hidden_dev, dx_dev, dw_gate_dev, dw_up_dev, dw_down_dev, ws, st)
                             : ffn_backward<VAE_BF16>(a, dy_dev, x_dev, w_gate_dev, w_up_dev, w_down_dev, gate_dev, up_dev,
                                                      hidden_dev, dx_dev, dw_gate_dev, dw_up_dev, dw_down_dev, ws, st);
}

}  // extern "C"
