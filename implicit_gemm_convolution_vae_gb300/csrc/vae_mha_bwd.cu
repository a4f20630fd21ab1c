// Gradient of multi-head attention (the C entry point is in vae_mha.cu).
//
//   P = 2^(S scale log2(e) - lse log2(e)),  dV = P^T dO,  dP = dO V^T,
//   D = rowsum(dO * O),  dS = P * (dP - D),  dQ = scale dS K,  dK = scale dS^T Q.
//
// Five products over every pair of tiles would do if one kernel could keep dQ,
// dK and dV at once; dQ's sum runs over the key tiles that other CTAs hold, so
// that form adds dQ with atomics, whose order changes the result. Here two
// kernels run over the pairs, one per key tile (S^T, dP^T, dV, dK: four
// products) and one per query tile (S, dP, dQ: three): seven products, P twice,
// no atomics on results and nothing of the pairs' size in memory.
//
// Key-tile kernel: lanes of TMEM are keys, columns are query rows. S^T = K Q^T
// and dP^T = V dO^T come from shared memory, eight softmax warps turn them into
// P^T and dS^T over the same TMEM columns, and these are the left operands of
// dV += P^T dO and dK += dS^T Q, for which the Q and dO tiles that TMA brought
// are read again with the rows as the contraction index. While the warps form
// dS^T, the tensor cores run dV and the next S^T; while they form the next
// P^T, dK and the next dP^T.
// Query-tile kernel: the same with lanes as query rows; P stays in registers,
// and the Q and dO rows lie in TMEM as the left operands of S and dP: M = N = 128
// MMAs with both operands in shared memory ran at 90 cycles each, bound by the
// 8 KB that each reads there, those with one in TMEM at 57 to 64.
//
// Both kernels read 64 KB of tiles per step of 128 channels, and L2 gives every SM
// 26 to 29 bytes a cycle (measured): the loads alone take 2280 to 2510 cycles.
//
// D = rowsum(dO * O) takes O as the forward rounded it. Rows that meet few keys
// (kExactTiles tiles at most) feel that rounding in dS: the query-tile kernel
// first runs over their keys once for D = rowsum(P * dP) itself, and hands it
// to the key-tile kernel after it. Over more keys the rounded O costs dq 1.44 to
// 1.46 times its own rounding at 96 and 128 channels instead of the 1.41 that one
// rounding of dS costs, up to 1.55 at 40 and 2.0 at 8; the pass over all keys would
// take two products more of seven.
//
// Measured on GB300: 16384 tokens x 9 heads x 128 in f16 2800 to 2980 us (1040 to
// 1100 TFLOP/s of the five products' flops). A step takes 2520 cycles in the
// query-tile kernel, as long as its loads (1536 at the tensor rate), and 3480 in
// the key-tile kernel (2600 with no hand-over between warps, 2048 at the tensor rate).
//
// 16 bits. P and dS are rounded to the tensors' type for the products, half a
// step of 2^-8 or 2^-11 relative, as the forward's P. f16 would lose long rows'
// P ~ 1/n below 2^-14, so it holds P 2^14 and dS c, with c the power of two
// that brings 2 max|dO| max|V| (a bound on |dP - D| by Cauchy-Schwarz, from a
// first kernel) to 2^14 .. 2^15; both factors leave in the epilogue. Every
// batch entry and key head has a c of its own: no gradient's digits hang on how
// large another's are. The maximum is taken by an atomic maximum, which has no order. Up to 64 rows of a
// head lie twice in their tile: the second copies' P and dS are what the first's
// rounding left of them.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "vae_mha_bwd.h"

namespace vae {

namespace {

constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 2) * 32;
constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr uint32_t kTmemCols = 512;
constexpr int kTargetCtas = 152;   // one CTA per SM
constexpr int kPLog2 = 14;         // f16: P is held as P 2^14
constexpr int kSideFloats = 256;   // of a row tile: 128 x (kPLog2 - lse log2(e)), 128 x D
constexpr int kSideBytes = kSideFloats * 4;

constexpr int kExactTiles = 2;     // key tiles up to which D is formed from P and dP

// Shared memory of a kernel: kRes resident tiles, a ring of kN stages of two
// tiles, kSideN side rows; the barriers behind them.
template <int kSteps, int kRes, int kN, int kSideN>
struct BwdCfg {
    static constexpr int kCh = kSteps > 4 ? 2 : 1;  // 64-channel chunks of the kSteps x 16 channels
    static constexpr int kTileBytes = kCh * kMhaChunkBytes;
    static constexpr int kStages = kN;
    static constexpr int kRing = kRes * kTileBytes;
    static constexpr int kSide = kRing + kStages * 2 * kTileBytes;
    static constexpr int kBars = kSide + kSideN * kSideBytes;
    static constexpr int kSmem = kBars + 512;
    static_assert(kSmem <= 232448, "attention shared memory over 227 KB");
};
template <int kSteps>
using KvCfg = BwdCfg<kSteps, 2, (kSteps > 4 ? 2 : 5), (kSteps > 4 ? 2 : 5)>;
template <int kSteps>
using QCfg = BwdCfg<kSteps, 0, (kSteps > 4 ? 3 : 6), 1>;  // (the side row: 256 floats for the rows' sums)

struct BwdParams {
    MhaShape s;
    float scale, scale_log2;
    int nsplit_q, nsplit_k;
    int twice;                  // at most 64 rows to a head: each lies twice in its tile, P and dS in two parts
    float* side;                // [b][hkv][nsub][ntile][256]
    const unsigned* maxima;     // f16: [b][hkv] x bits of max |dO|^2, max |V|^2
    const void *q, *dout;
    MhaStrides qs, gs;
    void *dq, *dk, *dv;
    MhaStrides dqs, dks, dvs;
    float *part_q, *part_kv;    // [nsplit_q][b][hq][sq][d], [nsplit_k][2][b][hkv][sk][d]
    DevStatus* status;
    unsigned long long timeout_ns;
};

// Where the maxima of entry e and key head hk lie.
__host__ __device__ __forceinline__ size_t maxima_at(const MhaShape& s, int e, int hk) {
    return 2 * (static_cast<size_t>(e) * s.hkv + hk);
}
// c of the file comment, from an entry's and key head's maxima.
template <int T>
__device__ __forceinline__ float ds_factor(const unsigned* maxima) {
    if constexpr (T == VAE_BF16) {
        return 1.f;
    } else {
        const float bound = 2.f * sqrtf(__uint_as_float(maxima[0])) * sqrtf(__uint_as_float(maxima[1]));
        if (!(bound > 0.f) || bound > 1e30f) return 1.f;
        const int k = 14 - ilogbf(bound);
        return scalbnf(1.f, k < -100 ? -100 : (k > 100 ? 100 : k));
    }
}

// ───────────────────────────── rows beforehand ─────────────────────────────

struct PrepParams {
    MhaShape s;
    const void *dout, *o, *v;
    MhaStrides gs, os, vs;
    const float* lse;
    float* side;
    unsigned* maxima;
    int row_tiles;  // of all heads; the key tiles' blocks (f16) follow
};

// A block per row tile: 16 lanes a row. Then (f16) a block per key tile for max |V|.
template <int T>
__global__ void __launch_bounds__(256) mha_prep_kernel(const PrepParams p) {
    pdl_wait();
    const MhaShape& s = p.s;
    const int part = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    float big = 0.f;
    unsigned* maximum;
    if (static_cast<int>(blockIdx.x) < p.row_tiles) {
        int x = blockIdx.x;
        const int tile = x % s.ntile;
        x /= s.ntile;
        const int sub = x % s.nsub;
        x /= s.nsub;
        const int hk = x % s.hkv, e = x / s.hkv;
        maximum = p.maxima + maxima_at(s, e, hk);
        const int ql = mha_len(s.q_len, e, s.sq);
        const int gp = 1 << s.gp_log2;
        float* side = p.side + static_cast<long long>(blockIdx.x) * kSideFloats;
#pragma unroll 2
        for (int k = 0; k < kMhaTile / 16; ++k) {
            const int rr = r0 + k * 16, r = tile * kMhaTile + rr;
            const int i = r >> s.gp_log2, h = hk * s.g + sub * gp + (r & (gp - 1));
            const bool live = i < ql;
            float d = 0.f, n = 0.f;
            if (live && part * 8 < s.d) {
                float a[8], b[8];
                load8<T>(static_cast<const typename Elem<T>::type*>(p.dout) + e * p.gs.b + i * p.gs.s + h * p.gs.h + part * 8, a);
                load8<T>(static_cast<const typename Elem<T>::type*>(p.o) + e * p.os.b + i * p.os.s + h * p.os.h + part * 8, b);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    d += a[u] * b[u];
                    n += a[u] * a[u];
                }
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) {
                d += __shfl_xor_sync(0xffffffffu, d, w);
                n += __shfl_xor_sync(0xffffffffu, n, w);
            }
            big = fmaxf(big, n);
            if (part == 0) {
                const float l = live ? p.lse[(static_cast<long long>(e) * s.hq + h) * s.sq + i] : -INFINITY;
                side[rr] = l == -INFINITY ? -INFINITY : (T == VAE_F16 ? kPLog2 : 0) - l * 1.4426950408889634074f;
                side[128 + rr] = live ? d : 0.f;
            }
        }
    } else {
        int x = blockIdx.x - p.row_tiles;
        const int kb = x % s.nkb;
        x /= s.nkb;
        const int hk = x % s.hkv, e = x / s.hkv;
        const int kl = mha_len(s.k_len, e, s.sk);
        maximum = p.maxima + maxima_at(s, e, hk) + 1;
#pragma unroll 4
        for (int k = 0; k < kMhaTile / 16; ++k) {
            const int j = kb * kMhaTile + r0 + k * 16;
            float n = 0.f;
            if (j < kl && part * 8 < s.d) {
                float a[8];
                load8<T>(static_cast<const typename Elem<T>::type*>(p.v) + e * p.vs.b + j * p.vs.s + hk * p.vs.h + part * 8, a);
#pragma unroll
                for (int u = 0; u < 8; ++u) n += a[u] * a[u];
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) n += __shfl_xor_sync(0xffffffffu, n, w);
            big = fmaxf(big, n);
        }
    }
    if constexpr (T == VAE_F16) {
        // (values >= 0: their bits order as unsigned numbers do)
        const unsigned b = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        if ((threadIdx.x & 31) == 0 && b != 0u) atomicMax(maximum, b);
    }
}

// ───────────────────────────── shared structure ─────────────────────────────

struct BwdSmem {
    uint8_t *res, *ring, *side;
    uint64_t *a_full, *b_full, *empty;  // [kStages]: first tile (+ side), second tile, both free
    uint64_t* fix;                      // [kStages]: both tiles, before their rows behind the length are zeroed
    uint64_t *res_full, *s_full, *x_full, *p_full, *ds_full, *done, *drain;
    uint64_t* x_bar;  // [4 quadrants]
    uint32_t* tmem_slot;
    int* abort_flag;
};

template <typename C>
__device__ __forceinline__ BwdSmem bwd_carve(uint8_t* base) {
    BwdSmem s;
    s.res = base;
    s.ring = base + C::kRing;
    s.side = base + C::kSide;
    uint64_t* b = reinterpret_cast<uint64_t*>(base + C::kBars);
    s.a_full = b;
    s.b_full = b + C::kStages;
    s.empty = b + 2 * C::kStages;
    s.fix = b + 3 * C::kStages;
    b += 4 * C::kStages;
    s.res_full = b;
    s.s_full = b + 1;
    s.x_full = b + 2;  // dP has been formed
    s.p_full = b + 3;  // key-tile kernel: P^T is in TMEM; query-tile kernel: S has been read
    s.ds_full = b + 4;
    s.done = b + 5;
    s.drain = b + 6;
    s.x_bar = b + 7;
    s.tmem_slot = reinterpret_cast<uint32_t*>(b + 11);
    s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
    return s;
}

__device__ __forceinline__ bool bwait(uint64_t* bar, uint32_t parity, const BwdSmem& s, const BwdParams& p) {
    return mbar_wait(smem_u32(bar), parity, s.abort_flag, p.timeout_ns, p.status, kWhereAttn);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// A 128-row tile as two boxes of 64 rows per chunk, into this CTA; `half` is the
// second box's distance in tokens.
template <int kChunks>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int head, int token, int half,
                                          int e, uint64_t pol) {
    for (int c = 0; c < kChunks; ++c)
        for (int r = 0; r < 2; ++r)
            tma_load_4d(smem_u32(dst + c * kMhaChunkBytes + r * (kMhaChunkBytes / 2)), map, bar, c * 64, head,
                        token + r * half, e, pol);
}
// Set-up and tear-down common to both kernels.
template <typename C>
__device__ __forceinline__ void bwd_begin(const BwdSmem& s, int warp, uint32_t res_arrivals) {
    if (threadIdx.x == 0) {
        *s.abort_flag = 0;
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&s.a_full[i]), 1u);
            mbar_init(smem_u32(&s.b_full[i]), 1u);
            mbar_init(smem_u32(&s.empty[i]), 1u);
            mbar_init(smem_u32(&s.fix[i]), 1u);
        }
        mbar_init(smem_u32(s.res_full), res_arrivals);
        mbar_init(smem_u32(s.s_full), 1u);
        mbar_init(smem_u32(s.x_full), 1u);
        mbar_init(smem_u32(s.p_full), kSoftWarps);
        mbar_init(smem_u32(s.ds_full), kSoftWarps);
        mbar_init(smem_u32(s.done), 1u);
        mbar_init(smem_u32(s.drain), 1u);
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.x_bar[i]), 2u);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(s.tmem_slot), kTmemCols);  // all 512 columns are this CTA's: they start at 0
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}
__device__ __forceinline__ void bwd_end(int warp) {
    pdl_launch_dependents();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(0u, kTmemCols);
    }
}

// The ring's producer state: what is in flight when a wait runs out has to
// land before the CTA may exit. A stage that has to be fixed completes on a
// barrier of its own and then on the stage's by hand.
template <int kN>
struct BwdRing {
    int stage = 0;
    uint32_t phase = 0, armed = 0, arm_par = 0, fixing = 0, fix_par = 0;
    __device__ __forceinline__ void arm() {
        armed |= 1u << stage;
        arm_par = (arm_par & ~(1u << stage)) | (phase << stage);
    }
    __device__ __forceinline__ void next() {
        if (++stage == kN) {
            stage = 0;
            phase ^= 1u;
        }
    }
    // Waits for the stage's copies (the whole warp), zeroes the rows behind the first `from` of both tiles (of each
    // half: twice) and hands it over.
    template <typename C>
    __device__ __forceinline__ bool fix(const BwdSmem& s, const BwdParams& p, int from, bool twice, int lane) {
        armed &= ~(1u << stage);
        fixing = 1u << stage;
        const uint32_t par = (fix_par >> stage) & 1u;
        __syncwarp();
        if (!warp_all(bwait(&s.fix[stage], par, s, p))) return false;
        fixing = 0u;
        fix_par ^= 1u << stage;
        uint8_t* dst = s.ring + stage * 2 * C::kTileBytes;
        for (int k = 0; k < 2; ++k, dst += C::kTileBytes) {
            mha_zero_rows(dst, from, twice ? kMhaTile / 2 : kMhaTile, C::kCh, lane);
            if (twice) mha_zero_rows(dst, kMhaTile / 2 + from, kMhaTile, C::kCh, lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&s.a_full[stage]));
            mbar_arrive(smem_u32(&s.b_full[stage]));
        }
        return true;
    }
    __device__ __forceinline__ void drain(const BwdSmem& s, const BwdParams& p, bool resident) const {
        int never = 0;
        const auto wait = [&](uint64_t* bar, uint32_t par) {
            (void)mbar_wait(smem_u32(bar), par, &never, p.timeout_ns, p.status, kWhereDrain);
        };
        if (resident) wait(s.res_full, 0u);
        for (int i = 0; i < kN; ++i) {
            if (fixing >> i & 1u) wait(&s.fix[i], (fix_par >> i) & 1u);
            if (armed >> i & 1u) {
                wait(&s.a_full[i], (arm_par >> i) & 1u);
                wait(&s.b_full[i], (arm_par >> i) & 1u);
            }
        }
    }
};

// (No CTA leaves while its MMAs still run.)
__device__ __forceinline__ void mma_finish(const BwdSmem& s, const BwdParams& p, bool ok) {
    if (elect_one()) {
        if (ok) umma_commit(smem_u32(s.done));
        umma_commit(smem_u32(s.drain));
        int never = 0;
        (void)mbar_wait(smem_u32(s.drain), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
    }
    __syncwarp();
}

// 64 columns of this warp's lanes.
__device__ __forceinline__ void load64(uint32_t t, uint32_t (&x)[4][16]) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld16(t + static_cast<uint32_t>(c * 16), x[c]);
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld_wait_regs(x[c]);
}

// A row of an accumulator (and of its second part, in shared memory), times `f`,
// to the 16-bit tensor or an f32 partial.
template <int T>
__device__ __forceinline__ void store_acc(uint32_t t, int d, bool live, bool any, float f, void* out, long long off, float* part,
                                          long long poff, const float* more = nullptr) {
    for (int c = 0; c < d; c += 16) {
        uint32_t r[16];
        if (any) {
            __syncwarp();
            tmem_ld16(t + static_cast<uint32_t>(c), r);
            tmem_ld_wait_regs(r);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) r[k] = 0u;  // no pair was met
        }
        if (!live) continue;
#pragma unroll
        for (int u = 0; u < 16; u += 8) {
            if (c + u >= d) continue;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = (more != nullptr ? __uint_as_float(r[u + k]) + more[(c + u + k) * 64] : __uint_as_float(r[u + k])) * f;
            if (part != nullptr) store8<VAE_F32>(part + poff + c + u, v);
            else store8<T>(static_cast<typename Elem<T>::type*>(out) + off + c + u, v);
        }
    }
}

// ───────────────────────────── dK and dV, per key tile ─────────────────────────────

struct KvWork {
    int e, hk, kb, split;
    int ql, kl;
    int t0, nt;      // row tiles [t0, nt) of each part of the group see the key tile
    int first, n;    // this split's share of the nsub * (nt - t0) tiles
};

__device__ __forceinline__ KvWork kv_work(const BwdParams& p) {
    const MhaShape& s = p.s;
    KvWork w;
    int r = blockIdx.x;
    w.kb = r % s.nkb;
    r /= s.nkb;
    w.split = r % p.nsplit_k;
    r /= p.nsplit_k;
    w.hk = r % s.hkv;
    w.e = r / s.hkv;
    w.ql = mha_len(s.q_len, w.e, s.sq);
    w.kl = mha_len(s.k_len, w.e, s.sk);
    const long long rows = static_cast<long long>(w.ql) << s.gp_log2;
    w.nt = static_cast<int>((rows + kMhaTile - 1) / kMhaTile);
    long long i0 = 0;  // the first query that sees a key of the tile
    if (s.block > 0) {
        i0 = static_cast<long long>(w.kb * kMhaTile / s.block * s.block) - (w.kl - w.ql);
        if (i0 < 0) i0 = 0;
    }
    const long long t0 = (i0 << s.gp_log2) / kMhaTile;
    w.t0 = t0 < w.nt ? static_cast<int>(t0) : w.nt;
    const int all = w.kb * kMhaTile < w.kl ? s.nsub * (w.nt - w.t0) : 0;
    const int per = (all + p.nsplit_k - 1) / p.nsplit_k;
    w.first = w.split * per < all ? w.split * per : all;
    w.n = (w.first + per < all ? w.first + per : all) - w.first;
    return w;
}

template <typename C>
__device__ void kv_producer(const BwdParams& p, const BwdSmem& s, const KvWork& w, const CUtensorMap* mq,
                            const CUtensorMap* mg, const CUtensorMap* mk, const CUtensorMap* mv, int lane) {
    const uint64_t pol = policy_evict_normal();
    const MhaShape& sh = p.s;
    const int gp = 1 << sh.gp_log2, half = p.twice ? 0 : 64 >> sh.gp_log2;
    if (lane == 0) {
        const uint32_t rb = smem_u32(s.res_full);
        mbar_arrive_expect_tx(rb, 2u * C::kTileBytes);
        load_tile<C::kCh>(s.res, mk, rb, w.hk, w.kb * kMhaTile, 64, w.e, pol);
        load_tile<C::kCh>(s.res + C::kTileBytes, mv, rb, w.hk, w.kb * kMhaTile, 64, w.e, pol);
    }
    BwdRing<C::kStages> r;
    const int per = w.nt - w.t0;
    for (int x = 0; x < w.n; ++x) {
        const int sub = (w.first + x) / per, tile = w.t0 + (w.first + x) % per;
        const int head = w.hk * sh.g + sub * gp, token = (tile * kMhaTile) >> sh.gp_log2;
        if (!warp_all(bwait(&s.empty[r.stage], r.phase ^ 1u, s, p))) break;
        uint8_t* dst = s.ring + r.stage * 2 * C::kTileBytes;
        uint8_t* sd = s.side + r.stage * kSideBytes;
        const float* src = p.side + (((static_cast<long long>(w.e) * sh.hkv + w.hk) * sh.nsub + sub) * sh.ntile + tile) * kSideFloats;
        // rows behind the length, inside the tensor, may hold anything: zeroed before the MMAs may read
        const long long valid = (static_cast<long long>(w.ql) << sh.gp_log2) - static_cast<long long>(tile) * kMhaTile;
        const bool fix = valid < kMhaTile && w.ql < sh.sq;
        const uint32_t ab = smem_u32(fix ? &s.fix[r.stage] : &s.a_full[r.stage]), bb = smem_u32(fix ? &s.fix[r.stage] : &s.b_full[r.stage]);
        if (lane == 0) {
            if (fix) {
                mbar_arrive_expect_tx(ab, 2u * C::kTileBytes + kSideBytes);
            } else {
                mbar_arrive_expect_tx(ab, C::kTileBytes + kSideBytes);
                mbar_arrive_expect_tx(bb, C::kTileBytes);
            }
            load_tile<C::kCh>(dst, mq, ab, head, token, half, w.e, pol);
            bulk_load(smem_u32(sd), src, kSideBytes, ab);
            load_tile<C::kCh>(dst + C::kTileBytes, mg, bb, head, token, half, w.e, pol);
        }
        if (fix) {
            if (!r.template fix<C>(s, p, static_cast<int>(valid), p.twice != 0, lane)) break;
        } else {
            r.arm();
        }
        r.next();
    }
    if (lane == 0) r.drain(s, p, true);
    __syncwarp();
}

template <int T, int kSteps>
__device__ void kv_mma(const BwdParams& p, const BwdSmem& s, const KvWork& w) {
    using C = KvCfg<kSteps>;
    constexpr uint32_t id_s = mha_idesc(T, 128, 128, false), id_o = mha_idesc(T, 128, kSteps * 16, true);
    constexpr uint32_t tS = 0u, tX = 128u, tV = 256u, tK = 384u;
    constexpr uint32_t stage_units = 2u * C::kTileBytes >> 4, second = C::kTileBytes >> 4;
    const uint64_t kdesc = sw128_kmajor_desc(smem_u32(s.res)), vdesc = kdesc + second;
    const uint64_t ring_k = sw128_kmajor_desc(smem_u32(s.ring)), ring_m = sw128_mnmajor_desc(smem_u32(s.ring));
    auto wait = [&](uint64_t* bar, uint32_t par) { return warp_all(bwait(bar, par, s, p)); };
    auto score = [&](uint32_t st) {
        mma_ss<kSteps>(tS, kdesc, ring_k + st * stage_units, id_s);
        umma_commit(smem_u32(s.s_full));
    };
    auto cross = [&](uint32_t st) {
        mma_ss<kSteps>(tX, vdesc, ring_k + st * stage_units + second, id_s);
        umma_commit(smem_u32(s.x_full));
    };
    uint32_t st = 0, ph = 0;
    bool ok = wait(s.res_full, 0u) && wait(&s.a_full[0], 0u) && wait(&s.b_full[0], 0u);
    if (ok) {
        tc_fence_after();
        if (elect_one()) {
            score(0);
            cross(0);
        }
        __syncwarp();
    }
    for (int x = 0; ok && x < w.n; ++x) {
        const uint32_t par = static_cast<uint32_t>(x) & 1u;
        const bool more = x + 1 < w.n;
        const bool wrap = st + 1 == C::kStages;
        const uint32_t st1 = wrap ? 0u : st + 1u, ph1 = wrap ? ph ^ 1u : ph;
        ok = wait(s.p_full, par);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) mma_ts<64>(tV, tS, ring_m + st * stage_units + second, id_o, x != 0 ? 1u : 0u);
        __syncwarp();
        if (more) {
            ok = wait(&s.a_full[st1], ph1);
            if (!ok) break;
            if (elect_one()) score(st1);
            __syncwarp();
        }
        ok = wait(s.ds_full, par);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            mma_ts<64>(tK, tX, ring_m + st * stage_units, id_o, x != 0 ? 1u : 0u);
            umma_commit(smem_u32(&s.empty[st]));
        }
        __syncwarp();
        if (more) {
            ok = wait(&s.b_full[st1], ph1);
            if (!ok) break;
            if (elect_one()) cross(st1);
            __syncwarp();
        }
        st = st1;
        ph = ph1;
    }
    mma_finish(s, p, ok);
}

// 64 values as 16-bit pairs in 32 columns, or what that rounding leaves of them.
template <int T>
__device__ __forceinline__ void store64(uint32_t t, const float (&v)[64], bool rest) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t h2[16];
        if (rest) {
#pragma unroll
            for (int u = 0; u < 16; ++u) h2[u] = pack2_rest<T>(v[k * 32 + 2 * u], v[k * 32 + 2 * u + 1]);
        } else {
#pragma unroll
            for (int u = 0; u < 16; ++u) h2[u] = pack2<T>(v[k * 32 + 2 * u], v[k * 32 + 2 * u + 1]);
        }
        tmem_st16(t + static_cast<uint32_t>(k * 16), h2);
    }
}

template <int T, int kSteps, bool kTwice>
__device__ void kv_softmax(const BwdParams& p, const BwdSmem& s, const KvWork& w, int warp, int lane) {
    using C = KvCfg<kSteps>;
    const int quad = warp & 3, half = warp >> 2;
    const MhaShape& sh = p.s;
    const int j = w.kb * kMhaTile + quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = lane_off + static_cast<uint32_t>(half * 64), tX = tS + 128u;
    const float c = ds_factor<T>(p.maxima + maxima_at(sh, w.e, w.hk));
    const float f = T == VAE_F16 ? c * (1.f / (1 << kPLog2)) : 1.f;  // dS c = (P 2^14) (dP - D) f
    // the first row of the group's packing that sees key j
    long long see = 0;
    if (sh.block > 0) see = (static_cast<long long>(j / sh.block * sh.block) - (w.kl - w.ql)) * (1 << sh.gp_log2);
    const int per = w.nt - w.t0;
    const bool rest = kTwice && half == 1;  // these columns hold the other half's rows again
    const int col0 = rest ? 0 : half * 64;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    bool ok = true;
    int st = 0;
    uint32_t ph = 0;
    for (int x = 0; x < w.n; ++x) {
        const uint32_t par = static_cast<uint32_t>(x) & 1u;
        const int tile = w.t0 + (w.first + x) % per;
        ok = warp_all(bwait(&s.a_full[st], ph, s, p));  // the side rows
        if (!ok) break;
        const float* side = reinterpret_cast<const float*>(s.side + st * kSideBytes) + col0;
        ok = warp_all(bwait(s.s_full, par, s, p));
        if (!ok) break;
        tc_fence_after();
        uint32_t xr[4][16];
        float pr[64];
        load64(tS, xr);
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
            const float4 nl = *reinterpret_cast<const float4*>(side + k);
            const uint32_t* y = xr[k >> 4] + (k & 15);
            const float2 a = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, make_float2(nl.x, nl.y));
            const float2 b = fma2(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), sc2, make_float2(nl.z, nl.w));
            pr[k] = mha_ex2(a.x);
            pr[k + 1] = mha_ex2(a.y);
            pr[k + 2] = mha_ex2(b.x);
            pr[k + 3] = mha_ex2(b.y);
        }
        const long long before = see - static_cast<long long>(tile) * kMhaTile - col0;
        const int hide = before > 64 ? 64 : (before < 0 ? 0 : static_cast<int>(before));  // columns that do not see the key
        if (__any_sync(0xffffffffu, hide > 0)) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
                if (k < hide) pr[k] = 0.f;
        }
        store64<T>(tS, pr, rest);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s.p_full));
        ok = warp_all(bwait(s.x_full, par, s, p));
        if (!ok) break;
        tc_fence_after();
        load64(tX, xr);
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
            const float4 D = *reinterpret_cast<const float4*>(side + 128 + k);
            uint32_t* y = xr[k >> 4] + (k & 15);
            float2 a = add2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), make_float2(-D.x, -D.y));
            float2 b = add2(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), make_float2(-D.z, -D.w));
            a = mul2(a, make_float2(pr[k], pr[k + 1]));
            b = mul2(b, make_float2(pr[k + 2], pr[k + 3]));
            if constexpr (T == VAE_F16) {
                a = mul2(a, make_float2(f, f));
                b = mul2(b, make_float2(f, f));
            }
            pr[k] = a.x;
            pr[k + 1] = a.y;
            pr[k + 2] = b.x;
            pr[k + 3] = b.y;
        }
        store64<T>(tX, pr, rest);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s.ds_full));
        if (++st == C::kStages) {
            st = 0;
            ph ^= 1u;
        }
    }
    if (ok) ok = warp_all(bwait(s.done, 0u, s, p));
    if (!ok) return;
    tc_fence_after();
    // dV by the first four warps, dK by the others
    const long long rows = static_cast<long long>(sh.b) * sh.hkv * sh.sk;
    const long long row = (static_cast<long long>(w.e) * sh.hkv + w.hk) * sh.sk + j;
    const bool split = p.nsplit_k > 1;
    const MhaStrides os = half == 0 ? p.dvs : p.dks;
    // (softmax over a single key is 1 whatever its score: that gradient is 0)
    const float g = half == 0 ? (T == VAE_F16 ? 1.f / (1 << kPLog2) : 1.f) : w.kl == 1 ? 0.f : p.scale / c;
    store_acc<T>(lane_off + 256u + static_cast<uint32_t>(half * 128), sh.d, j < w.kl, true, g,
                 half == 0 ? p.dv : p.dk, w.e * os.b + j * os.s + w.hk * os.h, split ? p.part_kv : nullptr,
                 ((w.split * 2 + half) * rows + row) * sh.d);
}

template <int T, int kSteps, bool kTwice>
__global__ void __launch_bounds__(kThreads, 1)
    mha_dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const BwdParams p) {
    using C = KvCfg<kSteps>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // (the swizzled tiles lie on 1024-byte boundaries)
    const BwdSmem s = bwd_carve<C>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();
    const KvWork w = kv_work(p);
    if (p.s.fill && p.nsplit_k == 1) {  // (else the joining kernel does)
        mha_fill_keys(p.s, w.e, w.hk, w.kb, w.kl, p.dk, p.dks.b, p.dks.s, p.dks.h);
        mha_fill_keys(p.s, w.e, w.hk, w.kb, w.kl, p.dv, p.dvs.b, p.dvs.s, p.dvs.h);
    }
    if (w.n == 0) {  // no query: zeros within the length
        const int j = w.kb * kMhaTile + (threadIdx.x & 127);
        if (threadIdx.x < 2 * kMhaTile && j < w.kl) {
            const int half = threadIdx.x / kMhaTile;
            const long long rows = static_cast<long long>(p.s.b) * p.s.hkv * p.s.sk;
            const long long row = (static_cast<long long>(w.e) * p.s.hkv + w.hk) * p.s.sk + j;
            const MhaStrides os = half == 0 ? p.dvs : p.dks;
            store_acc<T>(0u, p.s.d, true, false, 0.f, half == 0 ? p.dv : p.dk, w.e * os.b + j * os.s + w.hk * os.h,
                         p.nsplit_k > 1 ? p.part_kv : nullptr, ((w.split * 2 + half) * rows + row) * p.s.d);
        }
        return;
    }
    bwd_begin<C>(s, warp, 1u);
    if (warp < kSoftWarps) kv_softmax<T, kSteps, kTwice>(p, s, w, warp, lane);
    else if (warp == kTmaWarp) kv_producer<C>(p, s, w, &mq, &mg, &mk, &mv, lane);
    else kv_mma<T, kSteps>(p, s, w);
    bwd_end(warp);
}

// ───────────────────────────── dQ, per row tile ─────────────────────────────

struct QWork {
    int e, hk, sub, tile, split;
    int ql, kl;
    int kb0, n;  // this split's key tiles
    bool exact;  // D is formed here
};

__device__ __forceinline__ QWork q_work(const BwdParams& p) {
    const MhaShape& s = p.s;
    QWork w;
    int r = blockIdx.x;
    w.tile = s.ntile - 1 - r % s.ntile;  // the tiles that see the most keys first
    r /= s.ntile;
    w.split = r % p.nsplit_q;
    r /= p.nsplit_q;
    w.sub = r % s.nsub;
    r /= s.nsub;
    w.hk = r % s.hkv;
    w.e = r / s.hkv;
    w.ql = mha_len(s.q_len, w.e, s.sq);
    w.kl = mha_len(s.k_len, w.e, s.sk);
    // the tile's last row sees the most keys
    const int i0 = (w.tile * kMhaTile) >> s.gp_log2;
    int i1 = ((w.tile + 1) * kMhaTile - 1) >> s.gp_log2;
    if (i1 >= w.ql) i1 = w.ql - 1;
    const int lim = i0 < w.ql ? mha_key_limit(i1, w.ql, w.kl, s.block) : 0;
    const int all = (lim + kMhaTile - 1) / kMhaTile;
    // (few key tiles are one split's: it forms D over all of them)
    w.exact = all <= kExactTiles;
    const int per = w.exact ? all : (all + p.nsplit_q - 1) / p.nsplit_q;
    w.kb0 = w.split * per < all ? w.split * per : all;
    w.n = (w.kb0 + per < all ? w.kb0 + per : all) - w.kb0;
    return w;
}

template <typename C>
__device__ void q_producer(const BwdParams& p, const BwdSmem& s, const QWork& w, const CUtensorMap* mk,
                           const CUtensorMap* mv, int lane) {
    const uint64_t pol = policy_evict_normal();
    const MhaShape& sh = p.s;
    BwdRing<C::kStages> r;
    const int steps = w.exact ? 2 * w.n : w.n;
    for (int x = 0; x < steps; ++x) {
        const int kb = w.kb0 + (x < w.n ? x : x - w.n);
        if (!warp_all(bwait(&s.empty[r.stage], r.phase ^ 1u, s, p))) break;
        uint8_t* dst = s.ring + r.stage * 2 * C::kTileBytes;
        const bool fix = (kb + 1) * kMhaTile > w.kl && w.kl < sh.sk;  // the tile that the length ends in
        const uint32_t ab = smem_u32(fix ? &s.fix[r.stage] : &s.a_full[r.stage]), bb = smem_u32(fix ? &s.fix[r.stage] : &s.b_full[r.stage]);
        if (lane == 0) {
            mbar_arrive_expect_tx(ab, (fix ? 2u : 1u) * C::kTileBytes);
            if (!fix) mbar_arrive_expect_tx(bb, C::kTileBytes);
            load_tile<C::kCh>(dst, mk, ab, w.hk, kb * kMhaTile, 64, w.e, pol);
            load_tile<C::kCh>(dst + C::kTileBytes, mv, bb, w.hk, kb * kMhaTile, 64, w.e, pol);
        }
        if (fix) {
            if (!r.template fix<C>(s, p, w.kl - kb * kMhaTile, false, lane)) break;
        } else {
            r.arm();
        }
        r.next();
    }
    if (lane == 0) r.drain(s, p, false);
    __syncwarp();
}

constexpr uint32_t kTmemQ = 384u, kTmemG = 448u;  // the tile's Q and dO rows, 64 columns each

template <int T, int kSteps>
__device__ void q_mma(const BwdParams& p, const BwdSmem& s, const QWork& w) {
    using C = QCfg<kSteps>;
    constexpr uint32_t id_s = mha_idesc(T, 128, 128, false), id_o = mha_idesc(T, 128, kSteps * 16, true);
    constexpr uint32_t tS = 0u, tX = 128u, tQ = 256u;
    constexpr uint32_t stage_units = 2u * C::kTileBytes >> 4, second = C::kTileBytes >> 4;
    const uint64_t ring_k = sw128_kmajor_desc(smem_u32(s.ring)), ring_m = sw128_mnmajor_desc(smem_u32(s.ring));
    auto wait = [&](uint64_t* bar, uint32_t par) { return warp_all(bwait(bar, par, s, p)); };
    auto score = [&](uint32_t st) {
        mma_ts_k<kSteps>(tS, kTmemQ, ring_k + st * stage_units, id_s);
        umma_commit(smem_u32(s.s_full));
    };
    auto cross = [&](uint32_t st) {
        mma_ts_k<kSteps>(tX, kTmemG, ring_k + st * stage_units + second, id_s);
        umma_commit(smem_u32(s.x_full));
    };
    uint32_t st = 0, ph = 0;
    bool ok = wait(s.res_full, 0u) && wait(&s.a_full[0], 0u) && wait(&s.b_full[0], 0u);
    if (ok) {
        tc_fence_after();
        if (elect_one()) {
            score(0);
            cross(0);
        }
        __syncwarp();
    }
    const int from = w.exact ? w.n : 0, steps = from + w.n;
    for (int x = 0; ok && x < steps; ++x) {
        const uint32_t par = static_cast<uint32_t>(x) & 1u;
        const bool more = x + 1 < steps;
        const bool wrap = st + 1 == C::kStages;
        const uint32_t st1 = wrap ? 0u : st + 1u, ph1 = wrap ? ph ^ 1u : ph;
        if (more) {  // S has been read
            ok = wait(s.p_full, par) && wait(&s.a_full[st1], ph1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) score(st1);
            __syncwarp();
        }
        ok = wait(s.ds_full, par);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            if (x >= from) mma_ts<64>(tQ, tX, ring_m + st * stage_units, id_o, x != from ? 1u : 0u);
            umma_commit(smem_u32(&s.empty[st]));
        }
        __syncwarp();
        if (more) {
            ok = wait(&s.b_full[st1], ph1);
            if (!ok) break;
            if (elect_one()) cross(st1);
            __syncwarp();
        }
        st = st1;
        ph = ph1;
    }
    mma_finish(s, p, ok);
}

template <int T, int kSteps, bool kTwice>
__device__ void q_softmax(const BwdParams& p, const BwdSmem& s, const QWork& w, int warp, int lane) {
    const int quad = warp & 3, half = warp >> 2;
    const MhaShape& sh = p.s;
    const int gp = 1 << sh.gp_log2;
    const int at = quad * 32 + lane, rr = kTwice ? at & 63 : at, r = w.tile * kMhaTile + rr;
    const bool rest = kTwice && rr != at;  // these lanes hold the other half's rows again
    const int i = r >> sh.gp_log2, h = w.hk * sh.g + w.sub * gp + (r & (gp - 1));
    const bool live = i < w.ql;
    const int lim = live ? mha_key_limit(i, w.ql, w.kl, sh.block) : 0;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = lane_off + static_cast<uint32_t>(half * 64), tX = tS + 128u;
    // The row of Q (first four warps) or dO into TMEM, zeros behind the length and the channels.
    {
        const MhaStrides st = half == 0 ? p.qs : p.gs;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(half == 0 ? p.q : p.dout) +
                                                          (live ? w.e * st.b + i * st.s + h * st.h : 0));
#pragma unroll
        for (int c = 0; c < kSteps / 2; ++c) {
            uint32_t v[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 x = live && (c * 4 + k) * 8 < sh.d ? src[c * 4 + k] : make_uint4(0u, 0u, 0u, 0u);
                v[4 * k] = x.x;
                v[4 * k + 1] = x.y;
                v[4 * k + 2] = x.z;
                v[4 * k + 3] = x.w;
            }
            __syncwarp();
            tmem_st16((half == 0 ? kTmemQ : kTmemG) + lane_off + static_cast<uint32_t>(c * 16), v);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s.res_full));
    }
    float* side = p.side + (((static_cast<long long>(w.e) * sh.hkv + w.hk) * sh.nsub + w.sub) * sh.ntile + w.tile) * kSideFloats;
    const float nl = live ? side[rr] : -INFINITY;
    float D = live ? side[128 + rr] : 0.f;
    const float c = ds_factor<T>(p.maxima + maxima_at(sh, w.e, w.hk));
    const float f = T == VAE_F16 ? c * (1.f / (1 << kPLog2)) : 1.f;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(nl, nl);
    float2 D2 = make_float2(-D, -D), sum = make_float2(0.f, 0.f);
    const int from = w.exact ? w.n : 0, steps = from + w.n;
    bool ok = true;
    for (int x = 0; x < steps; ++x) {
        const uint32_t par = static_cast<uint32_t>(x) & 1u;
        if (w.exact && x == from) {
            // D = rowsum(P dP): this half's sum and the other's, for the key-tile kernel too
            float* trade = reinterpret_cast<float*>(s.side);
            trade[half * kMhaTile + at] = sum.x + sum.y;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.x_bar[quad]));
            ok = warp_all(bwait(&s.x_bar[quad], 0u, s, p));
            if (!ok) break;
            const float all = *static_cast<volatile float*>(trade + at) + *static_cast<volatile float*>(trade + kMhaTile + at);
            D = T == VAE_F16 ? all * (1.f / (1 << kPLog2)) : all;
            if (half == 0 && live && !rest) side[128 + rr] = D;
            D2 = make_float2(-D, -D);
        }
        ok = warp_all(bwait(s.s_full, par, s, p));
        if (!ok) break;
        tc_fence_after();
        uint32_t xr[4][16];
        float pr[64];
        load64(tS, xr);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s.p_full));
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
            const uint32_t* y = xr[k >> 4] + (k & 15);
            const float2 a = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, nl2);
            pr[k] = mha_ex2(a.x);
            pr[k + 1] = mha_ex2(a.y);
        }
        const int left = lim - (w.kb0 + (x < w.n ? x : x - w.n)) * kMhaTile - half * 64;
        if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
                if (k >= left) pr[k] = 0.f;
        }
        ok = warp_all(bwait(s.x_full, par, s, p));
        if (!ok) break;
        tc_fence_after();
        load64(tX, xr);
        if (x < from) {
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                const uint32_t* y = xr[k >> 4] + (k & 15);
                sum = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), make_float2(pr[k], pr[k + 1]), sum);
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t h2[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const int n = k * 32 + 2 * u;
                    const uint32_t* y = xr[n >> 4] + (n & 15);
                    float2 a = add2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), D2);
                    a = mul2(a, make_float2(pr[n], pr[n + 1]));
                    if constexpr (T == VAE_F16) a = mul2(a, make_float2(f, f));
                    h2[u] = pack2<T>(a.x, a.y);
                    if (kTwice && rest) h2[u] = pack2_rest<T>(a.x, a.y);
                }
                tmem_st16(tX + static_cast<uint32_t>(k * 16), h2);
            }
            tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(s.ds_full));
    }
    if (ok) ok = warp_all(bwait(s.done, 0u, s, p));
    if (half != 0) return;
    // the second copies' rows pass through the ring, which every MMA has read: [channel][64 rows]
    float* more = kTwice ? reinterpret_cast<float*>(s.ring) : nullptr;
    if constexpr (kTwice) {
        if (ok && quad >= 2) {
            tc_fence_after();
            for (int c0 = 0; c0 < sh.d; c0 += 16) {
                uint32_t v[16];
                __syncwarp();
                tmem_ld16(lane_off + 256u + static_cast<uint32_t>(c0), v);
                tmem_ld_wait_regs(v);
#pragma unroll
                for (int k = 0; k < 16; ++k) more[(c0 + k) * 64 + rr] = __uint_as_float(v[k]);
            }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // (the first four warps all come here, timed out or not)
        if (quad >= 2) return;
    }
    if (!ok) return;
    tc_fence_after();
    const long long rows = static_cast<long long>(sh.b) * sh.hq * sh.sq;
    const long long row = (static_cast<long long>(w.e) * sh.hq + h) * sh.sq + i;
    // (a row that sees a single key: P is 1 whatever the score, and dq 0)
    store_acc<T>(lane_off + 256u, sh.d, live, true, lim == 1 ? 0.f : p.scale / c, p.dq,
                 w.e * p.dqs.b + i * p.dqs.s + h * p.dqs.h, p.nsplit_q > 1 ? p.part_q : nullptr,
                 (w.split * rows + row) * sh.d, kTwice ? more + rr : nullptr);
}

template <int T, int kSteps, bool kTwice>
__global__ void __launch_bounds__(kThreads, 1)
    mha_dq_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const BwdParams p) {
    using C = QCfg<kSteps>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // (the swizzled tiles lie on 1024-byte boundaries)
    const BwdSmem s = bwd_carve<C>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_wait();
    const QWork w = q_work(p);
    if (p.s.fill && p.nsplit_q == 1)  // (else the joining kernel does)
        mha_fill_queries(p.s, w.e, w.hk, w.sub, w.tile, w.ql, p.dq, p.dqs.b, p.dqs.s, p.dqs.h, nullptr);
    if (w.n == 0) {  // no key: zeros within the length
        const int r = w.tile * kMhaTile + threadIdx.x;
        const int i = r >> p.s.gp_log2, h = w.hk * p.s.g + (w.sub << p.s.gp_log2) + (r & ((1 << p.s.gp_log2) - 1));
        if (threadIdx.x < kMhaTile && i < w.ql) {
            const long long rows = static_cast<long long>(p.s.b) * p.s.hq * p.s.sq;
            const long long row = (static_cast<long long>(w.e) * p.s.hq + h) * p.s.sq + i;
            store_acc<T>(0u, p.s.d, true, false, 0.f, p.dq, w.e * p.dqs.b + i * p.dqs.s + h * p.dqs.h,
                         p.nsplit_q > 1 ? p.part_q : nullptr, (w.split * rows + row) * p.s.d);
        }
        return;
    }
    bwd_begin<C>(s, warp, kSoftWarps);
    if (warp < kSoftWarps) q_softmax<T, kSteps, kTwice>(p, s, w, warp, lane);
    else if (warp == kTmaWarp) q_producer<C>(p, s, w, &mk, &mv, lane);
    else q_mma<T, kSteps>(p, s, w);
    bwd_end(warp);
}

// ───────────────────────────── joining the splits ─────────────────────────────

// out[row] = sum of the splits' partial rows in order, rounded once; four
// channels a thread. Rows [b][h][n], valid below the length.
template <int T>
__global__ void __launch_bounds__(256)
    mha_sum_kernel(const float* __restrict__ part, long long split_stride, int nsplit, int b, int h, int n, int d,
                   const int* len, int fill, void* out, MhaStrides os) {
    pdl_wait();
    const long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int d4 = d / 4;
    const long long row = x / d4;
    if (row >= static_cast<long long>(b) * h * n) return;
    const int c = static_cast<int>(x - row * d4) * 4;
    const int i = static_cast<int>(row % n), hh = static_cast<int>(row / n % h), e = static_cast<int>(row / n / h);
    if (i >= mha_len(len, e, n)) {
        if (fill)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + e * os.b + i * os.s + hh * os.h + c) = make_uint2(0u, 0u);
        return;
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < nsplit; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(part + k * split_stride + row * d + c);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
    }
    *reinterpret_cast<uint2*>(static_cast<typename Elem<T>::type*>(out) + e * os.b + i * os.s + hh * os.h + c) =
        make_uint2(pack2<T>(a.x, a.y), pack2<T>(a.z, a.w));
}

// The number of splits of the other side whose waves of CTAs take the shortest
// time, by what the parts measured on GB300 (microseconds): a tile of the other side 1.4 (query
// tiles) and 1.8 (key tiles), a CTA's set-up and end 5, the joining kernel 3 and
// its traffic at 6 TB/s.
struct BwdPlan {
    int nsplit_q, nsplit_k;
    long long q_items, k_items, row_tiles, key_tiles;
    size_t side, part_q, part_kv;  // floats
};
// heads x tiles CTAs against `other` tiles; `sum`: elements that a split writes and the join reads.
void split_plan(long long heads, int tiles, long long other, double tile_us, double sum, int most, int* nsplit, long long* items) {
    const long long each = heads * tiles;
    double least = 0.0;
    for (int n = 1; n == 1 || (n <= most && each * n <= 4 * kTargetCtas); ++n) {
        const double waves = static_cast<double>((each * n - 1) / kTargetCtas + 1);
        double t = waves * (static_cast<double>((other - 1) / n + 1) * tile_us + 5.0);
        if (n > 1) t += 3.0 + 8.0 * n * sum / 6e6;
        if (n == 1 || t < least) {
            least = t;
            *nsplit = n;
        }
    }
    *items = each * *nsplit;
}
BwdPlan bwd_plan(const MhaShape& s) {
    BwdPlan f;
    const long long q_heads = static_cast<long long>(s.b) * s.hkv * s.nsub, k_heads = static_cast<long long>(s.b) * s.hkv;
    const long long row_tiles = static_cast<long long>(s.nsub) * s.ntile;
    f.row_tiles = q_heads * s.ntile;
    f.key_tiles = k_heads * s.nkb;
    // (two tiles of the other side a CTA at least; rows that meet few keys are not split: they form their D)
    split_plan(q_heads, s.ntile, s.nkb, 1.4, static_cast<double>(s.b) * s.hq * s.sq * s.d,
               s.nkb <= kExactTiles ? 1 : s.nkb / 2, &f.nsplit_q, &f.q_items);
    split_plan(k_heads, s.nkb, row_tiles, 1.8, 2.0 * s.b * s.hkv * s.sk * s.d,
               static_cast<int>(std::min<long long>(row_tiles / 2, 1 << 20)), &f.nsplit_k, &f.k_items);
    f.side = static_cast<size_t>(f.row_tiles) * kSideFloats;
    f.part_q = f.nsplit_q > 1 ? static_cast<size_t>(f.nsplit_q) * s.b * s.hq * s.sq * s.d : 0;
    f.part_kv = f.nsplit_k > 1 ? static_cast<size_t>(f.nsplit_k) * 2 * s.b * s.hkv * s.sk * s.d : 0;
    return f;
}
// Words for the maxima; whole 256 bytes keep what follows aligned.
size_t maxima_floats(const MhaShape& s) { return (maxima_at(s, s.b, 0) + 63) / 64 * 64; }

template <int T, int kSteps, bool kTwice>
int bwd_launch(const vae_attention_desc* a, const BwdPlan& f, const CUtensorMap (&map)[4], const PrepParams& pp,
               const BwdParams& p, cudaStream_t st) {
    static CtxOnce once;
    static std::mutex mu;
    constexpr int kKvSmem = KvCfg<kSteps>::kSmem, kQSmem = QCfg<kSteps>::kSmem;
    {
        int dev;
        VAE_CUDA_CHECK(cudaGetDevice(&dev));
        std::lock_guard<std::mutex> lk(mu);
        if (!once.done(dev)) {
            VAE_CUDA_CHECK(cudaFuncSetAttribute(mha_dkv_kernel<T, kSteps, kTwice>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKvSmem));
            VAE_CUDA_CHECK(cudaFuncSetAttribute(mha_dq_kernel<T, kSteps, kTwice>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSmem));
            once.mark(dev);
        }
    }
    if (T == VAE_F16) VAE_CUDA_CHECK(cudaMemsetAsync(pp.maxima, 0, maxima_at(p.s, p.s.b, 0) * sizeof(unsigned), st));
    const long long prep = f.row_tiles + (T == VAE_F16 ? f.key_tiles : 0);
    VAE_CUDA_CHECK(launch_kernel(mha_prep_kernel<T>, dim3(static_cast<unsigned>(prep)), dim3(256), 0, st, pp));
    // (The query-tile kernel first: it may put its D into the side rows.)
    VAE_CUDA_CHECK(launch_kernel_as(false, mha_dq_kernel<T, kSteps, kTwice>, dim3(static_cast<unsigned>(f.q_items)),
                                    dim3(kThreads), kQSmem, st, map[2], map[3], p));
    VAE_CUDA_CHECK(launch_kernel_as(false, mha_dkv_kernel<T, kSteps, kTwice>, dim3(static_cast<unsigned>(f.k_items)),
                                    dim3(kThreads), kKvSmem, st, map[0], map[1], map[2], map[3], p));
    const MhaShape& s = p.s;
    if (f.nsplit_k > 1) {
        const long long rows = static_cast<long long>(s.b) * s.hkv * s.sk;
        const unsigned grid = static_cast<unsigned>((rows * (s.d / 4) + 255) / 256);
        for (int k = 0; k < 2; ++k)
            VAE_CUDA_CHECK(launch_kernel(mha_sum_kernel<T>, dim3(grid), dim3(256), 0, st,
                                         static_cast<const float*>(p.part_kv) + k * rows * s.d, 2 * rows * s.d, f.nsplit_k,
                                         s.b, s.hkv, s.sk, s.d, s.k_len, s.fill, k == 0 ? p.dv : p.dk, k == 0 ? p.dvs : p.dks));
    }
    if (f.nsplit_q > 1) {
        const long long rows = static_cast<long long>(s.b) * s.hq * s.sq;
        const unsigned grid = static_cast<unsigned>((rows * (s.d / 4) + 255) / 256);
        VAE_CUDA_CHECK(launch_kernel(mha_sum_kernel<T>, dim3(grid), dim3(256), 0, st, static_cast<const float*>(p.part_q),
                                     rows * s.d, f.nsplit_q, s.b, s.hq, s.sq, s.d, s.q_len, s.fill, p.dq, p.dqs));
    }
    return VAE_OK;
}

template <bool kTwice>
int bwd_by_type(const vae_attention_desc* a, const BwdPlan& f, const CUtensorMap (&map)[4], const PrepParams& pp,
                const BwdParams& p, cudaStream_t st) {
    const int d = p.s.d;
    if (a->type == VAE_F16)
        return d <= 64   ? bwd_launch<VAE_F16, 4, kTwice>(a, f, map, pp, p, st)
               : d <= 96 ? bwd_launch<VAE_F16, 6, kTwice>(a, f, map, pp, p, st)
                         : bwd_launch<VAE_F16, 8, kTwice>(a, f, map, pp, p, st);
    return d <= 64   ? bwd_launch<VAE_BF16, 4, kTwice>(a, f, map, pp, p, st)
           : d <= 96 ? bwd_launch<VAE_BF16, 6, kTwice>(a, f, map, pp, p, st)
                     : bwd_launch<VAE_BF16, 8, kTwice>(a, f, map, pp, p, st);
}

}  // namespace

size_t mha_bwd_bytes(const MhaShape& s) {
    const BwdPlan f = bwd_plan(s);
    return ((maxima_floats(s) + f.side + f.part_q + f.part_kv) * sizeof(float) + 15) / 16 * 16;
}

int mha_bwd_run(const vae_attention_desc* a, const MhaShape& s, const void* dout, const void* q, const void* k,
                const void* v, const void* o, const float* lse, void* dq, void* dk, void* dv, void* ws,
                cudaStream_t st) {
    const BwdPlan f = bwd_plan(s);
    if (f.q_items > 0x7fffffffLL || f.k_items > 0x7fffffffLL || f.row_tiles + f.key_tiles > 0x7fffffffLL)
        return set_error(VAE_ERR_SHAPE, "attention: too many tiles");
    const int gp = 1 << s.gp_log2;
    CUtensorMap map[4];
    int rc = mha_map(&map[0], a, q, a->q_stride, s.sq, s.hq, gp, 64 / gp);
    if (rc == VAE_OK) rc = mha_map(&map[1], a, dout, a->do_stride, s.sq, s.hq, gp, 64 / gp);
    if (rc == VAE_OK) rc = mha_map(&map[2], a, k, a->k_stride, s.sk, s.hkv, 1, 64);
    if (rc == VAE_OK) rc = mha_map(&map[3], a, v, a->v_stride, s.sk, s.hkv, 1, 64);
    if (rc != VAE_OK) return rc;
    float* w = static_cast<float*>(ws);
    PrepParams pp{};
    pp.s = s;
    pp.dout = dout;
    pp.o = o;
    pp.v = v;
    pp.gs = mha_strides(a->do_stride);
    pp.os = mha_strides(a->o_stride);
    pp.vs = mha_strides(a->v_stride);
    pp.lse = lse;
    pp.maxima = static_cast<unsigned*>(ws);
    pp.side = w + maxima_floats(s);
    pp.row_tiles = static_cast<int>(f.row_tiles);
    BwdParams p{};
    p.s = s;
    p.scale = a->scale;
    p.scale_log2 = a->scale * 1.4426950408889634074f;
    p.nsplit_q = f.nsplit_q;
    p.nsplit_k = f.nsplit_k;
    p.twice = static_cast<long long>(s.sq) * gp <= kMhaTile / 2;
    p.q = q;
    p.dout = dout;
    p.qs = mha_strides(a->q_stride);
    p.gs = mha_strides(a->do_stride);
    p.side = pp.side;
    p.maxima = pp.maxima;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dqs = mha_strides(a->dq_stride);
    p.dks = mha_strides(a->dk_stride);
    p.dvs = mha_strides(a->dv_stride);
    p.part_q = pp.side + f.side;
    p.part_kv = p.part_q + f.part_q;
    p.status = device_status_ptr();
    p.timeout_ns = wait_timeout_ns();
    if (p.status == nullptr) return VAE_ERR_CUDA;
    return p.twice ? bwd_by_type<true>(a, f, map, pp, p, st) : bwd_by_type<false>(a, f, map, pp, p, st);
}

}  // namespace vae
