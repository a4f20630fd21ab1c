// The norm of query and key heads with their rotary positions, and its gradient
// (public entry points at the end).
//
// A row is one head of one token, d channels: n = x (mean x^2 + eps)^-1/2,
// y = R (n gamma). Backward, with u = R^T dy and v = u gamma: dx = r (v - n mean(v n)),
// r the root, and dgamma = the sum of u n over the rows. A block takes some tokens,
// forms the (cos, sin) of their pairs once in shared memory and works on every
// query and key head of them: one read of each input and one write of each output,
// which bounds the call.
#include <algorithm>
#include <cmath>

#include "vae_overlap.h"
#include "vae_rope.cuh"
#include "vae_types.cuh"

namespace vae {

namespace {

constexpr int kQkMaxD = 256;
constexpr int kQkTokens = 8;     // tokens a block takes at a time, at most (a power of two, as fewer are)
constexpr int kQkThreads = 128;
constexpr int kQkWarps = kQkThreads / 32;
constexpr int kQkBlocks = 608;   // of the gradient, at most: each leaves a row of partial sums for dgamma
constexpr int kQkForward = 760;  // blocks of the forward, at most: five an SM
constexpr int kQkPitch = VAE_ROPE_MAX_PAIRS + 2;

struct QkPart {  // queries or keys
    const void *x, *dy;
    void* y;
    const float* gamma;
    float* dgamma;
    long long xs[3], gs[3], ys[3];
    int h;
};
struct QkParams {
    QkPart part[2];
    const void* pos;
    int tokens, s, d, tpb;
    int pos_int, pos_batch;
    int qblocks;  // in vectors: blocks of queries; the others are the keys'
    float eps;
    float* sums;  // a row of d for each block (in the plain form two, the queries' first): its part of dgamma
};

__device__ __forceinline__ float qk_pos(const QkParams& p, const vae_rope_plan& plan, int token, int pair) {
    const long long row = p.pos_batch > 1 ? token : token % p.s;
    const long long i = row * plan.naxes + plan.axis[pair];
    return p.pos_int ? static_cast<float>(static_cast<const int*>(p.pos)[i]) : static_cast<const float*>(p.pos)[i];
}

__device__ __forceinline__ long long qk_offset(const QkParams& p, int token, int head, const long long (&st)[3]) {
    const int e = token / p.s;
    return e * st[0] + (token - e * p.s) * st[1] + head * st[2];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Any d and any strides: a warp takes a row, channel by channel.
template <int T, bool kBack>
__global__ void __launch_bounds__(kQkThreads) qk_plain_kernel(const QkParams p, const __grid_constant__ vae_rope_plan plan) {
    using E = typename Elem<T>::type;
    constexpr int kEach = kQkMaxD / 32;
    __shared__ float2 cs[kQkTokens][kQkPitch];
    __shared__ float row[kQkWarps][kQkMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pairs = plan.pairs, rot = 2 * pairs;
    float acc[2][kEach] = {};
    pdl_wait();
    // the place of channel c's partner, and its pair
    auto turned = [&](const float* z, const float2* t, int c) {
        const float v = z[c];
        if (c >= rot) return v;
        const bool second = plan.interleaved ? (c & 1) != 0 : c >= pairs;
        const float2 a = t[plan.interleaved ? c >> 1 : second ? c - pairs : c];
        const float w = z[plan.interleaved ? c ^ 1 : second ? c - pairs : c + pairs];
        const float sn = second != kBack ? a.y : -a.y;  // (turned back, the sines change sign)
        return v * a.x + w * sn;
    };
    const int stride = static_cast<int>(gridDim.x) * p.tpb;  // (at most p.tokens and a turn: no sum below passes 31 bits)
    for (int t0 = static_cast<int>(blockIdx.x) * p.tpb; t0 < p.tokens; t0 = p.tokens - t0 > stride ? t0 + stride : p.tokens) {
        const int nt = p.tokens - t0 < p.tpb ? p.tokens - t0 : p.tpb;
        __syncthreads();
        for (int i = threadIdx.x; i < nt * pairs; i += kQkThreads) {
            const int pr = i / nt, t = i - pr * nt;
            cs[t][pr] = rope_cos_sin(plan, pr, qk_pos(p, plan, t0 + t, pr));
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const QkPart& part = p.part[w];
            for (int r = warp; r < nt * part.h; r += kQkWarps) {
                const int t = r / part.h, head = r - t * part.h;
                const E* x = static_cast<const E*>(part.x) + qk_offset(p, t0 + t, head, part.xs);
                E* y = static_cast<E*>(part.y) + qk_offset(p, t0 + t, head, part.ys);
                float v[kEach], ss = 0.f;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int c = lane + 32 * i;
                    v[i] = c < p.d ? to_f32<T>(x[c]) : 0.f;
                    ss += v[i] * v[i];
                }
                const float rs = rsqrtf(warp_sum(ss) / static_cast<float>(p.d) + p.eps);
                __syncwarp();
                if constexpr (!kBack) {
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (const int c = lane + 32 * i; c < p.d) row[warp][c] = v[i] * rs * (part.gamma != nullptr ? __ldg(part.gamma + c) : 1.f);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (const int c = lane + 32 * i; c < p.d) y[c] = from_f32<T>(turned(row[warp], cs[t], c));
                } else {
                    const E* dy = static_cast<const E*>(part.dy) + qk_offset(p, t0 + t, head, part.gs);
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (const int c = lane + 32 * i; c < p.d) row[warp][c] = to_f32<T>(dy[c]);
                    __syncwarp();
                    float along = 0.f, g[kEach];
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        const int c = lane + 32 * i;
                        g[i] = 0.f;
                        v[i] *= rs;
                        if (c < p.d) {
                            const float u = turned(row[warp], cs[t], c);
                            acc[w][i] += u * v[i];
                            g[i] = u * (part.gamma != nullptr ? __ldg(part.gamma + c) : 1.f);
                            along += g[i] * v[i];
                        }
                    }
                    along = warp_sum(along) / static_cast<float>(p.d);
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (const int c = lane + 32 * i; c < p.d) y[c] = from_f32<T>(rs * (g[i] - v[i] * along));
                }
            }
        }
    }
    if constexpr (kBack) {
        if (p.sums != nullptr)
            for (int w = 0; w < 2; ++w) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kEach; ++i) row[warp][lane + 32 * i] = acc[w][i];
                __syncthreads();
                for (int c = threadIdx.x; c < p.d; c += kQkThreads) {
                    float s = 0.f;
                    for (int k = 0; k < kQkWarps; ++k) s += row[k][c];
                    p.sums[(static_cast<long long>(w) * gridDim.x + blockIdx.x) * p.d + c] = s;
                }
            }
    }
    pdl_launch_dependents();
}

// Rows in 16-byte vectors. A row lies over G lanes (a power of two, 16 at most), two
// units of eight channels a lane, in one of three ways:
//   kLocal: units u and u + n of n lanes; interleaved pairs lie within a unit (or nothing turns);
//   kHalves: pairs (c, c + R/2) with R a multiple of 16: a lane holds a unit of each half;
//   kSwap: other halves: units u and u + n, the partners come through shared memory.
// Neighbouring lanes take neighbouring units, so that every access covers whole sectors
// (two neighbouring units a lane: 137 us instead of 127 for 36864 tokens of 36 heads of 128, when a
// block took eight tokens and its threads the next rows in registers).
// The tokens of a block are a power of two, so a group of G lanes stays with one token: its
// angles lie in registers, and the rows that it meets, every few heads, are a fixed step
// apart. (Rows dealt out over tokens and heads in turn, angles read from shared memory for each:
// 414 instructions a warp and four rows, which bound the call.)
enum : int { kLocal, kHalves, kSwap };

// Eight channels as they lie in memory.
template <int T>
struct QkUnit {
    static constexpr int kVecs = T == VAE_F32 ? 2 : 1;
    using E = typename Elem<T>::type;
    uint4 r[kVecs];
    // In shared memory the vectors of a unit lie kQkThreads apart. Without `in` zeros come.
    __device__ __forceinline__ static void fetch(uint4* at, const E* p, bool in) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(at + i * kQkThreads)), "l"(p + i * 4),
                         "r"(in ? 16 : 0)
                         : "memory");
    }
    __device__ __forceinline__ void take(const uint4* at) {
        r[0] = at[0];
        if constexpr (T == VAE_F32) r[1] = at[kQkThreads];
    }
    __device__ __forceinline__ void get(float2* v) const {
        if constexpr (T == VAE_F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[2 * i] = make_float2(__uint_as_float(r[i].x), __uint_as_float(r[i].y));
                v[2 * i + 1] = make_float2(__uint_as_float(r[i].z), __uint_as_float(r[i].w));
            }
        } else {
            v[0] = unpack2<T>(r[0].x);
            v[1] = unpack2<T>(r[0].y);
            v[2] = unpack2<T>(r[0].z);
            v[3] = unpack2<T>(r[0].w);
        }
    }
    __device__ __forceinline__ static void put(E* p, const float2* v) {
        if constexpr (T == VAE_F32) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
            *reinterpret_cast<float4*>(p + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y), pack2<T>(v[2].x, v[2].y),
                                                      pack2<T>(v[3].x, v[3].y));
        }
    }
};

// The tokens' (cos, sin): of pair 4 q + 2 i + j of a token at [i][q][j].
using QkAngles = float2[2][VAE_ROPE_MAX_PAIRS / 4][2];

// A lane's place in its row and among the rows of a block.
template <int kForm>
struct QkLane {
    int u, group, units, ca, cb, left_a, left_b, token, first, step;
    bool turns, has_a, has_b;
    __device__ __forceinline__ QkLane(const QkParams& p, int pairs, int glog2) {
        const int rot = 2 * pairs, nrot = pairs >> 3;
        group = 1 << glog2;
        u = threadIdx.x & (group - 1);
        units = (p.d + 15) / 16;  // lanes of a row
        turns = kForm == kHalves && u < nrot;
        if constexpr (kForm == kHalves) {
            units = nrot + (p.d - rot + 15) / 16;
            ca = turns ? 8 * u : rot + 8 * (u - nrot);
            cb = turns ? pairs + 8 * u : ca + 8 * (units - nrot);
        } else {
            ca = 8 * u;
            cb = 8 * (u + units);
        }
        has_a = u < units && ca < p.d;
        has_b = u < units && cb < p.d;
        left_a = pairs - ca / 2;  // kLocal: pairs that turn from this unit's first on
        left_b = pairs - cb / 2;
        const int mine = threadIdx.x >> glog2;
        token = mine & (p.tpb - 1);
        first = mine / p.tpb;  // its heads: first, first + step, ...
        step = (kQkThreads >> glog2) / p.tpb;
    }
    __device__ __forceinline__ float sum(float x) const {
        for (int o = group >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
    __device__ __forceinline__ float2 sum2(float2 x) const {
        for (int o = group >> 1; o > 0; o >>= 1)
            x = add2(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
        return x;
    }
};

// The angles of a lane's token, and the turn of a row's pairs by them (the table's sines have the direction's sign).
template <int kForm>
struct QkTurn {
    float2 c[4], s[4];  // kHalves: cosines and sines of two pairs each; kLocal: (cos, sin) of the pairs of both units
    __device__ __forceinline__ void take(const QkAngles& a, const QkLane<kForm>& l) {
        if constexpr (kForm == kHalves) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(&a[i & 1][l.turns ? 2 * l.u + (i >> 1) : 0][0]);
                c[i] = make_float2(x.x, x.z);
                s[i] = make_float2(x.y, x.w);
            }
        } else if constexpr (kForm == kLocal) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(&a[i][l.u][0]);
                const float4 y = *reinterpret_cast<const float4*>(&a[i][l.has_b ? l.u + l.units : 0][0]);
                c[2 * i] = make_float2(x.x, x.y);
                c[2 * i + 1] = make_float2(x.z, x.w);
                s[2 * i] = make_float2(y.x, y.y);
                s[2 * i + 1] = make_float2(y.z, y.w);
            }
        }
    }
    __device__ __forceinline__ void apply(float2 (&v)[8], const QkAngles& a, const QkLane<kForm>& l, int pairs, float* swap) const {
        if constexpr (kForm == kHalves) {
            if (l.turns) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 t = mul2(v[4 + i], s[i]);
                    const float2 b = fma2(v[i], s[i], mul2(v[4 + i], c[i]));
                    v[i] = fma2(v[i], c[i], make_float2(-t.x, -t.y));
                    v[4 + i] = b;
                }
            }
        } else if constexpr (kForm == kLocal) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < l.left_a) turn(v[i].x, v[i].y, c[i]);
                if (i < l.left_b) turn(v[4 + i].x, v[4 + i].y, s[i]);
            }
        } else {
            float* z = swap + (threadIdx.x & ~(l.group - 1)) * 16;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (l.has_a) *reinterpret_cast<float2*>(z + l.ca + 2 * i) = v[i];
                if (l.has_b) *reinterpret_cast<float2*>(z + l.cb + 2 * i) = v[4 + i];
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int ch = (k < 8 ? l.ca : l.cb - 8) + k;
                if ((k < 8 ? l.has_a : l.has_b) && ch < 2 * pairs) {
                    const bool second = ch >= pairs;
                    const int pr = second ? ch - pairs : ch;
                    const float2 t = a[(pr >> 1) & 1][pr >> 2][pr & 1];
                    float& x = (k & 1) != 0 ? v[k >> 1].y : v[k >> 1].x;
                    x = x * t.x + z[second ? pr : ch + pairs] * (second ? t.y : -t.y);
                }
            }
        }
    }
};

// The angles of the tokens from t0 on, by the whole block; turned back, the sines change sign.
template <bool kBack>
__device__ __forceinline__ void qk_angles(QkAngles* cs, const QkParams& p, const vae_rope_plan& plan, int t0, int nt) {
    for (int i = threadIdx.x; i < nt * plan.pairs; i += kQkThreads) {
        // neighbours take the tokens of one pair: its entries of the plan are one address for them
        const int pr = i / nt, t = i - pr * nt;
        const float2 c = rope_cos_sin(plan, pr, qk_pos(p, plan, t0 + t, pr));
        cs[t][(pr >> 1) & 1][pr >> 2][pr & 1] = make_float2(c.x, kBack ? -c.y : c.y);
    }
}

__device__ __forceinline__ void qk_gamma(float2 (&gamma)[8], const float* at, int ca, bool has_a, int cb, bool has_b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float* x = at + (i < 4 ? ca + 2 * i : cb + 2 * i - 8);
        gamma[i] = at != nullptr && (i < 4 ? has_a : has_b) ? make_float2(__ldg(x), __ldg(x + 1)) : make_float2(1.f, 1.f);
    }
}
__device__ __forceinline__ float qk_square(const float2 (&v)[8]) {
    float2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        s = fma2(v[i], v[i], s);
        t = fma2(v[i + 1], v[i + 1], t);
    }
    s = add2(s, t);
    return s.x + s.y;
}

// Blocks stay for many tokens, each with the queries or the keys, so that a thread keeps its channels of one gamma and, in
// the gradient, sums those of one dgamma. A thread has the next kDeep rows' units on their way into shared memory, which
// nobody else reads, over the ends of its tokens: 36864 tokens of 36 heads 107 us (6.4 TB/s), the gradient of 24 heads 122
// (5.6 TB/s; each row a chain of sums over its lanes, and registers for four blocks an SM). With rows ahead in registers 127
// and 184. Forward with 4, 5, 6, 7 blocks an SM 110, 107, 116, 113 us, with eight, whose registers spill, 118; gradient, when
// it took 142 with four (queries and keys shared out by heads alone), with five 149.
template <int T, bool kBack>
struct QkRing {
    static constexpr int kDeep = kBack || T == VAE_F32 ? 2 : 3;
    static constexpr int kVecs = (kBack ? 4 : 2) * QkUnit<T>::kVecs;  // of a row and thread
    static constexpr int kBytes = kDeep * kVecs * kQkThreads * 16;
    // tokens a turn: each costs two barriers and the angles' latency (gradient, then: 4: 193 us, 8: 151, 16: 142)
    static constexpr int kTokens = kBack && T != VAE_F32 ? 2 * kQkTokens : kQkTokens;
    static constexpr int kResident = kBack ? 4 : 5;  // blocks an SM
    static_assert(kBytes + kTokens * sizeof(QkAngles) + kQkThreads * 64 <= 48 * 1024, "more shared memory than a kernel has without asking");
    static_assert(!kBack || kBytes >= kQkWarps * kQkMaxD * 4, "the ring takes a row of sums for each warp at the end");
};

template <int T, int kForm, bool kBack>
__global__ void __launch_bounds__(kQkThreads, QkRing<T, kBack>::kResident)
    qk_vector_kernel(const QkParams p, const __grid_constant__ vae_rope_plan plan, const int glog2) {
    using E = typename Elem<T>::type;
    using Unit = QkUnit<T>;
    using Ring = QkRing<T, kBack>;
    constexpr int kDeep = Ring::kDeep, kVecs = Ring::kVecs, kUnits = kBack ? 4 : 2;
    extern __shared__ __align__(16) uint4 ring[];  // [kDeep][kVecs][threads]
    __shared__ __align__(16) QkAngles cs[Ring::kTokens];
    __shared__ float swap[kForm == kSwap ? kQkThreads * 16 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const QkLane<kForm> l(p, plan.pairs, glog2);
    const float inv_d = 1.f / static_cast<float>(p.d);
    const bool keys = static_cast<int>(blockIdx.x) >= p.qblocks;
    const QkPart& part = p.part[keys ? 1 : 0];
    const int stride = (keys ? static_cast<int>(gridDim.x) - p.qblocks : p.qblocks) * p.tpb;  // tokens from one turn of a block to the next
    const int t00 = (keys ? static_cast<int>(blockIdx.x) - p.qblocks : static_cast<int>(blockIdx.x)) * p.tpb;
    const int most = (part.h + l.step - 1) / l.step;  // rows of a turn, of any group: the warp stays together
    const int heads = l.first < part.h ? (part.h - l.first + l.step - 1) / l.step : 0;
    pdl_wait();

    // the next row to ask for
    int nt0 = t00, nrow = 0;
    const E *x = static_cast<const E*>(part.x), *g = static_cast<const E*>(part.dy);
    bool more = false;
    auto open = [&]() {
        nrow = 0;
        more = nt0 < p.tokens && nt0 + l.token < p.tokens;
        if (!more) return;
        const int e = (nt0 + l.token) / p.s, si = nt0 + l.token - e * p.s;
        x = static_cast<const E*>(part.x) + e * part.xs[0] + si * part.xs[1] + l.first * part.xs[2];
        if constexpr (kBack) g = static_cast<const E*>(part.dy) + e * part.gs[0] + si * part.gs[1] + l.first * part.gs[2];
    };
    auto fetch = [&](int slot) {
        constexpr int kUnit = Unit::kVecs * kQkThreads;
        uint4* at = ring + slot * kVecs * kQkThreads + threadIdx.x;
        const bool in = more && nrow < heads, a = in && l.has_a, b = in && l.has_b;
        Unit::fetch(at, x + (a ? l.ca : 0), a);
        Unit::fetch(at + kUnit, x + (b ? l.cb : 0), b);
        if constexpr (kBack) {
            Unit::fetch(at + 2 * kUnit, g + (a ? l.ca : 0), a);
            Unit::fetch(at + 3 * kUnit, g + (b ? l.cb : 0), b);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (in) {
            x += l.step * part.xs[2];
            if constexpr (kBack) g += l.step * part.gs[2];
        }
        if (++nrow == most && nt0 < p.tokens) {
            nt0 = p.tokens - nt0 > stride ? nt0 + stride : p.tokens;
            open();
        }
    };
    open();
#pragma unroll 1
    for (int k = 0; k < kDeep; ++k) fetch(k);
    float2 gamma[8], acc[kBack ? 8 : 1] = {};
    qk_gamma(gamma, part.gamma, l.ca, l.has_a, l.cb, l.has_b);
    int slot = 0;
    for (int t0 = t00; t0 < p.tokens; t0 = p.tokens - t0 > stride ? t0 + stride : p.tokens) {
        const int nt = p.tokens - t0 < p.tpb ? p.tokens - t0 : p.tpb;
        const bool here = l.token < nt;
        __syncthreads();  // (the last tokens' angles have been read)
        qk_angles<kBack>(cs, p, plan, t0, nt);
        __syncthreads();
        const QkAngles& angles = cs[here ? l.token : 0];
        QkTurn<kForm> turned;
        turned.take(angles, l);
        const int e = (t0 + l.token) / p.s;
        E* y = static_cast<E*>(part.y) + e * part.ys[0] + (t0 + l.token - e * p.s) * part.ys[1] + l.first * part.ys[2];
        const int rows = here ? heads : 0;
#pragma unroll 1
        for (int row = 0; row < most; ++row) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");  // (this thread's own copies: no barrier)
            const uint4* at = ring + slot * kVecs * kQkThreads + threadIdx.x;
            Unit r[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i) r[i].take(at + i * Unit::kVecs * kQkThreads);
            float2 v[8], q[8];
            r[0].get(v);
            r[1].get(v + 4);
            if constexpr (kBack) {
                r[2].get(q);
                r[3].get(q + 4);
            }
            fetch(slot);
            if (++slot == kDeep) slot = 0;
            if constexpr (kBack) {
                // the two sums side by side: of x x and of v x, before r is known
                turned.apply(q, angles, l, plan.pairs, swap);
                float2 along = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) along = fma2(mul2(q[i], gamma[i]), v[i], along);
                const float2 sums = l.sum2(make_float2(qk_square(v), along.x + along.y));
                const float rs = rsqrtf(sums.x * inv_d + p.eps), m = -(sums.y * rs) * inv_d;
                const float2 rs2 = make_float2(rs, rs), m2 = make_float2(m, m);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = mul2(v[i], rs2);
                    acc[i] = fma2(q[i], v[i], acc[i]);
                    q[i] = mul2(fma2(v[i], m2, mul2(q[i], gamma[i])), rs2);
                }
            } else {
                const float rs = rsqrtf(l.sum(qk_square(v)) * inv_d + p.eps);
                const float2 rs2 = make_float2(rs, rs);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = mul2(mul2(v[i], rs2), gamma[i]);
                turned.apply(q, angles, l, plan.pairs, swap);
            }
            if (row < rows) {
                if (l.has_a) Unit::put(y + l.ca, q);
                if (l.has_b) Unit::put(y + l.cb, q + 4);
                y += l.step * part.ys[2];
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (kBack) {
        if (p.sums != nullptr) {
            float* sums = reinterpret_cast<float*>(ring);  // [warps][kQkMaxD]
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                float s = (k & 1) != 0 ? acc[k >> 1].y : acc[k >> 1].x;
                for (int o = l.group; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane < l.group && (k < 8 ? l.has_a : l.has_b)) sums[warp * kQkMaxD + (k < 8 ? l.ca + k : l.cb + k - 8)] = s;
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.d; c += kQkThreads) {
                float s = 0.f;
                for (int k = 0; k < kQkWarps; ++k) s += sums[k * kQkMaxD + c];
                p.sums[static_cast<long long>(blockIdx.x) * p.d + c] = s;
            }
        }
    }
    pdl_launch_dependents();
}

// dgamma: the blocks' sums, 32 channels a block, 32 runs of them side by side. The queries' sums are the first `qblocks`
// rows, the keys' those from `kfirst` to `kend`.
__global__ void __launch_bounds__(1024) qk_join_kernel(const float* sums, int qblocks, int kfirst, int kend, int d, float* dgamma_q,
                                                       float* dgamma_k) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int w = blockIdx.y, c = static_cast<int>(blockIdx.x) * 32 + lane;
    const int end = w == 0 ? qblocks : kend;
    pdl_wait();
    float s = 0.f;
    if (c < d)
        for (int b = (w == 0 ? 0 : kfirst) + run; b < end; b += 32) s += sums[static_cast<long long>(b) * d + c];
    part[run][lane] = s;
    __syncthreads();
    s = warp_sum(part[lane][run]);  // (the transposed warp: run is the channel here)
    if (const int ch = static_cast<int>(blockIdx.x) * 32 + run; lane == 0 && ch < d) (w == 0 ? dgamma_q : dgamma_k)[ch] = s;
}

bool qk_vectors(const QkParams& p) {
    // Vectors where every row starts on 16 bytes and holds whole ones (a warp a row, channel by channel, otherwise)
    bool v8 = p.d % 8 == 0;
    for (const QkPart& t : p.part) {
        v8 = v8 && aligned16(t.x) && aligned16(t.dy) && aligned16(t.y);
        for (int i = 0; i < 3; ++i) v8 = v8 && t.xs[i] % 8 == 0 && t.gs[i] % 8 == 0 && t.ys[i] % 8 == 0;
    }
    return v8;
}

// The form that takes a plan's pairs, and log2 of the lanes that a row of d channels lies over.
struct QkForm {
    int form, glog2;
};
QkForm qk_form(int d, const vae_rope_plan& plan) {
    const bool halves = plan.pairs > 0 && !plan.interleaved;
    QkForm f{!halves ? kLocal : plan.pairs % 8 == 0 ? kHalves : kSwap, 0};
    const int lanes = f.form == kHalves ? plan.pairs / 8 + (d - 2 * plan.pairs + 15) / 16 : (d + 15) / 16;
    while ((1 << f.glog2) < lanes) ++f.glog2;
    return f;
}

template <int T, bool kBack>
cudaError_t qk_launch_type(unsigned grid, cudaStream_t s, const QkParams& p, const vae_rope_plan& plan) {
    if (!qk_vectors(p)) return launch_kernel(qk_plain_kernel<T, kBack>, dim3(grid), dim3(kQkThreads), 0, s, p, plan);
    const auto [form, glog2] = qk_form(p.d, plan);
    const auto go = [&, lanes = glog2](auto k) { return launch_kernel(k, dim3(grid), dim3(kQkThreads), QkRing<T, kBack>::kBytes, s, p, plan, lanes); };
    if (form == kLocal) return go(qk_vector_kernel<T, kLocal, kBack>);
    return form == kHalves ? go(qk_vector_kernel<T, kHalves, kBack>) : go(qk_vector_kernel<T, kSwap, kBack>);
}
template <bool kBack>
cudaError_t qk_launch(int type, unsigned grid, cudaStream_t s, const QkParams& p, const vae_rope_plan& plan) {
    if (type == VAE_F32) return qk_launch_type<VAE_F32, kBack>(grid, s, p, plan);
    return type == VAE_F16 ? qk_launch_type<VAE_F16, kBack>(grid, s, p, plan) : qk_launch_type<VAE_BF16, kBack>(grid, s, p, plan);
}

// A tensor of a call: what it is and whether it may be another one (given by its name and the same strides).
struct QkTensor {
    const char* name;
    const void* p;
    Extent at;
    bool written;
    const long long* stride;  // nullptr: dense
    const void *own0, *own1;  // inputs that a written tensor may be
    const long long *own0_stride, *own1_stride;
};

int qk_apart(const vae_qk_norm_rope_desc* a, const QkTensor* t, int count) {
    for (int i = 0; i < count; ++i) {
        if (t[i].p == nullptr || !t[i].written) continue;
        for (int j = 0; j < count; ++j) {
            if (j == i || t[j].p == nullptr || (t[j].written && j < i)) continue;
            if (t[j].p == t[i].p && (t[j].p == t[i].own0 || t[j].p == t[i].own1)) {
                const int dim[3] = {a->b, a->s, static_cast<int>(t[i].at.n[2])};
                const long long* st = t[j].stride;
                bool same = st != nullptr && t[j].at.n[2] == t[i].at.n[2] && (st == t[i].own0_stride || st == t[i].own1_stride);
                for (int k = 0; same && k < 3; ++k) same = dim[k] == 1 || st[k] == t[i].stride[k];
                if (same) continue;
                if (st != nullptr && (st == t[i].own0_stride || st == t[i].own1_stride))
                    return set_error(VAE_ERR_ARG, "qk norm: %s over %s needs the same strides", t[i].name, t[j].name);
            }
            if (extents_meet(t[i].at, t[j].at))
                return set_error(VAE_ERR_ARG, "qk norm: %s may not overlap %s", t[i].name, t[j].name);
        }
    }
    return VAE_OK;
}

int qk_check(const vae_qk_norm_rope_desc* a, bool backward) {
    if (a == nullptr) return set_error(VAE_ERR_ARG, "qk norm: NULL desc");
    if (!type_ok(a->type)) return set_error(VAE_ERR_ARG, "qk norm: unknown element type");
    if (a->b < 1 || a->s < 1 || a->hq < 1 || a->hk < 1)
        return set_error(VAE_ERR_SHAPE, "qk norm: b, s, hq, hk >= 1 are needed");
    if (static_cast<long long>(a->b) * a->s > 0x7fffff00LL || static_cast<long long>(a->hq) + a->hk >= (1 << 20))
        return set_error(VAE_ERR_SHAPE, "qk norm: over 2^31 - 256 tokens or 2^20 - 1 heads");
    if (a->d < 1 || a->d > kQkMaxD) return set_error(VAE_ERR_SHAPE, "qk norm: 1 <= d <= %d, got %d", kQkMaxD, a->d);
    if (!(a->eps > 0.f) || !std::isfinite(a->eps)) return set_error(VAE_ERR_ARG, "qk norm: eps must be > 0 and finite");
    const struct {
        const char* name;
        const long long* st;
        int h;
        bool written;
    } t[6] = {{"q", a->q_stride, a->hq, false},         {"k", a->k_stride, a->hk, false},
              {"q_out", a->q_out_stride, a->hq, true},  {"k_out", a->k_out_stride, a->hk, true},
              {"dq_out", a->dq_out_stride, a->hq, false}, {"dk_out", a->dk_out_stride, a->hk, false}};
    for (int i = 0; i < (backward ? 6 : 4); ++i) {
        const int dim[3] = {a->b, a->s, t[i].h};
        for (int k = 0; k < 3; ++k)
            if (t[i].st[k] < 0 || t[i].st[k] >= (1LL << 38) || (t[i].written && dim[k] > 1 && t[i].st[k] == 0))
                return set_error(VAE_ERR_SHAPE, "qk norm: %s's strides must be >= 0 (> 0 where it is written) and below 2^38", t[i].name);
        if (t[i].written && extent_folds(extent_tokens(nullptr, t[i].st, a->b, a->s, t[i].h, a->d, type_size(a->type))))
            return set_error(VAE_ERR_SHAPE, "qk norm: rows of %s lie in one another", t[i].name);
    }
    return VAE_OK;
}

int qk_check_plan(const vae_qk_norm_rope_desc* a, const void* pos, const vae_rope_plan* plan) {
    if ((pos == nullptr) != (plan == nullptr)) return set_error(VAE_ERR_ARG, "qk norm: positions and plan come together");
    if (plan == nullptr) return VAE_OK;
    if (plan->naxes < 1 || plan->naxes > 4 || plan->pairs < 1 || plan->pairs > VAE_ROPE_MAX_PAIRS)
        return set_error(VAE_ERR_ARG, "qk norm: the plan was not initialised");
    for (int i = 0; i < plan->pairs; ++i)
        if (plan->axis[i] >= plan->naxes) return set_error(VAE_ERR_ARG, "qk norm: the plan was not initialised");
    if (2 * plan->pairs > a->d)
        return set_error(VAE_ERR_SHAPE, "qk norm: the plan turns %d channels of a head of %d", 2 * plan->pairs, a->d);
    if (a->pos_batch != 1 && a->pos_batch != a->b)
        return set_error(VAE_ERR_SHAPE, "qk norm: positions of %d batch entries for a batch of %d", a->pos_batch, a->b);
    if (reinterpret_cast<uintptr_t>(pos) % 4) return set_error(VAE_ERR_ALIGN, "qk norm: positions are not aligned");
    return VAE_OK;
}

int qk_tiles(const vae_qk_norm_rope_desc* a, int* tpb) {
    const int tokens = a->b * a->s;
    // as many tokens as share one table, down to one when there are too few to give every SM a block
    *tpb = kQkTokens;
    while (*tpb > 1 && tokens / 304 < *tpb) *tpb /= 2;
    return (tokens - 1) / *tpb + 1;
}

// In vectors the queries and the keys have blocks of their own, `most` in all, shared out by what their turns cost: the rows
// of a group of lanes, and as much as kTurnRows rows for the angles and the barriers (36864 tokens of 32 heads and one of
// 128, bf16, with 0, 2, 4, 8: 245, 133, 110, 111 us, the gradient 461, 219, 176, 163; of 24 and 8 heads 119, 106, 104, 101
// and 174, 164, 161, 154).
constexpr int kTurnRows = 8;
int qk_share(const vae_qk_norm_rope_desc& a, const vae_rope_plan& plan, int tpb, int tiles, int most, int* qblocks) {
    const int step = (kQkThreads >> qk_form(a.d, plan).glog2) / tpb;
    const long long wq = (a.hq - 1) / step + 1 + kTurnRows, wk = (a.hk - 1) / step + 1 + kTurnRows;
    const int all = static_cast<int>(std::min<long long>(2LL * tiles, most));
    const int q = static_cast<int>((all * wq + (wq + wk) / 2) / (wq + wk));
    *qblocks = std::min(std::max(q, 1), std::min(all - 1, tiles));
    return *qblocks + std::min(all - *qblocks, tiles);
}

void qk_fill(const vae_qk_norm_rope_desc* a, QkParams* p, const void* q, const void* k, const void* gq, const void* gk, void* yq,
             void* yk, const float* gamma_q, const float* gamma_k, const void* pos) {
    const int dim[2][3] = {{a->b, a->s, a->hq}, {a->b, a->s, a->hk}};
    const long long* st[2][3] = {{a->q_stride, a->dq_out_stride, a->q_out_stride}, {a->k_stride, a->dk_out_stride, a->k_out_stride}};
    const void* x[2][2] = {{q, gq}, {k, gk}};
    void* y[2] = {yq, yk};
    for (int w = 0; w < 2; ++w) {
        QkPart& t = p->part[w];
        t.x = x[w][0];
        t.dy = x[w][1];
        t.y = y[w];
        t.gamma = w == 0 ? gamma_q : gamma_k;
        t.h = dim[w][2];
        for (int i = 0; i < 3; ++i) {
            const bool many = dim[w][i] > 1;
            t.xs[i] = many ? st[w][0][i] : 0;
            t.gs[i] = many && gq != nullptr ? st[w][1][i] : 0;
            t.ys[i] = many ? st[w][2][i] : 0;
        }
    }
    p->pos = pos;
    p->tokens = a->b * a->s;
    p->s = a->s;
    p->d = a->d;
    p->pos_int = a->pos_int != 0;
    p->pos_batch = a->pos_batch;
    p->eps = a->eps;
}

bool qk_aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" {

int vae_qk_norm_rope(const vae_qk_norm_rope_desc* desc, const void* q_dev, const void* k_dev, const float* gamma_q_dev,
                     const float* gamma_k_dev, const void* pos_dev, const vae_rope_plan* plan, void* q_out_dev,
                     void* k_out_dev, vae_stream_t stream) {
    clear_error();
    int rc = qk_check(desc, false);
    if (rc != VAE_OK) return rc;
    if (q_dev == nullptr || k_dev == nullptr || q_out_dev == nullptr || k_out_dev == nullptr)
        return set_error(VAE_ERR_ARG, "qk norm: NULL tensor");
    rc = qk_check_plan(desc, pos_dev, plan);
    if (rc != VAE_OK) return rc;
    const vae_qk_norm_rope_desc& a = *desc;
    const size_t es = type_size(a.type);
    if (!qk_aligned(q_dev, es) || !qk_aligned(k_dev, es) || !qk_aligned(q_out_dev, es) || !qk_aligned(k_out_dev, es) ||
        !qk_aligned(gamma_q_dev, 4) || !qk_aligned(gamma_k_dev, 4))
        return set_error(VAE_ERR_ALIGN, "qk norm: a pointer is not aligned to its elements");
    const auto heads = [&](const void* p, const long long* st, int h) { return extent_tokens(p, st, a.b, a.s, h, a.d, es); };
    const QkTensor t[] = {
        {"q_out", q_out_dev, heads(q_out_dev, a.q_out_stride, a.hq), true, a.q_out_stride, q_dev, nullptr, a.q_stride, nullptr},
        {"k_out", k_out_dev, heads(k_out_dev, a.k_out_stride, a.hk), true, a.k_out_stride, k_dev, nullptr, a.k_stride, nullptr},
        {"q", q_dev, heads(q_dev, a.q_stride, a.hq), false, a.q_stride},
        {"k", k_dev, heads(k_dev, a.k_stride, a.hk), false, a.k_stride},
        {"gamma_q", gamma_q_dev, extent_dense(gamma_q_dev, a.d * 4u), false},
        {"gamma_k", gamma_k_dev, extent_dense(gamma_k_dev, a.d * 4u), false},
        {"the positions", pos_dev, extent_dense(pos_dev, plan != nullptr ? static_cast<size_t>(a.pos_batch) * a.s * plan->naxes * 4 : 0), false}};
    rc = qk_apart(desc, t, 7);
    if (rc != VAE_OK) return rc;
    rc = check_device();
    if (rc != VAE_OK) return rc;
    QkParams p{};
    qk_fill(desc, &p, q_dev, k_dev, nullptr, nullptr, q_out_dev, k_out_dev, gamma_q_dev, gamma_k_dev, pos_dev);
    int grid = qk_tiles(desc, &p.tpb);
    const vae_rope_plan none{};
    const vae_rope_plan& pl = plan != nullptr ? *plan : none;
    if (qk_vectors(p)) grid = qk_share(a, pl, p.tpb, grid, kQkForward, &p.qblocks);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    VAE_CUDA_CHECK(qk_launch<false>(a.type, static_cast<unsigned>(grid), st, p, pl));
    return VAE_OK;
}

size_t vae_qk_norm_rope_backward_workspace_bytes(const vae_qk_norm_rope_desc* desc) {
    clear_error();
    if (qk_check(desc, true) != VAE_OK) return 0;
    int tpb;
    return static_cast<size_t>(std::min(qk_tiles(desc, &tpb), kQkBlocks)) * 2 * desc->d * sizeof(float);
}

int vae_qk_norm_rope_backward(const vae_qk_norm_rope_desc* desc, const void* dq_out_dev, const void* dk_out_dev,
                              const void* q_dev, const void* k_dev, const float* gamma_q_dev, const float* gamma_k_dev,
                              const void* pos_dev, const vae_rope_plan* plan, void* dq_dev, void* dk_dev,
                              float* dgamma_q_dev, float* dgamma_k_dev, void* workspace_dev, size_t workspace_bytes,
                              vae_stream_t stream) {
    clear_error();
    int rc = qk_check(desc, true);
    if (rc != VAE_OK) return rc;
    if (dq_out_dev == nullptr || dk_out_dev == nullptr || q_dev == nullptr || k_dev == nullptr || dq_dev == nullptr ||
        dk_dev == nullptr)
        return set_error(VAE_ERR_ARG, "qk norm: NULL tensor");
    rc = qk_check_plan(desc, pos_dev, plan);
    if (rc != VAE_OK) return rc;
    const vae_qk_norm_rope_desc& a = *desc;
    const bool weights = dgamma_q_dev != nullptr;
    if (weights != (dgamma_k_dev != nullptr)) return set_error(VAE_ERR_ARG, "qk norm: dgamma_q and dgamma_k come together");
    const size_t es = type_size(a.type), need = vae_qk_norm_rope_backward_workspace_bytes(desc);
    if (!qk_aligned(dq_out_dev, es) || !qk_aligned(dk_out_dev, es) || !qk_aligned(q_dev, es) || !qk_aligned(k_dev, es) ||
        !qk_aligned(dq_dev, es) || !qk_aligned(dk_dev, es) || !qk_aligned(gamma_q_dev, 4) || !qk_aligned(gamma_k_dev, 4) ||
        !qk_aligned(dgamma_q_dev, 4) || !qk_aligned(dgamma_k_dev, 4))
        return set_error(VAE_ERR_ALIGN, "qk norm: a pointer is not aligned to its elements");
    if (weights) {
        if (workspace_dev == nullptr) return set_error(VAE_ERR_ARG, "qk norm: a workspace is needed for dgamma");
        if (workspace_bytes < need)
            return set_error(VAE_ERR_NOMEM, "qk norm: workspace of %zu bytes, %zu are needed", workspace_bytes, need);
        if (!aligned16(workspace_dev)) return set_error(VAE_ERR_ALIGN, "qk norm: the workspace must be 16-byte aligned");
    }
    const auto heads = [&](const void* p, const long long* st, int h) { return extent_tokens(p, st, a.b, a.s, h, a.d, es); };
    const QkTensor t[] = {
        {"dq", dq_dev, heads(dq_dev, a.q_out_stride, a.hq), true, a.q_out_stride, q_dev, dq_out_dev, a.q_stride, a.dq_out_stride},
        {"dk", dk_dev, heads(dk_dev, a.k_out_stride, a.hk), true, a.k_out_stride, k_dev, dk_out_dev, a.k_stride, a.dk_out_stride},
        {"dgamma_q", dgamma_q_dev, extent_dense(dgamma_q_dev, a.d * 4u), true},
        {"dgamma_k", dgamma_k_dev, extent_dense(dgamma_k_dev, a.d * 4u), true},
        {"the workspace", weights ? workspace_dev : nullptr, extent_dense(workspace_dev, need), true},
        {"q", q_dev, heads(q_dev, a.q_stride, a.hq), false, a.q_stride},
        {"k", k_dev, heads(k_dev, a.k_stride, a.hk), false, a.k_stride},
        {"dq_out", dq_out_dev, heads(dq_out_dev, a.dq_out_stride, a.hq), false, a.dq_out_stride},
        {"dk_out", dk_out_dev, heads(dk_out_dev, a.dk_out_stride, a.hk), false, a.dk_out_stride},
        {"gamma_q", gamma_q_dev, extent_dense(gamma_q_dev, a.d * 4u), false},
        {"gamma_k", gamma_k_dev, extent_dense(gamma_k_dev, a.d * 4u), false},
        {"the positions", pos_dev, extent_dense(pos_dev, plan != nullptr ? static_cast<size_t>(a.pos_batch) * a.s * plan->naxes * 4 : 0), false}};
    rc = qk_apart(desc, t, 12);
    if (rc != VAE_OK) return rc;
    rc = check_device();
    if (rc != VAE_OK) return rc;
    QkParams p{};
    qk_fill(desc, &p, q_dev, k_dev, dq_out_dev, dk_out_dev, dq_dev, dk_dev, gamma_q_dev, gamma_k_dev, pos_dev);
    int tiles = qk_tiles(desc, &p.tpb);
    int grid = std::min(tiles, kQkBlocks), qblocks = grid, kend = 2 * grid;
    const vae_rope_plan none{};
    const vae_rope_plan& pl = plan != nullptr ? *plan : none;
    if (qk_vectors(p)) {
        if (p.tpb == kQkTokens && p.tokens / 608 >= kQkTokens && a.type != VAE_F32 && qk_form(a.d, pl).glog2 <= 3) {
            p.tpb = 2 * kQkTokens;
            tiles = (p.tokens - 1) / p.tpb + 1;
        }
        grid = kend = qk_share(a, pl, p.tpb, tiles, kQkBlocks, &qblocks);
    }
    p.qblocks = qblocks;
    p.sums = weights ? static_cast<float*>(workspace_dev) : nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    VAE_CUDA_CHECK(qk_launch<true>(a.type, static_cast<unsigned>(grid), st, p, pl));
    if (weights)
        VAE_CUDA_CHECK(launch_next(qk_join_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, st,
                                   static_cast<const float*>(p.sums), qblocks, qblocks, kend, a.d, dgamma_q_dev, dgamma_k_dev));
    return VAE_OK;
}

}  // extern "C"
