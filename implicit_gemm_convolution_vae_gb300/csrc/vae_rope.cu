// Rotary positions over several axes (public entry points at the end).
//
// A block computes the (cos, sin) of its tokens' pairs once in shared memory,
// then turns every head of those tokens: one read and one write of the tensor,
// which bounds the call. Measured on GB300 at 36864 tokens x 18 heads x 128 in f16 (340 MB): 70 us
// interleaved (4.9 TB/s), 60 us in halves (5.7 TB/s). Small blocks, so that the
// angles of some are formed while others move rows: 8 tokens, 128 threads, 12
// blocks an SM and two rows a thread in flight; 32 tokens and four blocks of 256
// threads with four rows in flight took 75 and 66 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vae_overlap.h"
#include "vae_rope.cuh"
#include "vae_types.cuh"

namespace vae {

namespace {

constexpr int kRopeMaxD = 256;
constexpr int kRopeTokens = 8;  // tokens per block, at most
// Threads of a block: a row's units (up to 255 one by one, 32 in vectors) have to fit.
__host__ __device__ constexpr int rope_threads(int unit) { return unit > 1 ? 128 : 256; }
constexpr int kRopePitch = VAE_ROPE_MAX_PAIRS + 2;  // of a token's (cos, sin) row: 16-byte aligned, few bank conflicts

struct RopeParams {
    const void* x;
    void* y;
    const void* pos;
    int tokens;        // b * s
    int s, h, d, tpb;  // tpb: tokens per block
    int pos_int, pos_batch, inverse;
    long long xs[3], ys[3];
};

// A unit as it lies in memory: sixteen or eight elements, or one.
template <int T, int kN>
struct RopeUnit {
    static constexpr bool kV8 = kN > 1;
    static constexpr int kRegs = kV8 ? (T == VAE_F32 ? kN / 4 : kN / 8) : 1;
    using Reg = std::conditional_t<kV8, uint4, typename Elem<T>::type>;
    Reg r[kRegs];
    __device__ __forceinline__ void load(const typename Elem<T>::type* p) {
#pragma unroll
        for (int i = 0; i < kRegs; ++i) r[i] = reinterpret_cast<const Reg*>(p)[i];
    }
    __device__ __forceinline__ void store(typename Elem<T>::type* p) const {
#pragma unroll
        for (int i = 0; i < kRegs; ++i) reinterpret_cast<Reg*>(p)[i] = r[i];
    }
    __device__ __forceinline__ void get(float (&v)[kN]) const {
        if constexpr (kV8) {
#pragma unroll
            for (int i = 0; i < kN / 8; ++i) load8<T>(r + i * kRegs / (kN / 8), *reinterpret_cast<float(*)[8]>(v + 8 * i));
        } else {
            v[0] = to_f32<T>(r[0]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[kN]) {
        if constexpr (kV8) {
#pragma unroll
            for (int i = 0; i < kN / 8; ++i) store8<T>(r + i * kRegs / (kN / 8), *reinterpret_cast<const float(*)[8]>(v + 8 * i));
        } else {
            r[0] = from_f32<T>(v[0]);
        }
    }
};

// kN: channels of a unit, 16 (interleaved) or 8 in 16-byte accesses, or 1.
// kInter: pairs (2p, 2p + 1), else (p, p + R/2).
// A row is one head of one token. Its units (vectors of interleaved pairs, or
// those of both halves, or both of a pair, together; then the copied ones: a
// thread turns 16 or 32 bytes a row) go to threads side by side, and a thread keeps its unit on every row it
// meets. The first rows are on their way while the angles are formed.
template <int T, int kN, bool kInter>
__global__ void __launch_bounds__(rope_threads(kN), 1536 / rope_threads(kN)) rope_kernel(const RopeParams p, const __grid_constant__ vae_rope_plan plan) {
    using E = typename Elem<T>::type;
    using Unit = RopeUnit<T, kN>;
    constexpr int kThreads = rope_threads(kN);
    constexpr bool kV8 = kN > 1;
    constexpr bool kTwo = !(kV8 && kInter);  // two units turn together
    constexpr int kRopeBatch = 2;  // rows whose loads a thread has in flight together
    __shared__ __align__(16) float2 cs[kRopeTokens][kRopePitch];
    pdl_wait();
    const int t0 = static_cast<int>(blockIdx.x) * p.tpb;
    const int nt = p.tokens - t0 < p.tpb ? p.tokens - t0 : p.tpb;
    const int b0 = t0 / p.s, s0 = t0 - b0 * p.s;
    const int pairs = plan.pairs, rot = 2 * pairs;
    const int nrot = kTwo ? pairs / kN : rot / kN;
    const int units = nrot + (p.d - rot) / kN;  // (kThreads at most)
    const int step = kThreads / units;          // rows that the block takes at a time
    const int u = threadIdx.x % units;
    const bool copied = u >= nrot;
    const int ia = copied ? rot + (u - nrot) * kN : (!kV8 && kInter ? 2 * u : u * kN);
    const int ib = kV8 ? ia + pairs : (kInter ? ia + 1 : ia + pairs);
    int hd = threadIdx.x / units, tk = hd < step ? 0 : nt;
    auto settle = [&]() {
        while (tk < nt && hd >= p.h) {
            hd -= p.h;
            ++tk;
        }
    };
    settle();
    auto offset = [&](int tok, int head, const long long (&st)[3]) {
        int si = s0 + tok, bi = b0;
        while (si >= p.s) {
            si -= p.s;
            ++bi;
        }
        return bi * st[0] + si * st[1] + head * st[2];
    };
    Unit a[kRopeBatch], b[kTwo ? kRopeBatch : 1];
    int at[kRopeBatch];  // the rows: token << 20 | head
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            at[k] = tk << 20 | hd;
            if (tk < nt) {
                const E* x = static_cast<const E*>(p.x) + offset(tk, hd, p.xs);
                a[k].load(x + ia);
                if constexpr (kTwo)
                    if (!copied) b[k].load(x + ib);
                hd += step;
                settle();
            }
        }
    };
    load();
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        // neighbours take the tokens of one pair: its entries of the plan are one address for them, and the constant
        // bank serves one address at a time (a pair per lane took 3/4 of the call on few heads)
        const int pr = i / nt, t = i - pr * nt;
        const long long row = p.pos_batch > 1 ? t0 + t : (s0 + t) % p.s;
        const long long i_pos = row * plan.naxes + plan.axis[pr];
        const float pos = p.pos_int ? static_cast<float>(static_cast<const int*>(p.pos)[i_pos])
                                    : static_cast<const float*>(p.pos)[i_pos];
        const float2 c = rope_cos_sin(plan, pr, pos);
        cs[t][pr] = make_float2(c.x, p.inverse ? -c.y : c.y);
    }
    __syncthreads();
    while (at[0] >> 20 < nt) {
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k)
            if (const int t = at[k] >> 20; t < nt) {
                E* y = static_cast<E*>(p.y) + offset(t, at[k] & 0xfffff, p.ys);
                if (!copied) {
                    float v[kN];
                    a[k].get(v);
                    if constexpr (kTwo) {
                        float w[kN];
                        b[k].get(w);
#pragma unroll
                        for (int e = 0; e < kN; ++e) turn(v[e], w[e], cs[t][u * kN + e]);
                        b[k].set(w);
                        b[k].store(y + ib);
                    } else {
#pragma unroll
                        for (int e = 0; e < kN / 2; ++e) turn(v[2 * e], v[2 * e + 1], cs[t][u * (kN / 2) + e]);
                    }
                    a[k].set(v);
                }
                a[k].store(y + ia);
            }
        load();
    }
}

template <int T>
cudaError_t rope_launch(int unit, bool inter, unsigned grid, cudaStream_t s, const RopeParams& p,
                        const vae_rope_plan& plan) {
    const auto go = [&](auto k) { return launch_kernel(k, dim3(grid), dim3(rope_threads(unit)), 0, s, p, plan); };
    if constexpr (T != VAE_F32)
        if (unit == 16) return go(rope_kernel<T, 16, true>);
    if (unit == 8) return inter ? go(rope_kernel<T, 8, true>) : go(rope_kernel<T, 8, false>);
    return inter ? go(rope_kernel<T, 1, true>) : go(rope_kernel<T, 1, false>);
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" {

int vae_rope_plan_init(vae_rope_plan* plan, int naxes, const int* dims, double theta, int interleaved) {
    clear_error();
    if (plan == nullptr || dims == nullptr) return set_error(VAE_ERR_ARG, "rope plan: NULL argument");
    if (naxes < 1 || naxes > 4) return set_error(VAE_ERR_SHAPE, "rope plan: 1 to 4 axes, got %d", naxes);
    if (!(theta >= 1.0) || !std::isfinite(theta))
        return set_error(VAE_ERR_ARG, "rope plan: theta must be >= 1 and finite");
    long long total = 0;
    for (int a = 0; a < naxes; ++a) {
        if (dims[a] < 0 || dims[a] % 2 != 0)
            return set_error(VAE_ERR_SHAPE, "rope plan: axis %d has %d channels; an even number >= 0 is needed", a,
                             dims[a]);
        total += dims[a];
    }
    if (total < 2 || total > kRopeMaxD)
        return set_error(VAE_ERR_SHAPE, "rope plan: 2 to %d channels turn, got %lld", kRopeMaxD, total);
    *plan = vae_rope_plan{};
    plan->naxes = naxes;
    plan->pairs = static_cast<int>(total / 2);
    plan->interleaved = interleaved != 0;
    int k = 0;
    for (int a = 0; a < naxes; ++a)
        for (int i = 0; i < dims[a] / 2; ++i, ++k) {
            const double turns = std::pow(theta, -2.0 * i / dims[a]) / 6.283185307179586476925286766559;
            plan->turns_hi[k] = static_cast<float>(turns);
            plan->turns_lo[k] = static_cast<float>(turns - static_cast<double>(plan->turns_hi[k]));
            plan->axis[k] = static_cast<unsigned char>(a);
        }
    return VAE_OK;
}

int vae_rope(const void* x_dev, int type, int b, int s, int h, int d, const long long x_stride[3],
             const void* pos_dev, int pos_int, int pos_batch, const vae_rope_plan* plan, int inverse, void* y_dev,
             const long long y_stride[3], vae_stream_t stream) {
    clear_error();
    if (x_dev == nullptr || y_dev == nullptr || pos_dev == nullptr || plan == nullptr || x_stride == nullptr ||
        y_stride == nullptr)
        return set_error(VAE_ERR_ARG, "rope: NULL argument");
    if (!type_ok(type)) return set_error(VAE_ERR_ARG, "rope: unknown element type");
    if (plan->naxes < 1 || plan->naxes > 4 || plan->pairs < 1 || plan->pairs > VAE_ROPE_MAX_PAIRS)
        return set_error(VAE_ERR_ARG, "rope: the plan was not initialised");
    for (int i = 0; i < plan->pairs; ++i)
        if (plan->axis[i] >= plan->naxes) return set_error(VAE_ERR_ARG, "rope: the plan was not initialised");
    if (b < 1 || s < 1 || h < 1) return set_error(VAE_ERR_SHAPE, "rope: b, s, h >= 1 are needed");
    if (static_cast<long long>(b) * s > 0x7fffff00LL || h >= (1 << 20))
        return set_error(VAE_ERR_SHAPE, "rope: over 2^31 - 256 tokens or 2^20 - 1 heads");
    if (d > kRopeMaxD || 2 * plan->pairs > d)
        return set_error(VAE_ERR_SHAPE, "rope: the plan turns %d channels of a head of %d (at most %d)",
                         2 * plan->pairs, d, kRopeMaxD);
    if (pos_batch != 1 && pos_batch != b)
        return set_error(VAE_ERR_SHAPE, "rope: positions of %d batch entries for a batch of %d", pos_batch, b);
    const int dim[3] = {b, s, h};
    for (int i = 0; i < 3; ++i)
        if (x_stride[i] < 0 || y_stride[i] < 0 || (dim[i] > 1 && y_stride[i] == 0))
            return set_error(VAE_ERR_SHAPE, "rope: strides must be >= 0, and y's > 0");
    if (x_dev == y_dev)
        for (int i = 0; i < 3; ++i)
            if (dim[i] > 1 && x_stride[i] != y_stride[i])
                return set_error(VAE_ERR_ARG, "rope: in place needs the same strides");
    const size_t es = type_size(type);
    if (reinterpret_cast<uintptr_t>(x_dev) % es || reinterpret_cast<uintptr_t>(y_dev) % es ||
        reinterpret_cast<uintptr_t>(pos_dev) % 4)
        return set_error(VAE_ERR_ALIGN, "rope: a pointer is not aligned to its elements");
    const Extent y_at = extent_tokens(y_dev, y_stride, b, s, h, d, es);
    if (extent_folds(y_at)) return set_error(VAE_ERR_SHAPE, "rope: rows of y lie in one another");
    if (x_dev != y_dev && extents_meet(extent_tokens(x_dev, x_stride, b, s, h, d, es), y_at))
        return set_error(VAE_ERR_ARG, "rope: y may not overlap x (but may be x)");
    if (extents_meet(extent_dense(pos_dev, static_cast<size_t>(pos_batch) * s * plan->naxes * 4), y_at))
        return set_error(VAE_ERR_ARG, "rope: y may not overlap the positions");
    int rc = check_device();
    if (rc != VAE_OK) return rc;
    RopeParams p{};
    p.x = x_dev;
    p.y = y_dev;
    p.pos = pos_dev;
    p.tokens = b * s;
    p.s = s;
    p.h = h;
    p.d = d;
    p.pos_int = pos_int != 0;
    p.pos_batch = pos_batch;
    p.inverse = inverse != 0;
    // Vectors where every row starts on 16 bytes and holds whole ones. Interleaved 16-bit pairs: sixteen channels a
    // thread where they fit (340 MB with blocks of 256: 74.6 us against 80.7 with eight; f32, 57 MB: 32.4 against 28.2,
    // and keeps eight).
    bool v8 = aligned16(x_dev) && aligned16(y_dev) && d % 8 == 0 &&
              (plan->interleaved ? 2 * plan->pairs : plan->pairs) % 8 == 0;
    for (int i = 0; i < 3; ++i) {
        p.xs[i] = dim[i] > 1 ? x_stride[i] : 0;
        p.ys[i] = dim[i] > 1 ? y_stride[i] : 0;
        v8 = v8 && p.xs[i] % 8 == 0 && p.ys[i] % 8 == 0;
    }
    // Tokens per block: as many as share one (cos, sin) table, down to one when
    // there are too few tokens to give every SM a block.
    p.tpb = std::min(kRopeTokens, std::max(1, p.tokens / 304));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned g = static_cast<unsigned>((p.tokens - 1) / p.tpb + 1);
    const bool in = plan->interleaved != 0;
    const int unit = !v8 ? 1 : (in && type != VAE_F32 && d % 16 == 0 && plan->pairs % 8 == 0 ? 16 : 8);
    VAE_CUDA_CHECK(type == VAE_F32   ? rope_launch<VAE_F32>(unit, in, g, st, p, *plan)
                   : type == VAE_F16 ? rope_launch<VAE_F16>(unit, in, g, st, p, *plan)
                                     : rope_launch<VAE_BF16>(unit, in, g, st, p, *plan));
    return VAE_OK;
}

}  // extern "C"
