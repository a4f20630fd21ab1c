// Rotary positions over several axes (public entry points at the end).
//
// The angle of pair p at position t is 2 pi t f_p with f_p turns per position.
// f_p comes from the host in two floats (hi + lo, 48 bits), so t f_hi is split
// exactly by one fma into whole turns and a fraction, t f_lo is added to the
// fraction, and sincospi of twice the fraction follows: far positions lose no
// digits and no 64-bit arithmetic runs on the device. A block computes the
// (cos, sin) of its tokens' pairs once in shared memory, then turns every head
// of those tokens: one read and one write of the tensor, which bounds the call.
#include <algorithm>
#include <cmath>

#include "vae_types.cuh"

namespace vae {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;
constexpr int kRopeTokens = 8;  // tokens per block, at most

struct RopeParams {
    const void* x;
    void* y;
    const void* pos;
    long long tokens;  // b * s
    int s, h, d, tpb;  // tpb: tokens per block
    int pos_int, pos_batch, inverse;
    long long xs[3], ys[3];
};

// Turns (a, b) by (cos, sin).
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
    const float x = a * cs.x - b * cs.y;
    b = a * cs.y + b * cs.x;
    a = x;
}

// kV8: eights of channels in 16-byte accesses; else one pair (or one copied
// channel) at a time. kInter: pairs (2p, 2p + 1), else (p, p + R/2).
template <int T, bool kV8, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, const __grid_constant__ vae_rope_plan plan) {
    using E = typename Elem<T>::type;
    __shared__ float2 cs[kRopeTokens][VAE_ROPE_MAX_PAIRS];
    pdl_wait();
    const long long t0 = static_cast<long long>(blockIdx.x) * p.tpb;
    const int nt = static_cast<int>(p.tokens - t0 < p.tpb ? p.tokens - t0 : p.tpb);
    const int pairs = plan.pairs;
    for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
        const int tk = i / pairs, pr = i - tk * pairs;
        const long long tok = t0 + tk;
        const long long prow = p.pos_batch > 1 ? tok : tok % p.s;
        const long long at = prow * plan.naxes + plan.axis[pr];
        const float pos = p.pos_int ? static_cast<float>(static_cast<const int*>(p.pos)[at])
                                    : static_cast<const float*>(p.pos)[at];
        // whole turns + fraction of pos * hi (the fma's product is exact), then the rest
        const float hi = plan.turns_hi[pr];
        const float whole = rintf(pos * hi);
        const float frac = fmaf(pos, hi, -whole) + pos * plan.turns_lo[pr];
        float sn, c;
        sincospif(2.f * frac, &sn, &c);
        cs[tk][pr] = make_float2(c, p.inverse ? -sn : sn);
    }
    __syncthreads();
    const int rot = 2 * pairs;
    // units of one token and head: kV8 interleaved: d / 8 eights; kV8 halves: the
    // eights of a pair of halves together, then the copied eights; scalar: pairs, then copied channels
    const int nrot = kV8 ? (kInter ? rot / 8 : pairs / 8) : pairs;
    const int units = nrot + (kV8 ? (p.d - rot) / 8 : p.d - rot);
    const int per_tok = p.h * units;
    for (int i = threadIdx.x; i < nt * per_tok; i += kRopeThreads) {
        const int tk = i / per_tok, r = i - tk * per_tok;
        const int hd = r / units, u = r - hd * units;
        const long long tok = t0 + tk;
        const long long bi = tok / p.s, si = tok - bi * p.s;
        const E* x = static_cast<const E*>(p.x) + bi * p.xs[0] + si * p.xs[1] + hd * p.xs[2];
        E* y = static_cast<E*>(p.y) + bi * p.ys[0] + si * p.ys[1] + hd * p.ys[2];
        if constexpr (kV8) {
            if (u >= nrot) {
                float v[8];
                const int at = rot + (u - nrot) * 8;
                load8<T>(x + at, v);
                store8<T>(y + at, v);
            } else if constexpr (kInter) {
                float v[8];
                load8<T>(x + u * 8, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) turn(v[2 * e], v[2 * e + 1], cs[tk][u * 4 + e]);
                store8<T>(y + u * 8, v);
            } else {
                float a[8], b[8];
                load8<T>(x + u * 8, a);
                load8<T>(x + pairs + u * 8, b);
#pragma unroll
                for (int e = 0; e < 8; ++e) turn(a[e], b[e], cs[tk][u * 8 + e]);
                store8<T>(y + u * 8, a);
                store8<T>(y + pairs + u * 8, b);
            }
        } else {
            if (u >= nrot) {
                y[rot + u - nrot] = x[rot + u - nrot];
            } else {
                const int ia = kInter ? 2 * u : u, ib = kInter ? 2 * u + 1 : u + pairs;
                float a = to_f32<T>(x[ia]), b = to_f32<T>(x[ib]);
                turn(a, b, cs[tk][u]);
                y[ia] = from_f32<T>(a);
                y[ib] = from_f32<T>(b);
            }
        }
    }
}

template <int T>
cudaError_t rope_launch(bool v8, bool inter, unsigned grid, cudaStream_t s, const RopeParams& p,
                        const vae_rope_plan& plan) {
    const auto go = [&](auto k) { return launch_kernel(k, dim3(grid), dim3(kRopeThreads), 0, s, p, plan); };
    if (v8) return inter ? go(rope_kernel<T, true, true>) : go(rope_kernel<T, true, false>);
    return inter ? go(rope_kernel<T, false, true>) : go(rope_kernel<T, false, false>);
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
    int rc = check_device();
    if (rc != VAE_OK) return rc;
    RopeParams p{};
    p.x = x_dev;
    p.y = y_dev;
    p.pos = pos_dev;
    p.tokens = static_cast<long long>(b) * s;
    p.s = s;
    p.h = h;
    p.d = d;
    p.pos_int = pos_int != 0;
    p.pos_batch = pos_batch;
    p.inverse = inverse != 0;
    bool v8 = aligned16(x_dev) && aligned16(y_dev) && d % 8 == 0 &&
              (plan->interleaved ? 2 * plan->pairs : plan->pairs) % 8 == 0;
    for (int i = 0; i < 3; ++i) {
        p.xs[i] = dim[i] > 1 ? x_stride[i] : 0;
        p.ys[i] = dim[i] > 1 ? y_stride[i] : 0;
        v8 = v8 && p.xs[i] % 8 == 0 && p.ys[i] % 8 == 0;
    }
    // Tokens per block: as many as share one (cos, sin) table, down to one when
    // there are too few tokens to give every SM a block.
    p.tpb = static_cast<int>(std::min<long long>(kRopeTokens, std::max<long long>(1, p.tokens / 304)));
    const long long grid = (p.tokens + p.tpb - 1) / p.tpb;
    if (grid > 0x7fffffffLL || static_cast<long long>(h) * d > (1 << 24))
        return set_error(VAE_ERR_SHAPE, "rope: too many tokens or heads");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned g = static_cast<unsigned>(grid);
    const bool in = plan->interleaved != 0;
    VAE_CUDA_CHECK(type == VAE_F32   ? rope_launch<VAE_F32>(v8, in, g, st, p, *plan)
                   : type == VAE_F16 ? rope_launch<VAE_F16>(v8, in, g, st, p, *plan)
                                     : rope_launch<VAE_BF16>(v8, in, g, st, p, *plan));
    return VAE_OK;
}

}  // extern "C"
