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
// rows of Wg, the odd one of Wu), so act(gate) o up never leaves the registers. The
// three weights' gradients and dx are one launch, whose tiles are dealt out by what
// they cost; rows of two tiles share one B where both accumulators can take them (512
// rows, "tall"); few tiles become narrow ones, or splits of the contraction, whose last
// one to finish adds them up.
//
// What bounds the products is the way from L2 to shared memory beside the tensor cores: a 256
// x 256 x 64 stage (32 KB a CTA) takes 578 cycles of it, more with every SM asking for long, and 512 of
// the tensor cores. Tall tiles read a quarter less. 16384 tokens of 1152 x 4608, bf16,
// in a graph: 292 to 302 us forward (1740 TFLOP/s; the first product 197), the gradient 673 to 713 on
// different machines (1460 to 1550). Of the gradient's first kernel (180 us) the products alone take
// 91, its stages' way 124, gate, up, dgate and dup 113. Small calls are chains of latencies: 256
// tokens of 512 x 2048 take 17.4 us, 8 of them in the first kernel.
#include <algorithm>
#include <cfloat>
#include <mutex>

#include "vae_ffn.cuh"
#include "vae_ffn_few.h"
#include "vae_ffn_plan.h"
#include "vae_overlap.h"

namespace vae {

namespace {

using namespace ffn;

constexpr int kOperand = kTile * kBk * 2;  // bytes
constexpr int kStage = 2 * kOperand;       // A, B
constexpr int kTallStage = 3 * kOperand;   // A, B, the other 256 rows' A
constexpr int kTallStages = 4;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kTmaWarp + 1;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;     // two accumulators
constexpr int kAmaxBlocks = 128;        // that look for the largest |dy|, at most

// Stages of the ring, and beside it what kBackGate's epilogue works in: boxes of 32 rows x 64 columns of gate and up,
// which become dgate and dup in place, three of each for every lane quadrant of TMEM. (Rows of 128 bytes through the
// copy engine: a lane that read and wrote its own row's 32 bytes took 125 us for 8192 tokens of 1152 x 4608, boxes of
// 64-byte rows 93; the number of requests counts.)
constexpr int kBox = 32 * 128;
constexpr int kBoxBufs = 3;
__host__ __device__ constexpr int ring_stages(int kind, bool tall = false) { return tall ? kTallStages : kind == kBackGate ? 4 : 7; }
__host__ __device__ constexpr int side_bytes(int kind) { return kind == kBackGate ? 4 * kBoxBufs * 2 * kBox : 0; }
__host__ __device__ constexpr int smem_bytes(int kind) { return 1024 + ring_stages(kind) * kStage + side_bytes(kind) + 512; }
static_assert(kTallStages * kTallStage <= ring_stages(kGrad) * kStage, "the ring holds the tall stages");
static_assert(smem_bytes(kGate) <= 232448 && smem_bytes(kBackGate) <= 232448, "shared memory over 227 KB");

struct Maps {
    CUtensorMap a[3];          // kGrad: dgate, dup, hidden
    CUtensorMap b[4];          // kGate: Wg, Wu; kGrad: Wg, Wu, x, dy
    CUtensorMap side[4];       // kBackGate: gate, up, dgate, dup
};

struct Params {
    Group group[2];
    Deal deal;
    int half;                  // kGrad: stages of dx's first segment
    void* out[4];              // kGate: hidden, gate, up; kDown: y; kGrad: dx, dWg, dWu, dWd
    float* parts[2];           // with splits: the sums of each problem and split (part_at)
    unsigned* arrived[2];      // with splits: how many of them have stored a warp's part of a tile, [tile][CTA of the pair][warp]
    unsigned* clear;           // counters of the kernel behind this one: set to 0 here
    int clear_n;
    int out_f32[2];
    const float* residual;
    const unsigned* amax;      // f16 gradients: the bits of the largest finite |dy|, from `amax_n` blocks
    int amax_n;
    unsigned* top;             // f16 gradients: the bits of the largest finite |dgate| or |dup| at that scale
    int again;                 // kBackGate: the second run, at the scale that `top` asks for
    int late;                  // kBackGate: only the epilogue needs the kernel before (that is the one that looks for the largest |dy|)
    int wide;                  // rows of D on 32 bytes
    DevStatus* status;
    unsigned long long timeout_ns;
};

struct Smem {
    uint8_t *ring, *side;
    uint64_t *full, *empty, *accf, *acce, *drain, *boxed, *done;
    uint32_t* tmem_slot;
    int* abort_flag;
};
template <int kKind>
__device__ __forceinline__ Smem carve(uint8_t* raw) {
    constexpr int kStages = ring_stages(kKind);
    Smem s;
    s.ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.side = s.ring + kStages * kStage;
    uint64_t* b = reinterpret_cast<uint64_t*>(s.side + side_bytes(kKind));
    s.full = b;
    s.empty = b + kStages;
    s.accf = b + 2 * kStages;
    s.acce = s.accf + 2;
    s.drain = s.acce + 2;
    s.boxed = s.drain + 1;  // [quadrants][kBoxBufs]
    s.done = s.boxed + 4 * kBoxBufs;
    s.tmem_slot = reinterpret_cast<uint32_t*>(s.done + 4 * kBoxBufs);
    s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
    return s;
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

// Rows of an operand that lies MN-major, in boxes of 64, 64 of the contraction from `k` on.
__device__ __forceinline__ void load_mn(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int row, int rows, int k) {
    tma_load_2d_pair(smem_u32(dst), map, bar, row, k);
    if (rows > 64) tma_load_2d_pair(smem_u32(dst + kOperand / 2), map, bar, row + 64, k);
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

// A launch's tiles have 256 rows, or (kTall) up to 512: four stages of 48 KB, one accumulator for each 256 rows. (One kernel
// for both, with the stages and the second rows' loads and products looked up at run time: 1024 tokens of 2048 x 5504, no tall
// tiles, second product 34 us and 28, dx and the weights' gradients 107 and 90; a loop over the rows in every kind: 16384
// tokens of 1152 x 4608, first product 225 us and 197.)
template <int kKind, bool kTall>
__device__ void role_producer(const Params& p, const Smem& s, const Maps& maps, int rank) {
    constexpr int stages = ring_stages(kKind, kTall), stage_bytes = kTall ? kTallStage : kStage;
    int stage = 0;
    uint32_t phase = 0, armed = 0, arm_par = 0;
    bool ok = true;
    const int pair = static_cast<int>(blockIdx.x >> 1);
    Tile ti;
    for (int i = 0; ok && tile_at(p.group, p.deal, pair, i, &ti); ++i) {
        const int row = ti.m0 + rank * kTile, col = kKind == kGate ? ti.n0 : ti.n0 + rank * (ti.n / 2);
        // rows of B that a CTA loads: those of a full tile where the map's box says so, else boxes of 64
        const int brows = b_mn(kKind) ? ti.n / 2 : kKind == kGate ? p.group[0].wide : p.group[0].wide / 2;
        const uint32_t bytes = static_cast<uint32_t>(kTall ? ti.subs : 1) * kOperand + (b_mn(kKind) ? (brows > 64 ? 2u : 1u) * 64 * 128 : static_cast<uint32_t>(brows) * 128);
        for (int kk = ti.k0; kk < ti.k1; ++kk) {
            ok = mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, s.abort_flag, p.timeout_ns, p.status, kWhereProducerEmpty);
            if (!ok) break;
            const uint32_t fb = smem_u32(&s.full[stage]);
            if (rank == 0) mbar_arrive_expect_tx(fb, 2u * bytes);
            const uint32_t fb0 = mapa_shared(fb, 0u);
            uint8_t *a = s.ring + stage * stage_bytes, *b = a + kOperand;
            if constexpr (kKind == kGrad) {
                const int seg = kk >= p.half ? 1 : 0, k = (kk - seg * p.half) * kBk;  // (dx)
                // dx: rows of dgate or dup as they lie, in boxes of 64
                const auto rows = [&](uint8_t* at, int r) {
                    if (ti.g != 0) return load_mn(at, &maps.a[ti.z - 1], fb0, r, kTile, kk * kBk);
                    tma_load_2d_pair(smem_u32(at), &maps.a[seg], fb0, k, r);
                    tma_load_2d_pair(smem_u32(at + kOperand / 2), &maps.a[seg], fb0, k, r + 64);
                };
                rows(a, row);
                if (ti.g == 0) load_mn(b, &maps.b[seg], fb0, col, brows, k);
                else load_mn(b, &maps.b[ti.z == 3 ? 3 : 2], fb0, col, brows, kk * kBk);
                if (kTall && ti.subs > 1) rows(a + kStage, row + 2 * kTile);
            } else {
                tma_load_2d_pair(smem_u32(a), &maps.a[0], fb0, kk * kBk, row);
                if constexpr (kKind == kBackGate) load_mn(b, &maps.b[0], fb0, col, brows, kk * kBk);
                else tma_load_2d_pair(smem_u32(b), &maps.b[kKind == kGate ? rank : 0], fb0, kk * kBk, col);
                if constexpr (kTall)
                    if (ti.subs > 1) tma_load_2d_pair(smem_u32(a + kStage), &maps.a[0], fb0, kk * kBk, row + 2 * kTile);
            }
            armed |= 1u << stage;
            arm_par = (arm_par & ~(1u << stage)) | (phase << stage);
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    // Every copy lands before the CTA can exit: the even CTA sees them on its full barriers, the odd one
    // on its empty barriers (the products that read a slot complete after its copies).
    int never = 0;
    for (int st = 0; st < stages; ++st)
        if (armed & (1u << st))
            (void)mbar_wait(smem_u32(rank == 0 ? &s.full[st] : &s.empty[st]), (arm_par >> st) & 1u, &never, p.timeout_ns,
                            p.status, kWhereDrain);
}

// The whole warp runs the loop and one lane issues: descriptors stay in uniform registers.
template <int T, int kKind, bool kTall>
__device__ void role_mma(const Params& p, const Smem& s, uint32_t tmem) {
    constexpr int stages = ring_stages(kKind, kTall);
    constexpr uint32_t stage_step = static_cast<uint32_t>(kTall ? kTallStage : kStage) >> 4;
    constexpr uint32_t ab = T == VAE_BF16 ? 1u : 0u;
    constexpr uint32_t idesc0 = (1u << 4) | (ab << 7) | (ab << 10) | ((b_mn(kKind) ? 1u : 0u) << 16) | ((2u * kTile >> 4) << 24);
    constexpr uint32_t bstep = b_mn(kKind) ? 2048 >> 4 : 2;
    const uint32_t ring = smem_u32(s.ring);
    const uint64_t ak = sw128_kmajor_desc(ring), am = mn_desc(ring);
    const uint64_t bd = b_mn(kKind) ? mn_desc(ring + kOperand) : sw128_kmajor_desc(ring + kOperand);
    int stage = 0, buf = 0;
    uint32_t phase = 0, accphase = 0;
    bool ok = true;
    const int pair = static_cast<int>(blockIdx.x >> 1);
    Tile ti;
    for (int i = 0; ok && tile_at(p.group, p.deal, pair, i, &ti); ++i) {
        const bool a_mn = kKind == kGrad && ti.g == 1;
        const uint64_t ad = a_mn ? am : ak;
        const uint32_t astep = a_mn ? 2048 >> 4 : 2;
        const uint32_t idesc = idesc0 | (a_mn ? 1u << 15 : 0u) | static_cast<uint32_t>((kKind == kGate ? 2 * ti.n : ti.n) >> 3) << 17;
        const int nk = ti.k1 - ti.k0;
        ok = warp_all(mbar_wait_cluster(smem_u32(&s.acce[buf]), accphase ^ 1u, s.abort_flag, p.timeout_ns, p.status, kWhereMmaAccEmpty));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * kMaxCols);
        for (int k = 0; k < nk; ++k) {
            ok = warp_all(mbar_wait(smem_u32(&s.full[stage]), phase, s.abort_flag, p.timeout_ns, p.status, kWhereMmaFull));
            if (!ok) break;
            tc_fence_after();
            const uint32_t off = static_cast<uint32_t>(stage) * stage_step;
            if (elect_one()) {
                if (kTall && ti.subs > 1) {
#pragma unroll
                    for (uint32_t j = 0; j < kBk / 16; ++j) {
                        umma_f16_pair(d, ad + (off + j * astep), bd + (off + j * bstep), idesc, j != 0 || k != 0 ? 1u : 0u);
                        umma_f16_pair(d + kMaxCols, ad + (off + (kStage >> 4) + j * astep), bd + (off + j * bstep), idesc, j != 0 || k != 0 ? 1u : 0u);
                    }
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kBk / 16; ++j)
                        umma_f16_pair(d, ad + (off + j * astep), bd + (off + j * bstep), idesc, j != 0 || k != 0 ? 1u : 0u);
                }
                umma_commit_pair(smem_u32(&s.empty[stage]));
                if (k + 1 == nk) umma_commit_pair(smem_u32(&s.accf[buf]));
            }
            __syncwarp();
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!kTall) buf ^= 1;
        if (buf == 0) accphase ^= 1u;
    }
    if (elect_one()) {
        umma_commit_pair(smem_u32(s.drain));
        int never = 0;
        (void)mbar_wait(smem_u32(s.drain), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
    }
    __syncwarp();
}

// The power of two that brings the largest finite |dy| to 4..8 (1 where there is none but 0). The whole warp.
__device__ __forceinline__ float dy_scale(const Params& p) {
    if (p.amax == nullptr) return 1.f;
    unsigned bits = 0u;
    for (int i = threadIdx.x & 31; i < p.amax_n; i += 32) bits = max(bits, p.amax[i]);
    bits = __reduce_max_sync(0xffffffffu, bits);
    const int e = static_cast<int>(bits >> 23) - 127;
    return bits == 0u ? 1.f : __uint_as_float(static_cast<unsigned>(2 - e + 127) << 23);
}

// The scale of dgate and dup: that of dy, or, where the largest of them would pass f16's range with it or lie so low that
// most are subnormal, the power of two that brings it to 2^14..2^15. (Nothing known ahead bounds dhidden up act' closely:
// the sum over c of |dy w_down| is some hundred times what dhidden comes to, and up may be any number of f16. So the first
// run looks, and a second one, which otherwise returns at once (2.4 us of a call), forms them anew.)
__device__ __forceinline__ unsigned far_top(const Params& p) {  // the largest, or 0 where the scale of dy serves
    if (p.top == nullptr) return 0u;
    const unsigned top = __ldcg(p.top);
    return top > __float_as_uint(65504.f) || top < __float_as_uint(0x1p-10f) ? top : 0u;
}
__device__ __forceinline__ float kept_scale(const Params& p) {
    const unsigned top = far_top(p);
    const float gain = dy_scale(p);
    return top == 0u ? gain : gain * __uint_as_float((127u + 14u + 127u - max(top >> 23, 127u - 60u)) << 23);
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
template <int T>
__device__ __forceinline__ B32 pack16(const float (&v)[16]) {
    B32 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.r[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    return r;
}

// Sixteen columns of a box (quarter q): rows of 128 bytes, a row per lane, 128-byte swizzle.
__device__ __forceinline__ B32 box_read(const uint8_t* box, int lane, int q) {
    const uint4 a = *reinterpret_cast<const uint4*>(box + sw128_off(lane, 2 * q));
    const uint4 b = *reinterpret_cast<const uint4*>(box + sw128_off(lane, 2 * q + 1));
    return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
__device__ __forceinline__ void box_write(uint8_t* box, int lane, int q, const B32& v) {
    *reinterpret_cast<uint4*>(box + sw128_off(lane, 2 * q)) = make_uint4(v.r[0], v.r[1], v.r[2], v.r[3]);
    *reinterpret_cast<uint4*>(box + sw128_off(lane, 2 * q + 1)) = make_uint4(v.r[4], v.r[5], v.r[6], v.r[7]);
}
// (what lies outside the tensor is not written)
__device__ __forceinline__ void box_store(const CUtensorMap* map, const uint8_t* box, int col, int row) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(box)), "r"(col), "r"(row)
                 : "memory");
}

// A quadrant's boxes of gate and up, asked for by its first warp up to kBoxBufs - 1 ahead of the one that its two warps
// work on (32 columns each).
struct Boxes {
    int i = 0, box = 0;  // the next one to ask for: of the pair's i-th tile
    Tile ti;
    bool more = false;
    int asked = 0, taken = 0;

    __device__ __forceinline__ void ask(const Params& p, const Smem& s, const Maps& maps, int pair, int quad, int lane, int rank) {
        if (!more) return;
        const int buf = quad * kBoxBufs + asked % kBoxBufs;
        if (lane == 0) {
            uint8_t* dst = s.side + buf * 2 * kBox;
            const uint32_t bar = smem_u32(&s.boxed[buf]);
            mbar_arrive_expect_tx(bar, 2u * kBox);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                        smem_u32(dst + k * kBox)),
                    "l"(reinterpret_cast<uint64_t>(&maps.side[k])), "r"(bar), "r"(ti.n0 + box * 64), "r"(ti.m0 + rank * kTile + quad * 32)
                    : "memory");
        }
        ++asked;
        if ((++box) * 64 >= ti.n) {
            box = 0;
            more = tile_at(p.group, p.deal, pair, ++i, &ti);
        }
    }
};

// Sixteen columns (eight where `left` is less) of a row of D from column n on, in its type. dWd comes as D^T = hidden^T dy:
// lanes are neighbours along its rows.
template <int T, int kKind>
__device__ __forceinline__ void put_out(const Params& p, const Tile& ti, int row, int n, int left, const float (&v)[16]) {
    const Group& gr = p.group[ti.g];
    const long long at = static_cast<long long>(row) * gr.cols + n;
    void* out = p.out[ti.z];
    if (kKind == kGrad && ti.z == 3) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (k >= left) continue;
            const long long o = static_cast<long long>(n + k) * gr.rows + row;
            if (p.out_f32[1]) static_cast<float*>(out)[o] = v[k];
            else static_cast<typename Elem<T>::type*>(out)[o] = from_f32<T>(v[k]);
        }
    } else if (p.out_f32[ti.g]) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            if (k >= left) continue;
            float4 r = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            if (kKind == kDown && p.residual != nullptr) {
                const float4 o = *reinterpret_cast<const float4*>(p.residual + at + k);
                r = make_float4(r.x + o.x, r.y + o.y, r.z + o.z, r.w + o.w);
            }
            *reinterpret_cast<float4*>(static_cast<float*>(out) + at + k) = r;
        }
    } else {
        store16(static_cast<uint16_t*>(out) + at, pack16<T>(v), left, p.wide);
    }
}
// Partial sums of splits lie as the epilogue holds them, so that every access is 512 bytes in a row and the lane that adds
// up has its row as from TMEM: [problem and split][tile of 256 rows][columns to the tile][CTA][warp], each warp's by
// sixteen columns, [quad of columns][lane][4]. (As D lies: 16 bytes of each row apart, read by one quad of lanes a row,
// 8 latencies one behind the other for 64 columns.)
__device__ __forceinline__ long long part_at(const Group& g, const Tile& ti, int rank, int warp, int lane) {
    return static_cast<long long>(ti.m0) * part_cols(g) + 2LL * kTile * ti.n0 + (rank * kEpiWarps + warp) * (32 * (ti.n / 2)) + lane * 4;
}
__device__ __forceinline__ void put_part(float* part, const float (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 16; k += 4) __stcg(reinterpret_cast<float4*>(part + k * 32), make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]));
}
// The sum of the splits' parts, in their order; four splits' loads are on their way at once.
__device__ __forceinline__ void add_parts(const float* part, long long each, int splits, float (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = 0.f;
#pragma unroll 1
    for (int s = 0; s < splits; s += 4) {
        float4 r[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r[q][k] = s + q < splits ? __ldcg(reinterpret_cast<const float4*>(part + (s + q) * each + k * 128)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[4 * k] += r[q][k].x;
                v[4 * k + 1] += r[q][k].y;
                v[4 * k + 2] += r[q][k].z;
                v[4 * k + 3] += r[q][k].w;
            }
    }
}

// Warp w: lane quadrant w % 4 of TMEM (a row per lane), half w / 4 of the columns.
template <int T, int kKind, int kAct, bool kTall>
__device__ void role_epilogue(const Params& p, const Smem& s, const Maps& maps, uint32_t tmem, int warp, int lane, int rank) {
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    int buf = 0;
    uint32_t phase = 0;
    const int pair = static_cast<int>(blockIdx.x >> 1);
    if (kKind == kBackGate && p.late) pdl_wait();
    const float gain = kKind == kGrad || (kKind == kBackGate && p.again) ? kept_scale(p) : kKind == kBackGate ? dy_scale(p) : 1.f;
    float top = 0.f;
    if (kKind == kGate || kKind == kBackGate)
        for (int i = static_cast<int>(blockIdx.x) * kEpiWarps * 32 + warp * 32 + lane; i < p.clear_n; i += static_cast<int>(gridDim.x) * kEpiWarps * 32)
            p.clear[i] = 0u;
    Boxes boxes;
    if constexpr (kKind == kBackGate) {
        boxes.more = half == 0 && tile_at(p.group, p.deal, pair, 0, &boxes.ti);
        for (int k = 0; k + 1 < kBoxBufs; ++k) boxes.ask(p, s, maps, pair, quad, lane, rank);
    }
    bool ok = true;
    Tile ti;
    for (int i = 0; ok && tile_at(p.group, p.deal, pair, i, &ti); ++i) {
        const Group& gr = p.group[ti.g];
        const int row = ti.m0 + rank * kTile + quad * 32 + lane, cols = gr.cols, rows = gr.rows;
        const bool live = row < rows;
        const long long at0 = static_cast<long long>(row) * cols;
        const int mine = ti.n / 2, n0 = ti.n0 + half * mine;  // this warp's columns
        ok = warp_all(mbar_wait_cluster(smem_u32(&s.accf[buf]), phase, s.abort_flag, p.timeout_ns, p.status, kWhereEpiAccFull));
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + lanes + static_cast<uint32_t>(buf * kMaxCols + half * mine);
        const float scale = kKind == kBackGate ? gain : kKind == kGrad && ti.z < 3 ? 1.f / gain : 1.f;
        if constexpr (kKind == kBackGate) {
            const int row0 = ti.m0 + rank * kTile + quad * 32;
            const uint32_t at = tmem + lanes + static_cast<uint32_t>(buf * kMaxCols + half * 32);
            for (int b = 0; ok && b * 64 < ti.n; ++b) {
                const int sbuf = quad * kBoxBufs + boxes.taken % kBoxBufs;
                const uint32_t turn = static_cast<uint32_t>(boxes.taken / kBoxBufs) & 1u;
                ok = warp_all(mbar_wait(smem_u32(&s.boxed[sbuf]), turn, s.abort_flag, p.timeout_ns, p.status, kWhereEpiAccFull));
                if (!ok) break;
                uint8_t* box = s.side + sbuf * 2 * kBox;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[16];
                    float v[16], w[16];
                    __syncwarp();
                    tmem_ld16(at + static_cast<uint32_t>(b * 64 + h * 16), x);
                    const B32 g = box_read(box, lane, half * 2 + h), u = box_read(box + kBox, lane, half * 2 + h);
                    tmem_ld_wait_regs(x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 g2 = unpack2<T>(g.r[k]), u2 = unpack2<T>(u.r[k]);
                        const float2 a0 = act_both<kAct>(g2.x), a1 = act_both<kAct>(g2.y);
                        const float d0 = __uint_as_float(x[2 * k]) * scale, d1 = __uint_as_float(x[2 * k + 1]) * scale;
                        v[2 * k] = d0 * u2.x * a0.y;
                        v[2 * k + 1] = d1 * u2.y * a1.y;
                        w[2 * k] = d0 * a0.x;
                        w[2 * k + 1] = d1 * a1.x;
                    }
                    if constexpr (T == VAE_F16) {
                        float most = 0.f;  // (columns and rows outside the tensors have gate = up = 0; fmaxf passes over NaN)
#pragma unroll
                        for (int k = 0; k < 16; ++k) most = fmaxf(most, fmaxf(fabsf(v[k]), fabsf(w[k])));
                        if (most > FLT_MAX) {  // an infinity, from one of the inputs: the finite ones
                            most = 0.f;
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                if (fabsf(v[k]) <= FLT_MAX) most = fmaxf(most, fabsf(v[k]));
                                if (fabsf(w[k]) <= FLT_MAX) most = fmaxf(most, fabsf(w[k]));
                            }
                        }
                        top = fmaxf(top, most);
                    }
                    box_write(box, lane, half * 2 + h, pack16<T>(v));
                    box_write(box + kBox, lane, half * 2 + h, pack16<T>(w));
                }
                ++boxes.taken;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.done[sbuf]));
                if (half == 0) {
                    ok = warp_all(mbar_wait(smem_u32(&s.done[sbuf]), turn, s.abort_flag, p.timeout_ns, p.status, kWhereEpiAccFull));
                    if (!ok) break;
                    if (lane == 0) {
                        if (ti.n0 + b * 64 < cols && row0 < rows) {
                            box_store(&maps.side[2], box, ti.n0 + b * 64, row0);
                            box_store(&maps.side[3], box + kBox, ti.n0 + b * 64, row0);
                        }
                        bulk_commit_group();
                        bulk_wait_read_1();  // the box before has left its buffer, which the next one takes
                    }
                    boxes.ask(p, s, maps, pair, quad, lane, rank);
                }
            }
        }
        if constexpr (kKind == kGate) {
#pragma unroll 1
            for (int c = 0; c < mine; c += 16) {
                const int n = n0 + c, left = cols - n;
                if (left <= 0) break;  // (the same for the whole warp)
                uint32_t x[16], y[16];
                float v[16];
                __syncwarp();
                tmem_ld16(acc + static_cast<uint32_t>(c), x);
                tmem_ld16(acc + static_cast<uint32_t>(ti.n + c), y);
                tmem_ld_wait_regs(x);
                tmem_ld_wait_regs(y);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = act_value<kAct>(__uint_as_float(x[k])) * __uint_as_float(y[k]);
                if (!live) continue;
                store16(static_cast<uint16_t*>(p.out[0]) + at0 + n, pack16<T>(v), left, p.wide);
                if (p.out[1] != nullptr) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(x[k]);
                    store16(static_cast<uint16_t*>(p.out[1]) + at0 + n, pack16<T>(v), left, p.wide);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(y[k]);
                    store16(static_cast<uint16_t*>(p.out[2]) + at0 + n, pack16<T>(v), left, p.wide);
                }
            }
        }
        if constexpr (kKind == kDown || kKind == kGrad) {
            for (int sub = 0; sub < (kTall ? ti.subs : 1); ++sub) {
                const int r = row + sub * 2 * kTile;
#pragma unroll 1
                for (int c = 0; c < mine; c += 16) {
                    const int n = n0 + c, left = cols - n;
                    if (left <= 0) break;  // (the same for the whole warp)
                    uint32_t x[16];
                    float v[16];
                    __syncwarp();
                    tmem_ld16(acc + static_cast<uint32_t>(sub * kMaxCols + c), x);
                    tmem_ld_wait_regs(x);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(x[k]) * scale;
                    if (r >= rows) continue;
                    if (!kTall && gr.splits > 1) put_part(p.parts[ti.g] + ti.part * part_size(gr) + part_at(gr, ti, rank, warp, lane) + c * 32, v);
                    else put_out<T, kKind>(p, ti, r, n, left, v);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.acce[buf]), 0u));
        if (!kTall) buf ^= 1;
        if (buf == 0) phase ^= 1u;
        if constexpr ((kKind == kDown || kKind == kGrad) && !kTall) {
            if (gr.splits > 1) {
                // The last split to store this warp's part of the tile adds them all up, in their order: nobody waits, and
                // the sum does not depend on who is last.
                __threadfence();
                __syncwarp();
                const int z = ti.part / gr.splits, tile = (z * gr.nm + ti.m0 / (2 * kTile)) * (gr.nfull + (gr.rest > 0 ? 1 : 0)) + ti.n0 / gr.wide;
                unsigned before = 0u;
                if (lane == 0) before = atomicAdd(p.arrived[ti.g] + (tile * 2 + rank) * kEpiWarps + warp, 1u);
                if (__shfl_sync(0xffffffffu, before, 0) + 1u != static_cast<unsigned>(gr.splits)) continue;
                __threadfence();
                if (row < rows) {
                    const float* part = p.parts[ti.g] + z * gr.splits * part_size(gr) + part_at(gr, ti, rank, warp, lane);
#pragma unroll 1
                    for (int c = 0; c < mine && n0 + c < cols; c += 16) {
                        float v[16];
                        add_parts(part + c * 32, part_size(gr), gr.splits, v);
                        put_out<T, kKind>(p, ti, row, n0 + c, cols - n0 - c, v);
                    }
                }
                __syncwarp();
            }
        }
    }
    if constexpr (kKind == kBackGate) {
        if (T == VAE_F16 && !p.again) {
            const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            if (lane == 0 && bits != 0u) atomicMax(p.top, bits);
        }
        if (half == 0) {  // boxes that a wait that ran out left on their way land before the CTA exits
            int never = 0;
            for (; boxes.taken < boxes.asked; ++boxes.taken)
                (void)mbar_wait(smem_u32(&s.boxed[quad * kBoxBufs + boxes.taken % kBoxBufs]),
                                static_cast<uint32_t>(boxes.taken / kBoxBufs) & 1u, &never, p.timeout_ns, p.status, kWhereDrain);
            if (lane == 0) bulk_wait_all();
            __syncwarp();
        }
    }
}

template <int T, int kKind, int kAct, bool kTall>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kStages = ring_stages(kKind);
    if constexpr (kKind == kBackGate && T == VAE_F16) {
        if (p.again) {  // (every thread of every CTA sees the same)
            pdl_wait();
            if (far_top(p) == 0u) return;
        }
    }
    const Smem s = carve<kKind>(smem_raw);
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
        for (int i = 0; i < 4 * kBoxBufs; ++i) {
            mbar_init(smem_u32(&s.boxed[i]), 1u);
            mbar_init(smem_u32(&s.done[i]), 2u);  // both warps of a quadrant
        }
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
    if (kKind != kBackGate || !p.late) pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM exist before any remote arrive or pair product
    tc_fence_after();
    const uint32_t tmem = *s.tmem_slot;
    if (warp < kEpiWarps) {
        role_epilogue<T, kKind, kAct, kTall>(p, s, maps, tmem, warp, lane, rank);
    } else if (warp == kTmaWarp) {
        if (lane == 0) role_producer<kKind, kTall>(p, s, maps, rank);
        __syncwarp();
    } else if (rank == 0) {
        role_mma<T, kKind, kTall>(p, s, tmem);
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

// (what is not finite counts as 0: it stays in its row, and the other rows keep their scale)
__device__ __forceinline__ unsigned finite_bits(float x) { return x <= FLT_MAX ? __float_as_uint(x) : 0u; }
// The largest finite |x| of f16 values, as the bits of an f32, one from each block; sets `zero` to 0.
__global__ void __launch_bounds__(512) amax_kernel(const uint4* x, long long n8, unsigned* amax, unsigned* zero) {
    __shared__ unsigned tops[16];
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *zero = 0u;
    pdl_launch_dependents();  // the next kernel's products may start: only its epilogue waits for this one
    unsigned top = 0u;
    for (long long i = static_cast<long long>(blockIdx.x) * 512 + threadIdx.x; i < n8; i += static_cast<long long>(gridDim.x) * 512) {
        const uint4 v = __ldg(x + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<VAE_F16>(u[k] & 0x7fff7fffu);
            top = max(top, max(finite_bits(f.x), finite_bits(f.y)));
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = __reduce_max_sync(0xffffffffu, threadIdx.x < 16 ? tops[threadIdx.x] : 0u);
        if (threadIdx.x == 0) amax[blockIdx.x] = top;
    }
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

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// A plan costs some tens of microseconds; it depends on the sizes alone, and calls of the same sizes follow one another.
Plan plan_for(int kind, const vae_gated_ffn_desc& a) {
    struct Known {
        int kind = -1, m, c, f;
        Plan plan;
    };
    thread_local Known known[8];
    thread_local int next = 0;
    for (const Known& k : known)
        if (k.kind == kind && k.m == a.m && k.c == a.c && k.f == a.f) return k.plan;
    Known& k = known[next];
    next = (next + 1) % 8;
    k.plan = make_plan(kind, a.m, a.c, a.f);
    k.kind = kind;
    k.m = a.m;
    k.c = a.c;
    k.f = a.f;
    return k.plan;
}

std::mutex g_mu;

template <int T, int kKind, int kAct, bool kTall>
int ffn_setup() {
    static CtxOnce once;
    int dev = 0;
    VAE_CUDA_CHECK(cudaGetDevice(&dev));
    std::lock_guard<std::mutex> lk(g_mu);
    if (!once.done(dev)) {
        VAE_CUDA_CHECK(cudaFuncSetAttribute(ffn_kernel<T, kKind, kAct, kTall>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kKind)));
        once.mark(dev);
    }
    return VAE_OK;
}

template <int T, int kKind, int kAct = VAE_ACT_SILU, bool kTall = false>
int ffn_launch(const Maps& maps, const Plan& plan, Params& p, bool ahead, cudaStream_t stream) {
    if constexpr ((kKind == kDown || kKind == kGrad) && !kTall)
        if (plan.group[0].tall > 1) return ffn_launch<T, kKind, kAct, true>(maps, plan, p, ahead, stream);
    int rc = ffn_setup<T, kKind, kAct, kTall>();
    if (rc != VAE_OK) return rc;
    p.status = device_status_ptr();
    if (p.status == nullptr) return VAE_ERR_CUDA;
    p.timeout_ns = wait_timeout_ns();
    p.group[0] = plan.group[0];
    p.group[1] = plan.group[1];
    p.deal = plan.deal;
    const int count = plan.group[1].problems > 0 ? 2 : 1;
    if (sm_count() < 2 * kPairs) deal_out(kKind, p.group, count, sm_count() / 2, &p.deal);
    int pairs = 0, at = 0;  // up to the last one with work
    for (int r = 0; r < p.deal.n; ++r) {
        at += p.deal.pairs[r];
        for (int c = 0; c < 4; ++c)
            if (p.deal.count[r][c] > 0) pairs = at;
    }
    VAE_CUDA_CHECK(launch_kernel_as(ahead || pdl_enabled(), ffn_kernel<T, kKind, kAct, kTall>, dim3(2 * pairs), dim3(kThreads), smem_bytes(kKind),
                                    stream, maps, p));
    return VAE_OK;
}

// The products whose epilogue knows the activation (a branch on it for every element took more of the instruction
// cache than there is: 295 us instead of 100 at 16384 tokens).
template <int T, int kKind>
int ffn_launch_act(int act, const Maps& maps, const Plan& plan, Params& p, bool ahead, cudaStream_t stream) {
    if (act == VAE_ACT_SILU) return ffn_launch<T, kKind, VAE_ACT_SILU>(maps, plan, p, ahead, stream);
    return act == VAE_ACT_GELU ? ffn_launch<T, kKind, VAE_ACT_GELU>(maps, plan, p, ahead, stream)
                               : ffn_launch<T, kKind, VAE_ACT_GELU_TANH>(maps, plan, p, ahead, stream);
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

size_t mc_bytes(const vae_gated_ffn_desc& a) { return static_cast<size_t>(a.m) * a.c * 2; }
size_t mf_bytes(const vae_gated_ffn_desc& a) { return static_cast<size_t>(a.m) * a.f * 2; }
size_t cf_bytes(const vae_gated_ffn_desc& a) { return static_cast<size_t>(a.c) * a.f * 2; }

#define VAE_TRY(expr)               \
    do {                            \
        const int rc_ = (expr);     \
        if (rc_ != VAE_OK) return rc_; \
    } while (0)

bool on32(const void* q) { return reinterpret_cast<uintptr_t>(q) % 32 == 0; }

template <int T>
int ffn_forward(const vae_gated_ffn_desc& a, const void* x, const void* wg, const void* wu, const void* wd, const float* residual,
                void* y, void* gate, void* up, void* hidden, char* ws, cudaStream_t stream) {
    Maps maps;
    Params p{};
    const Plan down = plan_for(kDown, a);
    unsigned* arrived = reinterpret_cast<unsigned*>(ws);
    p.clear = arrived;
    p.clear_n = arrivals(down.group[0]);
    const Plan plan = plan_for(kGate, a);
    VAE_TRY(ffn_map(&maps.a[0], T, x, a.m, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wg, a.f, a.c, plan.group[0].wide));
    VAE_TRY(ffn_map(&maps.b[1], T, wu, a.f, a.c, plan.group[0].wide));
    p.out[0] = hidden;
    p.out[1] = gate;
    p.out[2] = up;
    p.wide = a.f % 16 == 0 && on32(hidden) && on32(gate) && on32(up);
    VAE_TRY((ffn_launch_act<T, kGate>(a.activation, maps, plan, p, false, stream)));
    p = Params{};
    VAE_TRY(ffn_map(&maps.a[0], T, hidden, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wd, a.c, a.f, down.group[0].wide / 2));
    p.out[0] = y;
    p.arrived[0] = arrived;
    p.parts[0] = reinterpret_cast<float*>(ws + up256(arrivals(down.group[0]) * sizeof(unsigned)));
    p.out_f32[0] = a.y_type == VAE_F32;
    p.residual = residual;
    p.wide = a.c % 16 == 0 && on32(y);
    return ffn_launch<T, kDown>(maps, down, p, true, stream);
}

// Workspace of the gradient: the largest |dy|, the largest of dgate and dup, dgate, dup, the counters of splits, partial sums.
struct BackSpace {
    size_t dgate, dup, arrived[2], parts[2], bytes;
};
BackSpace back_space(const vae_gated_ffn_desc& a) {
    BackSpace s;
    s.dgate = up256((kAmaxBlocks + 1) * sizeof(unsigned));
    s.dup = s.dgate + up256(mf_bytes(a));
    const Plan plan = plan_for(kGrad, a);
    s.arrived[0] = s.dup + up256(mf_bytes(a));
    s.arrived[1] = s.arrived[0] + arrivals(plan.group[0]) * sizeof(unsigned);
    s.parts[0] = up256(s.arrived[1] + arrivals(plan.group[1]) * sizeof(unsigned));
    s.parts[1] = s.parts[0] + up256(parts_bytes(plan.group[0]));
    s.bytes = s.parts[1] + parts_bytes(plan.group[1]);
    return s;
}

template <int T>
int ffn_backward(const vae_gated_ffn_desc& a, const void* dy, const void* x, const void* wg, const void* wu, const void* wd,
                 const void* gate, const void* up, const void* hidden, void* dx, void* dwg, void* dwu, void* dwd, char* ws,
                 cudaStream_t stream) {
    const BackSpace at = back_space(a);
    void *dgate = ws + at.dgate, *dup = ws + at.dup;
    Params p{};
    if (T == VAE_F16) {
        unsigned* amax = reinterpret_cast<unsigned*>(ws);
        const long long n8 = static_cast<long long>(a.m) * a.c / 8;
        p.amax = amax;
        p.top = amax + kAmaxBlocks;
        p.amax_n = static_cast<int>(std::min<long long>((n8 + 511) / 512, kAmaxBlocks));
        p.late = 1;
        VAE_CUDA_CHECK(launch_kernel(amax_kernel, dim3(p.amax_n), dim3(512), 0, stream, static_cast<const uint4*>(dy), n8, amax, p.top));
    }
    Maps maps;
    VAE_TRY(ffn_map(&maps.a[0], T, dy, a.m, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wd, a.c, a.f, kBk));
    VAE_TRY(ffn_map(&maps.side[0], T, gate, a.m, a.f, 32));
    VAE_TRY(ffn_map(&maps.side[1], T, up, a.m, a.f, 32));
    VAE_TRY(ffn_map(&maps.side[2], T, dgate, a.m, a.f, 32));
    VAE_TRY(ffn_map(&maps.side[3], T, dup, a.m, a.f, 32));
    Plan plan = plan_for(kGrad, a);
    p.clear = reinterpret_cast<unsigned*>(ws + at.arrived[0]);
    p.clear_n = arrivals(plan.group[0]) + arrivals(plan.group[1]);
    const Plan first = plan_for(kBackGate, a);
    VAE_TRY((ffn_launch_act<T, kBackGate>(a.activation, maps, first, p, p.late != 0, stream)));
    p.late = 0;
    if (T == VAE_F16) {
        p.clear_n = 0;
        p.again = 1;
        VAE_TRY((ffn_launch_act<T, kBackGate>(a.activation, maps, first, p, true, stream)));
    }
    const bool weights = dwg != nullptr;
    VAE_TRY(ffn_map(&maps.a[0], T, dgate, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.a[1], T, dup, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.b[0], T, wg, a.f, a.c, kBk));
    VAE_TRY(ffn_map(&maps.b[1], T, wu, a.f, a.c, kBk));
    if (weights) {
        VAE_TRY(ffn_map(&maps.a[2], T, hidden, a.m, a.f, kBk));
        VAE_TRY(ffn_map(&maps.b[2], T, x, a.m, a.c, kBk));
        VAE_TRY(ffn_map(&maps.b[3], T, dy, a.m, a.c, kBk));
    }
    p.half = (a.f + kBk - 1) / kBk;
    p.out[0] = dx;
    p.out[1] = dwg;
    p.out[2] = dwu;
    p.out[3] = dwd;
    p.parts[0] = reinterpret_cast<float*>(ws + at.parts[0]);
    p.parts[1] = reinterpret_cast<float*>(ws + at.parts[1]);
    p.arrived[0] = reinterpret_cast<unsigned*>(ws + at.arrived[0]);
    p.arrived[1] = reinterpret_cast<unsigned*>(ws + at.arrived[1]);
    p.out_f32[1] = a.dw_type == VAE_F32;
    p.wide = a.c % 16 == 0 && on32(dx) && on32(dwg) && on32(dwu);
    if (!weights) {  // dx alone, cut the same way: the same bits
        plan.group[1] = Group{};
        deal_out(kGrad, plan.group, 1, kPairs, &plan.deal);
    }
    return ffn_launch<T, kGrad>(maps, plan, p, true, stream);
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" {

size_t vae_gated_ffn_workspace_bytes(const vae_gated_ffn_desc* desc) {
    clear_error();
    if (ffn_check(desc, false) != VAE_OK) return 0;
    // hidden, where it is not saved; of few tokens what its rounding left, else partial sums and their counters
    const size_t hidden = desc->save ? 0 : up256(mf_bytes(*desc));
    if (desc->m <= kFewTokens) return hidden + mf_bytes(*desc);
    const Group g = plan_for(kDown, *desc).group[0];
    return hidden + up256(arrivals(g) * sizeof(unsigned)) + parts_bytes(g);
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
    char* ws = static_cast<char*>(workspace_dev) + (save ? 0 : up256(mf_bytes(a)));
    if (a.m <= kFewTokens)
        return ffn_few(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, ws, st);
    return a.type == VAE_F16
               ? ffn_forward<VAE_F16>(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, ws, st)
               : ffn_forward<VAE_BF16>(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, ws, st);
}

size_t vae_gated_ffn_backward_workspace_bytes(const vae_gated_ffn_desc* desc) {
    clear_error();
    if (ffn_check(desc, true) != VAE_OK) return 0;
    return back_space(*desc).bytes;
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
