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

#include "vae_ffn.cuh"
#include "vae_ffn_few.h"
#include "vae_overlap.h"

namespace vae {

namespace {

constexpr int kTile = 128;              // rows of A per CTA
constexpr int kMaxCols = 256;           // columns of the pair's accumulator
constexpr int kBk = 64;                 // contraction per stage: one 128-byte swizzle row
constexpr int kOperand = kTile * kBk * 2;  // bytes
constexpr int kStage = 2 * kOperand;
constexpr int kEpiWarps = 8, kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;     // two accumulators
constexpr int kGroup = 8;               // row tiles that share their column tiles in L2
constexpr int kPairs = 76;              // that the plan counts with

// The products. A and B stand as [rows][contraction] (K-major) or [contraction][rows].
enum : int {
    kGate,      // x, (Wg, Wu) -> hidden (gate, up)
    kDown,      // hidden, Wd -> y
    kBackGate,  // dy, Wd^T -> dgate, dup
    kDx,        // (dgate, dup), (Wg, Wu)^T -> dx
    kDw,        // dgate^T, x^T -> dWg; dup^T, x^T -> dWu; hidden^T, dy^T -> dWd^T
};
__host__ __device__ constexpr bool a_mn(int kind) { return kind == kDw; }
__host__ __device__ constexpr bool b_mn(int kind) { return kind >= kBackGate; }

// Stages of the ring, and beside it what kBackGate's epilogue works in: boxes of 32 rows x 64 columns of gate and up,
// which become dgate and dup in place, three of each for every lane quadrant of TMEM. (Rows of 128 bytes through the
// copy engine: a lane that read and wrote its own row's 32 bytes took 125 us for 8192 tokens of 1152 x 4608, boxes of
// 64-byte rows 93; the number of requests counts.)
constexpr int kBox = 32 * 128;
constexpr int kBoxBufs = 3;
__host__ __device__ constexpr int ring_stages(int kind) { return kind == kBackGate ? 4 : 7; }
__host__ __device__ constexpr int side_bytes(int kind) { return kind == kBackGate ? 4 * kBoxBufs * 2 * kBox : 0; }
__host__ __device__ constexpr int smem_bytes(int kind) { return 1024 + ring_stages(kind) * kStage + side_bytes(kind) + 512; }
static_assert(smem_bytes(kGate) <= 232448 && smem_bytes(kBackGate) <= 232448, "shared memory over 227 KB");

struct Maps {
    CUtensorMap a[3], b[3];
    CUtensorMap side[4];       // kBackGate: gate, up, dgate, dup
};

// How a product is cut: column tiles of `wide` and what is left of the columns (`rest`, 0: nothing), the
// contraction in `splits`. `fit`: rest tiles that take about as long as a full one.
struct Cut {
    int wide, rest, splits, fit;
};

struct Params {
    int rows, cols, problems;  // of D
    Cut cut;
    int nm, nfull;             // row tiles, column tiles of full width
    int full, rests;           // tiles of full width, and of the rest
    int nk, segments;          // stages of a tile (per segment: products that add up)
    void* out[3];              // kGate: hidden, gate, up; kDown, kDx, kDw: D of each problem
    float* parts;              // with splits: D of each problem and split, [problems * splits][rows][cols]
    int out_f32;
    const float* residual;
    const unsigned* amax;      // f16 gradients: the largest |dy|'s bits
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

struct Tile {
    int z, m0, n0, n;  // problem (and split: problem * splits + split), the pair's first row, the columns [n0, n0 + n)
    int k0, k1;        // stages
};
// The i-th tile of pair `pair` of `pairs`; false behind its last. Tiles of full width are dealt out in turn;
// what is left of the columns goes first to the pairs that have one full tile less (as many as fit into one), so
// that it costs no turn of its own. Row tiles lie in groups of kGroup, their column tiles side by side: the
// pairs at work share rows of A and of B in L2.
__device__ __forceinline__ bool tile_at(const Params& p, int pair, int pairs, int i, Tile* r) {
    const int q = p.full / pairs, heavy = p.full - q * pairs;
    const int mine = q + (pair < heavy ? 1 : 0);
    int t = -1;
    if (i < mine) {
        t = pair + i * pairs;
    } else {
        i -= mine;
        const int light = heavy > 0 ? pairs - heavy : 0;
        const int first = light * p.cut.fit < p.rests ? light * p.cut.fit : p.rests;
        const int own = pair >= heavy && light > 0 && first > pair - heavy ? (first - (pair - heavy) + light - 1) / light : 0;
        const int j = i < own ? pair - heavy + i * light : first + pair + (i - own) * pairs;
        if (j >= p.rests) return false;
        t = p.full + j;
    }
    int nt;
    if (t < p.full) {
        const int each = p.nm * p.nfull;
        r->z = t / each;
        t -= r->z * each;
        const int g = t / (kGroup * p.nfull), in = t - g * kGroup * p.nfull;
        const int tall = p.nm - g * kGroup < kGroup ? p.nm - g * kGroup : kGroup;
        nt = in / tall;
        r->m0 = (g * kGroup + in - nt * tall) * 2 * kTile;
        r->n = p.cut.wide;
    } else {
        t -= p.full;
        r->z = t / p.nm;
        r->m0 = (t - r->z * p.nm) * 2 * kTile;
        nt = p.nfull;
        r->n = p.cut.rest;
    }
    r->n0 = nt * p.cut.wide;
    const int s = r->z % p.cut.splits, all = p.nk * p.segments;
    r->k0 = static_cast<int>(static_cast<long long>(all) * s / p.cut.splits);
    r->k1 = static_cast<int>(static_cast<long long>(all) * (s + 1) / p.cut.splits);
    return true;
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

// One operand of a stage: `rows` rows (a K-major map's boxes hold as many) from `row` on, 64 of the contraction from `k` on.
template <bool kMn>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, uint32_t bar, int row, int rows, int k) {
    if constexpr (kMn) {  // boxes of 64 rows each, as they lie
        tma_load_2d_pair(smem_u32(dst), map, bar, row, k);
        if (rows > 64) tma_load_2d_pair(smem_u32(dst + kOperand / 2), map, bar, row + 64, k);
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
    constexpr int kStages = ring_stages(kKind);
    int stage = 0;
    uint32_t phase = 0, armed = 0, arm_par = 0;
    bool ok = true;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    // rows of B that a CTA loads, always those of a full tile
    const int brows = kKind == kGate ? p.cut.wide : p.cut.wide / 2;
    const uint32_t bytes = kOperand + (b_mn(kKind) ? (brows > 64 ? 2u : 1u) * 64 * 128 : static_cast<uint32_t>(brows) * 128);
    Tile ti;
    for (int i = 0; ok && tile_at(p, pair, pairs, i, &ti); ++i) {
        const int row = ti.m0 + rank * kTile, col = kKind == kGate ? ti.n0 : ti.n0 + rank * (ti.n / 2);
        const int z = ti.z / p.cut.splits;
        for (int kk = ti.k0; kk < ti.k1; ++kk) {
            const int seg = kKind == kDx && kk >= p.nk ? 1 : 0, k = kk - seg * p.nk;
            const CUtensorMap* ma = &maps.a[kKind == kDx ? seg : z];
            const CUtensorMap* mb = &maps.b[kKind == kDx ? seg : kKind == kGate ? rank : z];
            ok = mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, s.abort_flag, p.timeout_ns, p.status, kWhereProducerEmpty);
            if (!ok) break;
            const uint32_t fb = smem_u32(&s.full[stage]);
            if (rank == 0) mbar_arrive_expect_tx(fb, 2u * bytes);
            const uint32_t fb0 = mapa_shared(fb, 0u);
            uint8_t* a = s.ring + stage * kStage;
            load_operand<a_mn(kKind)>(a, ma, fb0, row, kTile, k * kBk);
            load_operand<b_mn(kKind)>(a + kOperand, mb, fb0, col, brows, k * kBk);
            armed |= 1u << stage;
            arm_par = (arm_par & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
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
    constexpr int kStages = ring_stages(kKind);
    constexpr uint32_t ab = T == VAE_BF16 ? 1u : 0u;
    constexpr uint32_t idesc0 = (1u << 4) | (ab << 7) | (ab << 10) | ((a_mn(kKind) ? 1u : 0u) << 15) |
                                ((b_mn(kKind) ? 1u : 0u) << 16) | ((2u * kTile >> 4) << 24);
    constexpr uint32_t astep = a_mn(kKind) ? 2048 >> 4 : 2, bstep = b_mn(kKind) ? 2048 >> 4 : 2;
    const uint32_t ring = smem_u32(s.ring);
    const uint64_t ad = a_mn(kKind) ? mn_desc(ring) : sw128_kmajor_desc(ring);
    const uint64_t bd = b_mn(kKind) ? mn_desc(ring + kOperand) : sw128_kmajor_desc(ring + kOperand);
    int stage = 0, buf = 0;
    uint32_t phase = 0, accphase = 0;
    bool ok = true;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    Tile ti;
    for (int i = 0; ok && tile_at(p, pair, pairs, i, &ti); ++i) {
        const uint32_t idesc = idesc0 | static_cast<uint32_t>((kKind == kGate ? 2 * ti.n : ti.n) >> 3) << 17;
        const int nk = ti.k1 - ti.k0;
        ok = warp_all(mbar_wait_cluster(smem_u32(&s.acce[buf]), accphase ^ 1u, s.abort_flag, p.timeout_ns, p.status, kWhereMmaAccEmpty));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * kMaxCols);
        for (int k = 0; k < nk; ++k) {
            ok = warp_all(mbar_wait(smem_u32(&s.full[stage]), phase, s.abort_flag, p.timeout_ns, p.status, kWhereMmaFull));
            if (!ok) break;
            tc_fence_after();
            const uint32_t off = static_cast<uint32_t>(stage) * (kStage >> 4);
            if (elect_one()) {
#pragma unroll
                for (uint32_t j = 0; j < kBk / 16; ++j)
                    umma_f16_pair(d, ad + (off + j * astep), bd + (off + j * bstep), idesc, j != 0 || k != 0 ? 1u : 0u);
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

    __device__ __forceinline__ void ask(const Params& p, const Smem& s, const Maps& maps, int pair, int pairs, int quad, int lane, int rank) {
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
            more = tile_at(p, pair, pairs, ++i, &ti);
        }
    }
};

// Warp w: lane quadrant w % 4 of TMEM (a row per lane), half w / 4 of the columns.
template <int T, int kKind, int kAct>
__device__ void role_epilogue(const Params& p, const Smem& s, const Maps& maps, uint32_t tmem, int warp, int lane, int rank) {
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    int buf = 0;
    uint32_t phase = 0;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    Boxes boxes;
    if constexpr (kKind == kBackGate) {
        boxes.more = half == 0 && tile_at(p, pair, pairs, 0, &boxes.ti);
        for (int k = 0; k + 1 < kBoxBufs; ++k) boxes.ask(p, s, maps, pair, pairs, quad, lane, rank);
    }
    bool ok = true;
    Tile ti;
    for (int i = 0; ok && tile_at(p, pair, pairs, i, &ti); ++i) {
        const int row = ti.m0 + rank * kTile + quad * 32 + lane, cols = p.cols;
        const bool live = row < p.rows;
        const long long at0 = static_cast<long long>(row) * cols;
        const int mine = ti.n / 2, n0 = ti.n0 + half * mine;  // this warp's columns
        ok = warp_all(mbar_wait_cluster(smem_u32(&s.accf[buf]), phase, s.abort_flag, p.timeout_ns, p.status, kWhereEpiAccFull));
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + lanes + static_cast<uint32_t>(buf * kMaxCols + half * mine);
        const int z = ti.z / p.cut.splits;
        float scale = 1.f;
        if constexpr (kKind == kBackGate) scale = dy_scale(p.amax);
        if constexpr (kKind == kDx || kKind == kDw) scale = z < 2 ? 1.f / dy_scale(p.amax) : 1.f;
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
                        if (ti.n0 + b * 64 < cols && row0 < p.rows) {
                            box_store(&maps.side[2], box, ti.n0 + b * 64, row0);
                            box_store(&maps.side[3], box + kBox, ti.n0 + b * 64, row0);
                        }
                        bulk_commit_group();
                        bulk_wait_read_1();  // the box before has left its buffer, which the next one takes
                    }
                    boxes.ask(p, s, maps, pair, pairs, quad, lane, rank);
                }
            }
        }
#pragma unroll 1
        for (int c = 0; kKind != kBackGate && c < mine; c += 16) {
            const int n = n0 + c, left = cols - n;
            if (left <= 0) break;  // (the same for the whole warp)
            uint32_t x[16];
            float v[16];
            __syncwarp();
            tmem_ld16(acc + static_cast<uint32_t>(c), x);
            if constexpr (kKind == kGate) {
                uint32_t y[16];
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
            } else {
                    tmem_ld_wait_regs(x);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(x[k]) * scale;
                    if (!live) continue;
                    const bool split = p.cut.splits > 1;
                    float* part = p.parts + static_cast<long long>(ti.z) * p.rows * cols;
                    if (kKind == kDw && z == 2) {
                        // D^T = hidden^T dy: lanes are neighbours along a row of dWd
                        const long long at = static_cast<long long>(n) * p.rows + row;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            if (k >= left) continue;
                            const long long o = at + static_cast<long long>(k) * p.rows;
                            if (split) part[o] = v[k];
                            else if (p.out_f32) static_cast<float*>(p.out[2])[o] = v[k];
                            else static_cast<typename Elem<T>::type*>(p.out[2])[o] = from_f32<T>(v[k]);
                        }
                    } else if (split || p.out_f32) {
                        float* y = split ? part : static_cast<float*>(p.out[z]);
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            if (k >= left) continue;
                            float4 r = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                            if (kKind == kDown && !split && p.residual != nullptr) {
                                const float4 o = *reinterpret_cast<const float4*>(p.residual + at0 + n + k);
                                r = make_float4(r.x + o.x, r.y + o.y, r.z + o.z, r.w + o.w);
                            }
                            *reinterpret_cast<float4*>(y + at0 + n + k) = r;
                        }
                    } else {
                        store16(static_cast<uint16_t*>(p.out[z]) + at0 + n, pack16<T>(v), left, p.wide);
                    }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.acce[buf]), 0u));
        buf ^= 1;
        if (buf == 0) phase ^= 1u;
    }
    if constexpr (kKind == kBackGate) {
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

template <int T, int kKind, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kStages = ring_stages(kKind);
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
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM exist before any remote arrive or pair product
    tc_fence_after();
    const uint32_t tmem = *s.tmem_slot;
    if (warp < kEpiWarps) {
        role_epilogue<T, kKind, kAct>(p, s, maps, tmem, warp, lane, rank);
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

// The splits' sums, in order, eight elements a thread: D of each problem in its type.
template <int T>
__global__ void __launch_bounds__(256) join_kernel(const float* parts, int splits, long long n8, int out_f32, void* out0, void* out1,
                                                   void* out2, const float* residual) {
    pdl_wait();
    const int z = blockIdx.y;
    void* out = z == 0 ? out0 : z == 1 ? out1 : out2;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<long long>(gridDim.x) * 256) {
        float v[8];
        load8<VAE_F32>(parts + (static_cast<long long>(z) * splits * n8 + i) * 8, v);
        for (int s = 1; s < splits; ++s) {
            float w[8];
            load8<VAE_F32>(parts + ((static_cast<long long>(z) * splits + s) * n8 + i) * 8, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += w[k];
        }
        if (residual != nullptr) {
            float w[8];
            load8<VAE_F32>(residual + i * 8, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += w[k];
        }
        if (out_f32) store8<VAE_F32>(static_cast<float*>(out) + i * 8, v);
        else store8<T>(static_cast<typename Elem<T>::type*>(out) + i * 8, v);
    }
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

// Cycles that a pair takes for a stage of a tile of n accumulator columns, as measured: the stage's bytes from L2, 64 a
// cycle and CTA, or below that the hand-over between loads and products.
double stage_cycles(int n) { return std::max(430.0, 1.13 * (256 + n)); }

// How D (rows x cols, `problems` of them) with `nk` stages in all is cut: the tile width and the number of splits with
// the least time, counted in cycles of the busiest pair. Wide tiles read the least; narrow ones and splits give work
// to more SMs. Splits cost a second kernel (4000 cycles) that reads the f32 sums that they write (2700 bytes a cycle
// both ways).
Cut plan_cut(int kind, int rows, int cols, int nk, int problems) {
    const bool gated = kind == kGate || kind == kBackGate;
    const int per = kind == kGate ? 2 : 1, unit = 32;  // accumulator columns per column; widths are multiples of it
    const long long nm = (rows + 2 * kTile - 1) / (2 * kTile);
    Cut best{};
    double least = 0;
    for (int wide = kMaxCols / per; wide >= 64 / per && wide >= unit; wide -= 64 / per) {
        if (wide % unit != 0) continue;
        for (int splits = 1; splits <= 8 && splits <= std::max(1, nk / 4) && (splits == 1 || !gated); ++splits) {
            Cut c;
            c.wide = wide;
            c.splits = splits;
            c.rest = (cols % wide + unit - 1) / unit * unit;
            const long long each = nm * problems * splits, full = each * (cols / wide), rests = c.rest > 0 ? each : 0;
            const double one = stage_cycles(wide * per), part = c.rest > 0 ? stage_cycles(c.rest * per) : one;
            c.fit = c.rest > 0 ? std::max(1, static_cast<int>(one / part)) : 0;
            const long long q = full / kPairs, heavy = full % kPairs, light = heavy > 0 ? kPairs - heavy : 0;
            const long long first = std::min(rests, light * c.fit), over = rests - first;
            double turns = std::max((q + (heavy > 0)) * one, q * one + (light > 0 ? (first + light - 1) / light : 0) * part);
            turns += (over + kPairs - 1) / kPairs * part;
            double t = turns * ((nk + splits - 1) / splits) + 10.0 * wide;  // (the last tile's epilogue)
            if (splits > 1) t += 4000 + 8.0 * splits * problems * rows * cols / 2700;
            if (best.wide == 0 || t < least) {
                best = c;
                least = t;
            }
        }
    }
    return best;
}
size_t parts_bytes(const Cut& c, int rows, int cols, int problems) {
    return c.splits > 1 ? static_cast<size_t>(c.splits) * problems * rows * cols * sizeof(float) : 0;
}

std::mutex g_mu;

template <int T, int kKind, int kAct>
int ffn_setup() {
    static CtxOnce once;
    int dev = 0;
    VAE_CUDA_CHECK(cudaGetDevice(&dev));
    std::lock_guard<std::mutex> lk(g_mu);
    if (!once.done(dev)) {
        VAE_CUDA_CHECK(cudaFuncSetAttribute(ffn_kernel<T, kKind, kAct>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kKind)));
        once.mark(dev);
    }
    return VAE_OK;
}

template <int T, int kKind, int kAct = VAE_ACT_SILU>
int ffn_launch(const Maps& maps, Params& p, bool ahead, cudaStream_t stream) {
    int rc = ffn_setup<T, kKind, kAct>();
    if (rc != VAE_OK) return rc;
    p.status = device_status_ptr();
    if (p.status == nullptr) return VAE_ERR_CUDA;
    p.timeout_ns = wait_timeout_ns();
    p.nm = (p.rows + 2 * kTile - 1) / (2 * kTile);
    p.nfull = p.cols / p.cut.wide;
    const int each = p.nm * p.problems * p.cut.splits;
    p.full = each * p.nfull;
    p.rests = p.cut.rest > 0 ? each : 0;
    const int pairs = std::min(p.full + p.rests, sm_count() / 2);
    VAE_CUDA_CHECK(launch_kernel_as(ahead || pdl_enabled(), ffn_kernel<T, kKind, kAct>, dim3(2 * pairs), dim3(kThreads), smem_bytes(kKind),
                                    stream, maps, p));
    if (p.cut.splits > 1) {
        const long long n8 = static_cast<long long>(p.rows) * p.cols / 8;
        const unsigned grid = static_cast<unsigned>(std::min<long long>((n8 + 255) / 256, 152 * 8));
        VAE_CUDA_CHECK(launch_next(join_kernel<T>, dim3(grid, p.problems), dim3(256), 0, stream, static_cast<const float*>(p.parts),
                                   p.cut.splits, n8, p.out_f32, p.out[0], p.out[1], p.out[2], p.residual));
    }
    return VAE_OK;
}
// The products whose epilogue knows the activation (a branch on it for every element took more of the instruction
// cache than there is: 295 us instead of 100 at 16384 tokens).
template <int T, int kKind>
int ffn_launch_act(int act, const Maps& maps, Params& p, bool ahead, cudaStream_t stream) {
    if (act == VAE_ACT_SILU) return ffn_launch<T, kKind, VAE_ACT_SILU>(maps, p, ahead, stream);
    return act == VAE_ACT_GELU ? ffn_launch<T, kKind, VAE_ACT_GELU>(maps, p, ahead, stream)
                               : ffn_launch<T, kKind, VAE_ACT_GELU_TANH>(maps, p, ahead, stream);
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

int stages(int k) { return (k + kBk - 1) / kBk; }
Cut cut_gate(const vae_gated_ffn_desc& a) { return plan_cut(kGate, a.m, a.f, stages(a.c), 1); }
Cut cut_down(const vae_gated_ffn_desc& a) { return plan_cut(kDown, a.m, a.c, stages(a.f), 1); }
Cut cut_back_gate(const vae_gated_ffn_desc& a) { return plan_cut(kBackGate, a.m, a.f, stages(a.c), 1); }
Cut cut_dx(const vae_gated_ffn_desc& a) { return plan_cut(kDx, a.m, a.c, 2 * stages(a.f), 1); }
Cut cut_dw(const vae_gated_ffn_desc& a) { return plan_cut(kDw, a.f, a.c, stages(a.m), 3); }

bool on32(const void* q) { return reinterpret_cast<uintptr_t>(q) % 32 == 0; }

template <int T>
int ffn_forward(const vae_gated_ffn_desc& a, const void* x, const void* wg, const void* wu, const void* wd, const float* residual,
                void* y, void* gate, void* up, void* hidden, float* parts, cudaStream_t stream) {
    Maps maps;
    Params p{};
    p.cut = cut_gate(a);
    VAE_TRY(ffn_map(&maps.a[0], T, x, a.m, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wg, a.f, a.c, p.cut.wide));
    VAE_TRY(ffn_map(&maps.b[1], T, wu, a.f, a.c, p.cut.wide));
    p.rows = a.m;
    p.cols = a.f;
    p.problems = 1;
    p.nk = stages(a.c);
    p.segments = 1;
    p.out[0] = hidden;
    p.out[1] = gate;
    p.out[2] = up;
    p.wide = a.f % 16 == 0 && on32(hidden) && on32(gate) && on32(up);
    VAE_TRY((ffn_launch_act<T, kGate>(a.activation, maps, p, false, stream)));
    p = Params{};
    p.cut = cut_down(a);
    VAE_TRY(ffn_map(&maps.a[0], T, hidden, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wd, a.c, a.f, p.cut.wide / 2));
    p.rows = a.m;
    p.cols = a.c;
    p.problems = 1;
    p.nk = stages(a.f);
    p.segments = 1;
    p.out[0] = y;
    p.parts = parts;
    p.out_f32 = a.y_type == VAE_F32;
    p.residual = residual;
    p.wide = a.c % 16 == 0 && on32(y);
    return ffn_launch<T, kDown>(maps, p, true, stream);
}

// Workspace of the gradient: the largest |dy|, dgate, dup, partial sums.
struct BackSpace {
    size_t dgate, dup, parts, bytes;
};
BackSpace back_space(const vae_gated_ffn_desc& a) {
    BackSpace s;
    s.dgate = 256;
    s.dup = s.dgate + up256(mf_bytes(a));
    s.parts = s.dup + up256(mf_bytes(a));
    s.bytes = s.parts + std::max(parts_bytes(cut_dx(a), a.m, a.c, 1), parts_bytes(cut_dw(a), a.f, a.c, 3));
    return s;
}

template <int T>
int ffn_backward(const vae_gated_ffn_desc& a, const void* dy, const void* x, const void* wg, const void* wu, const void* wd,
                 const void* gate, const void* up, const void* hidden, void* dx, void* dwg, void* dwu, void* dwd, char* ws,
                 cudaStream_t stream) {
    const BackSpace at = back_space(a);
    unsigned* amax = nullptr;
    void *dgate = ws + at.dgate, *dup = ws + at.dup;
    float* parts = reinterpret_cast<float*>(ws + at.parts);
    bool ahead = false;
    if (T == VAE_F16) {
        amax = reinterpret_cast<unsigned*>(ws);
        VAE_CUDA_CHECK(cudaMemsetAsync(amax, 0, sizeof(unsigned), stream));
        const long long n8 = static_cast<long long>(a.m) * a.c / 8;
        const unsigned grid = static_cast<unsigned>(std::min<long long>((n8 + 255) / 256, 152 * 8));
        VAE_CUDA_CHECK(launch_kernel(amax_kernel, dim3(grid), dim3(256), 0, stream, static_cast<const uint4*>(dy), n8, amax));
        ahead = true;
    }
    Maps maps;
    Params p{};
    p.cut = cut_back_gate(a);
    VAE_TRY(ffn_map(&maps.a[0], T, dy, a.m, a.c, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wd, a.c, a.f, kBk));
    p.rows = a.m;
    p.cols = a.f;
    p.problems = 1;
    p.nk = stages(a.c);
    p.segments = 1;
    VAE_TRY(ffn_map(&maps.side[0], T, gate, a.m, a.f, 32));
    VAE_TRY(ffn_map(&maps.side[1], T, up, a.m, a.f, 32));
    VAE_TRY(ffn_map(&maps.side[2], T, dgate, a.m, a.f, 32));
    VAE_TRY(ffn_map(&maps.side[3], T, dup, a.m, a.f, 32));
    p.amax = amax;
    VAE_TRY((ffn_launch_act<T, kBackGate>(a.activation, maps, p, ahead, stream)));
    p = Params{};
    p.cut = cut_dx(a);
    VAE_TRY(ffn_map(&maps.a[0], T, dgate, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.a[1], T, dup, a.m, a.f, kTile));
    VAE_TRY(ffn_map(&maps.b[0], T, wg, a.f, a.c, kBk));
    VAE_TRY(ffn_map(&maps.b[1], T, wu, a.f, a.c, kBk));
    p.rows = a.m;
    p.cols = a.c;
    p.problems = 1;
    p.nk = stages(a.f);
    p.segments = 2;
    p.out[0] = dx;
    p.parts = parts;
    p.amax = amax;
    p.wide = a.c % 16 == 0 && on32(dx);
    VAE_TRY((ffn_launch<T, kDx>(maps, p, true, stream)));
    if (dwg == nullptr) return VAE_OK;
    p = Params{};
    p.cut = cut_dw(a);
    VAE_TRY(ffn_map(&maps.a[0], T, dgate, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.a[1], T, dup, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.a[2], T, hidden, a.m, a.f, kBk));
    VAE_TRY(ffn_map(&maps.b[0], T, x, a.m, a.c, kBk));
    maps.b[1] = maps.b[0];
    VAE_TRY(ffn_map(&maps.b[2], T, dy, a.m, a.c, kBk));
    p.rows = a.f;
    p.cols = a.c;
    p.problems = 3;
    p.nk = stages(a.m);
    p.segments = 1;
    p.out[0] = dwg;
    p.out[1] = dwu;
    p.out[2] = dwd;
    p.parts = parts;
    p.out_f32 = a.dw_type == VAE_F32;
    p.amax = amax;
    p.wide = a.c % 16 == 0 && on32(dwg) && on32(dwu);
    return ffn_launch<T, kDw>(maps, p, true, stream);
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" {

size_t vae_gated_ffn_workspace_bytes(const vae_gated_ffn_desc* desc) {
    clear_error();
    if (ffn_check(desc, false) != VAE_OK) return 0;
    // hidden, where it is not saved, and partial sums
    return (desc->save ? 0 : up256(mf_bytes(*desc))) + (desc->m <= kFewTokens ? 0 : parts_bytes(cut_down(*desc), desc->m, desc->c, 1));
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
    if (a.m <= kFewTokens)
        return ffn_few(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, st);
    float* parts = reinterpret_cast<float*>(static_cast<char*>(workspace_dev) + (save ? 0 : up256(mf_bytes(a))));
    return a.type == VAE_F16
               ? ffn_forward<VAE_F16>(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, parts, st)
               : ffn_forward<VAE_BF16>(a, x_dev, w_gate_dev, w_up_dev, w_down_dev, residual_dev, y_dev, gate_dev, up_dev, hidden, parts, st);
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
