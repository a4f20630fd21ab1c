// Multi-head attention, forward (the C entry point is in vae_mha.cu).
//
// o = softmax(scale q k^T) v in one pass over the keys: S = Q K^T of a 128-row
// and a 128-key tile accumulates in TMEM, four softmax warps (a row per thread)
// read it, keep the running maximum m and sum l, and write P = 2^(S - m) back
// over S as 16-bit pairs; O += P V takes P from TMEM and V as TMA left it
// (MN-major), so that nothing but Q, K and V passes through shared memory.
//
// A CTA runs two such streams, because one stream alone would leave the tensor
// cores idle while its softmax runs: while the MMA thread issues PV and the
// next S of one stream, the softmax warps of the other work.
//   Two query tiles (pair): both streams meet the same key tiles; K and V are
//   read once for 256 rows.
//   One query tile (alt, where there are too few tiles to fill the GPU): the
//   streams take every other key tile and their (m, l, O) join at the end
//   through shared memory.
//   Few rows (narrow: 32 at most, as for single tokens): one tile holds its rows
//   four times, once per TMEM lane quadrant, and each quadrant's warp takes a
//   quarter of the keys, so that the softmax of a few rows is not one warp's
//   chain of 128 keys; eight partial (m, l, O) join at the end. Up to 16 rows lie
//   twice in each quadrant, for P in two 16-bit parts.
// In either form the keys may be split over CTAs, whose f32 partial rows a
// second kernel joins in a fixed order: for single tokens over a long cache, and
// where a last wave of CTAs would leave most SMs without work.
//
// P is held as 2^(S - m + kBias) with m moved only when the new maximum is 2^8
// over it: at most 2^14, exact scaling, and f16 keeps P down to 2^-20 of the
// row's largest at full precision. O is scaled when m moves (rare); the S of a
// stream is issued behind the PV before it, so S having arrived means that O
// may be touched. Rows and keys of tensors behind their lengths may hold NaN:
// masked scores are replaced before the maximum, and V's rows are zeroed in
// shared memory on the one tile that the length ends in.
//
// A row sees no key exactly where its sum l is 0: the key of a row's first maximum
// adds 2^kBias to it, and l is scaled down only when a new one does. (The maximum
// does not tell: it passes over NaN. A NaN score leaves l, O and so o and lse NaN,
// through every join.)
//
// Measured on GB300: 16384 tokens x 9 heads x 128 in f16 840 to 920 us (1340 to
// 1470 TFLOP/s; with the softmax left out 786, with no hand-over between warps
// 717). Bound by the MMAs: S reads both operands from shared memory, 8 KB in 64
// cycles, which is all that it gives; the products alone take 2400 cycles of a
// step of both streams, which took 2970 before the registers were moved (below).
// Eight softmax warps and not sixteen (half a row each, maxima traded: 1282 us);
// a tile's PV whole and not from its first half of P on (918 against 876 us), a
// tile whole and not S and P in halves of 64 keys (1193 against 882 us). One
// token over four caches of up to 32760 keys (201 MB): 45 us a call in a graph,
// 6.3 TB/s while it streams.
#include <cmath>

#include "vae_mha_fwd.h"

namespace vae {

namespace {

constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 4) * 32;  // whole warpgroups; the last two warps wait at the end
constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
// A softmax thread holds a row's 128 scores, which 168 registers (65536 over
// three warpgroups) do not fit without spilling: the other warpgroup gives some
// of its own up. 16384 tokens, 9 heads of 128: 876 us without, 216 + 72 841,
// 208 + 88 875, 224 + 56 902 (the MMA warp's group spills); of 64, whose ring has
// more stages: 738, 698, 677, 693. (Narrow, a thread holds 32 scores: not needed.)
constexpr int kLaunchRegs = 168;
template <int kSteps>
struct FwdRegs {
    static constexpr int kSoft = kSteps > 4 ? 216 : 208, kOther = kSteps > 4 ? 72 : 88;
    static_assert(kSoftWarps * kSoft + 4 * kOther <= (kSoftWarps + 4) * kLaunchRegs, "more registers than the launch has");
};
constexpr uint32_t kTmemCols = 512;  // S0 | S1 | O0 | O1, 128 columns each
constexpr int kTargetCtas = 152;     // one CTA per SM

template <int kSteps>  // 16-channel steps of a row
struct FwdCfg {
    static constexpr int kCh = kSteps > 4 ? 2 : 1;  // 64-channel chunks
    static constexpr int kTileBytes = kCh * kMhaChunkBytes;
    static constexpr int kStages = kCh == 2 ? 5 : 8;
    static constexpr int kRing = 2 * kTileBytes;  // behind the two Q tiles
    static constexpr int kBars = kRing + kStages * kTileBytes;
    static constexpr int kSmem = 1024 + kBars + 512;
};
static_assert(FwdCfg<8>::kSmem <= 232448 && FwdCfg<4>::kSmem <= 232448, "attention shared memory over 227 KB");

struct FwdParams {
    MhaShape s;
    int alt;
    int twice;        // narrow, the rows twice in each quadrant: the second copies' P is what the first rounded off
    int nsplit;       // with nsplit > 1: nsplit * b pieces of key tiles, shared out by the entries' lengths
    float scale_log2;
    void* o;
    MhaStrides os;
    float* lse;
    float *po, *plse;  // the pieces' partial rows: [nsplit * b][hq * sq][d], [nsplit * b][hq * sq] (log2)
    DevStatus* status;
    unsigned long long timeout_ns;
};

struct FwdSmem {
    uint8_t *q, *ring;
    uint64_t *full, *empty;             // [kStages]
    uint64_t *s_full, *p_full, *o_full;  // [2 streams]
    uint64_t *q_full, *fix, *drain;
    uint32_t* tmem_slot;
    int* abort_flag;
    float* ml;  // [2][128]: (m, l) of the second stream's rows (alt)
};

template <int kSteps>
__device__ __forceinline__ FwdSmem fwd_carve(uint8_t* raw) {
    using C = FwdCfg<kSteps>;
    FwdSmem s;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.q = base;
    s.ring = base + C::kRing;
    uint64_t* b = reinterpret_cast<uint64_t*>(base + C::kBars);
    s.full = b;
    s.empty = b + C::kStages;
    s.s_full = b + 2 * C::kStages;
    s.p_full = s.s_full + 2;
    s.o_full = s.p_full + 2;
    s.q_full = s.o_full + 2;
    s.fix = s.q_full + 1;
    s.drain = s.fix + 1;
    s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
    s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
    s.ml = reinterpret_cast<float*>(s.ring + 128 * 128 * 4 / (C::kCh == 2 ? 1 : 2));  // behind the exchanged O
    return s;
}

__device__ __forceinline__ bool fwait(uint64_t* bar, uint32_t parity, const FwdSmem& s, const FwdParams& p) {
    return mbar_wait(smem_u32(bar), parity, s.abort_flag, p.timeout_ns, p.status, kWhereAttn);
}

// What a CTA works on; the same values in every thread.
struct FwdWork {
    int e, hk, sub;   // batch entry, key head, part of the group
    int tile[2];      // the streams' 128-row tiles (alt: the same)
    int piece;        // which partial rows (nsplit > 1)
    int ql, kl;
    int kb0, n;       // key tiles [kb0, kb0 + n)
    int streams;
};

__device__ __forceinline__ int tile_limit(const MhaShape& s, int tile, int ql, int kl) {
    const int i0 = (tile * kMhaTile) >> s.gp_log2;
    int i1 = ((tile + 1) * kMhaTile - 1) >> s.gp_log2;
    if (tile >= s.ntile || i0 >= ql) return 0;
    if (i1 >= ql) i1 = ql - 1;
    return mha_key_limit(i1, ql, kl, s.block);
}

// How nsplit * b pieces are shared out: each entry's key tiles in runs of
// `run`, the shortest for which the runs of all entries are no more than the
// pieces. Long caches beside short ones then give every CTA about as much.
// (The whole warp, converged; `first` of an entry is the number of runs before it.)
struct Pieces {
    int run, first, count, e;
};
__device__ __forceinline__ int key_tiles(const MhaShape& s, int e) {
    return (mha_len(s.k_len, e, s.sk) + kMhaTile - 1) / kMhaTile;
}
__device__ __forceinline__ int piece_run(const MhaShape& s, int pieces) {
    const int lane = threadIdx.x & 31;
    int all = 0;
    for (int e = lane; e < s.b; e += 32) all += key_tiles(s, e);
    all = __reduce_add_sync(0xffffffffu, all);
    for (int run = all > pieces ? (all - 1) / pieces + 1 : 1;; ++run) {  // (ends: one run an entry is enough at last)
        int n = 0;
        for (int e = lane; e < s.b; e += 32) n += (key_tiles(s, e) + run - 1) / run;
        if (__reduce_add_sync(0xffffffffu, n) <= pieces) return run;
    }
}
// The entry that piece `at` belongs to (e = b: none), or the runs of entry `of` (at < 0).
__device__ __forceinline__ Pieces find_piece(const MhaShape& s, int pieces, int at, int of) {
    const int lane = threadIdx.x & 31;
    Pieces r;
    r.run = piece_run(s, pieces);
    r.e = s.b;
    r.first = r.count = 0;
    int before = 0;
    for (int e0 = 0; e0 < s.b; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < s.b ? (key_tiles(s, e) + r.run - 1) / r.run : 0;
        int upto = n;  // inclusive scan
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const int first = before + upto - n;
        const unsigned hit = __ballot_sync(0xffffffffu, at < 0 ? e == of : (at >= first && at < first + n));
        if (hit != 0u) {
            const int l = __ffs(static_cast<int>(hit)) - 1;
            r.first = __shfl_sync(0xffffffffu, first, l);
            r.count = __shfl_sync(0xffffffffu, n, l);
            r.e = e0 + l;
            return r;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return r;
}

__device__ __forceinline__ FwdWork fwd_work(const FwdParams& p) {
    const MhaShape& s = p.s;
    FwdWork w;
    const int nt = p.alt ? s.ntile : (s.ntile + 1) / 2;
    int r = blockIdx.x;
    const int t = nt - 1 - r % nt;  // the last tiles see the most keys where blocks limit them: first
    r /= nt;
    w.piece = r % (p.nsplit * s.b);
    r /= p.nsplit * s.b;
    w.sub = r % s.nsub;
    w.hk = r / s.nsub;
    int run = s.nkb, at = 0;
    w.e = w.piece;
    w.n = 0;
    w.streams = 0;
    w.tile[0] = p.alt ? t : 2 * t;
    w.tile[1] = p.alt ? t : 2 * t + 1;
    if (p.nsplit > 1) {
        const Pieces x = find_piece(s, p.nsplit * s.b, w.piece, 0);
        w.e = x.e;
        run = x.run;
        at = w.piece - x.first;
        if (w.e == s.b) return w;  // no piece left
    }
    w.ql = mha_len(s.q_len, w.e, s.sq);
    w.kl = mha_len(s.k_len, w.e, s.sk);
    const int l0 = tile_limit(s, w.tile[0], w.ql, w.kl), l1 = p.alt ? 0 : tile_limit(s, w.tile[1], w.ql, w.kl);
    const int nb = ((l0 > l1 ? l0 : l1) + kMhaTile - 1) / kMhaTile;
    w.kb0 = at * run;
    const int end = w.kb0 + run < nb ? w.kb0 + run : nb;
    w.n = end > w.kb0 ? end - w.kb0 : 0;
    w.streams = p.alt ? (w.n >= 2 ? 2 : 1) : ((w.tile[1] * kMhaTile) >> s.gp_log2) < w.ql && w.tile[1] < s.ntile ? 2 : 1;
    return w;
}

template <int kSteps, bool kNarrow>
__device__ void fwd_producer(const FwdParams& p, const FwdSmem& s, const FwdWork& w, const CUtensorMap* mq,
                             const CUtensorMap* mk, const CUtensorMap* mv, int lane) {
    using C = FwdCfg<kSteps>;
    const uint64_t pol = policy_evict_normal();
    const int gp = 1 << p.s.gp_log2;
    const int h0 = w.hk * p.s.g + w.sub * gp;
    const int nq = p.alt ? 1 : w.streams;
    uint32_t armed = 0, arm_par = 0;
    if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(s.q_full), static_cast<uint32_t>(nq * C::kTileBytes));
        for (int t = 0; t < nq; ++t)
            for (int c = 0; c < C::kCh; ++c)
                for (int r = 0; r < (!kNarrow ? 1 : p.twice ? 8 : 4); ++r)  // (the map's boxes are 128, 16 or 32 rows)
                    tma_load_4d(smem_u32(s.q + t * C::kTileBytes + c * kMhaChunkBytes + r * (kMhaChunkBytes / (p.twice ? 8 : 4))), mq,
                                smem_u32(s.q_full), c * 64, h0, (w.tile[t] * kMhaTile) >> p.s.gp_log2, w.e, pol);
    }
    const int ahead = p.alt ? 2 : 1;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true, fixed = false;
    // K tiles run `ahead` tiles before V: the order in which the MMA thread takes them
    auto load = [&](bool is_v, int j) {
        const int kb = w.kb0 + j;
        if (!warp_all(fwait(&s.empty[stage], phase ^ 1u, s, p))) return false;
        // the tile that a length ends in, inside the tensor: rows behind it may hold anything
        const bool fix = is_v && (kb + 1) * kMhaTile > w.kl && w.kl < p.s.sk;
        const uint32_t fb = smem_u32(fix ? s.fix : &s.full[stage]);
        uint8_t* dst = s.ring + stage * C::kTileBytes;
        if (lane == 0) {
            mbar_arrive_expect_tx(fb, static_cast<uint32_t>(C::kTileBytes));
            for (int c = 0; c < C::kCh; ++c)
                tma_load_4d(smem_u32(dst + c * kMhaChunkBytes), is_v ? mv : mk, fb, c * 64, w.hk, kb * kMhaTile, w.e, pol);
        }
        if (fix) {
            armed &= ~(1u << stage);  // (its copy completes on the fix barrier)
            fixed = true;
            __syncwarp();
            if (!warp_all(fwait(s.fix, 0u, s, p))) return false;
            mha_zero_rows(dst, w.kl - kb * kMhaTile, kMhaTile, C::kCh, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.full[stage]));
        } else {
            armed |= 1u << stage;
            arm_par = (arm_par & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
        }
        return true;
    };
    for (int j = 0; ok && j < ahead && j < w.n; ++j) ok = load(false, j);
    __syncthreads();  // the first tiles are on their way while the CTA is set up
    for (int j = 0; ok && j < w.n; ++j) {
        ok = load(true, j);
        if (ok && j + ahead < w.n) ok = load(false, j + ahead);
    }
    // Every copy lands before the CTA can exit.
    if (lane == 0) {
        int never = 0;
        (void)mbar_wait(smem_u32(s.q_full), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
        if (fixed) (void)mbar_wait(smem_u32(s.fix), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
        for (int i = 0; i < C::kStages; ++i)
            if (armed & (1u << i))
                (void)mbar_wait(smem_u32(&s.full[i]), (arm_par >> i) & 1u, &never, p.timeout_ns, p.status, kWhereDrain);
    }
    __syncwarp();
}

template <int T, int kSteps>
__device__ void fwd_mma(const FwdParams& p, const FwdSmem& s, const FwdWork& w) {
    using C = FwdCfg<kSteps>;
    constexpr uint32_t id_s = mha_idesc(T, 128, 128, false), id_o = mha_idesc(T, 128, kSteps * 16, true);
    const uint64_t qd = sw128_kmajor_desc(smem_u32(s.q));
    const uint64_t kdesc = sw128_kmajor_desc(smem_u32(s.ring)), vdesc = sw128_mnmajor_desc(smem_u32(s.ring));
    int stage = 0;
    uint32_t phase = 0;
    uint32_t pp[2] = {0u, 0u};
    auto wait = [&](uint64_t* bar, uint32_t par) { return warp_all(fwait(bar, par, s, p)); };
    auto next = [&]() {
        if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    };
    auto issue_s = [&](int t, int st) {
        mma_ss<kSteps>(static_cast<uint32_t>(t * 128), qd + (p.alt ? 0u : static_cast<uint32_t>(t) * (C::kTileBytes >> 4)),
                       kdesc + static_cast<uint32_t>(st) * (C::kTileBytes >> 4), id_s);
        umma_commit(smem_u32(&s.s_full[t]));
    };
    bool ok = wait(s.q_full, 0u);
    const int ahead = p.alt ? 2 : 1;
    for (int j = 0; ok && j < ahead && j < w.n; ++j) {
        ok = wait(&s.full[stage], phase);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            if (p.alt) {
                issue_s(j & 1, stage);
            } else {
                issue_s(0, stage);
                if (w.streams == 2) issue_s(1, stage);
            }
            umma_commit(smem_u32(&s.empty[stage]));
        }
        __syncwarp();
        next();
    }
    for (int j = 0; ok && j < w.n; ++j) {
        ok = wait(&s.full[stage], phase);
        if (!ok) break;
        const int vst = stage;
        next();
        const bool more = j + ahead < w.n;
        const int kst = stage;
        const uint32_t kph = phase;
        if (more) next();
        const int t0 = p.alt ? j & 1 : 0, t1 = p.alt ? t0 + 1 : w.streams;
        for (int t = t0; ok && t < t1; ++t) {
            ok = wait(&s.p_full[t], t == 0 ? pp[0] : pp[1]);
            if (!ok) break;
            if (t == 0) pp[0] ^= 1u;
            else pp[1] ^= 1u;
            if (more && t == t0) {
                ok = wait(&s.full[kst], kph);
                if (!ok) break;
            }
            tc_fence_after();
            if (elect_one()) {
                mma_ts<32>(256u + static_cast<uint32_t>(t * 128), static_cast<uint32_t>(t * 128),
                           vdesc + static_cast<uint32_t>(vst) * (C::kTileBytes >> 4), id_o, (p.alt ? j < 2 : j == 0) ? 0u : 1u);
                if (t + 1 == t1) umma_commit(smem_u32(&s.empty[vst]));
                if (more) {
                    issue_s(t, kst);
                    if (t + 1 == t1) umma_commit(smem_u32(&s.empty[kst]));
                } else {
                    umma_commit(smem_u32(&s.o_full[t]));
                }
            }
            __syncwarp();
        }
    }
    if (elect_one()) {
        umma_commit(smem_u32(s.drain));
        int never = 0;
        (void)mbar_wait(smem_u32(s.drain), 0u, &never, p.timeout_ns, p.status, kWhereDrain);
    }
    __syncwarp();
}

// One row's result: `inv` scales O, lse2 is in units of log 2.
template <int T, int kSteps>
__device__ void fwd_store(const FwdParams& p, const FwdWork& w, uint32_t tO, int i, int h, bool live, float w0,
                          const float* o1, float w1, float inv, float lse2) {
    const int d = p.s.d;
    const long long row = (static_cast<long long>(w.e) * p.s.hq + h) * p.s.sq + i;
    const long long prow = (static_cast<long long>(w.piece) * p.s.hq + h) * p.s.sq + i;
    for (int c = 0; c < d; c += 16) {
        uint32_t r[16];
        __syncwarp();
        tmem_ld16(tO + static_cast<uint32_t>(c), r);
        tmem_ld_wait_regs(r);
        if (!live) continue;
#pragma unroll
        for (int u = 0; u < 16; u += 8) {
            if (c + u >= d) continue;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = __uint_as_float(r[u + k]) * w0;
                if (o1 != nullptr) v[k] += o1[(c + u + k) * 128] * w1;
                v[k] *= inv;
            }
            if (p.nsplit > 1)
                store8<VAE_F32>(p.po + prow * d + c + u, v);
            else
                store8<T>(static_cast<typename Elem<T>::type*>(p.o) + w.e * p.os.b + i * p.os.s + h * p.os.h + c + u, v);
        }
    }
    if (!live) return;
    if (p.nsplit > 1) p.plse[prow] = lse2;
    else p.lse[row] = lse2 * 0.69314718055994530942f;
}

// The weight of a part whose maximum is m and sum l beside the maximum mm of all parts: 0 where it saw no key. (m and mm
// are -infinity where every score that a part saw is NaN, and l is NaN then.)
__device__ __forceinline__ float part_weight(float m, float l, float mm) {
    return l == 0.f ? 0.f : m == mm ? 1.f : mha_ex2(m - mm);
}

template <int T, int kSteps>
__device__ void fwd_softmax(const FwdParams& p, const FwdSmem& s, const FwdWork& w, uint32_t tmem, int warp, int lane) {
    // f16 holds P 2^kBias high (the sum l too): 2^(8 + 6) at most
    constexpr float kBias = T == VAE_F16 ? 6.f : 0.f;
    const int t = warp >> 2, quad = warp & 3;
    const int gp = 1 << p.s.gp_log2;
    const int r = w.tile[t] * kMhaTile + quad * 32 + lane;
    const int i = r >> p.s.gp_log2, h = w.hk * p.s.g + w.sub * gp + (r & (gp - 1));
    const bool live = i < w.ql;
    const int lim = live ? mha_key_limit(i, w.ql, w.kl, p.s.block) : 0;
    const int wmin = __reduce_min_sync(0xffffffffu, live ? lim : 0x7fffffff);  // (no live row: nothing is computed)
    const bool any_live = __any_sync(0xffffffffu, live);
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * 128), tO = tS + 256u;
    const int dn = (p.s.d + 15) / 16 * 16;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int step = p.alt ? 2 : 1;
    uint32_t par = 0;
    const bool runs = t < w.streams;
    for (int j = p.alt ? t : 0; runs && j < w.n; j += step, par ^= 1u) {
        ok = warp_all(fwait(&s.s_full[t], par, s, p));
        if (!ok) break;
        if (any_live) {
            tc_fence_after();
            uint32_t x[8][16];
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) tmem_ld16(tS + static_cast<uint32_t>(c * 16), x[c]);
#pragma unroll
            for (int c = 0; c < 8; ++c) tmem_ld_wait_regs(x[c]);
            const int k0 = (w.kb0 + j) * kMhaTile;
            if (k0 + kMhaTile > wmin) {
                const int left = lim - k0;
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (c * 16 + k >= left) x[c][k] = 0xff800000u;  // -infinity
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int k = 0; k < 16; k += 2)
                    mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
            if (j < step) {  // the stream's first tile
                m = top;
            } else {
                const bool up = top > m + 8.f;
                if (__any_sync(0xffffffffu, up)) {
                    const float alpha = up ? mha_ex2(m - top) : 1.f;
                    if (up) m = top;
                    l *= alpha;
                    for (int c = 0; c < dn; c += 16) {
                        uint32_t o[16];
                        __syncwarp();
                        tmem_ld16(tO + static_cast<uint32_t>(c), o);
                        tmem_ld_wait_regs(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        tmem_st16(tO + static_cast<uint32_t>(c), o);
                    }
                }
            }
            const float sub = m == -INFINITY ? 0.f : kBias - m;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), sub2 = make_float2(sub, sub);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                uint32_t h2[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint32_t* y = x[c + (k >> 3)] + 2 * (k & 7);
                    float2 f = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, sub2);
                    f.x = mha_ex2(f.x);
                    f.y = mha_ex2(f.y);
                    sum[k & 1] = add2(sum[k & 1], f);
                    h2[k] = pack2<T>(f.x, f.y);
                }
                tmem_st16(tS + static_cast<uint32_t>(c * 8), h2);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_st_wait();
            tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.p_full[t]));
    }
    const bool join = p.alt && w.streams == 2;
    if (runs && ok) ok = warp_all(fwait(&s.o_full[t], 0u, s, p));
    if (join) {
        // the second stream's rows pass through the ring, which every MMA has read by then
        if (ok && t == 1) ok = warp_all(fwait(&s.o_full[0], 0u, s, p));
        float* o1 = reinterpret_cast<float*>(s.ring);
        const int rr = quad * 32 + lane;
        if (t == 1 && ok && any_live) {
            tc_fence_after();
            for (int c = 0; c < dn; c += 16) {
                uint32_t o[16];
                __syncwarp();
                tmem_ld16(tO + static_cast<uint32_t>(c), o);
                tmem_ld_wait_regs(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o1[(c + k) * 128 + rr] = __uint_as_float(o[k]);
            }
            s.ml[rr] = m;
            s.ml[128 + rr] = l;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // (every softmax warp comes here, timed out or not)
        if (t == 0 && ok && any_live && *static_cast<volatile int*>(s.abort_flag) == 0) {
            tc_fence_after();
            const float m1 = s.ml[rr], l1 = s.ml[128 + rr];
            const float mm = fmaxf(m, m1);
            const float w0 = part_weight(m, l, mm), w1 = part_weight(m1, l1, mm);
            const float ll = w0 * l + w1 * l1;
            fwd_store<T, kSteps>(p, w, tO, i, h, live, w0, o1 + rr, w1, ll == 0.f ? 0.f : 1.f / ll,
                              ll == 0.f ? -INFINITY : mm - kBias + log2f(ll));
        }
    } else if (runs && ok && any_live) {
        tc_fence_after();
        const bool none = l == 0.f;
        fwd_store<T, kSteps>(p, w, tO, i, h, live, 1.f, nullptr, 0.f, none ? 0.f : 1.f / l,
                          none ? -INFINITY : m - kBias + log2f(l));
    }
}

// The narrow form's softmax: every quadrant holds the same 32 rows; its warp
// takes 32 of a tile's 128 keys.
template <int T, int kSteps>
__device__ void fwd_softmax_narrow(const FwdParams& p, const FwdSmem& s, const FwdWork& w, int warp, int lane) {
    constexpr float kBias = T == VAE_F16 ? 6.f : 0.f;
    const int t = warp >> 2, quad = warp & 3;
    const int gp = 1 << p.s.gp_log2;
    const int rr = p.twice ? lane & 15 : lane;
    const int i = rr >> p.s.gp_log2, h = w.hk * p.s.g + w.sub * gp + (rr & (gp - 1));
    const bool live = i < w.ql;
    const int lim = live ? mha_key_limit(i, w.ql, w.kl, p.s.block) : 0;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = lane_off + static_cast<uint32_t>(t * 128), tO = tS + 256u;
    const int dn = (p.s.d + 15) / 16 * 16;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    uint32_t par = 0;
    for (int j = t; j < w.n; j += 2, par ^= 1u) {
        ok = warp_all(fwait(&s.s_full[t], par, s, p));
        if (!ok) break;
        tc_fence_after();
        uint32_t x[2][16];
        __syncwarp();
        tmem_ld16(tS + static_cast<uint32_t>(quad * 32), x[0]);
        tmem_ld16(tS + static_cast<uint32_t>(quad * 32 + 16), x[1]);
        tmem_ld_wait_regs(x[0]);
        tmem_ld_wait_regs(x[1]);
        const int left = lim - (w.kb0 + j) * kMhaTile - quad * 32;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if (k >= left) x[0][k] = 0xff800000u;  // -infinity
            if (16 + k >= left) x[1][k] = 0xff800000u;
            mx[0] = fmaxf(mx[0], __uint_as_float(x[0][k]));
            mx[1] = fmaxf(mx[1], __uint_as_float(x[1][k]));
        }
        const float top = fmaxf(mx[0], mx[1]) * p.scale_log2;
        if (j < 2) {
            m = top;
        } else {
            const bool up = top > m + 8.f;
            if (__any_sync(0xffffffffu, up)) {
                const float alpha = up ? mha_ex2(m - top) : 1.f;
                if (up) m = top;
                l *= alpha;
                for (int c = 0; c < dn; c += 16) {
                    uint32_t o[16];
                    __syncwarp();
                    tmem_ld16(tO + static_cast<uint32_t>(c), o);
                    tmem_ld_wait_regs(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    tmem_st16(tO + static_cast<uint32_t>(c), o);
                }
            }
        }
        const float sub = m == -INFINITY ? 0.f : kBias - m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), sub2 = make_float2(sub, sub);
        float2 sum = make_float2(0.f, 0.f);
        uint32_t h2[16], zero[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const uint32_t* y = x[k >> 3] + 2 * (k & 7);
            float2 f = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, sub2);
            f.x = mha_ex2(f.x);
            f.y = mha_ex2(f.y);
            sum = add2(sum, f);
            h2[k] = rr == lane ? pack2<T>(f.x, f.y) : pack2_rest<T>(f.x, f.y);
            zero[k] = 0u;
        }
        l += sum.x + sum.y;
        __syncwarp();
        // the other quadrants' keys count as 0 in these lanes
        tmem_st16(tS + static_cast<uint32_t>(quad * 16), h2);
        tmem_st16(tS + static_cast<uint32_t>((quad ^ 1) * 16), zero);
        tmem_st16(tS + static_cast<uint32_t>((quad ^ 2) * 16), zero);
        tmem_st16(tS + static_cast<uint32_t>((quad ^ 3) * 16), zero);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.p_full[t]));
    }
    // The parts pass through the ring, which every MMA has read once both streams are done: [part][channel][32 rows].
    const int parts = w.streams * 4;
    const bool runs = t < w.streams;
    if (ok) ok = warp_all(fwait(&s.o_full[0], 0u, s, p) && (w.streams == 1 || fwait(&s.o_full[1], 0u, s, p)));
    float* o = reinterpret_cast<float*>(s.ring);
    float* ml = o + 8 * dn * 32;  // [2][8 parts][32 rows]
    if (ok && runs) {
        tc_fence_after();
        for (int c = 0; c < dn; c += 16) {
            uint32_t v[16];
            __syncwarp();
            tmem_ld16(tO + static_cast<uint32_t>(c), v);
            tmem_ld_wait_regs(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[(warp * dn + c + k) * 32 + lane] = __uint_as_float(v[k]);
        }
        ml[warp * 32 + lane] = m;
        ml[256 + warp * 32 + lane] = l;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");  // (every softmax warp comes here, timed out or not)
    if (!ok || *static_cast<volatile int*>(s.abort_flag) != 0) return;
    // a row per lane, a slice of the channels per warp
    float mm = -INFINITY;
    for (int k = 0; k < parts; ++k) mm = fmaxf(mm, ml[k * 32 + lane]);
    float wt[8], ll = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float lk = k < parts ? ml[256 + k * 32 + lane] : 0.f;
        wt[k] = k < parts ? part_weight(ml[k * 32 + lane], lk, mm) : 0.f;
        ll += wt[k] * lk;
    }
    if (!live || rr != lane) return;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const long long row = (static_cast<long long>(w.e) * p.s.hq + h) * p.s.sq + i;
    const long long prow = (static_cast<long long>(w.piece) * p.s.hq + h) * p.s.sq + i;
    for (int c = warp * 8; c < p.s.d; c += 64) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < parts) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float* x = o + (k * dn + c + u) * 32 + lane;
                    v[u] += wt[k] * (p.twice ? x[0] + x[16] : x[0]);
                }
            }
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= inv;
        if (p.nsplit > 1)
            store8<VAE_F32>(p.po + prow * p.s.d + c, v);
        else
            store8<T>(static_cast<typename Elem<T>::type*>(p.o) + w.e * p.os.b + i * p.os.s + h * p.os.h + c, v);
    }
    if (warp == 0) {
        const float lse2 = ll == 0.f ? -INFINITY : mm - kBias + log2f(ll);
        if (p.nsplit > 1) p.plse[prow] = lse2;
        else p.lse[row] = lse2 * 0.69314718055994530942f;
    }
}

// The third warpgroup: it sets up the barriers and TMEM, loads and issues the products.
template <int T, int kSteps, bool kNarrow>
__device__ __forceinline__ void fwd_feed(const FwdParams& p, const FwdSmem& s, const FwdWork& w, const CUtensorMap& mq,
                                         const CUtensorMap& mk, const CUtensorMap& mv, int warp, int lane) {
    using C = FwdCfg<kSteps>;
    if (warp == kTmaWarp) {
        if (lane == 0) {
            *s.abort_flag = 0;
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(smem_u32(&s.full[i]), 1u);
                mbar_init(smem_u32(&s.empty[i]), 1u);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&s.s_full[i]), 1u);
                mbar_init(smem_u32(&s.p_full[i]), 4u);
                mbar_init(smem_u32(&s.o_full[i]), 1u);
            }
            mbar_init(smem_u32(s.q_full), 1u);
            mbar_init(smem_u32(s.fix), 1u);
            mbar_init(smem_u32(s.drain), 1u);
            fence_mbar_init();
            fence_proxy_async_smem();
        }
        __syncwarp();
        fwd_producer<kSteps, kNarrow>(p, s, w, &mq, &mk, &mv, lane);  // (meets the others' __syncthreads)
    } else {
        if (warp == kMmaWarp) {
            tmem_alloc(smem_u32(s.tmem_slot), kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == kMmaWarp) fwd_mma<T, kSteps>(p, s, w);
    }
}

template <int T, int kSteps, bool kNarrow>
__global__ void __launch_bounds__(kThreads, 1)
    mha_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const FwdParams p) {
    using C = FwdCfg<kSteps>;
    extern __shared__ uint8_t smem_raw[];
    const FwdSmem s = fwd_carve<kSteps>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
    }
    pdl_wait();
    const FwdWork w = fwd_work(p);
    if (w.e == p.s.b) return;  // more pieces than runs of key tiles
    if (p.s.fill && p.nsplit == 1)  // (else the joining kernel does)
        for (int t = 0; t < (p.alt ? 1 : 2); ++t)
            mha_fill_queries(p.s, w.e, w.hk, w.sub, w.tile[t], w.ql, p.o, p.os.b, p.os.s, p.os.h, p.lse);
    if (w.n == 0) {  // no key: rows within the length give 0 and -infinity
        const int gp = 1 << p.s.gp_log2;
        for (int t = 0; t < (p.alt ? 1 : 2); ++t) {
            const int r = w.tile[t] * kMhaTile + threadIdx.x;
            const int i = r >> p.s.gp_log2, h = w.hk * p.s.g + w.sub * gp + (r & (gp - 1));
            if (threadIdx.x >= kMhaTile || w.tile[t] >= p.s.ntile || i >= w.ql) continue;
            const long long row = (static_cast<long long>(w.e) * p.s.hq + h) * p.s.sq + i;
            if (p.nsplit > 1) {
                p.plse[(static_cast<long long>(w.piece) * p.s.hq + h) * p.s.sq + i] = -INFINITY;
            } else {
                const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                for (int c = 0; c < p.s.d; c += 8)
                    store8<T>(static_cast<typename Elem<T>::type*>(p.o) + w.e * p.os.b + i * p.os.s + h * p.os.h + c, z);
                p.lse[row] = -INFINITY;
            }
        }
        return;
    }
    constexpr uint32_t tmem = 0u;  // all 512 columns are this CTA's: they start at 0
    if (warp < kSoftWarps) {
        if constexpr (!kNarrow) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FwdRegs<kSteps>::kSoft));
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if constexpr (kNarrow) fwd_softmax_narrow<T, kSteps>(p, s, w, warp, lane);
        else fwd_softmax<T, kSteps>(p, s, w, tmem, warp, lane);
    } else {
        if constexpr (!kNarrow) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FwdRegs<kSteps>::kOther));
        fwd_feed<T, kSteps, kNarrow>(p, s, w, mq, mk, mv, warp, lane);
    }
    pdl_launch_dependents();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the pieces' partial rows: a warp per row, pieces in order.
template <int T>
__global__ void __launch_bounds__(128) mha_join_kernel(const FwdParams p) {
    pdl_wait();
    const MhaShape& s = p.s;
    const long long rows = static_cast<long long>(s.b) * s.hq * s.sq, per = static_cast<long long>(s.hq) * s.sq;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= rows) return;
    const int i = static_cast<int>(row % s.sq), h = static_cast<int>(row / s.sq % s.hq);
    const int e = static_cast<int>(row / per);
    if (i >= mha_len(s.q_len, e, s.sq)) {
        if (s.fill) {
            if (lane < 4) mha_fill_row(p.o, e * p.os.b + i * p.os.s + h * p.os.h, s.d, lane);
            if (lane == 0) p.lse[row] = -INFINITY;
        }
        return;
    }
    const Pieces x = find_piece(s, p.nsplit * s.b, -1, e);
    const long long row0 = x.first * per + (row - e * per);  // its place in the entry's first piece
    float mm = -INFINITY;
    for (int k = lane; k < x.count; k += 32) mm = fmaxf(mm, p.plse[k * per + row0]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    // Eight pieces' loads in flight together; a piece that the row sees nothing of has written nothing but its -infinity.
    float ll = 0.f;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const int c = lane * 4 < s.d ? lane * 4 : 0;
    for (int k0 = 0; k0 < x.count; k0 += 8) {
        float y[8];
        float4 f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = k0 + u < x.count ? k0 + u : x.count - 1;
            y[u] = p.plse[k * per + row0];
            f[u] = *reinterpret_cast<const float4*>(p.po + (k * per + row0) * s.d + c);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (k0 + u >= x.count || y[u] == -INFINITY) continue;
            const float wt = mha_ex2(y[u] - mm);
            ll += wt;
            v[0] += f[u].x * wt;
            v[1] += f[u].y * wt;
            v[2] += f[u].z * wt;
            v[3] += f[u].w * wt;
        }
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;  // (a piece's NaN passes through its weight)
    if (lane * 4 < s.d) {
        uint2* dst = reinterpret_cast<uint2*>(static_cast<typename Elem<T>::type*>(p.o) + e * p.os.b + i * p.os.s +
                                              h * p.os.h + lane * 4);
        *dst = make_uint2(pack2<T>(v[0] * inv, v[1] * inv), pack2<T>(v[2] * inv, v[3] * inv));
    }
    if (lane == 0) p.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
}

// The form and the number of splits whose waves of CTAs take the shortest time,
// by what the parts measured on GB300 (microseconds): a key tile 1.65 in the
// pair form (two row tiles) and 1.2 in the other, a CTA's set-up and end 4, the
// joining kernel 3 and its traffic at 6 TB/s.
struct FwdPlan {
    int alt, narrow, nsplit;
    long long items;
};
FwdPlan fwd_plan(const MhaShape& s) {
    FwdPlan best{};
    double least = 0.0;
    const long long heads = static_cast<long long>(s.hkv) * s.nsub;
    for (int alt = s.ntile == 1; alt < 2; ++alt) {
        const long long items = heads * s.b * (alt ? s.ntile : (s.ntile + 1) / 2);
        const int most = s.nkb / 2;  // two key tiles a CTA at least
        for (int n = 1; n == 1 || (n <= most && items * n <= 4 * kTargetCtas); ++n) {
            const double waves = static_cast<double>((items * n - 1) / kTargetCtas + 1);
            double t = waves * (((s.nkb - 1) / n + 1) * (alt ? 1.2 : 1.65) + 4.0);
            if (n > 1) t += 3.0 + 8.0 * n * s.b * s.hq * s.sq * s.d / 6e6;
            if (best.items == 0 || t < least) {
                least = t;
                best = {alt, alt && s.sq << s.gp_log2 <= 32, n, items * n};
            }
        }
    }
    return best;
}

template <int T, int kSteps, bool kNarrow>
int fwd_launch(const vae_attention_desc* a, const FwdPlan& f, const CUtensorMap (&map)[3], const FwdParams& p,
               cudaStream_t st) {
    static CtxOnce once;
    static std::mutex mu;
    using C = FwdCfg<kSteps>;
    {
        int dev;
        VAE_CUDA_CHECK(cudaGetDevice(&dev));
        std::lock_guard<std::mutex> lk(mu);
        if (!once.done(dev)) {
            VAE_CUDA_CHECK(cudaFuncSetAttribute(mha_fwd_kernel<T, kSteps, kNarrow>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                C::kSmem));
            cudaFuncAttributes at;
            VAE_CUDA_CHECK(cudaFuncGetAttributes(&at, mha_fwd_kernel<T, kSteps, kNarrow>));
            if (!kNarrow && at.numRegs < kLaunchRegs)  // the softmax warps would wait for registers that the block does not have
                return set_error(VAE_ERR_CUDA, "attention: compiled to %d registers a thread, its split needs %d",
                                 at.numRegs, kLaunchRegs);
            once.mark(dev);
        }
    }
    VAE_CUDA_CHECK(launch_kernel(mha_fwd_kernel<T, kSteps, kNarrow>, dim3(static_cast<unsigned>(f.items)), dim3(kThreads), C::kSmem,
                                 st, map[0], map[1], map[2], p));
    if (f.nsplit > 1) {
        const long long rows = static_cast<long long>(a->b) * a->hq * a->sq;
        VAE_CUDA_CHECK(launch_next(mha_join_kernel<T>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, st, p));
    }
    return VAE_OK;
}

template <bool kNarrow>
int fwd_by_type(const vae_attention_desc* a, const FwdPlan& f, const CUtensorMap (&map)[3], const FwdParams& p, cudaStream_t st) {
    const int d = p.s.d;
    if (a->type == VAE_F16)
        return d <= 64   ? fwd_launch<VAE_F16, 4, kNarrow>(a, f, map, p, st)
               : d <= 96 ? fwd_launch<VAE_F16, 6, kNarrow>(a, f, map, p, st)
                         : fwd_launch<VAE_F16, 8, kNarrow>(a, f, map, p, st);
    return d <= 64   ? fwd_launch<VAE_BF16, 4, kNarrow>(a, f, map, p, st)
           : d <= 96 ? fwd_launch<VAE_BF16, 6, kNarrow>(a, f, map, p, st)
                     : fwd_launch<VAE_BF16, 8, kNarrow>(a, f, map, p, st);
}

}  // namespace

size_t mha_fwd_bytes(const MhaShape& s) {
    const FwdPlan f = fwd_plan(s);
    if (f.nsplit == 1) return 0;
    const size_t rows = static_cast<size_t>(s.b) * s.hq * s.sq;
    return static_cast<size_t>(f.nsplit) * rows * s.d * sizeof(float) + (f.nsplit * rows * sizeof(float) + 15) / 16 * 16;
}

int mha_fwd_run(const vae_attention_desc* a, const MhaShape& s, const void* q, const void* k, const void* v, void* o,
                float* lse, void* ws, cudaStream_t st) {
    const FwdPlan f = fwd_plan(s);
    if (f.items > 0x7fffffffLL) return set_error(VAE_ERR_SHAPE, "attention: too many tiles");
    const int gp = 1 << s.gp_log2;
    CUtensorMap map[3];
    const bool twice = f.narrow && static_cast<long long>(s.sq) * gp <= 16;
    int rc = mha_map(&map[0], a, q, a->q_stride, s.sq, s.hq, gp, (twice ? 16 : f.narrow ? 32 : kMhaTile) / gp);
    if (rc == VAE_OK) rc = mha_map(&map[1], a, k, a->k_stride, s.sk, s.hkv, 1, kMhaTile);
    if (rc == VAE_OK) rc = mha_map(&map[2], a, v, a->v_stride, s.sk, s.hkv, 1, kMhaTile);
    if (rc != VAE_OK) return rc;
    FwdParams p{};
    p.s = s;
    p.alt = f.alt;
    p.twice = twice;
    p.nsplit = f.nsplit;
    p.scale_log2 = a->scale * 1.4426950408889634074f;
    p.o = o;
    p.os = mha_strides(a->o_stride);
    p.lse = lse;
    p.po = static_cast<float*>(ws);
    p.plse = p.po + static_cast<size_t>(f.nsplit) * s.b * s.hq * s.sq * s.d;
    p.status = device_status_ptr();
    p.timeout_ns = wait_timeout_ns();
    if (p.status == nullptr) return VAE_ERR_CUDA;
    if (f.narrow) return fwd_by_type<true>(a, f, map, p, st);
    return fwd_by_type<false>(a, f, map, p, st);
}

}  // namespace vae
