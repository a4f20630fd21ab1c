// How the products of the gated feed-forward block are cut into tiles and dealt out to
// pairs of CTAs: the kernel's way from a pair's turn to its tile, and the host's choice.
#pragma once

#include <algorithm>
#include <cstddef>

#ifdef __CUDACC__
#define VAE_BOTH __host__ __device__ __forceinline__
#else
#define VAE_BOTH inline
#endif

namespace vae {
namespace ffn {

constexpr int kTile = 128;              // rows of A per CTA
constexpr int kMaxCols = 256;           // columns of the pair's accumulator
constexpr int kBk = 64;                 // contraction per stage: one 128-byte swizzle row
constexpr int kEpiWarps = 8;
constexpr int kGroup = 8;               // row tiles that share their column tiles in L2
constexpr int kPairs = 76;              // that the plan counts with
constexpr int kMaxSplits = 8;

// The products. A and B stand as [rows][contraction] (K-major) or [contraction][rows].
enum : int {
    kGate,      // x, (Wg, Wu) -> hidden (gate, up)
    kDown,      // hidden, Wd -> y
    kBackGate,  // dy, Wd^T -> dgate, dup
    kGrad,      // (dgate, dup), (Wg, Wu)^T -> dx; dgate^T, x^T -> dWg; dup^T, x^T -> dWu; hidden^T, dy^T -> dWd^T
};
constexpr bool b_mn(int kind) { return kind >= kBackGate; }

// Products of one shape and how they are cut: column tiles of `wide` and what is left of the columns (`rest`, 0:
// nothing), the contraction of `nk` stages in `splits`. kGrad has two of them (dx; the weights' gradients), the
// others one.
struct Group {
    int rows, cols, problems, nk;
    int wide, rest, splits;
    int tall;                  // tiles have 256 rows, or (2) 512, which read a quarter less
    int nm, nfull;             // row tiles, column tiles of full width
};

// Which pair computes what: the tiles of the four classes (group 0's full ones and rests, group 1's) go to the least
// laden pairs, the longest ones first. Pairs that got the same lie side by side: `n` runs of them, with a count of each class.
constexpr int kRuns = 6;
struct Deal {
    int n;
    int order[4];
    int pairs[kRuns], count[kRuns][4];
};

struct Tile {
    int g, z, part;    // group, problem (in Params::out's order), partial sums
    int m0, n0, n;     // the pair's first row, the columns [n0, n0 + n)
    int subs;          // times 256 rows (the last tile of 512 may have 256)
    int k0, k1;        // stages
};
// The i-th tile of pair `pair`; false behind its last. Row tiles lie in groups of kGroup, their column tiles side by
// side: the pairs at work share rows of A and of B in L2.
VAE_BOTH bool tile_at(const Group* groups, const Deal& deal, int pair, int i, Tile* r) {
    int run = 0, before = 0;
    while (pair >= before + deal.pairs[run]) before += deal.pairs[run++];
    int c = -1;
    for (int o = 0; o < 4; ++o) {
        const int n = deal.count[run][deal.order[o]];
        if (i < n) {
            c = deal.order[o];
            break;
        }
        i -= n;
    }
    if (c < 0) return false;
    // the class's tiles are dealt out round by round, over the pairs that have as many
    int t = pair - before;
    for (int q = 0; q < deal.n; ++q) {
        const int n = deal.count[q][c];
        t += (n < i ? n : i) * deal.pairs[q] + (q < run && n > i ? deal.pairs[q] : 0);
    }
    const Group& g = groups[c >> 1];
    int nt;
    if ((c & 1) == 0) {
        const int each = g.nm * g.nfull;
        r->part = t / each;
        t -= r->part * each;
        const int w = t / (kGroup * g.nfull), in = t - w * kGroup * g.nfull;
        const int tall = g.nm - w * kGroup < kGroup ? g.nm - w * kGroup : kGroup;
        nt = in / tall;
        r->m0 = (w * kGroup + in - nt * tall) * g.tall * 2 * kTile;
        r->n = g.wide;
    } else {
        r->part = t / g.nm;
        r->m0 = (t - r->part * g.nm) * g.tall * 2 * kTile;
        nt = g.nfull;
        r->n = g.rest;
    }
    r->n0 = nt * g.wide;
    r->subs = r->m0 + 2 * kTile < g.rows ? g.tall : 1;
    r->g = c >> 1;
    const int z = r->part / g.splits, s = r->part - z * g.splits;
    r->z = r->g + z;
    r->k0 = static_cast<int>(static_cast<long long>(g.nk) * s / g.splits);
    r->k1 = static_cast<int>(static_cast<long long>(g.nk) * (s + 1) / g.splits);
    return true;
}

VAE_BOTH int part_cols(const Group& g) { return g.nfull * g.wide + g.rest; }
VAE_BOTH long long part_size(const Group& g) { return static_cast<long long>(g.nm) * 2 * kTile * part_cols(g); }

// Cycles that a pair takes for a stage of a tile of n accumulator columns, as measured: the stage's bytes from L2 (with
// every SM asking, 46 a cycle and CTA), or the hand-over between loads and products; of a tall tile the products
// themselves. An operand that lies MN-major comes in boxes of 64 rows for each CTA.
inline int stage_cycles(int kind, int n, int tall) {
    const int rows = 256 * tall + (b_mn(kind) ? (n > 128 ? 256 : 128) : n);
    return std::max(std::max(430, rows * 7 / 5), tall > 1 ? n * 17 / 4 : 0);
}

inline int class_tiles(const Group& g, int rest) {
    return rest != 0 ? (g.rest > 0 ? g.problems * g.splits * g.nm : 0) : g.problems * g.splits * g.nm * g.nfull;
}
// Deals the classes' tiles out over `pairs` pairs; returns the cycles of the one with the most.
inline long long deal_out(int kind, const Group* groups, int count, int pairs, Deal* d) {
    const int per = kind == kGate ? 2 : 1;  // accumulator columns per column
    long long cost[4] = {}, load[kRuns] = {};
    int tiles[4] = {};
    *d = Deal{};
    d->n = 1;
    d->pairs[0] = pairs;
    for (int c = 0; c < 4; ++c) {
        d->order[c] = c;
        if (c >> 1 >= count) continue;
        const Group& g = groups[c >> 1];
        tiles[c] = class_tiles(g, c & 1);
        // its stages, or where they are few its way out of TMEM (which runs under the next tile's stages, but for the tall ones)
        const int n = ((c & 1) != 0 ? g.rest : g.wide) * per;
        const long long part = g.splits > 1 ? 22LL * n : 0;  // a split's sums, written and read; beside much other work that hides
        const long long in = 400 + (kind == kDown ? part : 0) + static_cast<long long>(stage_cycles(kind, n, g.tall)) * ((g.nk + g.splits - 1) / g.splits);
        const long long out = 600 + part + 12LL * n;
        cost[c] = g.tall > 1 ? in + 2 * out : std::max(in, out);
    }
    std::sort(d->order, d->order + 4, [&](int a, int b) { return cost[a] != cost[b] ? cost[a] > cost[b] : a < b; });
    for (int c : d->order) {
        if (tiles[c] == 0) continue;
        const long long k = cost[c];
        // the highest level that the pairs can be filled to with these tiles: within two of them of what they all come to
        long long most = 0, all = k * tiles[c];
        for (int r = 0; r < d->n; ++r) {
            most = std::max(most, load[r]);
            all += load[r] * d->pairs[r];
        }
        long long lo = std::max(0LL, all / pairs - 2 * k), hi = std::max(all / pairs, most) + 2 * k;
        const auto filled = [&](long long level) {
            long long n = 0;
            for (int r = 0; r < d->n; ++r) n += level > load[r] ? (level - load[r]) / k * d->pairs[r] : 0;
            return n;
        };
        if (filled(lo) > tiles[c]) lo = 0;
        while (hi - lo > 1) {
            const long long mid = (lo + hi) / 2;
            (filled(mid) <= tiles[c] ? lo : hi) = mid;
        }
        int left = tiles[c] - static_cast<int>(filled(lo));
        for (int r = 0; r < d->n; ++r) {
            const int n = lo > load[r] ? static_cast<int>((lo - load[r]) / k) : 0;
            d->count[r][c] = n;
            load[r] += n * k;
        }
        // one more each for the least laden
        while (left > 0) {
            int r = -1;
            for (int q = 0; q < d->n; ++q)
                if (d->count[q][c] >= 0 && (r < 0 || load[q] < load[r])) r = q;
            if (d->pairs[r] > left) {  // a part of this run
                for (int q = d->n++; q > r; --q) {
                    d->pairs[q] = d->pairs[q - 1];
                    load[q] = load[q - 1];
                    std::copy(d->count[q - 1], d->count[q - 1] + 4, d->count[q]);
                }
                d->pairs[r] = left;
                d->pairs[r + 1] -= left;
            }
            left -= d->pairs[r];
            ++d->count[r][c];
            load[r] += k;
        }
    }
    return *std::max_element(load, load + d->n);
}

// How the products of a kernel are cut and dealt out.
struct Plan {
    Group group[2];
    Deal deal;
};
inline Group cut_group(const Group& base, int wide, int splits, int tall) {
    Group g{base.rows, base.cols, base.problems, base.nk, wide, (base.cols % wide + 31) / 32 * 32, splits, tall};
    g.nm = (g.rows - 1) / (2 * kTile * tall) + 1;
    g.nfull = g.cols / wide;
    return g;
}
inline size_t parts_bytes(const Group& g) {
    return g.splits > 1 ? g.splits * g.problems * part_size(g) * sizeof(float) : 0;
}
// Counters of a group's splits: for each tile, CTA of the pair and epilogue warp.
inline int arrivals(const Group& g) { return g.splits > 1 ? g.problems * g.nm * (g.nfull + (g.rest > 0 ? 1 : 0)) * 2 * kEpiWarps : 0; }
// The tile width and the splits with the least time, counted in cycles of the busiest pair. Wide tiles read the least;
// narrow ones and splits give work to more SMs. Splits cost, beside each tile's sums, the last one's way through all of
// them: as measured 4000 cycles and 40 for each column (kDown, with splits and without, bf16: 256 tokens of 512 x 2048
// 19.7 and 21.0 us, of 1152 x 4608 25.7 and 36.1, 512 of 2048 x 5504 48 and 55; 4096 of 1152 x 4608, whole, 101 and not 109),
// of the gradients 80 and 10 for each split (one token of 512 x 2048 25.5 us, 28 with fewer, which splits more; the
// whole one 38).
inline Plan make_plan(int kind, int m, int c, int f) {
    const int kc = (c + kBk - 1) / kBk, kf = (f + kBk - 1) / kBk, km = (m + kBk - 1) / kBk, count = kind == kGrad ? 2 : 1;
    Group base[2] = {};
    if (kind == kGate || kind == kBackGate) {
        base[0] = Group{m, f, 1, kc};
    } else if (kind == kDown) {
        base[0] = Group{m, c, 1, kf};
    } else {
        base[0] = Group{m, c, 1, 2 * kf};
        base[1] = Group{f, c, 3, km};
    }
    const int per = kind == kGate ? 2 : 1;  // accumulator columns per column
    const bool whole = kind == kGate || kind == kBackGate;  // (their epilogues need the whole sums)
    Plan best{};
    long long least = -1;
    const auto look = [&](int wide, const int (&splits)[2], int tall) {
        Plan p{};
        for (int g = 0; g < count; ++g) p.group[g] = cut_group(base[g], wide / per, splits[g], tall);
        long long t = deal_out(kind, p.group, count, kPairs, &p.deal) + 10 * wide;  // (the last tile's epilogue)
        const int most = std::max(splits[0], count > 1 ? splits[1] : 1);
        if (most > 1) t += 4000 + (kind == kDown ? 40 : 80 + 10LL * most) * wide;
        if (least >= 0 && t >= least) return false;
        best = p;
        least = t;
        return true;
    };
    if (!whole) look(kMaxCols, {1, 1}, 2);
    for (int wide = kMaxCols; wide >= 64; wide -= 64) {
        int splits[2] = {1, 1};
        look(wide, splits, 1);
        bool many = true;  // with many tiles neither splits nor narrow ones can win
        for (int g = count - 1; g >= 0; --g) {  // one group's splits, then the other's beside them
            const Group cut = cut_group(base[g], wide / per, 1, 1);
            if (class_tiles(cut, 0) + class_tiles(cut, 1) >= 4 * kPairs) continue;
            many = false;
            int own = 1;
            for (int s : {2, 3, 4, 6, 8}) {
                if (whole || s > kMaxSplits || s * 4 > base[g].nk) break;
                splits[g] = s;
                if (look(wide, splits, 1)) own = s;
            }
            splits[g] = own;
        }
        if (many) break;
    }
    return best;
}

}  // namespace ffn
}  // namespace vae
