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

// Cycles that a pair takes for a stage of a tile of n accumulator columns, as measured: the stage's bytes from L2, 57 a
// cycle and CTA, or the hand-over between loads and products; of a tall tile the products themselves. An operand that lies
// MN-major comes in boxes of 64 rows for each CTA, the others as the rows of a full tile (`wide`).
inline int stage_cycles(int kind, int n, int wide, int tall) {
    const int rows = 256 * tall + (b_mn(kind) ? (n > 128 ? 256 : 128) : wide);
    return std::max(std::max(430, rows * 113 / 100), tall > 1 ? n * 17 / 4 : 0);
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
        const long long in = 400 + (kind == kDown ? part : 0) + static_cast<long long>(stage_cycles(kind, n, g.wide * per, g.tall)) * ((g.nk + g.splits - 1) / g.splits);
        const long long out = 600 + part + 12LL * n;
        // (a tall tile takes a little less, of dx and the weights' gradients a seventh: with every SM asking for long sums the
        // others' stages come slower than counted, and these read a quarter less)
        cost[c] = g.tall > 1 ? (in + out) * (kind == kGrad ? 86 : 94) / 100 : std::max(in, out);
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
// The tile widths and the splits with the least time, counted in cycles of the busiest pair. Wide tiles read the least;
// narrow ones and splits give work to more SMs. Splits cost, beside each tile's sums, the last one's way through all of
// them. Of the gradients each group has its own width and splits: dx is long sums over few tiles, the weights' gradients of
// few tokens short ones over many, whose way out of TMEM counts. What splits and tall tiles cost is fitted to the measured
// times of the widths with every number of splits at 174 shapes, 1 to 32768 tokens and 256 x 1024 to 4096 x 11008 (bf16, in
// a graph): the plan taken is 0.7 % over the best of them on average for the second product, 8 % at most, and 2.5 %, 13 %,
// for the gradients. (One width for both groups of the gradients and a higher charge: one token of 1152 x 4608 52 us and 44,
// 1024 tokens 95 and 68, 256 of 2048 x 5504 88 and 69; 256 of 512 x 2048 forward, in eight splits and in four, 19.0 us and
// 17.4.)
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
    struct Cut {
        int wide[2], splits[2], tall;
    };
    const auto look = [&](const Cut& c, Plan* p) {
        long long sums = 0, join = 0;
        for (int g = 0; g < count; ++g) {
            const Group& r = p->group[g] = cut_group(base[g], c.wide[g] / per, c.splits[g], c.tall);
            if (r.splits == 1) continue;
            sums += 1LL * r.splits * r.problems * r.rows * r.cols;
            join = std::max(join, kind == kDown ? 3000 + (40LL + 8 * r.splits) * c.wide[g] : (8LL + 4 * r.splits) * c.wide[g]);
        }
        // (kGrad: the sums' way through L2, beside what else is on it; the others: the last tile's epilogue)
        const long long end = kind == kGrad ? sums * 3 / (20 * kPairs) : kind == kDown ? 0 : 10LL * c.wide[0];
        return deal_out(kind, p->group, count, kPairs, &p->deal) + join + end;
    };
    Plan best{};
    long long least = -1;
    const auto take = [&](const Cut& c) {
        Plan p{};
        const long long t = look(c, &p);
        if (least >= 0 && t >= least) return false;
        best = p;
        least = t;
        return true;
    };
    // with many tiles neither splits nor narrow ones can win
    const auto many = [&](int g, int wide) {
        const Group cut = cut_group(base[g], wide / per, 1, 1);
        return class_tiles(cut, 0) + class_tiles(cut, 1) >= 4 * kPairs;
    };
    if (!whole) take({{kMaxCols, kMaxCols}, {1, 1}, 2});
    if (count == 1) {
        for (int wide = kMaxCols; wide >= 64; wide -= 64) {
            take({{wide, wide}, {1, 1}, 1});
            if (many(0, wide)) break;
            for (int s : {2, 3, 4, 6, 8})
                if (!whole && s <= kMaxSplits && s * 4 <= base[0].nk) take({{wide, wide}, {s, 1}, 1});
        }
        return best;
    }
    // both groups alike first, then one's width and splits beside the other's
    Cut now{{kMaxCols, kMaxCols}, {1, 1}, 1};
    for (int wide = kMaxCols; wide >= 64; wide -= 64)
        if (const Cut c{{wide, wide}, {1, 1}, 1}; take(c)) now = c;
    for (int g = count - 1; g >= 0; --g) {
        Cut own = now;
        long long t = -1;
        for (int wide = kMaxCols; wide >= 64; wide -= 64)
            for (int s : {1, 2, 3, 4, 6, 8}) {
                if (s > 1 && (s > kMaxSplits || s * 4 > base[g].nk || many(g, wide))) break;
                Cut c = now;
                c.wide[g] = wide;
                c.splits[g] = s;
                Plan p{};
                if (const long long k = look(c, &p); t < 0 || k < t) {
                    t = k;
                    own = c;
                    if (k < least) {
                        best = p;
                        least = k;
                    }
                }
            }
        now = own;
    }
    return best;
}

}  // namespace ffn
}  // namespace vae
