// Whether strided tensors share memory (host): the checks behind "what is
// written lies apart from what is read".
//
// A tensor is runs of `run` bytes at p + sum of i_k stride_k, 0 <= i_k < n_k. Two
// of them share a byte where some sum of index differences times strides brings
// their runs together. Tensors apart as a whole, the usual case, take two
// comparisons. Views that lie in one another (the parts of a joint projection)
// are searched stride by stride, the largest first, over the index differences
// that the smaller strides can still make up for: one or two a stride where a
// larger stride steps over all that the smaller ones span. Layouts that do not
// nest could take many more; over kOverlapSteps of them the answer is "shared".
#pragma once

#include <cstddef>
#include <cstdint>

namespace vae {

using Wide = __int128;  // (an index times a stride may pass 64 bits)

constexpr int kOverlapSteps = 1 << 14;

struct Extent {
    uintptr_t p;
    Wide stride[3];
    long long n[3];
    Wide run;
};

inline Extent extent_dense(const void* p, size_t bytes) {
    return {reinterpret_cast<uintptr_t>(p), {0, 0, 0}, {1, 1, 1}, static_cast<Wide>(bytes)};
}
// [b][n][h][d] elements of `size` bytes, strides {batch, token, head} in elements (of a dimension of one: never used).
inline Extent extent_tokens(const void* p, const long long* stride, int b, int n, int h, int d, size_t size) {
    Extent e{reinterpret_cast<uintptr_t>(p), {0, 0, 0}, {b, n, h}, static_cast<Wide>(d) * size};
    for (int k = 0; k < 3; ++k) e.stride[k] = e.n[k] > 1 ? static_cast<Wide>(stride[k]) * size : 0;
    return e;
}
inline Wide extent_span(const Extent& e) {
    Wide s = e.run;
    for (int k = 0; k < 3; ++k) s += e.stride[k] * (e.n[k] - 1);
    return s;
}

// sum of k_i stride_i, lo_i <= k_i <= hi_i, within (low, high), with some k_i other than 0 where `moved` is asked for.
struct StrideSearch {
    struct Term {
        Wide stride;
        long long lo, hi;
    };
    Term t[6];
    Wide least[7], most[7];  // what the terms from i on can add
    int count = 0, steps = 0;
    Wide low, high;
    bool moved;

    void add(Wide stride, long long lo, long long hi) {
        if (stride == 0 || lo == hi) return;
        int i = 0;
        while (i < count && t[i].stride > stride) ++i;
        if (i < count && t[i].stride == stride) {
            t[i].lo += lo;
            t[i].hi += hi;
            return;
        }
        for (int j = count++; j > i; --j) t[j] = t[j - 1];
        t[i] = {stride, lo, hi};
    }
    bool run() {
        least[count] = most[count] = 0;
        for (int i = count - 1; i >= 0; --i) {
            least[i] = least[i + 1] + t[i].stride * t[i].lo;
            most[i] = most[i + 1] + t[i].stride * t[i].hi;
        }
        return from(0, 0, false);
    }
    static Wide floor_div(Wide a, Wide b) { return a / b - (a % b != 0 && a < 0 ? 1 : 0); }
    bool from(int i, Wide at, bool any) {
        if (++steps > kOverlapSteps) return true;
        if (i == count) return at > low && at < high && (any || !moved);
        // at + k stride + (what follows) within (low, high)
        Wide lo = -floor_div(-(low + 1 - most[i + 1] - at), t[i].stride), hi = floor_div(high - 1 - least[i + 1] - at, t[i].stride);
        if (lo < t[i].lo) lo = t[i].lo;
        if (hi > t[i].hi) hi = t[i].hi;
        for (Wide k = lo; k <= hi; ++k)
            if (from(i + 1, at + k * t[i].stride, any || k != 0)) return true;
        return false;
    }
};

inline bool extents_meet(const Extent& a, const Extent& b) {
    const Wide apart = static_cast<Wide>(a.p) - static_cast<Wide>(b.p);
    if (apart >= extent_span(b) || -apart >= extent_span(a)) return false;
    StrideSearch s;
    for (int k = 0; k < 3; ++k) {
        s.add(a.stride[k], 0, a.n[k] - 1);
        s.add(b.stride[k], -(b.n[k] - 1), 0);
    }
    // a's run at `apart` + the sum, b's at 0
    s.low = -a.run - apart;
    s.high = b.run - apart;
    s.moved = false;
    return s.run();
}

// Whether two runs of one tensor meet (a stride of 0 over several indexes too).
inline bool extent_folds(const Extent& e) {
    StrideSearch s;
    for (int k = 0; k < 3; ++k) {
        if (e.n[k] > 1 && e.stride[k] == 0) return true;
        s.add(e.stride[k], 0, e.n[k] - 1);
    }
    // nested strides: each steps over all that the smaller ones span (equal ones were joined by add)
    Wide inner = e.run;
    int dims = 0;
    for (int k = 0; k < 3; ++k) dims += e.n[k] > 1;
    bool nested = dims == s.count;
    for (int i = s.count - 1; nested && i >= 0; --i) {
        nested = s.t[i].stride >= inner;
        inner += s.t[i].stride * s.t[i].hi;
    }
    if (nested) return false;
    if (dims != s.count) return true;  // two dimensions of one stride: index (1, 0) lies on (0, 1)
    for (int i = 0; i < s.count; ++i) s.t[i].lo = -s.t[i].hi;
    s.low = -e.run;
    s.high = e.run;
    s.moved = true;
    return s.run();
}

}  // namespace vae
