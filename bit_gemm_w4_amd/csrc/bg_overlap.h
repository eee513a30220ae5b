// bg_overlap.h -- whether operands of a call share memory (host code).
#pragma once
#include <cstdint>
#include <utility>

namespace bg {

// `bytes` bytes from p on.
struct Span {
    uintptr_t at;
    uint64_t bytes;

    Span(const void* p, uint64_t n) : at(reinterpret_cast<uintptr_t>(p)), bytes(n) {}
};

inline bool apart(const Span& a, const Span& b) {
    return a.bytes == 0 || b.bytes == 0 || (a.at < b.at ? b.at - a.at >= a.bytes : a.at - b.at >= b.bytes);
}

// Rows of `run` bytes: n[0] groups stride[0] apart of n[1] rows stride[1] <= stride[0] apart.
struct RowSet {
    uintptr_t at;
    uint64_t run, n[2] = {1, 1}, stride[2] = {0, 0};
    bool repeated = false;                    // some row counts more than once

    // Strides in bytes, of either sign.
    RowSet(const void* p, int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t run_bytes)
        : at(reinterpret_cast<uintptr_t>(p)), run((uint64_t)run_bytes) {
        axis(0, tokens, token_stride);
        axis(1, heads, head_stride);
        if (stride[1] > stride[0]) {
            std::swap(stride[0], stride[1]);
            std::swap(n[0], n[1]);
        }
    }
    uint64_t inner() const { return (n[1] - 1) * stride[1] + run; }
    Span span() const { return Span(reinterpret_cast<const void*>(at), (n[0] - 1) * stride[0] + inner()); }
    bool same(const RowSet& o) const {
        return at == o.at && run == o.run && n[0] == o.n[0] && n[1] == o.n[1] && stride[0] == o.stride[0] && stride[1] == o.stride[1];
    }
    // No row lies in another.
    bool distinct() const { return !repeated && (n[1] == 1 || stride[1] >= run) && (n[0] == 1 || stride[0] >= inner()); }

private:
    void axis(int i, int64_t count, int64_t by) {
        if (count <= 1) return;
        repeated |= by == 0;
        if (by == 0) return;
        if (by < 0) at -= (uint64_t)(count - 1) * (0 - (uint64_t)by);
        n[i] = (uint64_t)count;
        stride[i] = by < 0 ? 0 - (uint64_t)by : (uint64_t)by;
    }
};

// True where the two surely have no byte in common: one behind the other; in different parts of a common outer
// stride (slices of a fused row, or of a fused block of heads); or in different parts of a common inner one (heads of each kind in turn).
inline bool apart(const RowSet& a, const RowSet& b) {
    if (apart(a.span(), b.span())) return true;
    auto parts = [&](uint64_t period, uint64_t x, uint64_t y) {
        const uint64_t d = (b.at >= a.at ? (b.at - a.at) % period : (period - (a.at - b.at) % period) % period);
        return d >= x && period - d >= y;
    };
    if (a.stride[0] != b.stride[0] || a.stride[0] == 0) return false;
    if (parts(a.stride[0], a.inner(), b.inner())) return true;
    return a.stride[1] == b.stride[1] && a.stride[1] != 0 && a.stride[0] % a.stride[1] == 0 && parts(a.stride[1], a.run, b.run);
}

}  // namespace bg
