// bg_kvquant.h -- a row of keys or values to the cache's codes, in the D / 8 lanes
// that hold it (the rules are in k_kvcache.hip).
#pragma once
#include <type_traits>

#include "bg_device.h"
#include "bg_kv.h"

namespace bg {

// First element of slot `slot`'s row of head h, in rows of the code and record arrays.
__device__ __forceinline__ int64_t kv_row(const KvCache& c, int64_t slot, int h) {
    const int64_t page = slot >> c.page_shift, in = slot & ((1 << c.page_shift) - 1);
    return ((page * c.heads + h) << c.page_shift) + in;
}

// f over the L lanes of a row (8, 16 or 32), in all of them; f commutes.  Up to 16
// lanes exchange in the vector unit (within 4, 8 and 16 lanes), not through LDS.
template <int L, typename T, typename F>
__device__ __forceinline__ T over_row(T v, F&& f) {
    struct Words {
        int w[sizeof(T) / 4];
    };
    auto from = [&](auto CTRL) {
        Words x = __builtin_bit_cast(Words, v);
        for (int& w : x.w) w = __builtin_amdgcn_update_dpp(0, w, CTRL(), 0xF, 0xF, true);
        return __builtin_bit_cast(T, x);
    };
    v = f(v, from(std::integral_constant<int, 0xB1>{}));        // lane ^ 1
    v = f(v, from(std::integral_constant<int, 0x4E>{}));        // lane ^ 2
    v = f(v, from(std::integral_constant<int, 0x141>{}));       // 8 lanes mirrored
    if constexpr (L >= 16) v = f(v, from(std::integral_constant<int, 0x140>{}));       // 16 lanes mirrored
    if constexpr (L == 32) v = f(v, __shfl_xor(v, 16, 64));
    return v;
}

// Two finite quotients to E4M3: as e4m3x2, without its NaN.
__device__ __forceinline__ uint32_t finite_e4m3x2(float a, float b) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_fmed3f(a, -448.0f, 448.0f),
                                                     __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f), 0, false) & 0xFFFFu;
}

// A lane's eight codes (4 bits: all in w[0], element i in nibble i; else elements 0 to 3
// and 4 to 7) and the row's record.
struct RowCodes {
    uint32_t w[2], record;
};

// e: the lane's elements of the row; which eight of them it holds does not matter.
template <int FMT, int D>
__device__ __forceinline__ RowCodes quantize_row(const float (&e)[8]) {
#pragma clang fp contract(off)
    constexpr int L = D / 8;
    // The largest magnitude, as bits: infinities and NaN come out on top.
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = __float_as_uint(e[i]) & 0x7FFFFFFFu;
        bits = m > bits ? m : bits;
    }
    bits = over_row<L>(bits, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    const bool bad = bits >= 0x7F800000u;
    if constexpr (FMT == KV_U4) {
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = __builtin_fminf(lo, e[i]);
            hi = __builtin_fmaxf(hi, e[i]);
        }
        lo = over_row<L>(lo, [](float a, float b) { return __builtin_fminf(a, b); });
        hi = over_row<L>(hi, [](float a, float b) { return __builtin_fmaxf(a, b); });
        float s = (float)(_Float16)__builtin_fminf(__builtin_fmaxf((hi - lo) / 15.0f, 0x1p-24f), 65504.0f);
        if (hi == lo) s = 1.0f;
        const float z = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(-lo / s), 0.0f), 15.0f);
        float d[8];
        quotients8(e, QScale{s, 1.0f / s, true}, d);        // 2^-24 <= s <= 65504
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __builtin_amdgcn_fmed3f(__builtin_rintf(d[i]) + z, 0.0f, 15.0f);
            w |= (uint32_t)u << (4 * i);
        }
        return RowCodes{{bad ? 0u : w, 0u}, bad ? 0x00007E00u : (uint32_t)f32_to_f16(s) | (uint32_t)f32_to_f16(z) << 16};
    } else {
        float s = (bad ? 0.0f : __uint_as_float(bits)) / (FMT == KV_I8 ? 127.0f : 448.0f);
        if (s == 0.0f) s = 1.0f;
        float d[8];
        quotients8(e, QScale{s, 1.0f / s, s >= 0x1p-80f && s <= 0x1p100f}, d);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            uint32_t p;
            if constexpr (FMT == KV_I8) {
                const int a = (int)__builtin_amdgcn_fmed3f(__builtin_rintf(d[i]), -127.0f, 127.0f);
                const int b = (int)__builtin_amdgcn_fmed3f(__builtin_rintf(d[i + 1]), -127.0f, 127.0f);
                p = ((uint32_t)a & 0xFFu) | ((uint32_t)b & 0xFFu) << 8;
            } else {
                p = finite_e4m3x2(d[i], d[i + 1]);
            }
            w[i / 4] |= p << (8 * (i % 4));
        }
        return RowCodes{{bad ? 0u : w[0], bad ? 0u : w[1]}, bad ? 0x7FC00000u : __float_as_uint(s)};
    }
}

}  // namespace bg
