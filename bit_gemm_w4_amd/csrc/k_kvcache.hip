// k_kvcache.hip -- writing rows into the quantized KV cache and reading them
// back.
//
// A row is one token's key (or value) of one head, D elements.  Its scale
// follows the activation quantizers' rules (symmetric INT8 s = amax / 127,
// E4M3 s = amax / 448; 4-bit s = fp16((max - min) / 15) with the range widened
// to hold 0 and z = rne(-min / s)); an all-zero row has s = 1.  Every float
// expression is one correctly rounded operation, so codes do not depend on how
// the work is split.
//
// Bound by HBM: a row is read once and its codes written once.  D / 8 lanes
// hold a row, 8 elements (16 bytes of a 16-bit type) each, so a wave loads
// 1 KB and the row's statistics are log2(D / 8) lane exchanges; one launch
// does keys and values, which for a decode step's few rows is what counts.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kv.h"

namespace bg {
namespace {

constexpr int kBlock = 256;

// First element of slot `slot`'s row of head h, in rows of the code and record arrays.
__device__ __forceinline__ int64_t kv_row(const KvCache& c, int64_t slot, int h) {
    const int64_t page = slot >> c.page_shift, in = slot & ((1 << c.page_shift) - 1);
    return ((page * c.heads + h) << c.page_shift) + in;
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kBlock) k_kv_write(KvCache c, KvRows x, int64_t tokens, const int64_t* slots) {
#pragma clang fp contract(off)
    constexpr int L = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * kBlock + threadIdx.x) / L;
    const int lane = threadIdx.x % L;
    const int64_t per = 2 * c.heads;
    const int64_t t = row / per;
    if (t >= tokens) return;
    const int kv = (int)((row - t * per) / c.heads), h = (int)((row - t * per) % c.heads);
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= (c.pages << c.page_shift)) return;   // whole rows leave together

    float e[8];
    load8_f32<DT>(kv ? x.v : x.k, (kv ? t * x.v_ts + h * x.v_hs : t * x.k_ts + h * x.k_hs) + lane * 8, e);
    const int64_t at = kv_row(c, slot, h);
    uint8_t* codes = (kv ? c.v : c.k) + at * (FMT == KV_U4 ? D / 2 : D);
    uint32_t* record = (kv ? c.vs : c.ks) + at;
    const float inf = __builtin_inff();
    if constexpr (FMT == KV_U4) {
        float lo = 0.0f, hi = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = __builtin_fminf(lo, e[i]);
            hi = __builtin_fmaxf(hi, e[i]);
            top = __builtin_fmaxf(top, __builtin_isfinite(e[i]) ? 0.0f : inf);
        }
        lo = wave_min<L>(lo);
        hi = wave_max<L>(hi);
        const bool bad = wave_max<L>(top) == inf;
        float s = (float)(_Float16)__builtin_fminf(__builtin_fmaxf((hi - lo) / 15.0f, 0x1p-24f), 65504.0f);
        if (hi == lo) s = 1.0f;
        const float z = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(-lo / s), 0.0f), 15.0f);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(e[i] / s) + z, 0.0f), 15.0f);
            w |= (uint32_t)u << (4 * i);
        }
        reinterpret_cast<uint32_t*>(codes)[lane] = bad ? 0u : w;
        if (lane == 0) *record = bad ? 0x00007E00u : (uint32_t)f32_to_f16(s) | (uint32_t)f32_to_f16(z) << 16;
    } else {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, __builtin_isfinite(e[i]) ? __builtin_fabsf(e[i]) : inf);
        top = wave_max<L>(top);
        const bool bad = top == inf;
        float s = top / (FMT == KV_I8 ? 127.0f : 448.0f);
        if (s == 0.0f) s = 1.0f;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            uint32_t p;
            if constexpr (FMT == KV_I8) {
                const int a = (int)__builtin_fminf(__builtin_fmaxf(__builtin_rintf(e[i] / s), -127.0f), 127.0f);
                const int b = (int)__builtin_fminf(__builtin_fmaxf(__builtin_rintf(e[i + 1] / s), -127.0f), 127.0f);
                p = ((uint32_t)a & 0xFFu) | ((uint32_t)b & 0xFFu) << 8;
            } else {
                p = e4m3x2(e[i] / s, e[i + 1] / s);
            }
            w[i / 4] |= p << (8 * (i % 4));
        }
        reinterpret_cast<uint2*>(codes)[lane] = bad ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
        if (lane == 0) *record = bad ? 0x7FC00000u : __float_as_uint(s);
    }
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kBlock) k_kv_read(KvCache c, const int64_t* slots, int64_t tokens, void* k, void* v) {
#pragma clang fp contract(off)
    constexpr int L = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * kBlock + threadIdx.x) / L;
    const int lane = threadIdx.x % L;
    const int64_t per = 2 * c.heads;
    const int64_t t = row / per;
    if (t >= tokens) return;
    const int kv = (int)((row - t * per) / c.heads), h = (int)((row - t * per) % c.heads);
    const int64_t slot = slots[t];
    float e[8];
    if (slot < 0 || slot >= (c.pages << c.page_shift)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = 0.0f;
    } else {
        const int64_t at = kv_row(c, slot, h);
        const uint8_t* codes = (kv ? c.v : c.k) + at * (FMT == KV_U4 ? D / 2 : D);
        const uint32_t record = (kv ? c.vs : c.ks)[at];
        if constexpr (FMT == KV_U4) {
            const float s = f16_to_f32(record & 0xFFFFu), z = f16_to_f32(record >> 16);
            const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = ((float)(w >> (4 * i) & 15u) - z) * s;
        } else {
            const float s = __uint_as_float(record);
            const uint2 r = reinterpret_cast<const uint2*>(codes)[lane];
            const uint32_t w[2] = {r.x, r.y};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = w[i / 4] >> (8 * (i % 4)) & 0xFFu;
                if constexpr (FMT == KV_I8) e[i] = (float)(int8_t)b * s;
                else e[i] = __builtin_amdgcn_cvt_f32_fp8((int)b, 0) * s;
            }
        }
    }
    const int64_t o = (t * c.heads + h) * D + lane * 8;
    if constexpr (DT == DT_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(kv ? v : k) + o);
        p[0] = make_float4(e[0], e[1], e[2], e[3]);
        p[1] = make_float4(e[4], e[5], e[6], e[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = DT == DT_BF16 ? (uint32_t)f32_to_bf16(e[2 * i]) | (uint32_t)f32_to_bf16(e[2 * i + 1]) << 16
                                 : (uint32_t)f32_to_f16(e[2 * i]) | (uint32_t)f32_to_f16(e[2 * i + 1]) << 16;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? v : k) + o) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// f(DT, FMT, D) over the supported types, formats and head sizes.
template <typename F>
void for_kv(int dt, int fmt, int dim, F&& f) {
    auto on_dim = [&](auto DT, auto FMT) {
        if (dim == 64) f(DT, FMT, std::integral_constant<int, 64>{});
        else if (dim == 128) f(DT, FMT, std::integral_constant<int, 128>{});
        else f(DT, FMT, std::integral_constant<int, 256>{});
    };
    auto on_fmt = [&](auto DT) {
        if (fmt == KV_I8) on_dim(DT, std::integral_constant<int, KV_I8>{});
        else if (fmt == KV_FP8) on_dim(DT, std::integral_constant<int, KV_FP8>{});
        else on_dim(DT, std::integral_constant<int, KV_U4>{});
    };
    if (dt == DT_F32) on_fmt(std::integral_constant<int, DT_F32>{});
    else if (dt == DT_F16) on_fmt(std::integral_constant<int, DT_F16>{});
    else on_fmt(std::integral_constant<int, DT_BF16>{});
}

unsigned row_blocks(const KvCache& c, int64_t tokens) {
    const int per_block = kBlock / (c.dim / 8);
    return (unsigned)((tokens * 2 * c.heads + per_block - 1) / per_block);
}

}  // namespace

const char* launch_kv_write(const KvCache& c, const KvRows& x, int dt, int64_t tokens, const int64_t* slots, hipStream_t s) {
    for_kv(dt, c.fmt, c.dim, [&](auto DT, auto FMT, auto D) {
        k_kv_write<DT(), FMT(), D()><<<row_blocks(c, tokens), kBlock, 0, s>>>(c, x, tokens, slots);
    });
    return kname("k_kv_write", dt, c.fmt, c.dim);
}

const char* launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, int dt, void* k, void* v, hipStream_t s) {
    for_kv(dt, c.fmt, c.dim, [&](auto DT, auto FMT, auto D) {
        k_kv_read<DT(), FMT(), D()><<<row_blocks(c, tokens), kBlock, 0, s>>>(c, slots, tokens, k, v);
    });
    return kname("k_kv_read", dt, c.fmt, c.dim);
}

}  // namespace bg
