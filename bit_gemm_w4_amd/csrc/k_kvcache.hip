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
// Quotients are taken through the row's reciprocal with Markstein's correction,
// rows are found without a 64-bit division, and a row's lanes exchange without
// LDS: with divisions for the first two and LDS for the third, 16,383 tokens of
// 8 heads of 128 in E4M3 took 38 us to write with the rows in the last-level cache,
// 22 now; 27 from memory (101 MB at 3.8 TB/s; reading them back 19 us at 5.3 TB/s; a
// large copy runs at 4.8).  4 bits at 4 heads of 256 are bound by the vector units
// still: 16,000 tokens 29 us, 2.8 TB/s.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kv.h"
#include "bg_kvquant.h"

namespace bg {
namespace {

constexpr int kBlock = 256;

// A block's rows: `group` tokens from its first, all heads, keys (blockIdx.y 0) or
// values (1).  f(t, h, lane) for each row of this thread, D / 8 lanes together.
template <int D, typename F>
__device__ __forceinline__ void for_rows(int heads, int group, int64_t tokens, F&& f) {
    constexpr uint32_t L = D / 8, R = kBlock / L;
    const int64_t first = (int64_t)blockIdx.x * group;
    const uint32_t left = (uint32_t)(tokens - first < group ? tokens - first : group), rows = left * heads;
    for (uint32_t i = threadIdx.x / L; i < rows; i += R) f(first + i / heads, (int)(i % heads), (int)(threadIdx.x % L));
}

template <int DT, int FMT, int D>
__device__ __forceinline__ void write_row(const KvCache& c, const KvRows& x, int kv, int64_t t, int h, int lane, const int64_t* slots) {
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= (c.pages << c.page_shift)) return;   // whole rows leave together

    float e[8];
    load8_f32<DT>(kv ? x.v : x.k, (kv ? t * x.v_ts + h * x.v_hs : t * x.k_ts + h * x.k_hs) + lane * 8, e);
    const int64_t at = kv_row(c, slot, h);
    uint8_t* codes = (kv ? c.v : c.k) + at * (FMT == KV_U4 ? D / 2 : D);
    const RowCodes r = quantize_row<FMT, D>(e);
    if constexpr (FMT == KV_U4) reinterpret_cast<uint32_t*>(codes)[lane] = r.w[0];
    else reinterpret_cast<uint2*>(codes)[lane] = make_uint2(r.w[0], r.w[1]);
    if (lane == 0) (kv ? c.vs : c.ks)[at] = r.record;
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kBlock) k_kv_write(KvCache c, KvRows x, int64_t tokens, int group, const int64_t* slots) {
    for_rows<D>(c.heads, group, tokens, [&](int64_t t, int h, int lane) { write_row<DT, FMT, D>(c, x, (int)blockIdx.y, t, h, lane, slots); });
}

template <int DT, int FMT, int D>
__device__ __forceinline__ void read_row(const KvCache& c, int kv, int64_t t, int h, int lane, const int64_t* slots, void* k, void* v) {
#pragma clang fp contract(off)
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

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kBlock) k_kv_read(KvCache c, const int64_t* slots, int64_t tokens, int group, void* k, void* v) {
    for_rows<D>(c.heads, group, tokens, [&](int64_t t, int h, int lane) { read_row<DT, FMT, D>(c, (int)blockIdx.y, t, h, lane, slots, k, v); });
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

// Tokens of a block: as many as give each thread a row (one token of many heads: several),
// two from 2^23 on, since a launch holds less than 2^32 threads along an axis.
int token_group(const KvCache& c, int64_t tokens) {
    const int rows = kBlock / (c.dim / 8), group = c.heads < rows ? rows / c.heads : 1;
    return group < 2 && tokens > (1 << 23) ? 2 : group;
}

dim3 grid_of(const KvCache& c, int64_t tokens) {
    const int group = token_group(c, tokens);
    return dim3((unsigned)((tokens + group - 1) / group), 2);
}

}  // namespace

const char* launch_kv_write(const KvCache& c, const KvRows& x, int dt, int64_t tokens, const int64_t* slots, hipStream_t s) {
    for_kv(dt, c.fmt, c.dim, [&](auto DT, auto FMT, auto D) {
        k_kv_write<DT(), FMT(), D()><<<grid_of(c, tokens), kBlock, 0, s>>>(c, x, tokens, token_group(c, tokens), slots);
    });
    return kname("k_kv_write", dt, c.fmt, c.dim);
}

const char* launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, int dt, void* k, void* v, hipStream_t s) {
    for_kv(dt, c.fmt, c.dim, [&](auto DT, auto FMT, auto D) {
        k_kv_read<DT(), FMT(), D()><<<grid_of(c, tokens), kBlock, 0, s>>>(c, slots, tokens, token_group(c, tokens), k, v);
    });
    return kname("k_kv_read", dt, c.fmt, c.dim);
}

}  // namespace bg
