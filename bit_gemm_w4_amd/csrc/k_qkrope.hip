// k_qkrope.hip -- norms of each head of queries and keys and the rotation by their
// positions, the keys quantized into the KV cache with the values in the same launch.
//
//   y = x / sqrt(mean x^2 + eps) (offset + w)             per head, optional
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t)      pairs of the first `rot` elements
// t = position * frequency.  Frequencies come as turns a position in units of 2^-64, so
// that position * frequency mod 2^64 is the angle's fraction of a turn: exact for every
// position, where a binary32 product is off by 0.06 at 10^6.
//
// Bound by HBM: rows are read once, queries and codes written once.  A block takes a run
// of rows of one kind (queries, keys or values; a row is one token's head, D / 8 lanes of
// eight elements), puts the cosines and sines of its tokens into LDS, once for all heads,
// and asks for the next row before it turns the last.  A lane holds four whole pairs: in
// halves elements 4 l .. 4 l + 3 and rot / 2 + 4 l .. (two loads of 8 bytes, each
// contiguous over lanes, and no exchange), as neighbours 8 l .. 8 l + 7.
//
// Keys on their way to codes are computed in binary64 up to one rounding to binary32, and
// quantized from there as kv_cache_write does: a code sits next to a border of its rounding, so
// in binary32 some codes would follow the order of a row's sum.  So they are those of the
// formula, whatever the split, and they can be tested bit for bit.  Binary64 multiply-adds run
// at the rate of binary32 ones here; in binary32 the case below takes 78 us.
//
// 16,383 tokens of 32 query and 8 + 8 key and value heads of 128, BF16 into E4M3: 82 us for
// 370 MB, 4.6 TB/s (a large copy runs at 5.1); queries alone 45 us, 6.0 TB/s with part of them in the
// last-level cache; keys and values 33 us, where kv_cache_write takes 27.  First form 105 us: with roots and
// quotients by the compiler's sequences, a division and 64-bit products for each row, and binary64 copies of rows and
// weights that stayed in registers (118 of them, four waves a SIMD; 76 now).  16 tokens: 4.5 us.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kv.h"
#include "bg_kvquant.h"

namespace bg {
namespace {

constexpr int kBlock = 256;
constexpr int kPhases = 1152;             // cosines and sines of a block; grid_of keeps to it

enum { ROW_Q = 0, ROW_K = 1, ROW_V = 2 };

struct RopeGrid {
    unsigned blocks[3];                   // of queries, keys and values, in this order
    int rows[3];                          // of a block
};

// cos and sin of 2 pi u 2^-64: to the nearest quarter turn, and from there by their series,
// whose first terms left out are below 2^-54.
__device__ __forceinline__ void cos_sin(uint64_t u, double& c, double& s) {
    const uint32_t quarter = (uint32_t)((u + (1ull << 61)) >> 62);
    const double t = (double)(int64_t)(u - ((uint64_t)quarter << 62)) * 0x1.921fb54442d18p-62;      // 2 pi 2^-64
    const double z = t * t;
    constexpr double S[] = {-1.0 / 6, 1.0 / 120, -1.0 / 5040, 1.0 / 362880, -1.0 / 39916800, 1.0 / 6227020800.0, -1.0 / 1307674368000.0};
    constexpr double C[] = {-1.0 / 2, 1.0 / 24, -1.0 / 720, 1.0 / 40320, -1.0 / 3628800, 1.0 / 479001600.0, -1.0 / 87178291200.0,
                            1.0 / 20922789888000.0};
    double a = S[6], b = C[7];
#pragma unroll
    for (int i = 5; i >= 0; --i) a = __builtin_fma(a, z, S[i]);
#pragma unroll
    for (int i = 6; i >= 0; --i) b = __builtin_fma(b, z, C[i]);
    a = __builtin_fma(a * z, t, t);
    b = __builtin_fma(b, z, 1.0);
    const double x = quarter & 1 ? a : b, y = quarter & 1 ? b : a;
    c = (quarter + 1) & 2 ? -x : x;
    s = quarter & 2 ? -y : y;
}

// Four elements of a row as they lie.
template <int DT>
using Four = std::conditional_t<DT == DT_F32, uint4, uint2>;

template <int DT>
__device__ __forceinline__ Four<DT> load4(const void* p, int64_t at) {
    if constexpr (DT == DT_F32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    else return *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
}

template <int DT>
__device__ __forceinline__ void floats4(const Four<DT>& x, float* f) {
    if constexpr (DT == DT_F32) {
        f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y); f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
    } else if constexpr (DT == DT_BF16) {
        f[0] = __uint_as_float(x.x << 16); f[1] = __uint_as_float(x.x & 0xFFFF0000u);
        f[2] = __uint_as_float(x.y << 16); f[3] = __uint_as_float(x.y & 0xFFFF0000u);
    } else {
        f[0] = f16_to_f32(x.x & 0xFFFFu); f[1] = f16_to_f32(x.x >> 16);
        f[2] = f16_to_f32(x.y & 0xFFFFu); f[3] = f16_to_f32(x.y >> 16);
    }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t at, const float* f) {
    if constexpr (DT == DT_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        auto half = [](float x) { return (uint32_t)(DT == DT_BF16 ? f32_to_bf16(x) : f32_to_f16(x)); };
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = make_uint2(half(f[0]) | half(f[1]) << 16, half(f[2]) | half(f[3]) << 16);
    }
}

// 1 / sqrt(x): the hardware's estimate and a step of Newton's (in binary64 of third order: the
// estimate is good for 2^-23), 5 operations where the root and the quotient take 20 and more.
__device__ __forceinline__ float inverse_root(float x) {
    const float r = __builtin_amdgcn_rsqf(x), e = __builtin_fmaf(-x * r, r, 1.0f);
    float y = __builtin_fmaf(0.5f * r, e, r);
    const bool plain = x >= 0x1p-100f && x <= 0x1p100f;
    if (__any(!plain)) y = plain ? y : 1.0f / __builtin_sqrtf(x);
    return y;
}

__device__ __forceinline__ double inverse_root(double x) {
    const double r = __builtin_amdgcn_rsq(x), e = __builtin_fma(-x * r, r, 1.0);
    return __builtin_fma(r * e, __builtin_fma(0.375, e, 0.5), r);
}

// Norm and rotation of a lane's eight elements, in T, a pair at a time; pair n's cosine and sine lie at phase[n * step].
// Without a norm w is 1 and offset 0; a lane that does not turn takes what lies in LDS and drops the result: no
// branches between the pairs.
template <typename T, int D, typename P>
__device__ __forceinline__ void turn_row(const RopeArgs& a, float (&x)[8], const float (&w)[8], bool norm, double offset, bool turns, const P* phase, int step) {
    T r = 1;
    if (norm) {
        T sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_elementwise_fma((T)x[i], (T)x[i], sum);
        sum = over_row<D / 8>(sum, [](T p, T q) { return p + q; });
        r = inverse_root(sum * (T)(1.0 / D) + (T)a.eps);
    }
    auto pair = [&](int i, int j, int n) {
        float xi = x[i], xj = x[j], wi = w[i], wj = w[j];
        // binary64 copies that wait in registers would cost waves
        if constexpr (sizeof(T) == 8) asm volatile("" : "+v"(xi), "+v"(xj), "+v"(wi), "+v"(wj));
        T p = (T)xi * r * ((T)wi + (T)offset), q = (T)xj * r * ((T)wj + (T)offset);
        const P z = phase[n * step];
        const T c = z.x, s = z.y, u = __builtin_elementwise_fma(p, c, -(q * s)), v = __builtin_elementwise_fma(p, s, q * c);
        p = turns ? u : p;
        q = turns ? v : q;
        x[i] = (float)p;
        x[j] = (float)q;
    };
    if (a.interleaved) {
#pragma unroll
        for (int n = 0; n < 4; ++n) pair(2 * n, 2 * n + 1, n);
    } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) pair(n, n + 4, n);
    }
}

// FMT 0: no cache, keys go to k_out.
template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kBlock) k_qk_rope(RopeArgs a, KvCache cache, RopeGrid grid) {
    constexpr int L = D / 8, SLOTS = kBlock / L;
    __shared__ double2 phase[kPhases];
    const int lane = threadIdx.x % L;
    unsigned block = blockIdx.x;
    int kind = ROW_Q;
    for (; kind < ROW_V && block >= grid.blocks[kind]; ++kind) block -= grid.blocks[kind];
    const int heads = kind == ROW_Q ? a.q_heads : a.kv_heads, pairs = a.rot / 2;
    const uint32_t per = (uint32_t)grid.rows[kind], r0 = block * per, all = (uint32_t)a.tokens * heads;
    const uint32_t rows = all - r0 < per ? all - r0 : per;
    const uint32_t t0 = r0 / heads, h0 = r0 - t0 * heads;             // the first row's token and head
    const void* src = kind == ROW_Q ? a.q : kind == ROW_K ? a.k : a.v;
    const int64_t ts = kind == ROW_Q ? a.q_ts : kind == ROW_K ? a.k_ts : a.v_ts, hs = kind == ROW_Q ? a.q_hs : kind == ROW_K ? a.k_hs : a.v_hs;
    const bool wide = FMT != 0 && kind == ROW_K;
    // the lane's two runs of four elements
    const bool halves = kind != ROW_V && !a.interleaved && lane < a.rot / 8;
    const int e0 = halves ? 4 * lane : 8 * lane, e1 = halves ? pairs + 4 * lane : 8 * lane + 4;
    const bool turns = kind != ROW_V && lane < a.rot / 8;

    // The lane's next row: token and head from the block's first, where it lies and where it goes.  SLOTS rows
    // on is dt tokens and dh heads on, or a token more and the heads less: no division or product a row.
    constexpr int SIZE = DT == DT_F32 ? 4 : 2;
    const bool rows_out = kind == ROW_Q || (FMT == 0 && kind == ROW_K);
    const int64_t ots = kind == ROW_Q ? a.qo_ts : a.ko_ts, ohs = kind == ROW_Q ? a.qo_hs : a.ko_hs;
    const uint32_t dt = SLOTS / (uint32_t)heads, dh = SLOTS - dt * heads;
    const int64_t on = (dt * ts + dh * hs) * SIZE, over = (ts - heads * hs) * SIZE;
    const int64_t out_on = (dt * ots + dh * ohs) * SIZE, out_over = (ots - heads * ohs) * SIZE;
    uint32_t i = threadIdx.x / L, next_t = (h0 + i) / (uint32_t)heads, next_h = h0 + i - next_t * heads;
    const char* from = static_cast<const char*>(src) + ((int64_t)(t0 + next_t) * ts + (int64_t)next_h * hs + e0) * SIZE;
    char* to = static_cast<char*>(kind == ROW_Q ? a.q_out : a.k_out) + ((int64_t)(t0 + next_t) * ots + (int64_t)next_h * ohs + e0) * SIZE;
    const int apart = (e1 - e0) * SIZE;
    Four<DT> x0{}, x1{};
    int64_t next_slot = -1;
    auto ask = [&]() {
        x0 = load4<DT>(from, 0);
        x1 = load4<DT>(from + apart, 0);
        if (FMT != 0 && kind != ROW_Q) next_slot = a.slots[t0 + next_t];
    };
    if (i < rows) ask();
    const void* weight = kind == ROW_Q ? a.q_weight : kind == ROW_K ? a.k_weight : nullptr;
    float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    const double offset = weight ? a.offset : 0.0;
    if (weight) {
        if (a.weight_f32) {
            floats4<DT_F32>(load4<DT_F32>(weight, e0), w);
            floats4<DT_F32>(load4<DT_F32>(weight, e1), w + 4);
        } else {
            floats4<DT>(load4<DT>(weight, e0), w);
            floats4<DT>(load4<DT>(weight, e1), w + 4);
        }
    }
    // pair n of token t: phase[t pairs + (n % 4) pairs / 4 + n / 4], so that lanes read next to each other
    if (kind != ROW_V && pairs > 0 && rows > 0) {
        const uint32_t some = ((h0 + rows - 1) / (uint32_t)heads + 1) * pairs;
        for (uint32_t n = threadIdx.x; n < some; n += kBlock) {
            const uint32_t t = n / pairs, p = n - t * pairs;
            double c, s;
            cos_sin((uint64_t)(int64_t)a.positions[t0 + t] * a.freqs[p], c, s);
            const uint32_t to = t * pairs + (p & 3) * (pairs / 4) + (p >> 2);
            if (wide) phase[to] = make_double2(c, s);
            else reinterpret_cast<float2*>(phase)[to] = make_float2((float)c, (float)s);
        }
        __syncthreads();
    }
    for (; i < rows; i += SLOTS) {
        float x[8];
        floats4<DT>(x0, x);
        floats4<DT>(x1, x + 4);
        const uint32_t t = next_t, h = next_h;
        const int64_t slot = next_slot;
        char* const here = to;
        if (i + SLOTS < rows) {
            next_t += dt;
            next_h += dh;
            const bool wrap = next_h >= (uint32_t)heads;
            next_t += wrap ? 1 : 0;
            next_h -= wrap ? heads : 0;
            from += wrap ? on + over : on;
            to += wrap ? out_on + out_over : out_on;
            ask();
        }
        const uint32_t turn = t * pairs + (turns ? lane : 0);
        if (rows_out) {
            turn_row<float, D>(a, x, w, weight != nullptr, offset, turns, reinterpret_cast<const float2*>(phase) + turn, pairs / 4);
            store4<DT>(here, 0, x);
            store4<DT>(here + apart, 0, x + 4);
        }
        if constexpr (FMT != 0) {
            if (kind == ROW_Q || slot < 0 || slot >= (cache.pages << cache.page_shift)) continue;       // whole rows skip together
            if (wide) turn_row<double, D>(a, x, w, weight != nullptr, offset, turns, phase + turn, pairs / 4);
            const int64_t row = kv_row(cache, slot, (int)h);
            uint8_t* codes = (kind == ROW_V ? cache.v : cache.k) + row * (FMT == KV_U4 ? D / 2 : D);
            const RowCodes q = quantize_row<FMT, D>(x);
            if constexpr (FMT == KV_U4) {
                *reinterpret_cast<uint16_t*>(codes + e0 / 2) = (uint16_t)q.w[0];
                *reinterpret_cast<uint16_t*>(codes + e1 / 2) = (uint16_t)(q.w[0] >> 16);
            } else {
                *reinterpret_cast<uint32_t*>(codes + e0) = q.w[0];
                *reinterpret_cast<uint32_t*>(codes + e1) = q.w[1];
            }
            if (lane == 0) (kind == ROW_V ? cache.vs : cache.ks)[row] = q.record;
        }
    }
}

// Rows of a block: up to eight for each of its row slots while that leaves 2,048 blocks, and no more tokens than
// their cosines and sines have room in LDS.  (So the largest call, 2^28 rows of either, stays below 2^32 threads.)
RopeGrid grid_of(const RopeArgs& a, int dim, bool cache) {
    const int slots = kBlock * 8 / dim, heads[3] = {a.q_heads, a.kv_heads, cache ? a.kv_heads : 0};
    const int64_t all = a.tokens * (heads[0] + heads[1] + heads[2]);
    RopeGrid g;
    for (int n = 0; n < 3; ++n) {
        const int64_t pairs = n == ROW_V ? 0 : a.rot / 2;
        int each = heads[n] ? 8 : 1;
        while (each > 1 && (all / (each * slots) < 2048 || ((each * slots - 1) / heads[n] + 2) * pairs > kPhases)) each /= 2;
        g.rows[n] = each * slots;
        g.blocks[n] = (unsigned)((a.tokens * heads[n] + g.rows[n] - 1) / g.rows[n]);
    }
    return g;
}

}  // namespace

const char* launch_qk_rope(const RopeArgs& a, int dt, int dim, const KvCache* cache, hipStream_t s) {
    const RopeGrid g = grid_of(a, dim, cache != nullptr);
    const KvCache c = cache ? *cache : KvCache{};
    const int fmt = cache ? cache->fmt : 0;
    auto go = [&](auto DT, auto FMT, auto D) { k_qk_rope<DT(), FMT(), D()><<<g.blocks[0] + g.blocks[1] + g.blocks[2], kBlock, 0, s>>>(a, c, g); };
    auto on_dim = [&](auto DT, auto FMT) {
        if (dim == 64) go(DT, FMT, std::integral_constant<int, 64>{});
        else if (dim == 128) go(DT, FMT, std::integral_constant<int, 128>{});
        else go(DT, FMT, std::integral_constant<int, 256>{});
    };
    auto on_fmt = [&](auto DT) {
        if (fmt == KV_I8) on_dim(DT, std::integral_constant<int, KV_I8>{});
        else if (fmt == KV_FP8) on_dim(DT, std::integral_constant<int, KV_FP8>{});
        else if (fmt == KV_U4) on_dim(DT, std::integral_constant<int, KV_U4>{});
        else on_dim(DT, std::integral_constant<int, 0>{});
    };
    if (dt == DT_F32) on_fmt(std::integral_constant<int, DT_F32>{});
    else if (dt == DT_F16) on_fmt(std::integral_constant<int, DT_F16>{});
    else on_fmt(std::integral_constant<int, DT_BF16>{});
    return kname("k_qk_rope", dt, fmt, dim);
}

}  // namespace bg
