// bg_kvattn.h -- what the attention kernels over the KV cache share: which
// positions a row sees, and codes on their way to FP16 matrix operands.
#pragma once
#include <type_traits>

#include "bg_device.h"
#include "bg_kv.h"

namespace bg {

// Positions are split into `splits` runs of `tiles` visible tiles; the last
// run takes whatever is left.
struct KvSplit {
    int splits, tiles;
};

// A sequence: its queries are rows q0 .. q0 + len - 1 of q and stand at
// positions first .. first + len - 1 = kv - 1.
// Each query sees positions below `prefix` whatever its own (SCORED; else 0).
struct KvSeq {
    int64_t q0;
    int len, kv, first, prefix;
};

template <bool SCORED>
__device__ __forceinline__ KvSeq kv_seq(const KvAttnArgs& a, int b) {
    KvSeq q;
    int64_t q0 = b, q1 = b + 1;
    if (a.cu_q) {
        q0 = a.cu_q[b];
        q1 = a.cu_q[b + 1];
        q0 = q0 < 0 ? 0 : q0 > a.tokens ? a.tokens : q0;
        q1 = q1 < q0 ? q0 : q1 > a.tokens ? a.tokens : q1;
    }
    const int64_t room = a.max_pages << a.c.page_shift, kv = a.kv_lens[b];
    q.q0 = q0;
    q.kv = (int)(kv < 0 ? 0 : kv > room ? room : kv);
    q.len = (int)(q1 - q0);
    q.first = q.kv - q.len;
    q.prefix = 0;
    if constexpr (SCORED) {
        if (a.prefix) {
            const int n = a.prefix[b];
            q.prefix = n < 0 ? 0 : n > q.kv ? q.kv : n;
        }
    }
    return q;
}

// The sequence's rows of a kv head: those of its first max_q queries.
__device__ __forceinline__ int kv_rows(const KvAttnArgs& a, const KvSeq& q) {
    return (q.len < (int)a.max_q ? q.len : (int)a.max_q) * (a.q_heads / a.c.heads);
}

// The rows r0 .. rows - 1 of sequence b, of which a block takes its first.
struct KvBlock {
    int b, r0, rows;
    KvSeq q;
};

// Row block rb of blockIdx.z: of sequence z, of its first `chunk` queries if that is set; past
// the batch, of those queries from `chunk` on whose sequence holds token (z - batch) chunk,
// up to the next such token.  Between two such tokens no sequence has queries from `chunk`
// on but the one that holds the first.  False: none.
template <bool SCORED>
__device__ __forceinline__ bool kv_block(const KvAttnArgs& a, int rb, int per_block, KvBlock& o) {
    const int G = a.q_heads / a.c.heads, z = blockIdx.z;
    if (z < (int)a.batch) {
        o.b = z;
        o.q = kv_seq<SCORED>(a, z);
        o.rows = kv_rows(a, o.q);
        if (a.chunk && o.rows > (int)a.chunk * G) o.rows = (int)a.chunk * G;
        o.r0 = rb * per_block;
    } else {
        const int64_t t = (z - a.batch) * a.chunk;
        int low = 0, high = (int)a.batch - 1;              // the last sequence that starts at t or before
        while (low < high) {
            const int mid = (low + high + 1) >> 1;
            if (a.cu_q[mid] <= t) low = mid;
            else high = mid - 1;
        }
        o.b = low;
        o.q = kv_seq<SCORED>(a, low);
        const int64_t at = t - o.q.q0;
        if (at < 0 || at >= o.q.len) return false;
        const int64_t first = at < a.chunk ? a.chunk : at, end = at + a.chunk < o.q.len ? at + a.chunk : o.q.len;
        o.rows = (int)end * G;
        o.r0 = (int)first * G + rb * per_block;
    }
    return o.r0 < o.rows;
}

// Whether query i of the sequence sees position j < kv (its page aside).
template <bool SCORED>
__device__ __forceinline__ bool kv_sees(const KvAttnArgs& a, const KvSeq& q, int i, int j) {
    if (a.tree) {
        const int e = j - q.first;
        if (e < 0) return j < q.kv;
        return j < q.kv && e < 64 * a.tree_words && (a.tree[(q.q0 + i) * a.tree_words + (e >> 6)] >> (e & 63) & 1);
    }
    const int at = q.first + i;
    return (j <= at || (SCORED && j < q.prefix)) && (a.window == 0 || j > at - (int)a.window || j < (int)a.sinks);
}

// What queries i0 .. i1 see between them: positions [0, sink) and [low, high),
// as `tiles` tiles of T positions; tile n is tile(n).
struct KvRange {
    int low, high, sink, sink_tiles, low_tile, tiles;
    int all_high, all_low;     // every one of the queries sees [0, all_high), of these but [sink, all_low)

    // Some query may see j.
    __device__ __forceinline__ bool live(int j) const { return (j < high) & ((j >= low) | (j < sink)); }
    // Every query sees all of [base, base + n).
    __device__ __forceinline__ bool whole(int base, int n) const {
        return (base + n <= all_high) & ((base >= all_low) | (base + n <= sink));
    }
    __device__ __forceinline__ int tile(int n) const { return n < sink_tiles ? n : n - sink_tiles + low_tile; }
};

template <int T, bool SCORED>
__device__ __forceinline__ KvRange kv_range(const KvAttnArgs& a, const KvSeq& q, int i0, int i1) {
    KvRange r;
    if (a.tree) {
        r.low = r.all_low = r.sink = 0;
        r.high = q.kv;
        r.all_high = q.first;
    } else {
        const int at0 = q.first + i0, at1 = q.first + i1;
        r.high = at1 + 1 > 0 ? at1 + 1 : 0;
        r.all_high = at0 + 1;
        if constexpr (SCORED) {
            r.high = r.high > q.prefix ? r.high : q.prefix;
            r.all_high = r.all_high > q.prefix ? r.all_high : q.prefix;
        }
        const int w = (int)a.window;
        r.low = w && at0 - w + 1 > 0 ? at0 - w + 1 : 0;
        r.all_low = w && at1 - w + 1 > 0 ? at1 - w + 1 : 0;
        r.sink = (int)(a.sinks < r.high ? a.sinks : r.high);
    }
    r.sink_tiles = (r.sink + T - 1) / T;
    r.low_tile = r.low / T;
    if (r.low_tile <= r.sink_tiles) r.sink_tiles = r.low_tile = 0;     // no gap between the two
    const int end = (r.high + T - 1) / T;
    r.tiles = r.sink_tiles + (end > r.low_tile ? end - r.low_tile : 0);
    return r;
}

// A block's tiles [t0, t1): its split's share.  A prefix may show a block far more tiles past its window than the host
// counted on from the mean of the queries (kv_attn_workspace_bytes does not know of it): then the splits share them
// equally, else the last takes what is left.  3,000 queries of one of 8 sequences, window 64, prefix 2,990, D = 64, INT8, five
// splits: 48 us with what is left to the last (2,481 positions), 33 so; 8,000 of one of 2, four heads of 128, two splits: 232 and 170.
template <bool SCORED>
__device__ __forceinline__ void kv_run(const KvAttnArgs& a, const KvSplit& sp, const KvRange& rg, int split, int& t0, int& t1) {
    int run = sp.tiles;
    if constexpr (SCORED) {
        if (a.prefix && rg.tiles > run * sp.splits) run = (rg.tiles + sp.splits - 1) / sp.splits;
    }
    t0 = split * run;
    t1 = split + 1 == sp.splits || t0 + run > rg.tiles ? rg.tiles : t0 + run;
}

// How a 16-lane row group holds a row of codes: a key's D codes over 4 lanes,
// KC chunks of KB bytes each; a value's over 16 lanes, VB bytes each.  Operands
// hold UNIT^-1 times the code.
template <int FMT, int D>
struct KvLayout {
    static constexpr int PER = FMT == KV_U4 ? 2 : 1;          // codes per byte
    static constexpr int ROW = D / PER;
    static constexpr int KB = ROW / 4 < 16 ? ROW / 4 : 16, KC = ROW / (4 * KB), KW = KC * KB / 4;
    static constexpr int VB = ROW / 16, VW = VB < 4 ? 1 : VB / 4;
    static constexpr float UNIT = FMT == KV_FP8 ? 1.0f : 512.0f;
};

template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* w) {
    if constexpr (N == 32) {
        load_bytes<16>(p, w);
        load_bytes<16>(p + 16, w + 4);
    } else if constexpr (N == 1) {
        w[0] = *p;
    } else if constexpr (N == 2) {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (N == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 8) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x; w[1] = x.y;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
}

template <int FMT>
__device__ __forceinline__ float kv_scale(uint32_t record) {
    return FMT == KV_U4 ? f16_to_f32(record & 0xFFFFu) : __uint_as_float(record);
}

// A value record for rows that may not see it: a zero-point that is not finite
// moves to the scale, which only the rows that see the token take.
template <int FMT>
__device__ __forceinline__ uint32_t kv_masked_record(uint32_t record) {
    if constexpr (FMT == KV_U4) return (record & 0x7C000000u) == 0x7C000000u ? 0x7E00u : record;
    return record;
}

// A row's references.  Its weights are over 2^m: w = 2^(score - m); its weights times their
// value scales, which the second product takes in FP16, over 2^n, n = m + log2(1 / fb):
// w s fb.  Both are powers of two, so that moving one is exact, and follow what the row
// itself sees and nothing else: n the largest w |s|, which lies in 2^(T - 1) .. 2^T when
// found and stays below FP16's 2^16; m is n (fb = 1), but for value scales so large or
// small that the weights would leave binary32: within 2^40 of the largest weight.  With
// one reference of the weights and one of the scales instead, a first token with 90 %
// of the weight and a value near zero left the others' weights below FP16's range: 20 %
// off and more at 40,000 tokens in a block.
constexpr float kNoRef = -0x1.fffffep127f;         // of a row that has seen nothing
constexpr float kMaxWeight = 0x1p50f;

// log2 of a scale's magnitude (infinities and NaN aside); those below binary32's normal range count as its least.
__device__ __forceinline__ float scale_log2(float s) { return __builtin_fmaxf(__builtin_amdgcn_logf(__builtin_fabsf(s)), -126.0f); }

// a b, not fused with what takes it.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
    return a * b;
}

// The record that kv_cache_write gives a row of zeros (scale 1, zero-point 0).  Its products
// are 0 whatever the weight, so it must not raise a reference: next to a first token of
// zeros that takes most of the weight, the others would fall below FP16's range.
template <int FMT>
__device__ __forceinline__ bool kv_maybe_zeros(uint32_t record) {
    return record == (FMT == KV_U4 ? 0x3C00u : 0x3F800000u);
}

// Codes that are not 0 (E4M3: of either sign).
template <int FMT>
__device__ __forceinline__ uint32_t kv_some(uint32_t codes) {
    return FMT == KV_FP8 ? codes & 0x7F7F7F7Fu : codes;
}

struct RowStep {
    float l, o;                // what the move makes of the sum and of the outputs
};

// Moves a row's references: ty is the largest score so far, tp the largest score + log2
// |value scale| of the tile, -infinity if there are none.
template <int T>
__device__ __forceinline__ RowStep raise_row(float& m, float& fb, float ty, float tp) {
    const float n = m + (float)(127 - (int)(__float_as_uint(fb) >> 23));
    const float n1 = tp > n + (T + 1) ? __builtin_ceilf(tp) - T : n;
    const float y = __builtin_fmaxf(__builtin_ceilf(ty), kNoRef);
    const float m1 = __builtin_fminf(__builtin_fmaxf(n1, y - 40.0f), y + 40.0f);
    const float b = __builtin_fminf(__builtin_fmaxf(n1 - m1, -120.0f), 100.0f);
    const RowStep f{__builtin_amdgcn_exp2f(m - m1), __builtin_amdgcn_exp2f(n - (m1 + b))};
    m = m1;
    fb = __uint_as_float((uint32_t)(127 - (int)b) << 23);
    return f;
}

// The slope of a head's bias, in units of the scores before their last factor, a.cap.  With slopes the
// tiles are taken from the last one back: a query's nearest positions usually hold its largest scores, so its
// references seldom move after the first (forwards, in every tile of a steep head: 2,048 queries over a window
// of 4,096, E4M3, 32 heads of 128, slopes 2^(-i / 4): 395 us, 171 so).
// It stays finite, as the bias of a query's own position is 0 times it; NaN stays NaN.
__device__ __forceinline__ float head_slope(const KvAttnArgs& a, int head) {
    const float s = a.slopes[head] * 0x1.715476p0f * (a.cap_inv != 0.0f ? a.cap_inv : 1.0f);
    return __builtin_fabsf(s) == __builtin_inff() ? __builtin_copysignf(0x1.fffffep127f, s) : s;
}

// Caps up to kCapExp are taken as tanh(u) = 1 - 2 / (1 + 2^x), x = 2 log2(e) u (a factor that the tokens'
// scales take along): within 2^-21, so a score errs by 2^-21 of its cap, a weight by 2^-13 of itself at most, of
// which FP16 takes 2^-11.  Larger ones (FAR) as polynomials, within 2^-21 of tanh(u).  Those have fewer vector
// instructions, 6 a score against what 10 take, but they need their largest score looked at: with a branch
// on it in the loop the above chunk with a cap of 50 took 288 us, by the power it takes 211.
constexpr float kCapExp = 256.0f;
__device__ __forceinline__ float cap_unit(const KvAttnArgs& a) { return a.cap_far ? a.cap_inv : a.cap_inv * 0x1.715476p1f; }

// tanh(u) / u for z = u^2 (minimax polynomials): |u| up to kTanhSmall, off by 2^-22.2, and up to 1, by 2^-22.6.
constexpr float kTanhSmall = 0.4f;

__device__ __forceinline__ float tanh_ratio_small(float z) {
    float p = -0x1.858f22p-5f;
    p = __builtin_fmaf(p, z, 0x1.0fca24p-3f);
    p = __builtin_fmaf(p, z, -0x1.55502ap-2f);
    return __builtin_fmaf(p, z, 0x1.fffffcp-1f);
}

__device__ __forceinline__ float tanh_ratio(float z) {
    float p = 0x1.10e5d6p-10f;
    p = __builtin_fmaf(p, z, -0x1.968b6cp-8f);
    p = __builtin_fmaf(p, z, 0x1.4c6e58p-6f);
    p = __builtin_fmaf(p, z, -0x1.b5eb84p-5f);
    p = __builtin_fmaf(p, z, 0x1.10e672p-3f);
    p = __builtin_fmaf(p, z, -0x1.55540ap-2f);
    return __builtin_fmaf(p, z, 0x1.fffffep-1f);
}

// u to tanh(u).  FAR: where scores under large caps lie, by a polynomial; if some score of the wave is larger, by
// another up to 1 and as below beyond, for all.
template <bool FAR, int N>
__device__ __forceinline__ void cap_scores(float (&u)[N]) {
    float top = 0.0f;
    if constexpr (FAR) {
#pragma unroll
        for (int j = 0; j < N; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(u[j]));
    }
    if constexpr (!FAR) {
#pragma unroll
        for (int j = 0; j < N; ++j) u[j] = __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u[j])), 1.0f);
    } else if (__any(top > kTanhSmall)) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float x = u[j], y = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(__builtin_fabsf(x) * 0x1.715476p1f));
            u[j] = __builtin_fabsf(x) > 1.0f ? __builtin_copysignf(y, x) : x * tanh_ratio(x * x);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) u[j] *= tanh_ratio_small(u[j] * u[j]);
    }
}

// Two small unsigned integers in the halves of w, read as FP16 subnormals
// n 2^-24, to n * mul 2^-24 + add: exact.
__device__ __forceinline__ half2_t small_pair(uint32_t w, _Float16 mul, half2_t add) {
    return __builtin_elementwise_fma(__builtin_bit_cast(half2_t, w), half2_t{mul, mul}, add);
}

__device__ __forceinline__ half8_t join4(half2_t a, half2_t b, half2_t c, half2_t d) {
    return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The zero-point part of a 4-bit operand: -z 2^-9 in both halves.
__device__ __forceinline__ half2_t minus_zero(uint32_t record) {
    const _Float16 z = __builtin_bit_cast(_Float16, (uint16_t)(record >> 16)) * (_Float16)-0x1p-9f;
    return half2_t{z, z};
}

// Eight codes (one or two words) to FP16.  4-bit codes come in the order
// 0 4 1 5 2 6 3 7, which load_query follows.
template <int FMT>
__device__ __forceinline__ half8_t codes8(const uint32_t* w, half2_t z) {
    if constexpr (FMT == KV_FP8) {
        return join4(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], 1.0f, true),
                     __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], 1.0f, true));
    } else if constexpr (FMT == KV_I8) {
        const half2_t off{(_Float16)-0.25f, (_Float16)-0.25f};        // -128 2^-9
        const uint32_t a = w[0] ^ 0x80808080u, b = w[1] ^ 0x80808080u;
        const _Float16 up = (_Float16)0x1p15f;
        return join4(small_pair(__builtin_amdgcn_perm(0u, a, 0x0c010c00u), up, off), small_pair(__builtin_amdgcn_perm(0u, a, 0x0c030c02u), up, off),
                     small_pair(__builtin_amdgcn_perm(0u, b, 0x0c010c00u), up, off), small_pair(__builtin_amdgcn_perm(0u, b, 0x0c030c02u), up, off));
    } else {
        const _Float16 u0 = (_Float16)0x1p15f, u1 = (_Float16)0x1p11f;
        const uint32_t a = w[0], b = w[0] >> 8;
        return join4(small_pair(a & 0x000F000Fu, u0, z), small_pair(a & 0x00F000F0u, u1, z),
                     small_pair(b & 0x000F000Fu, u0, z), small_pair(b & 0x00F000F0u, u1, z));
    }
}

// A key's fragments, one per 32 head elements.
template <int FMT, int D>
__device__ __forceinline__ void key_fragments(const uint32_t* w, uint32_t record, half8_t* f) {
    const half2_t z = FMT == KV_U4 ? minus_zero(record) : half2_t{(_Float16)0.0f, (_Float16)0.0f};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) f[i] = codes8<FMT>(w + i * (FMT == KV_U4 ? 1 : 2), z);
}

// -z 2^-9 of the value tokens of k-slots 2 n, 2 n + 1.
__device__ __forceinline__ void value_zeros(const uint32_t* r, uint32_t* vz) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint32_t w = r[2 * n] >> 16 | (r[2 * n + 1] & 0xFFFF0000u);
        vz[n] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, w) * half2_t{(_Float16)-0x1p-9f, (_Float16)-0x1p-9f});
    }
}

// Element d of a lane's value codes, 8 tokens, to FP16.
template <int FMT, int D, int VW>
__device__ __forceinline__ half8_t value_fragment(const uint32_t (&v)[8][VW], const uint32_t* vz, int d) {
    half2_t x[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        if constexpr (FMT == KV_FP8) {
            // both elements of a byte pair come from one permute: the compiler shares it
            const int w = d / 4, i = d % 4 & 2;
            const uint32_t sel = (uint32_t)(5 + i) << 24 | (uint32_t)(1 + i) << 16 | (uint32_t)(4 + i) << 8 | (uint32_t)i;
            const uint32_t y = __builtin_amdgcn_perm(v[2 * n + 1][w], v[2 * n][w], sel);
            x[n] = d & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y, 1.0f, false);
        } else {
            const int byte = FMT == KV_U4 ? d / 2 : d, w = byte / 4, i = byte % 4;
            const uint32_t sel = 0x0c000c00u | (uint32_t)(4 + i) << 16 | (uint32_t)i;
            if constexpr (FMT == KV_I8) {
                const uint32_t y = __builtin_amdgcn_perm(v[2 * n + 1][w] ^ 0x80808080u, v[2 * n][w] ^ 0x80808080u, sel);
                x[n] = small_pair(y, (_Float16)0x1p15f, half2_t{(_Float16)-0.25f, (_Float16)-0.25f});
            } else {
                const uint32_t y = __builtin_amdgcn_perm(v[2 * n + 1][w], v[2 * n][w], sel);
                const half2_t z = __builtin_bit_cast(half2_t, vz[n]);
                x[n] = d & 1 ? small_pair(y & 0x00F000F0u, (_Float16)0x1p11f, z) : small_pair(y & 0x000F000Fu, (_Float16)0x1p15f, z);
            }
        }
    }
    return join4(x[0], x[1], x[2], x[3]);
}

typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));

// The larger of each half's magnitude, as bits (the order of FP16's and of BF16's).
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, a), __builtin_bit_cast(ushort2_t, b & 0x7FFF7FFFu)));
}

__device__ __forceinline__ uint32_t max_magnitude(uint4 x) {
    return max_magnitude(max_magnitude(max_magnitude(max_magnitude(0u, x.x), x.y), x.z), x.w);
}

// The exponent e of the largest of BF16 magnitudes (the larger half of m), at least
// -100; 13, which leaves them as they are, if that is 0 or not finite.
__device__ __forceinline__ int scale_exponent(uint32_t m) {
    const uint32_t top = m >> 16 > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu;
    const int e = (int)(top >> 7) - 127;
    return top == 0u || e == 128 ? 13 : e < -100 ? -100 : e;
}

// Eight query elements as an FP16 fragment, BF16 ones times `up` (FP16 ones are exact as
// they are), in the order of the format's codes.
template <int FMT>
__device__ __forceinline__ half8_t query8(bool bf16, uint4 x, float up) {
    half2_t y[4];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (bf16) {
#pragma unroll
        for (int n = 0; n < 4; ++n) y[n] = half2_t{(_Float16)(__uint_as_float(w[n] << 16) * up), (_Float16)(__uint_as_float(w[n] & 0xFFFF0000u) * up)};
    } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) y[n] = __builtin_bit_cast(half2_t, w[n]);
    }
    return FMT == KV_U4 ? half8_t{y[0][0], y[2][0], y[0][1], y[2][1], y[1][0], y[3][0], y[1][1], y[3][1]} : join4(y[0], y[1], y[2], y[3]);
}

// The factor that takes a product of operands to a base-2 exponent, queries scaled so
// that 2^e comes to 2^13.
template <int FMT, int D>
__device__ __forceinline__ float query_unit(const KvAttnArgs& a, int e) {
    return a.scale * 0x1.715476p0f * KvLayout<FMT, D>::UNIT * __uint_as_float((uint32_t)(127 - 13 + e) << 23);
}

// The row's query fragments for lane group g of four, BF16 ones scaled by a power of
// two so that FP16 holds them; returns the factor that takes a product of
// operands to a base-2 exponent.  Rows that are not there are zeros.
template <int FMT, int D>
__device__ __forceinline__ float load_query(const KvAttnArgs& a, int64_t at, int g, bool ok, half8_t* f) {
    using L = KvLayout<FMT, D>;
    constexpr int N = D / 32, CHUNK = FMT == KV_U4 ? 2 * L::KB : L::KB;    // elements a lane holds in a run
    uint4 w[N];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int in = i * 8 % CHUNK, c = i * 8 / CHUNK;
        const int d = c * 4 * CHUNK + g * CHUNK + in;
        w[i] = make_uint4(0, 0, 0, 0);
        if (ok) w[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + d);
    }
    int e = 13;
    if (a.bf16) {
#pragma unroll
        for (int i = 0; i < N; ++i) top = max_magnitude(top, max_magnitude(w[i]));
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) top = max_magnitude(top, (uint32_t)__shfl_xor((int)top, o, 64));
        e = scale_exponent(top);
    }
    const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = query8<FMT>(a.bf16, w[i], up);
    return query_unit<FMT, D>(a, e);
}

// A wave's 32 rows, two lane groups, as they lie in memory: fragment c is elements
// 16 c + 8 g .. 16 c + 8 g + 7.
template <int D>
__device__ __forceinline__ void load_queries(const KvAttnArgs& a, int64_t at, int g, bool ok, half8_t* f) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint4 y = make_uint4(0, 0, 0, 0);
        if (ok) y = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + 16 * c + 8 * g);
        f[c] = __builtin_bit_cast(half8_t, y);
    }
}

// ... and to FP16, BF16 ones scaled by a power of two: the largest element of the block's
// rows (WAVES waves; rows that hold an infinity or NaN aside) lands in [2^15, 2^16).  A row
// that lies more than 2^16 below takes its own, and `own`, which its scores then lack, is
// not 1: another row never costs it bits.
template <int FMT, int D, int WAVES>
__device__ __forceinline__ float scale_queries(const KvAttnArgs& a, int wave, uint32_t* lds, half8_t* f, float& own) {
    constexpr int N = D / 16;
    int e = 15, block = 15;
    if (a.bf16) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < N; ++c) top = max_magnitude(top, max_magnitude(__builtin_bit_cast(uint4, f[c])));
        top = max_magnitude(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const uint32_t t = top >> 16 > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu;
        const bool some = t != 0u && t < 0x7F80u;
        e = scale_exponent(top);
        uint32_t most = some ? (uint32_t)(e + 128) : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = (uint32_t)__shfl_xor((int)most, o, 64);
            most = x > most ? x : most;
        }
        if ((threadIdx.x & 63) == 0) lds[wave] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) most = lds[w] > most ? lds[w] : most;
        block = __builtin_amdgcn_readfirstlane(most == 0u ? 15 : (int)most - 128);
        e = !some || e >= block - 16 ? block : e < block - 126 ? block - 126 : e;
    }
    own = __uint_as_float((uint32_t)(127 + e - block) << 23);
    const float up = __uint_as_float((uint32_t)(127 + 15 - e) << 23);
#pragma unroll
    for (int c = 0; c < N; ++c) f[c] = query8<FMT>(a.bf16, __builtin_bit_cast(uint4, f[c]), up);
    return query_unit<FMT, D>(a, block - 2);
}

template <int N>
__device__ __forceinline__ void store_out(const KvAttnArgs& a, int64_t at, const float* y) {
    uint16_t* p = static_cast<uint16_t*>(a.out) + at;
    if constexpr (N == 1) {
        *p = a.bf16 ? f32_to_bf16(y[0]) : f32_to_f16(y[0]);
    } else {
        uint32_t w[N / 2];
        if (a.bf16) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) w[i] = (uint32_t)f32_to_bf16(y[2 * i]) | (uint32_t)f32_to_bf16(y[2 * i + 1]) << 16;
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) w[i] = (uint32_t)f32_to_f16(y[2 * i]) | (uint32_t)f32_to_f16(y[2 * i + 1]) << 16;
        }
        if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else {
#pragma unroll
            for (int i = 0; i < N / 8; ++i) reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
}

// f(FMT, D) over the formats and head sizes.
template <typename F>
void for_format(int fmt, int dim, F&& f) {
    auto on_dim = [&](auto FMT) {
        if (dim == 64) f(FMT, std::integral_constant<int, 64>{});
        else if (dim == 128) f(FMT, std::integral_constant<int, 128>{});
        else f(FMT, std::integral_constant<int, 256>{});
    };
    if (fmt == KV_I8) on_dim(std::integral_constant<int, KV_I8>{});
    else if (fmt == KV_FP8) on_dim(std::integral_constant<int, KV_FP8>{});
    else on_dim(std::integral_constant<int, KV_U4>{});
}

constexpr int64_t kGridZ = 65535;        // blocks along the grid's third axis

// Sequences, and the tokens past the batch of kv_block.
inline unsigned kv_grid_z(const KvAttnArgs& a) { return (unsigned)(a.batch + (a.chunk ? (a.tokens + a.chunk - 1) / a.chunk : 0)); }

// Many query rows per kv head, rows of row_blocks blocks of 8 waves (4 at D = 256; either at D = 64) (k_kvattn_many.hip).
const char* launch_kv_attn_many(const KvAttnArgs& a, const KvSplit& sp, unsigned row_blocks, int waves, float* po, float* pl, hipStream_t s);
// With other scores (k_kvattn_many_*.hip): biased (or none but a prefix), capped, both, far caps with or without a bias.
void launch_kv_attn_many_bias(const KvAttnArgs& a, const KvSplit& sp, dim3 grid, int waves, float* po, float* pl, hipStream_t s);
void launch_kv_attn_many_cap(const KvAttnArgs& a, const KvSplit& sp, dim3 grid, int waves, float* po, float* pl, hipStream_t s);
void launch_kv_attn_many_cap_bias(const KvAttnArgs& a, const KvSplit& sp, dim3 grid, int waves, float* po, float* pl, hipStream_t s);
void launch_kv_attn_many_far_cap(const KvAttnArgs& a, const KvSplit& sp, dim3 grid, int waves, float* po, float* pl, hipStream_t s);

}  // namespace bg
