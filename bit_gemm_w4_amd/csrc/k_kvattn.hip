// k_kvattn.hip -- attention over the paged, quantized KV cache for few query
// rows per kv head (decode steps, small draft trees), and the join of split
// sequences.
//
// Rows are (query token, query head) pairs of one sequence and kv head: the
// G = q_heads / kv_heads heads of a token share the cache's keys and values,
// so a block's rows read them once.
//
// Bound by HBM: a cache token is 2 D codes and 8 bytes of records per kv
// head.  A wave takes 32 tokens at a time straight from memory into registers
// (no LDS, no barrier in the loop), with the next 32 in flight where registers allow:
//   S^T = K Q^T   v_mfma_f32_16x16x32_f16, A = 16 tokens' codes, B = 16 rows
//   O^T += V^T P^T  the same instruction, A = 16 head elements of 32 tokens
// The tile's pages are looked up two tiles ahead; 8 waves a CU with two tiles each
// keep about 130 KB of codes in flight, and 8-bit caches stream at 5.4 TB/s (decode
// of 32 x 8192 tokens, 554 MB: 103 us; a large copy runs at 4.8 TB/s).  4 bits
// have half the bytes for the same instructions: 4 x 131072 tokens 571 MB in
// 114 us, 5.0 TB/s, and a block's start (6 us) weighs more.
//
// The accumulator of S^T holds, in lane (row r, g), tokens 4 g .. 4 g + 3 of
// each 16; those of two S^T tiles are exactly the 8 k-slots that lane feeds to
// the second product if V's k-slots are numbered the same way, so the weights
// go from one product to the next without leaving the lane.  V's codes are
// loaded as they lie ([token][D], D / 16 codes per lane and token); a byte
// permute pairs two tokens' codes of one element, which any conversion to FP16
// needs anyway, and the elements a lane holds become rows of different MFMAs.
//
// Numerics.  Codes are exact in FP16 (INT8 and 4-bit codes less their offset,
// E4M3 values); queries too, each row scaled by a power of two so BF16's range
// fits (elements below 2^-38 of their row's largest lose bits).  Scales stay in
// binary32: the key's on the score, the value's on the weight.  The weight w times
// the value's scale s is what is rounded to FP16 for the second product: off by
// 2^-11 at most, against 2^-8 for BF16, or, where w s lies more than 2^20 below the
// largest that the row has seen, by 2^-31 of that largest (raise_row in bg_kvattn.h).
// A row's references follow what it sees itself: taken over all rows of a wave, a
// value that one row sees took the others' weights out of FP16's range (at 2^24 times
// their scale all of it).  They move only when a w s passes them by 2^8, so in the
// steady state a tile needs no lane exchange.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kvattn.h"

namespace bg {
namespace {

constexpr int kWaves = 4;

// One 32-token tile of a wave: codes and records of lane (r = lane % 16,
// g = lane / 16): keys of tokens r and 16 + r, values of its 8 k-slots.
template <int FMT, int D>
struct Tile {
    using L = KvLayout<FMT, D>;
    uint32_t k[2][L::KW];
    uint32_t v[8][L::VW];
    uint32_t ks[8], vs[8];   // records of its k-slots: tokens 4 g .. 4 g + 3 of each 16
    uint32_t kz[2];          // 4-bit: the record of the token whose key this lane holds
    uint32_t there;          // bit s: 16 tokens s lie in a page that exists

    // page: those of the tile's two halves.
    __device__ __forceinline__ void load(const KvAttnArgs& a, const int (&page)[2], int h, int tile, int r, int g) {
        there = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const bool ok = page[s] >= 0 && page[s] < a.c.pages;
            there |= (ok ? 1u : 0u) << s;
            const int in = (tile * 32 + 16 * s) & ((1 << a.c.page_shift) - 1);
            const int64_t run = ok ? (((int64_t)page[s] * a.c.heads + h) << a.c.page_shift) + in : 0;
            const uint8_t* kp = a.c.k + run * L::ROW;
            const uint8_t* vp = a.c.v + run * L::ROW;
#pragma unroll
            for (int c = 0; c < L::KC; ++c)
                load_bytes<L::KB>(kp + (uint32_t)(r * L::ROW + c * 4 * L::KB + g * L::KB), &k[s][c * (L::KB / 4)]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_bytes<L::VB>(vp + (uint32_t)((4 * g + j) * L::ROW + r * L::VB), v[4 * s + j]);
            load_bytes<16>(reinterpret_cast<const uint8_t*>(a.c.ks + run + 4 * g), ks + 4 * s);
            load_bytes<16>(reinterpret_cast<const uint8_t*>(a.c.vs + run + 4 * g), vs + 4 * s);
            if constexpr (FMT == KV_U4) kz[s] = a.c.ks[run + r];
        }
    }
};

// RT row tiles of 16 rows per wave.
template <int FMT, int D, int RT>
__global__ void __launch_bounds__(kWaves * 64, 2) k_kv_attn_few(KvAttnArgs a, KvSplit sp, float* po, float* pl) {
    using L = KvLayout<FMT, D>;
    constexpr int DT = D / 16, ST = D / 32, PAD = D + 4;
    // One tile in flight, not two; there a branch spares the products' 8 multiplications by fb for each
    // 16 rows, 2 to 4 % (48 rows of 64 x 2000 tokens 83 -> 79 us).  With two tiles its code costs more
    // than it spares (8 x 24-token trees in 4 bits, D = 64: 29.2 -> 29.9).
    constexpr bool kOne = RT * D > 128;
    __shared__ float o_lds[kWaves][16][PAD];
    __shared__ float m_lds[kWaves][16], l_lds[kWaves][16];

    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = blockIdx.x % a.c.heads, split = blockIdx.y;
    KvBlock own;
    if (!kv_block(a, blockIdx.x / a.c.heads, 16 * RT, own)) return;
    const KvSeq q = own.q;
    const int G = a.q_heads / a.c.heads, rows = own.rows, r0 = own.r0, b = own.b;
    const int last = (rows < r0 + 16 * RT ? rows : r0 + 16 * RT) - 1;
    const KvRange rg = kv_range<32>(a, q, r0 / G, last / G);
    const int t0 = split * sp.tiles, t1 = split + 1 == sp.splits || t0 + sp.tiles > rg.tiles ? rg.tiles : t0 + sp.tiles;
    const int32_t* table = a.table + b * a.max_pages;

    if (t0 >= t1 && split > 0) {          // nothing left for this split
        for (int i = threadIdx.x; i <= last - r0; i += kWaves * 64) {
            const int row = r0 + i;
            pl[((int64_t)split * a.tokens + q.q0 + row / G) * a.q_heads + h * G + row % G] = -__builtin_inff();
        }
        return;
    }

    // a tile's pages are looked up two tiles before its codes are asked for
    auto find = [&](int (&page)[2], int i) {
        const int base = rg.tile(i < t1 ? i : t1 - 1) * 32;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t p = (base + 16 * s) >> a.c.page_shift;
            page[s] = table[p < a.max_pages ? p : a.max_pages - 1];     // past the table: past the sequence, masked
        }
    };
    int pa[2] = {}, pb[2] = {};
    int i = t0 + wave;
    if (t0 < t1) {
        find(pa, i);
        find(pb, i + kWaves);
    }

    half8_t qf[RT][ST];
    // of each row: weights are over 2^m, weights times value scales over 2^m / fb
    float rq[RT], m[RT], l[RT], fb[RT];
    bool apart = false;                   // some fb is not 1
    int qi[RT];
    float4_t o[RT][DT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const int row = r0 + 16 * x + r;
        const bool ok = row < rows;
        qi[x] = (ok ? row : rows - 1) / G;
        const int64_t at = (q.q0 + qi[x]) * a.q_ts + (h * G + (ok ? row % G : 0)) * a.q_hs;
        rq[x] = load_query<FMT, D>(a, at, g, ok, qf[x]);
        m[x] = kNoRef;
        l[x] = 0.0f;
        fb[x] = 1.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[x][d] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    auto compute = [&](Tile<FMT, D>& t, int tile) {
        const int base = tile * 32;
        const bool whole = rg.whole(base, 32) && t.there == 3u;
        const int first_token = base + 4 * g;   // k-slot j: token first_token + (j & 3) + 16 (j >> 2)
        if (!whole) {
            // what no row sees may hold anything: its weight is 0, and so is its value
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool live = (t.there >> (j >> 2) & 1) && rg.live(first_token + (j & 3) + 16 * (j >> 2));
                t.vs[j] = live ? kv_masked_record<FMT>(t.vs[j]) : 0u;
#pragma unroll
                for (int w = 0; w < L::VW; ++w) t.v[j][w] = live ? t.v[j][w] : 0u;
            }
        }
        // scores
        float4_t s[RT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            half8_t kf[ST];
            key_fragments<FMT, D>(t.k[u], FMT == KV_U4 ? t.kz[u] : 0u, kf);
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                s[x][u] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < ST; ++c) s[x][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[c], qf[x][c], s[x][u], 0, 0, 0);
            }
        }
        half8_t p[RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            // score j is y[j] kr[j]; what the row does not see weighs 0, whatever its scales hold
            float y[8], kr[8], sv[8], pv[8], sum;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = s[x][j >> 2][j & 3];
                kr[j] = kv_scale<FMT>(t.ks[j]) * rq[x];
                sv[j] = kv_scale<FMT>(t.vs[j]);
            }
            if (!whole) {
                uint32_t see = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    see |= (uint32_t)((t.there >> (j >> 2) & 1) && kv_sees(a, q, qi[x], first_token + (j & 3) + 16 * (j >> 2))) << j;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool in = see >> j & 1;
                    y[j] = in ? y[j] : -__builtin_inff();
                    kr[j] = in ? kr[j] : 1.0f;
                    sv[j] = in ? sv[j] : 0.0f;
                }
            }
            for (bool moved = false;; moved = true) {
                float top = 0.0f;
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(y[j], kr[j], -m[x]));
                    pv[j] = kOne ? w * sv[j] : w * (sv[j] * fb[x]);
                    sum += w;
                    if constexpr (!kOne) top = __builtin_fmaxf(top, __builtin_fabsf(pv[j]));
                }
                if constexpr (kOne) {
                    if (apart) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) pv[j] *= fb[x];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(pv[j]));
                }
                if (moved || !__any((top > 0x1p15f) | (sum > kMaxWeight))) break;
                uint32_t zeros = 0;           // bit j: k-slot j's value row may be of zeros
#pragma unroll
                for (int j = 0; j < 8; ++j) zeros |= (uint32_t)kv_maybe_zeros<FMT>(t.vs[j]) << j;
                if (__any(zeros)) {
                    uint32_t some = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t codes = 0;
#pragma unroll
                        for (int w = 0; w < L::VW; ++w) codes |= kv_some<FMT>(t.v[j][w]);
                        some |= (uint32_t)(codes != 0u) << j;
                    }
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) some |= (uint32_t)__shfl_xor((int)some, o, 64);
                    zeros &= ~some;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sv[j] = zeros >> j & 1 ? 0.0f : sv[j];
                }
                float ty = m[x] + __builtin_amdgcn_logf(l[x]), tp = -__builtin_inff();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // rounded, as the reference is: past 2^31 a product's last half step would be a weight of infinity
                    y[j] = rounded_product(y[j], kr[j]);
                    kr[j] = 1.0f;
                    ty = __builtin_fmaxf(ty, y[j]);
                    tp = __builtin_fmaxf(tp, y[j] + scale_log2(sv[j]));
                }
#pragma unroll
                for (int o = 16; o < 64; o <<= 1) {
                    ty = __builtin_fmaxf(ty, __shfl_xor(ty, o, 64));
                    tp = __builtin_fmaxf(tp, __shfl_xor(tp, o, 64));
                }
                const RowStep f = raise_row<7>(m[x], fb[x], ty, tp);
                apart = apart || __any(fb[x] != 1.0f);
                l[x] *= f.l;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[x][d] *= f.o;
            }
            l[x] += sum;
#pragma unroll
            for (int j = 0; j < 8; ++j) p[x][j] = (_Float16)pv[j];
        }
        // O^T += V^T P^T
        uint32_t vz[4];
        if constexpr (FMT == KV_U4) value_zeros(t.vs, vz);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const half8_t vf = value_fragment<FMT, D>(t.v, vz, d);
#pragma unroll
            for (int x = 0; x < RT; ++x) o[x][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[x], o[x][d], 0, 0, 0);
        }
    };

    if constexpr (kOne) {
        // One tile at a time leaves registers for two waves a SIMD, which cover each other's
        // waits: 64 rows of 16 x 8192 tokens (ragged, as below), E4M3, D = 128, 110 us with two
        // tiles and one wave, 184 with two of each (spills), 82 so; 48 rows of 64 x 2000, INT8,
        // 113, 172 and 79; 18 x 2 queries of 4668, 4 bits, D = 256, 55, 44 and 45.
        Tile<FMT, D> t;
        for (; i < t1; i += kWaves) {
            t.load(a, pa, h, rg.tile(i), r, g);
            pa[0] = pb[0];
            pa[1] = pb[1];
            find(pb, i + 2 * kWaves);
            compute(t, rg.tile(i));
        }
    } else {
        Tile<FMT, D> ta, tb;
        if (i < t1) {
            ta.load(a, pa, h, rg.tile(i), r, g);
            find(pa, i + 2 * kWaves);
        }
        for (; i < t1; i += 2 * kWaves) {
            if (i + kWaves < t1) tb.load(a, pb, h, rg.tile(i + kWaves), r, g);
            find(pb, i + 3 * kWaves);
            compute(ta, rg.tile(i));
            if (i + kWaves >= t1) break;
            if (i + 2 * kWaves < t1) ta.load(a, pa, h, rg.tile(i + 2 * kWaves), r, g);
            find(pa, i + 4 * kWaves);
            compute(tb, rg.tile(i + kWaves));
        }
    }

    // join the waves, 16 rows at a time: each wave's result times its share of the sum
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        l[x] += __shfl_xor(l[x], 16, 64);
        l[x] += __shfl_xor(l[x], 32, 64);
        if (x > 0) __syncthreads();
        if (g == 0) {
            m_lds[wave][r] = m[x];
            l_lds[wave][r] = l[x];
        }
        __syncthreads();
        float base = m_lds[0][r], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) base = __builtin_fmaxf(base, m_lds[w][r]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += l_lds[w][r] * __builtin_amdgcn_exp2f(m_lds[w][r] - base);
        const float f = __builtin_amdgcn_exp2f(m[x] - base) / sum, unit = L::UNIT / fb[x];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int d = 0; d < DT; d += 4) {
                float4_t y;
#pragma unroll
                for (int c = 0; c < 4; ++c) y[c] = l[x] == 0.0f ? 0.0f : o[x][d + c][n] * f * unit;
                *reinterpret_cast<float4_t*>(&o_lds[wave][r][(4 * g + n) * DT + d]) = y;
            }
        __syncthreads();
        const int row = r0 + 16 * x + threadIdx.x / 16, part = threadIdx.x % 16;
        if (row < rows) {
            const int rr = threadIdx.x / 16;
            float base = m_lds[0][rr], sum = 0.0f;
#pragma unroll
            for (int w = 1; w < kWaves; ++w) base = __builtin_fmaxf(base, m_lds[w][rr]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) sum += l_lds[w][rr] * __builtin_amdgcn_exp2f(m_lds[w][rr] - base);
            float y[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) y[d] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
#pragma unroll
                for (int d = 0; d < DT; d += 4) {
                    const float4_t z = *reinterpret_cast<const float4_t*>(&o_lds[w][rr][part * DT + d]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) y[d + c] += z[c];
                }
            const int64_t to = (q.q0 + row / G) * a.q_heads + h * G + row % G;
            const float ls = sum == 0.0f ? -__builtin_inff() : base + __builtin_log2f(sum);
            if (sp.splits > 1) {
                float* to_o = po + ((int64_t)split * a.tokens * a.q_heads + to) * D + part * DT;
#pragma unroll
                for (int d = 0; d < DT; d += 4) *reinterpret_cast<float4_t*>(to_o + d) = float4_t{y[d], y[d + 1], y[d + 2], y[d + 3]};
                if (part == 0) pl[(int64_t)split * a.tokens * a.q_heads + to] = ls;
            } else {
                store_out<DT>(a, to * D + part * DT, y);
                if (part == 0 && a.lse) a.lse[to] = ls * 0x1.62e43p-1f;
            }
        }
    }
}

// Joins the splits of a row: o = sum_s 2^(ls_s - max) o_s / sum_s 2^(ls_s - max).
// WPR waves take a row's splits in turn (64 splits one after the other: 18 us), eight
// partials in flight each.  A split without tokens wrote no partial: its weight is 0
// and what lies there is not used.  TURNS: the grid counts on fewer queries than a
// sequence may have, so its rows come in turns.
template <int D, int WPR, bool TURNS>
__global__ void __launch_bounds__(256) k_kv_attn_join(KvAttnArgs a, int splits, const float* po, const float* pl) {
    __shared__ float part[WPR == 1 ? 1 : 4][D];
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.y;
    const KvSeq q = kv_seq(a, b);
    const int64_t n = a.tokens * a.q_heads, rows = (int64_t)kv_rows(a, q) * a.c.heads, first_row = (int64_t)blockIdx.x * (4 / WPR) + wave / WPR;
    int64_t row = first_row;
    if (row >= rows) return;
    do {
        const int64_t to = q.q0 * a.q_heads + row;
        auto load = [&](int s) { return s < splits ? pl[s * n + to] : -__builtin_inff(); };
        const float first = load(lane);
        float top = first;
        for (int s = lane + 64; s < splits; s += 64) top = __builtin_fmaxf(top, load(s));
        top = wave_max<64>(top);
        const float base = top == -__builtin_inff() ? 0.0f : top;
        float y[E] = {}, sum = __builtin_amdgcn_exp2f(first - base);
        for (int s = lane + 64; s < splits; s += 64) sum += __builtin_amdgcn_exp2f(load(s) - base);
        sum = wave_sum<64>(sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int s0 = 0; s0 < splits; s0 += 64) {
            const float w = __builtin_amdgcn_exp2f((s0 == 0 ? first : load(s0 + lane)) - base) * inv;
            const int last = splits - s0 < 64 ? splits - s0 : 64;
            for (int s = wave % WPR; s < last; s += 8 * WPR) {
                float p[8][E], ws[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int sx = s + x * WPR < last ? s + x * WPR : s;
                    ws[x] = s + x * WPR < last ? __shfl(w, sx, 64) : 0.0f;
                    const float* at = po + ((int64_t)(s0 + sx) * n + to) * D + lane * E;
#pragma unroll
                    for (int d = 0; d < E; ++d) p[x][d] = at[d];
                }
#pragma unroll
                for (int x = 0; x < 8; ++x)
#pragma unroll
                    for (int d = 0; d < E; ++d) y[d] += ws[x] == 0.0f ? 0.0f : ws[x] * p[x][d];
            }
        }
        if constexpr (WPR > 1) {
            // WPR = 4: the block's waves share the row and its turns
            if (TURNS && row > first_row) __syncthreads();
#pragma unroll
            for (int d = 0; d < E; ++d) part[wave][lane * E + d] = y[d];
            __syncthreads();
            if (wave > 0) continue;
#pragma unroll
            for (int w = 1; w < 4; ++w)
#pragma unroll
                for (int d = 0; d < E; ++d) y[d] += part[w][lane * E + d];
        }
        store_out<E>(a, to * D + lane * E, y);
        if (a.lse && lane == 0) a.lse[to] = sum == 0.0f ? -__builtin_inff() : (base + __builtin_log2f(sum)) * 0x1.62e43p-1f;
    } while (TURNS && (row += (int64_t)gridDim.x * (4 / WPR)) < rows);
}

// The kernel, rows of a block, and how positions are split over blocks.
struct Plan {
    int waves;                            // of a block of the many-row kernel; 0: the few-row kernel
    int rt;
    unsigned row_blocks;
    int64_t chunk;                        // KvAttnArgs::chunk
    KvSplit sp;
    double us;
};

// Queries a sequence is taken to have: the bound, or where that is all of the call's and so
// says nothing of one sequence, their mean; further ones are found by the blocks past
// the batch (kv_block).  With a grid for the bound itself, a decode step of 32 x 8192
// tokens that gave none took 237 us (81 with one), and 64 x 2000 206 (37).
int64_t usual_q(const KvAttnArgs& a) { return a.batch > 1 && a.max_q == a.tokens ? (a.tokens + a.batch - 1) / a.batch : a.max_q; }

// The plan with one of the kernels that takes the least time by this model: rounds of the
// blocks that the device holds at once, each a start and its tiles; the join; and the
// partials' way to memory and back at 4 TB/s.  Many rows: one block a CU (two of four
// waves at D = 64), a start worth 3 tiles.  Few: two blocks a CU, each wave a quarter of the tiles, a start worth 2 of its.
// As many splits as fill the device, for which this stands, ran 136 blocks of 16 tiles as
// two rounds of 8 tiles in 94 us (one of 16: 58), and 35 sequences of 11687 tokens,
// D = 256, in 64 (47).
Plan plan_with(const KvAttnArgs& a, int waves) {
    Plan p;
    const int64_t G = a.q_heads / a.c.heads, usual = usual_q(a), rows = usual * G;
    const bool many = waves > 0, wide = a.c.dim == 256, narrow = a.c.dim == 64;
    p.waves = waves;
    p.rt = rows <= 16 || wide ? 1 : 2;
    const int per_block = many ? 32 * waves : 16 * p.rt, tile = many ? 64 : 32;
    p.chunk = 0;
    if (usual < a.max_q && a.batch < kGridZ) {
        // a block's queries at least, and as many as keep the blocks past the batch within the grid
        const int64_t least = (a.tokens + kGridZ - a.batch - 1) / (kGridZ - a.batch);
        p.chunk = usual > per_block / G ? usual : per_block / G;
        p.chunk = p.chunk > least ? p.chunk : least;
        if (p.chunk >= a.max_q) p.chunk = 0;
    }
    p.row_blocks = (unsigned)(((p.chunk ? p.chunk : a.max_q) * G + per_block - 1) / per_block);
    // positions a row block can see, in tiles
    int64_t seen = a.max_kv;
    if (a.window) {
        const int64_t most = a.window + (p.chunk ? p.chunk : a.max_q) + 64 + (a.sinks ? a.sinks + 64 : 0);
        seen = most < seen ? most : seen;
    }
    const int64_t tiles = (seen + tile - 1) / tile > 0 ? (seen + tile - 1) / tile : 1;
    const int64_t blocks = a.batch * a.c.heads * ((rows + per_block - 1) / per_block), room = many && (waves == 8 || wide) ? 256 : 512;
    const double tile_us = many ? (wide ? 3.5 : !narrow ? 2.1 : waves == 8 ? 1.65 : 1.85) : (wide ? 3.0 : 2.1);      // measured, device full
    const double partials = (double)(a.tokens * a.q_heads * a.c.dim) * 8.0 / 4.0e6;
    int64_t splits = 1;
    p.us = 1e30;
    for (int64_t s = 1; s <= 256 && s <= tiles; ++s) {
        const int64_t run = (tiles + s - 1) / s, rounds = (blocks * s + room - 1) / room;
        const double us = (double)(rounds * (many ? 3 + run : 2 + (run + 3) / 4)) * tile_us + (s == 1 ? 0.0 : (many ? 4.0 : 3.0) + (double)s * (partials + 0.03));
        if (us < p.us) {
            p.us = us;
            splits = s;
        }
        if (blocks * s > 4 * room) break;
    }
    p.sp.tiles = (int)((tiles + splits - 1) / splits);
    p.sp.splits = (int)((tiles + p.sp.tiles - 1) / p.sp.tiles);
    return p;
}

// Up to 32 rows (16 at D = 256: one block's) the few-row kernel reads each code once; from
// there on by the model.  16 x 8192 tokens, E4M3, D = 128: 96 rows 104 us with few, 119 with
// many; 192 rows 151 and 146; 65536 tokens in 4 bits, 192 rows: 116 and 94; 1000 tokens,
// INT8, 192 rows: 19 and 27; 4 x 8192, INT8, D = 256, 128 rows: 98 and 75.  D = 64, blocks of
// eight waves and of four: 112 rows of 12 x 26287 tokens in 4 bits 238 and 189 us, 800 of
// 9 x 6000, E4M3, 69 and 62; 256 of 16 x 8192 122 and 136, 8192 of 2 x 4096 190 and 202.
Plan plan_of(const KvAttnArgs& a) {
    Plan best = plan_with(a, 0);
    if (usual_q(a) * (a.q_heads / a.c.heads) <= (a.c.dim == 256 ? 16 : 32)) return best;
    for (int waves : {8, 4}) {
        if (a.c.dim != 64 && waves != (a.c.dim == 256 ? 4 : 8)) continue;
        const Plan p = plan_with(a, waves);
        if (p.us < best.us) best = p;
    }
    return best;
}

}  // namespace

int64_t kv_attn_workspace(const KvAttnArgs& a) {
    const Plan p = plan_of(a);
    return p.sp.splits > 1 ? (int64_t)p.sp.splits * a.tokens * a.q_heads * (a.c.dim + 1) * 4 : 0;
}

const char* launch_kv_attn(const KvAttnArgs& given, void* ws, hipStream_t s) {
    const Plan p = plan_of(given);
    KvAttnArgs a = given;
    a.chunk = p.chunk;
    float* po = static_cast<float*>(ws);
    float* pl = po + (int64_t)p.sp.splits * a.tokens * a.q_heads * a.c.dim;
    const dim3 grid((unsigned)a.c.heads * p.row_blocks, (unsigned)p.sp.splits, kv_grid_z(a));
    const char* name = nullptr;
    if (p.waves) name = launch_kv_attn_many(a, p.sp, p.row_blocks, p.waves, po, pl, s);
    else for_format(a.c.fmt, a.c.dim, [&](auto FMT, auto D) {
        if (p.rt == 1) k_kv_attn_few<FMT(), D(), 1><<<grid, kWaves * 64, 0, s>>>(a, p.sp, po, pl);
        else if constexpr (D() != 256) k_kv_attn_few<FMT(), D(), 2><<<grid, kWaves * 64, 0, s>>>(a, p.sp, po, pl);
    });
    if (p.sp.splits > 1) {
        const bool wide = p.sp.splits > 8;
        const int64_t rows = (p.chunk ? p.chunk : a.max_q) * a.q_heads;
        const dim3 join((unsigned)(wide ? rows : (rows + 3) / 4), (unsigned)a.batch);
        auto go = [&](auto D) {
            auto with = [&](auto TURNS) {
                if (wide) k_kv_attn_join<D(), 4, TURNS()><<<join, 256, 0, s>>>(a, p.sp.splits, po, pl);
                else k_kv_attn_join<D(), 1, TURNS()><<<join, 256, 0, s>>>(a, p.sp.splits, po, pl);
            };
            if (p.chunk) with(std::true_type{});
            else with(std::false_type{});
        };
        if (a.c.dim == 64) go(std::integral_constant<int, 64>{});
        else if (a.c.dim == 128) go(std::integral_constant<int, 128>{});
        else go(std::integral_constant<int, 256>{});
    }
    return name ? name : kname("k_kv_attn_few", a.c.fmt, a.c.dim, p.rt);
}

}  // namespace bg
