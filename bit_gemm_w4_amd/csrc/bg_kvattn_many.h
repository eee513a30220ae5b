// bg_kvattn_many.h -- the kernel body of k_kvattn_many.hip and k_kvattn_many_*.hip.
#pragma once
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kvattn.h"

namespace bg {
namespace {

constexpr int kT = 64, kRows = 32;          // positions of a tile, rows of a wave

// A lane's part of a key row (KB bytes) and of a value row (VB bytes, E elements; LR lanes).
template <int FMT, int D>
struct ManyLayout {
    static constexpr int ROW = KvLayout<FMT, D>::ROW, PER = KvLayout<FMT, D>::PER;
    static constexpr int KB = ROW / 8, KW = KB / 4, KF = D / 64;               // bytes, words, fragments
    static constexpr int VB = ROW >= 64 ? ROW / 64 : 1, E = VB * PER, LR = D / E;
};

template <int FMT, int D>
struct ManyLds {
    static constexpr int KRING = D == 256 ? 4 : 8, VRING = D == 256 ? 5 : 8;       // of 5 and 6 needed at D <= 128, 8 cost no division
    half8_t k[KRING][D / 8][32];      // [step mod KRING][8 elements][token]
    half8_t v[VRING][2][2][D];        // [step mod VRING][16 tokens][lane half][element e of lane r at e LR + r]
    float ks[4][kT], vs[4][kT];       // [tile mod 4]: key scales times the queries' unit, value scales
    float lv[4][kT];                  // log2 of the value scales' magnitude
    float most[4];                    // [tile mod 4]: sums of weights up to this stay in FP16's range with the tile's value scales
    uint32_t top[8];
    uint16_t vz[4][kT];               // 4 bits: -2^-9 times the zero-points of values, FP16
};

// Where a sequence's tokens of one head lie.
struct ManyPages {
    const int32_t* table;
    int last, shift;           // last entry of the table
    uint32_t pages, rows, row; // pages of the cache, rows of a page, first row of the head in it

    __device__ __forceinline__ ManyPages(const KvAttnArgs& a, int b, int h)
        : table(a.table + b * a.max_pages), last((int)a.max_pages - 1), shift(a.c.page_shift), pages((uint32_t)a.c.pages),
          rows((uint32_t)a.c.heads << a.c.page_shift), row((uint32_t)h << a.c.page_shift) {}
    // Positions past the table are past every sequence: what is read for them is masked.
    __device__ __forceinline__ uint32_t page(int position) const {
        const int p = position >> shift;
        return (uint32_t)table[p < last ? p : last];
    }
    __device__ __forceinline__ bool there(uint32_t page) const { return page < pages; }
    // Offset in an array of `unit` bytes per token and head (in page 0 if the page does not exist); a page's bytes fit 32 bits.
    __device__ __forceinline__ uint64_t at(uint32_t page, int position, uint32_t unit) const {
        return (uint64_t)(there(page) ? page : 0u) * (rows * unit) + (row + (uint32_t)(position & ((1 << shift) - 1))) * unit;
    }
};

// Bit j: the row sees position base + j.
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

template <bool SCORED>
__device__ __forceinline__ uint64_t seen_bits(const KvAttnArgs& a, const KvSeq& q, int i, int base, uint64_t there) {
    uint64_t m;
    if (a.tree) {
        m = low_bits(q.first - base);
        const int e = base - q.first;            // bit 0's drafted token
        const uint64_t* w = a.tree + (q.q0 + i) * a.tree_words;
        const int n = e >> 6, sh = e & 63;
        // The index in a vector register: as a scalar it became part of 16 words of arguments, which were spilled and
        // brought back as one, 50 lane moves in each masked tile (16 trees of 64, 4 bits: 161 us, 156 so).
        int at = n;
        asm("" : "+v"(at));
        uint64_t bits = n >= 0 && n < a.tree_words ? w[at] >> sh : 0;
        if (sh && n + 1 >= 0 && n + 1 < a.tree_words) bits |= w[at + 1] << (64 - sh);
        m |= bits & ~low_bits(-e);
        m &= low_bits(q.kv - base);
    } else {
        const int at = q.first + i;
        m = low_bits(at + 1 - base);
        if constexpr (SCORED) m |= low_bits(q.prefix - base);
        if (a.window) m &= ~low_bits(at - base - (int)a.window + 1) | low_bits((int)a.sinks - base);
    }
    return m & there;
}

// Scores are capped (CAP; FAR: see cap_scores), biased by their distance (BIAS; slopes may be NULL), or see a
// prefix (either).
template <int FMT, int D, int WAVES, bool CAP, bool BIAS, bool FAR>
__device__ __forceinline__ void attend_many(const KvAttnArgs& a, const KvSplit& sp, float* po, float* pl) {
    using L = KvLayout<FMT, D>;
    using M = ManyLayout<FMT, D>;
    constexpr int DT = D / 32, ST = D / 16, PARTS = 8 / WAVES;
    constexpr bool SCORED = CAP || BIAS, NEAR = CAP && !FAR;
    __shared__ ManyLds<FMT, D> lds;

    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = blockIdx.x % a.c.heads, split = blockIdx.y;
    KvBlock own_rows;
    if (!kv_block<SCORED>(a, gridDim.x / a.c.heads - 1 - blockIdx.x / a.c.heads, WAVES * kRows, own_rows)) return;     // the longest first
    const KvSeq q = own_rows.q;
    const int G = a.q_heads / a.c.heads, rows = own_rows.rows, r0 = own_rows.r0, b = own_rows.b;
    const int last = (rows < r0 + WAVES * kRows ? rows : r0 + WAVES * kRows) - 1;
    const KvRange rg = kv_range<kT, SCORED>(a, q, r0 / G, last / G);
    int t0, t1;
    kv_run<SCORED>(a, sp, rg, split, t0, t1);
    const int nt = t1 - t0;               // tiles of this block: number i is tile t0 + i of the range
    if (nt <= 0 && split > 0) {          // nothing left for this split
        for (int i = threadIdx.x; i <= last - r0; i += WAVES * 64) {
            const int row = r0 + i;
            pl[((int64_t)split * a.tokens + q.q0 + row / G) * a.q_heads + h * G + row % G] = -__builtin_inff();
        }
        return;
    }

    const int w0 = r0 + wave * kRows;     // the wave's first row
    const bool has_rows = w0 < rows;
    const int wlast = rows < w0 + kRows ? rows - 1 : w0 + kRows - 1;
    const KvRange wr = kv_range<kT, SCORED>(a, q, (has_rows ? w0 : rows - 1) / G, wlast / G);
    const int row = w0 + r;
    const bool ok = row < rows;
    const int qi = (ok ? row : rows - 1) / G;

    half8_t qf[ST];
    float unit_s = 0.0f;
    float16_t o[DT], s[2];
    // of the lane's row: its sum, weights over 2^m, weights times value scales over 2^m / fb;
    // own: what its scores lack (scale_queries); apart: some row of the wave has an fb or own other than 1
    float m = kNoRef, fb = 1.0f, l = 0.0f, own = 1.0f;
    bool apart = false;
    float slope = 0.0f;                    // of the row's head, over `unit`
    if constexpr (BIAS) slope = a.slopes ? head_slope(a, h * G + (ok ? row - qi * G : 0)) * (NEAR ? 0.5f : -1.0f) : 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = float16_t{} ;

    // Step n is tokens 32 (n % 2) of the block's tile n / 2.  At step n the matrix cores take the
    // scores of step n + 1 and the values of step n - 1 in turn, and the vector units the
    // weights of step n.  A fragment's register (keys: elements 16 c of 32 tokens;
    // values: elements 32 d of 16 tokens t at t DT + d) takes the one FK (FV) further on
    // as soon as its product is issued.
    constexpr int FK = D == 256 ? ST : FAR && D == 128 ? 2 : 4, FV = SCORED && D == 128 ? 2 : 4;
    half8_t fk[FK], fv[FV], p[2][2];
    float4_t kr, vr;                                   // scales of the 4 tokens that come next
    auto key = [&](int n, int c) { return lds.k[(uint32_t)(n + 40) % lds.KRING][2 * c + g][r]; };
    auto value = [&](int n, int j) { return lds.v[(uint32_t)(n + 40) % lds.VRING][j / DT][g][32 * (j % DT) + r]; };
    auto k_scale = [&](int n, int x) { return *reinterpret_cast<const float4_t*>(&lds.ks[n >> 1 & 3][32 * (n & 1) + 8 * x + 4 * g]); };
    auto v_scale = [&](int n, int x) { return *reinterpret_cast<const float4_t*>(&lds.vs[n >> 1 & 3][32 * (n & 1) + 8 * x + 4 * g]); };
    // The scores of an even step n, with the fragments that follow; step n - 1 weighs nothing.
    auto start = [&](int n) {
        half8_t f[ST];
#pragma unroll
        for (int c = 0; c < ST; ++c) f[c] = key(n, c);
        s[0] = float16_t{};
#pragma unroll
        for (int c = 0; c < ST; ++c) s[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[c], qf[c], s[0], 0, 0, 0);
#pragma unroll
        for (int c = 0; c < FK; ++c) fk[c] = key(n + 1, c);
#pragma unroll
        for (int j = 0; j < FV; ++j) fv[j] = half8_t{};
        p[1][0] = p[1][1] = half8_t{};
        kr = k_scale(n, 0);
        vr = v_scale(n, 0);
    };
    // The values of an odd step, of which FV fragments are here.
    auto finish = [&](int n) {
#pragma unroll
        for (int j = 0; j < ST; ++j)
            o[j % DT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(j < FV ? fv[j % FV] : value(n, j), p[1][j / DT], o[j % DT], 0, 0, 0);
        p[1][0] = p[1][1] = half8_t{};
    };
    auto attend = [&](int i, auto U, bool whole, uint64_t seen, float most, int base, auto&& beside) {
        constexpr int u = U();
        const int n = 2 * i + u;
        float sum = 0.0f;
        s[1 - u] = float16_t{};
        auto products = [&](int c) {
            s[1 - u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fk[c % FK], qf[c], s[1 - u], 0, 0, 0);
            fk[c % FK] = c + FK < ST ? key(n + 1, c + FK) : key(n + 2, c + FK - ST);
            o[c % DT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fv[c % FV], p[1 - u][c / DT], o[c % DT], 0, 0, 0);
            fv[c % FV] = c + FV < ST ? value(n - 1, c + FV) : value(n, c + FV - ST);
        };
        // A product times its token's scale, t, to what unit t + zero is the score of (see cap_scores and head_slope).
        // Near caps: t = 1 / (1 + 2^t) and the score cap - 2 cap t, which spares an instruction.
        const float unit = NEAR ? -2.0f * a.cap : a.cap, zero = NEAR ? a.cap : 0.0f, from = zero - m;
        float top = 0.0f;                  // FAR: the largest t that the first pass takes for a small one
        auto scores = [&](auto AGAIN, int x, float (&t)[4]) {
            if constexpr (NEAR) {
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t[j]));
            } else if constexpr (CAP && AGAIN()) {
                cap_scores<true>(t);
            } else if constexpr (CAP) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    top = __builtin_fmaxf(top, __builtin_fabsf(t[j]));
                    t[j] *= tanh_ratio_small(t[j] * t[j]);
                }
            }
            if constexpr (BIAS) {
                const float away = (float)(q.first + qi - base - 32 * u - 4 * g);
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = __builtin_fmaf(__builtin_fabsf(away - (float)(8 * x + j)), slope, t[j]);
            }
        };
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float4_t kn = kr, vn = vr;
            if (x < 3) {
                kr = k_scale(n, x + 1);
                vr = v_scale(n, x + 1);
            }
#pragma unroll
            for (int c = x * ST / 4; c < (x + 1) * ST / 4; ++c) products(c);
            beside(x);
            if constexpr (SCORED) {
                float t[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = rounded_product(s[u][4 * x + j], kn[j]);
                scores(std::false_type{}, x, t);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(t[j], unit, from));
                    sum += w;
                    p[u][x >> 1][4 * (x & 1) + j] = (_Float16)(w * vn[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][4 * x + j], kn[j], -m));
                    sum += w;
                    p[u][x >> 1][4 * (x & 1) + j] = (_Float16)(w * vn[j]);
                }
            }
            if (x < 3) __builtin_amdgcn_sched_barrier(0);
        }
        bool again = (uint32_t)!whole | (uint32_t)apart;
        if constexpr (FAR) again |= __any(top > kTanhSmall);
#pragma unroll
        for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(p[u][j]));
        if (__ballot(!(sum <= most)) != 0 && !again) {
            // some product may have left FP16's range
            const half8_t top = __builtin_elementwise_max(__builtin_elementwise_abs(p[u][0]), __builtin_elementwise_abs(p[u][1]));
            bool left = sum > kMaxWeight;
#pragma unroll
            for (int j = 0; j < 8; ++j) left |= top[j] == (_Float16)__builtin_inff();
            again = __any(left);
        }
        kr = k_scale(n + 1, 0);
        vr = v_scale(n + 1, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (again) {
            const uint32_t see = (uint32_t)(seen >> (32 * u + 4 * g));     // bit 8 (j / 4) + j % 4: the row sees k-slot j
            auto in = [&](int x, int j) { return see >> (8 * x + j) & 1; };
            float ty = -__builtin_inff(), tp = -__builtin_inff();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4_t kn = k_scale(n, x), lv = *reinterpret_cast<const float4_t*>(&lds.lv[n >> 1 & 3][32 * (n & 1) + 8 * x + 4 * g]);
                // scores are rounded, as the reference is: past 2^31 a product's last half step would be a weight of infinity
                float t[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = rounded_product(s[u][4 * x + j], kn[j] * own);
                if constexpr (SCORED) {
                    scores(std::true_type{}, x, t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[u][4 * x + j] = t[j] = __builtin_fmaf(t[j], unit, zero);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ty = in(x, j) ? __builtin_fmaxf(ty, t[j]) : ty;
                    tp = in(x, j) ? __builtin_fmaxf(tp, t[j] + lv[j]) : tp;
                }
            }
            ty = __builtin_fmaxf(ty, m + __builtin_amdgcn_logf(l));
            ty = __builtin_fmaxf(ty, __shfl_xor(ty, 32, 64));
            tp = __builtin_fmaxf(tp, __shfl_xor(tp, 32, 64));
            const RowStep f = raise_row<4>(m, fb, ty, tp);
            apart = __any((fb != 1.0f) | (own != 1.0f));
            l *= f.l;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f.o;
            sum = 0.0f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4_t kn = k_scale(n, x), vn = v_scale(n, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float y = SCORED ? s[u][4 * x + j] : rounded_product(s[u][4 * x + j], kn[j] * own);
                    // what the row does not see weighs 0, whatever its scales hold
                    const float w = in(x, j) ? __builtin_amdgcn_exp2f(y - m) : 0.0f;
                    sum += w;
                    p[u][x >> 1][4 * (x & 1) + j] = (_Float16)(in(x, j) ? w * (vn[j] * fb) : 0.0f);
                }
            }
        }
        l += sum;
    };

    // Each wave carries an eighth of a tile from memory to LDS: part w is the keys of
    // tokens 8 w .. 8 w + 7, and the values of k-slots (16 tokens w / 2, half w % 2).  Keys
    // go two tiles ahead, values one; each is asked for a tile before it is stored.
    const ManyPages pages(a, b, h);
    uint32_t kc[PARTS][M::KW], kz[PARTS], vc[PARTS][8][M::VB < 4 ? 1 : M::VB / 4];
    // Past the last tile the last one is carried again, into parts that nothing reads.
    auto base_of = [&](int i) {
        const int n = i < nt ? i : nt - 1;
        return rg.tile(BIAS && a.slopes ? t1 - 1 - n : t0 + n) * kT;
    };
    auto part = [&](int x) { return wave * PARTS + x; };
    auto find = [&](int base) { return pages.page(base + lane); };                 // token `lane`'s page
    // Bit n: token n lies in a page that exists and some row of the block sees it.
    auto live_of = [&](int base, uint32_t page) -> uint64_t { return __ballot(pages.there(page) & rg.live(base + lane)); };
    auto load_keys = [&](auto& c, auto& z, int base, uint32_t page) {
#pragma unroll
        for (int x = 0; x < PARTS; ++x) {
            const int first = base + 8 * part(x) + (lane & 7);
            const uint32_t own = __builtin_amdgcn_readlane(page, 8 * part(x));
            load_bytes<M::KB>(a.c.k + (pages.at(own, first, L::ROW) + (uint32_t)((lane >> 3) * M::KB)), c[x]);
            if constexpr (FMT == KV_U4) load_bytes<4>(reinterpret_cast<const uint8_t*>(a.c.ks) + pages.at(own, first, 4), &z[x]);
        }
    };
    auto store_keys = [&](const auto& c, const auto& z, int i) {
#pragma unroll
        for (int x = 0; x < PARTS; ++x) {
            auto& t = lds.k[(uint32_t)(2 * i + (part(x) >> 2) + 40) % lds.KRING];
            const half2_t mz = FMT == KV_U4 ? minus_zero(z[x]) : half2_t{(_Float16)0.0f, (_Float16)0.0f};
#pragma unroll
            for (int f = 0; f < M::KF; ++f)
                t[(lane >> 3) * M::KF + f][8 * (part(x) & 3) + (lane & 7)] = codes8<FMT>(c[x] + f * (FMT == KV_U4 ? 1 : 2), mz);
        }
    };
    auto load_values = [&](auto& c, int base, uint32_t page) {
#pragma unroll
        for (int x = 0; x < PARTS; ++x) {
            const int first = base + 16 * (part(x) >> 1) + 4 * (part(x) & 1);
            const uint32_t own = __builtin_amdgcn_readlane(page, 16 * (part(x) >> 1));
            const uint8_t* vp = a.c.v + (pages.at(own, first, L::ROW) + (uint32_t)((M::LR < 64 ? lane & (M::LR - 1) : lane) * M::VB));
#pragma unroll
            for (int j = 0; j < 8; ++j) load_bytes<M::VB>(vp + ((j & 3) + 8 * (j >> 2)) * L::ROW, c[x][j]);
        }
    };
    // What no row sees may hold anything: its value becomes 0.
    auto store_values = [&](const auto& c, int i, uint64_t live) {
#pragma unroll
        for (int x = 0; x < PARTS; ++x) {
            auto& t = lds.v[(uint32_t)(2 * i + (part(x) >> 2) + 40) % lds.VRING][part(x) >> 1 & 1][part(x) & 1];
            const int first = 16 * (part(x) >> 1) + 4 * (part(x) & 1);
            const uint32_t own = (uint32_t)(live >> first);
            uint32_t v[8][M::VB < 4 ? 1 : M::VB / 4], z[4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t keep = 0u - (own >> ((j & 3) + 8 * (j >> 2)) & 1u);
#pragma unroll
                for (int n = 0; n < (M::VB < 4 ? 1 : M::VB / 4); ++n) v[j][n] = c[x][j][n] & keep;
            }
            if constexpr (FMT == KV_U4) {
                const uint2 lo = *reinterpret_cast<const uint2*>(&lds.vz[i & 3][first]), hi = *reinterpret_cast<const uint2*>(&lds.vz[i & 3][first + 8]);
                z[0] = lo.x; z[1] = lo.y; z[2] = hi.x; z[3] = hi.y;
            }
#pragma unroll
            for (int e = 0; e < M::E; ++e) {
                const half8_t y = value_fragment<FMT, D>(v, z, e);
                if (M::LR == 64 || lane < M::LR) t[e * M::LR + lane] = y;
            }
        }
    };
    // Wave 0: the records of token `lane`, with the keys.
    uint32_t k_rec = 0, v_rec = 0;
    float top_v = 0.0f, most_v = 0.0f;                 // a power of two above the tile's value scales, 2^15 over it
    auto load_records = [&](uint32_t& kr, uint32_t& vr, int base, uint32_t page) {
        const uint64_t at = pages.at(page, base + lane, 4);
        load_bytes<4>(reinterpret_cast<const uint8_t*>(a.c.ks) + at, &kr);
        load_bytes<4>(reinterpret_cast<const uint8_t*>(a.c.vs) + at, &vr);
    };
    auto store_records = [&](uint32_t kr, uint32_t vr, int i, uint64_t live, int base, uint32_t page) {
        vr = live >> lane & 1 ? kv_masked_record<FMT>(vr) : 0u;
        if (__any(kv_maybe_zeros<FMT>(vr))) {
            const uint8_t* row = a.c.v + pages.at(page, base + lane, L::ROW);
            uint32_t some = 0;
            for (int n = 0; n < L::ROW; n += 16) {
                uint32_t w[4];
                load_bytes<16>(row + n, w);
                some |= kv_some<FMT>(w[0] | w[1] | w[2] | w[3]);
            }
            if (kv_maybe_zeros<FMT>(vr) && some == 0u) vr = 0u;
        }
        const float sv = kv_scale<FMT>(vr), size = __builtin_fabsf(sv);
        if (__any(size >= top_v) || !__any(size >= top_v * 0x1p-3f)) {
            const uint32_t e = __builtin_amdgcn_readfirstlane(__float_as_uint(wave_max<64>(size))) >> 23;
            top_v = __uint_as_float((e < 254u ? e + 1u : 255u) << 23);
            most_v = __builtin_fminf(0x1p15f / top_v, kMaxWeight);
        }
        lds.ks[i & 3][lane] = kv_scale<FMT>(kr) * unit_s;
        lds.vs[i & 3][lane] = sv;
        lds.lv[i & 3][lane] = scale_log2(sv);
        lds.most[i & 3] = most_v;
        if constexpr (FMT == KV_U4) lds.vz[i & 3][lane] = __builtin_bit_cast(uint16_t, (_Float16)(__builtin_bit_cast(_Float16, (uint16_t)(vr >> 16)) * (_Float16)-0x1p-9f));
    };

    // Of tiles i to i + 3: first position, pages (from i + 2) and live tokens (to i + 2).
    int b0 = base_of(0), b1 = base_of(1), b2 = base_of(2), b3 = base_of(3);
    uint32_t pg2 = 0, pg3 = 0;
    uint64_t th0 = 0, th1 = 0, th2 = 0;
    {
        // the first tiles' pages, codes and queries are all asked for before any is waited for
        uint32_t k0[PARTS][M::KW], k1[PARTS][M::KW], z0[PARTS], z1[PARTS], v0[PARTS][8][M::VB < 4 ? 1 : M::VB / 4], r0k = 0, r0v = 0, r1k = 0, r1v = 0;
        const uint32_t p0 = nt > 0 ? find(b0) : 0, p1 = nt > 0 ? find(b1) : 0;
        if (nt > 0) pg2 = find(b2);
        load_queries<D>(a, (q.q0 + qi) * a.q_ts + (h * G + (ok ? row - qi * G : 0)) * a.q_hs, g, ok, qf);
        if (nt > 0) {
            load_keys(k0, z0, b0, p0);
            load_values(v0, b0, p0);
            load_keys(k1, z1, b1, p1);
            load_values(vc, b1, p1);
            load_keys(kc, kz, b2, pg2);
            if (wave == 0) {
                load_records(r0k, r0v, b0, p0);
                load_records(r1k, r1v, b1, p1);
                load_records(k_rec, v_rec, b2, pg2);
            }
            th0 = live_of(b0, p0);
            th1 = live_of(b1, p1);
            th2 = live_of(b2, pg2);
            pg3 = find(b3);
        }
        // the step before the first: no weight, but products with its values are taken
        half8_t* before = &lds.v[39 % lds.VRING][0][0][0];
        for (int x = threadIdx.x; x < 4 * D; x += WAVES * 64) before[x] = half8_t{};
        unit_s = scale_queries<FMT, D, WAVES>(a, wave, lds.top, qf, own);
        if constexpr (CAP) unit_s *= cap_unit(a);
        apart = __any(own != 1.0f);
        if (nt > 0) {
            if (wave == 0) {
                store_records(r0k, r0v, 0, th0, b0, p0);
                store_records(r1k, r1v, 1, th1, b1, p1);
            }
            store_keys(k0, z0, 0);
            store_keys(k1, z1, 1);
            if constexpr (FMT == KV_U4) __syncthreads();         // its values' zero-points come from the records
            store_values(v0, 0, th0);
        }
    }
    __syncthreads();
    start(0);
    float most = lds.most[0];
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
        // Into what the last tile left, beside the products: keys and records of tile i + 2,
        // values of tile i + 1.
        auto carry_keys = [&](int x) {
            if (x == 0) store_keys(kc, kz, i + 2);
            if (x == 1) load_keys(kc, kz, b3, pg3);
        };
        auto carry_values = [&](int x) {
            if (x == 0) store_values(vc, i + 1, th1);
            if (x == 2) load_values(vc, b2, pg2);
        };
        if (wave == 0) {
            store_records(k_rec, v_rec, i + 2, th2, b2, pg2);
            load_records(k_rec, v_rec, b3, pg3);
        }
        const uint64_t th3 = live_of(b3, pg3);
        // a tile that none of the wave's rows sees takes part with no weight
        const int base = b0;
        const bool whole = (th0 == ~0ull) & wr.whole(base, kT);
        uint64_t seen = ~0ull;
        const float next = lds.most[(i + 1) & 3];
        if (!whole) seen = seen_bits<SCORED>(a, q, qi, base, th0);
        if (has_rows) {
            attend(i, std::integral_constant<int, 0>{}, whole, seen, most, base, carry_keys);
            attend(i, std::integral_constant<int, 1>{}, whole, seen, most, base, carry_values);
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) carry_keys(x);
#pragma unroll
            for (int x = 0; x < 4; ++x) carry_values(x);
        }
        most = next;
        b0 = b1;
        b1 = b2;
        b2 = b3;
        b3 = base_of(i + 4);
        pg2 = pg3;
        pg3 = find(b3);
        th0 = th1;
        th1 = th2;
        th2 = th3;
        __syncthreads();
    }

    if (has_rows) finish(2 * nt - 1);
    l += __shfl_xor(l, 32, 64);
    if (!ok) return;
    const int64_t to = (q.q0 + qi) * a.q_heads + h * G + row - qi * G;      // here, and not two registers through the loop
    const float inv = 1.0f / l, unit = L::UNIT / fb;
    const float ls = l == 0.0f ? -__builtin_inff() : __builtin_log2f(l) + m;
    constexpr int HB = M::LR / 32, RUN = 4 * M::E;          // accumulator row m of O[e HB + x] is element e of lane 32 x + m
#pragma unroll
    for (int x = 0; x < HB; ++x)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float y[RUN];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < M::E; ++e) y[j * M::E + e] = l == 0.0f ? 0.0f : o[e * HB + x][4 * n + j] * inv * unit;
            const int64_t d = to * D + (32 * x + 8 * n + 4 * g) * M::E;
            if (sp.splits > 1) {
                float* p = po + (int64_t)split * a.tokens * a.q_heads * D + d;
#pragma unroll
                for (int e = 0; e < RUN; e += 4) *reinterpret_cast<float4_t*>(p + e) = float4_t{y[e], y[e + 1], y[e + 2], y[e + 3]};
            } else {
                store_out<RUN>(a, d, y);
            }
        }
    if (g == 0) {
        if (sp.splits > 1) pl[(int64_t)split * a.tokens * a.q_heads + to] = ls;
        else if (a.lse) a.lse[to] = ls * 0x1.62e43p-1f;
    }
}

// f(FMT, D, WAVES) for the form of the call.
template <typename F>
void for_many(const KvAttnArgs& a, int waves, F&& f) {
    for_format(a.c.fmt, a.c.dim, [&](auto FMT, auto D) {
        if constexpr (D() != 256) {
            if (waves == 8) f(FMT, D, std::integral_constant<int, 8>{});
        }
        if constexpr (D() != 128) {
            if (waves == 4) f(FMT, D, std::integral_constant<int, 4>{});
        }
    });
}

}  // namespace
}  // namespace bg
