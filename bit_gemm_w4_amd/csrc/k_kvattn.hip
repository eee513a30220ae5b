// k_kvattn.hip -- attention over the paged, quantized KV cache.
//
// One wave per (query token, query head): 64 cache tokens at a time, one per
// lane for the scores, then D / 64 elements per lane for the weighted sum of
// the values, with the running maximum and sum of the softmax in binary32.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kv.h"

namespace bg {
namespace {

template <int FMT>
__device__ __forceinline__ float kv_value(const uint8_t* codes, uint32_t record, int i) {
    if constexpr (FMT == KV_U4) {
        const uint32_t u = codes[i / 2] >> (4 * (i % 2)) & 15u;
        return ((float)u - f16_to_f32(record >> 16)) * f16_to_f32(record & 0xFFFFu);
    } else if constexpr (FMT == KV_I8) {
        return (float)(int8_t)codes[i] * __uint_as_float(record);
    } else {
        return __builtin_amdgcn_cvt_f32_fp8((int)codes[i], 0) * __uint_as_float(record);
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(64) k_kv_attn_row(KvAttnArgs a) {
    __shared__ float qs[D];
    __shared__ float ps[64];
    __shared__ int64_t rows[64];
    const int lane = threadIdx.x, hq = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
    int64_t q0 = b, q1 = b + 1;
    if (a.cu_q) {
        q0 = a.cu_q[b];
        q1 = a.cu_q[b + 1];
        q0 = q0 < 0 ? 0 : q0 > a.tokens ? a.tokens : q0;
        q1 = q1 < q0 ? q0 : q1 > a.tokens ? a.tokens : q1;
    }
    if (i >= q1 - q0) return;
    const int64_t t = q0 + i;
    int64_t len = a.kv_lens[b];
    const int64_t room = a.max_pages << a.c.page_shift;
    len = len < 0 ? 0 : len > room ? room : len;
    const int64_t first = len - (q1 - q0), pos = first + i;
    const int h = hq / (a.q_heads / a.c.heads);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_ts + hq * a.q_hs;
    for (int d = lane; d < D; d += 64) qs[d] = a.bf16 ? bf16_to_f32(q[d]) : f16_to_f32(q[d]);
    __syncthreads();
    constexpr int W = FMT == KV_U4 ? D / 2 : D;
    float m = -__builtin_inff(), l = 0.0f, o[D / 64] = {};
    for (int64_t base = 0; base < len; base += 64) {
        const int64_t j = base + lane;
        bool seen = j < len;
        if (a.tree) {
            const int64_t e = j - first;
            if (e >= 0) seen = seen && e < 64 * (int64_t)a.tree_words && (a.tree[t * a.tree_words + (e >> 6)] >> (e & 63) & 1);
        } else {
            seen = seen && j <= pos && (a.window == 0 || j > pos - a.window || j < a.sinks);
        }
        int64_t row = 0;
        if (seen) {
            const int page = a.table[b * a.max_pages + (j >> a.c.page_shift)];
            seen = page >= 0 && page < a.c.pages;
            row = (((int64_t)page * a.c.heads + h) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        }
        float s = -__builtin_inff();
        if (seen) {
            const uint8_t* k = a.c.k + row * W;
            const uint32_t rec = a.c.ks[row];
            float acc = 0.0f;
            for (int d = 0; d < D; ++d) acc += qs[d] * kv_value<FMT>(k, rec, d);
            s = acc * a.scale;
        }
        float mt = wave_max<64>(s);
        if (!__any(seen)) continue;
        const float mn = __builtin_fmaxf(m, mt);
        const float base_m = mn == -__builtin_inff() ? 0.0f : mn;
        const float alpha = __builtin_expf(m - base_m);
        const float p = seen ? __builtin_expf(s - base_m) : 0.0f;
        l = l * alpha + wave_sum<64>(p);
        m = mn;
        ps[lane] = p;
        rows[lane] = seen ? row : -1;
        __syncthreads();
        for (int x = 0; x < D / 64; ++x) o[x] *= alpha;
        for (int n = 0; n < 64; ++n) {
            if (rows[n] < 0) continue;
            const uint32_t rec = a.c.vs[rows[n]];
            for (int x = 0; x < D / 64; ++x) o[x] += ps[n] * kv_value<FMT>(a.c.v + rows[n] * W, rec, x * 64 + lane);
        }
        __syncthreads();
    }
    for (int x = 0; x < D / 64; ++x) {
        const float y = l == 0.0f ? 0.0f : o[x] / l;
        static_cast<uint16_t*>(a.out)[(t * a.q_heads + hq) * D + x * 64 + lane] = a.bf16 ? f32_to_bf16(y) : f32_to_f16(y);
    }
    if (a.lse && lane == 0) a.lse[t * a.q_heads + hq] = l == 0.0f ? -__builtin_inff() : m + __builtin_logf(l);
}

}  // namespace

int64_t kv_attn_workspace(const KvAttnArgs&) { return 0; }

const char* launch_kv_attn(const KvAttnArgs& a, void*, hipStream_t s) {
    const dim3 grid((unsigned)a.q_heads, (unsigned)a.max_q, (unsigned)a.batch);
    auto on_dim = [&](auto FMT) {
        if (a.c.dim == 64) k_kv_attn_row<FMT(), 64><<<grid, 64, 0, s>>>(a);
        else if (a.c.dim == 128) k_kv_attn_row<FMT(), 128><<<grid, 64, 0, s>>>(a);
        else k_kv_attn_row<FMT(), 256><<<grid, 64, 0, s>>>(a);
    };
    if (a.c.fmt == KV_I8) on_dim(std::integral_constant<int, KV_I8>{});
    else if (a.c.fmt == KV_FP8) on_dim(std::integral_constant<int, KV_FP8>{});
    else on_dim(std::integral_constant<int, KV_U4>{});
    return kname("k_kv_attn_row", a.c.fmt, a.c.dim);
}

}  // namespace bg
