// k_kvattn_many_bias.hip -- the many-row kernel (k_kvattn_many.hip) with scores biased by distance, or a prefix.
#include "bg_kvattn_many.h"

namespace bg {
namespace {

template <int FMT, int D, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, D == 256 ? 1 : 2) k_kv_attn_many_bias(KvAttnArgs a, KvSplit sp, float* po, float* pl) {
    attend_many<FMT, D, WAVES, false, true, false>(a, sp, po, pl);
}

}  // namespace

void launch_kv_attn_many_bias(const KvAttnArgs& a, const KvSplit& sp, dim3 grid, int waves, float* po, float* pl, hipStream_t s) {
    for_many(a, waves, [&](auto FMT, auto D, auto WAVES) { k_kv_attn_many_bias<FMT(), D(), WAVES()><<<grid, WAVES() * 64, 0, s>>>(a, sp, po, pl); });
}

}  // namespace bg
