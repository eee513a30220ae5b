// k_kvattn_many.hip -- attention over the paged, quantized KV cache for many
// query rows per kv head (prompt chunks, large draft trees).
//
// A block of eight waves takes 256 rows of one sequence and kv head, 32 to a wave
// (head size 256: four waves, 128 rows; head size 64: that or two blocks of four
// waves a CU, where 256 rows would leave most of a block empty), and walks the positions some row sees
// in tiles of 64.  With this many rows per cache byte the matrix cores bound it:
//   S^T = K Q^T     v_mfma_f32_32x32x16_f16, A = 32 tokens, B = 32 rows
//   O^T += V^T P^T  A = 32 head elements of 16 tokens, B = the weights in place
// (the k-slots of V are numbered as the accumulator of S^T holds its tokens).
// 32x32x16 and not 16x16x32: beside the latter's 16-cycle products the vector
// units issue little (16 products with 4 multiply-adds after each: 444 ns of two
// waves, against 433 ns for the products alone; the same work in 16x16x32: 658 ns).
//
// What else there is to do runs beside the products:
// * A tile's codes turn to FP16 once per block, in LDS, as the fragments that the
//   waves' products take (16 bytes per lane, contiguous over lanes: no bank
//   conflicts in either direction).  Each wave carries an eighth of a tile (a quarter
//   in blocks of four), keys two tiles ahead and values one, between its products; one barrier a tile.
// * The products of the next step's scores and of the last step's values alternate
//   (two chains that do not wait for one another), with this step's weights in the
//   vector units' slots between them.
// A tile of 64 positions takes a block 2.1 us (4,200 cycles, 2,048 of them in each SIMD's
// matrix core); a block's start (pages, first codes, queries) 6 us.  2,048 queries
// over a window of 4,096 in E4M3 (8 kv heads of 4, D = 128): 165 us, 835 TFLOP/s; the
// few-row kernel takes 460 us, a library product of 8192^3 in FP16 runs at 1,064
// TFLOP/s.  In 16x16x32, a barrier and codes of a tile at a time: 245 us; with half of
// the waves carrying keys and half values outside the products: 175 us.  At D = 128 a
// lane's 256 registers are full and 9 to 20 more lie in scratch, of what the loop seldom
// asks for.
//
// Numerics as in the few-row kernel: codes exact in FP16, scales and statistics
// in binary32.  Two things differ, both to spare vector instructions.  Queries are
// scaled by one power of two per block, so the score's factors fold into the token's
// scale; a row that lies more than 2^16 below the block's largest keeps its own, and its
// wave takes every tile's weights as a masked one's (twice the time; above that, a
// query element errs by 2^-24 of its row's largest at most).  The weights are taken
// against the running references before their maxima are known, and only if one of
// them times its value's scale left FP16's range (which is looked at if a lane's sum
// times the tile's largest value scale passes 2^15) are the maxima found, the row's
// references moved and the weights taken again; a wave that has a row with two
// references (raise_row in bg_kvattn.h: value scales beyond 2^+-40) takes them so
// always, too.  A row's largest w s lies at 2^3 at least, so one that falls below
// FP16's normal range errs by 2^-28 of it.
//
// Other scores (k_kvattn_many_*.hip) cost vector instructions, which bound them: the chunk above 176 us as it is
// with queries of four times the size, 171 with slopes, 211 with a cap of 50, 202 with both, 240 with a cap of 1000.
// A form each, as what a form does not need costs registers: with caps and slopes behind branches in one kernel 250
// us (cap) where this takes 211, and at D = 128 value fragments are read two products ahead there, not four (ragged
// chunks with slopes 193 -> 163 us).
#include "bg_kvattn_many.h"

namespace bg {
namespace {

template <int FMT, int D, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, D == 256 ? 1 : 2) k_kv_attn_many(KvAttnArgs a, KvSplit sp, float* po, float* pl) {
    attend_many<FMT, D, WAVES, false, false, false>(a, sp, po, pl);
}

}  // namespace

const char* launch_kv_attn_many(const KvAttnArgs& a, const KvSplit& sp, unsigned row_blocks, int waves, float* po, float* pl, hipStream_t s) {
    const dim3 grid((unsigned)a.c.heads * row_blocks, (unsigned)sp.splits, kv_grid_z(a));
    if (!a.scored) {
        for_many(a, waves, [&](auto FMT, auto D, auto WAVES) { k_kv_attn_many<FMT(), D(), WAVES()><<<grid, WAVES() * 64, 0, s>>>(a, sp, po, pl); });
        return kname("k_kv_attn_many", a.c.fmt, a.c.dim, waves);
    }
    const char* name = a.cap_far ? "k_kv_attn_many_far_cap" : a.cap_inv == 0.0f ? "k_kv_attn_many_bias" : a.slopes ? "k_kv_attn_many_cap_bias" : "k_kv_attn_many_cap";
    (a.cap_far ? launch_kv_attn_many_far_cap : a.cap_inv == 0.0f ? launch_kv_attn_many_bias : a.slopes ? launch_kv_attn_many_cap_bias : launch_kv_attn_many_cap)(
        a, sp, grid, waves, po, pl, s);
    return kname(name, a.c.fmt, a.c.dim, waves);
}

}  // namespace bg
