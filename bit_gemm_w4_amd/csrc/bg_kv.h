// bg_kv.h -- the paged, quantized key/value cache: its layout and the
// arguments of the kernels that write, read and attend over it.
//
// Codes of a page are [kv_heads][page][D] (4-bit: [D / 2] bytes, element 2i in
// the low nibble), so one head's tokens of a page are one contiguous run;
// records are [kv_heads][page], 4 bytes per token and head: a binary32 scale,
// or for 4 bits the FP16 scale (low half) and FP16 zero-point (high half).
// A token's codes are always finite: a row that holds an infinity or NaN is
// stored as codes 0 with a NaN scale.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bg {

enum { KV_I8 = 3, KV_FP8 = 4, KV_U4 = 6 };   // bg_dtype values of the formats

struct KvCache {
    uint8_t* k;
    uint8_t* v;
    uint32_t* ks;
    uint32_t* vs;
    int64_t pages;
    int page_shift;      // page size = 1 << page_shift, at least 16
    int heads, dim, fmt;
};

// Rows of new keys and values: element (t, h, i) at t * ts + h * hs + i.
struct KvRows {
    const void* k;
    const void* v;
    int64_t k_ts, k_hs, v_ts, v_hs;
};

const char* launch_kv_write(const KvCache& c, const KvRows& x, int dt, int64_t tokens, const int64_t* slots, hipStream_t s);
const char* launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, int dt, void* k, void* v, hipStream_t s);

// Norms and rotation of queries and keys: element (t, h, i) of each at t * ts + h * hs + i.
struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;             // with a cache
    void* q_out;
    void* k_out;               // without a cache
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    const void* q_weight;      // [D] of the rows' type, or binary32 (weight_f32); NULL: no norm
    const void* k_weight;
    const int32_t* positions;  // [tokens]
    const uint64_t* freqs;     // [rot / 2] turns a position, in units of 2^-64
    const int64_t* slots;      // [tokens], with a cache
    int64_t tokens;
    int q_heads, kv_heads;     // either may be 0
    int rot;                   // elements that are rotated, a multiple of 8
    bool interleaved;          // pairs are neighbours, else i and i + rot / 2
    bool weight_f32;
    double eps, offset;
};

// cache NULL: keys go to k_out.
const char* launch_qk_rope(const RopeArgs& a, int dt, int dim, const KvCache* cache, hipStream_t s);

struct KvAttnArgs {
    KvCache c;
    const void* q;             // element (t, h, i) at t * q_ts + h * q_hs + i
    int64_t q_ts, q_hs;
    bool bf16;                 // q and out are BF16, else FP16
    int64_t tokens;            // rows of q and out
    int q_heads;
    const int32_t* table;      // [batch][max_pages]
    int64_t max_pages;
    const int32_t* kv_lens;    // [batch]
    const int32_t* cu_q;       // [batch + 1], or NULL: sequence b owns query b
    int64_t batch, max_q, max_kv;
    int64_t chunk;             // queries of a sequence that its own blocks take, if not max_q (0); set by launch_kv_attn
    int64_t window, sinks;     // window 0: every earlier token is visible
    const uint64_t* tree;      // [tokens][tree_words] ancestor bits, or NULL: causal
    int tree_words;
    float scale;
    void* out;                 // [tokens][q_heads][D]
    float* lse;                // [tokens][q_heads], or NULL
    bool scored;               // any of the following
    float cap, cap_inv;        // scores (base 2) are capped: cap tanh(score cap_inv); cap_inv 0: not, cap 1
    bool cap_far;              // a cap of kCapExp (bg_kvattn.h) or more
    const float* slopes;       // [q_heads]: less slope times distance; or NULL
    const int32_t* prefix;     // [batch]: positions below it are seen from before, too; or NULL
};

// The pages of a cache that sequences do not hold, and those that they do.
struct KvPool {
    int32_t* table;            // [batch][max_pages]
    int32_t* lens;             // [batch] tokens held
    int32_t* gone;             // [batch] with a window: pages from the sinks' to this one were given back
    int32_t* free;             // [pages], the first state[0] of them are free
    int32_t* state;            // free pages; blocks that are done with a launch (0 between launches)
    int64_t batch, max_pages, pages;
    int page_shift, window, sinks;
};

// A step of new tokens: q_lens [batch] in, the rest out.
struct KvPlan {
    const int32_t* q_lens;
    int64_t tokens;            // rows of positions and slots
    bool advance;              // the pool is left as after the step
    int32_t* cu_q;             // [batch + 1]
    int32_t* kv_lens;          // [batch]
    int32_t* served;           // [batch]
    int32_t* positions;        // [tokens]
    int64_t* slots;            // [tokens]
};

const char* launch_kv_plan(const KvPool& p, const KvPlan& o, hipStream_t s);
const char* launch_kv_release(const KvPool& p, const int32_t* keep, hipStream_t s);

int64_t kv_attn_workspace(const KvAttnArgs& a);
const char* launch_kv_attn(const KvAttnArgs& a, void* ws, hipStream_t s);

}  // namespace bg
