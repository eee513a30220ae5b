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
};

int64_t kv_attn_workspace(const KvAttnArgs& a);
const char* launch_kv_attn(const KvAttnArgs& a, void* ws, hipStream_t s);

}  // namespace bg
