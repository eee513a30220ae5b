// k_kvplan.hip -- a serving step's page table, slots, positions and row offsets, and
// pages given back.
//
// A pool's free pages are a stack: free[0 .. count).  A step gives sequence b its
// n = q_lens[b] new tokens: rows start .. start + n - 1 of the step (start: the sum of
// the n before it), positions len .. len + n - 1, and need = ceil((len + n) / page) -
// ceil(len / page) new pages, the sequences' in order: new page i of all is
// free[count - 1 - i].  Giving back walks the same order backwards, so that a step taken
// back leaves the stack as it was.
//
// Bound by latency: a step reads 12 bytes a sequence and writes 12 a row.  One launch, so
// that nothing waits for a second: every block (1,024 items: rows of a step, pages to give
// back) takes the sums over all sequences itself, 4,096 at a time, from the lengths in its
// cache; a block leaves a mark where a sequence's items begin among its own, and the
// running maximum of the marks gives each item its sequence without a search.  The state
// that others still read (lengths, count) is written by the block that comes last.
// Sums saturate, so that no length, however large, passes 32 bits.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kv.h"

namespace bg {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kEach = 4, kSeqs = kThreads * kEach;
constexpr uint32_t kMost = 0x7FFFFFFFu;

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return a + b < kMost ? a + b : kMost; }

// The sum over the block's threads before this one; v becomes the sum over all.
// part: words that no thread reads any more.
__device__ __forceinline__ uint32_t sum_before(uint32_t& v, uint32_t* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = (uint32_t)__shfl_up((int)x, o, 64);
        if (lane >= o) x = add_sat(x, y);
    }
    const uint32_t up = (uint32_t)__shfl_up((int)x, 1, 64);
    if (lane == 63) part[wave] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t p = part[w];
        before = w < wave ? add_sat(before, p) : before;
        all = add_sat(all, p);
    }
    v = all;
    return lane ? add_sat(before, up) : before;
}

// The largest of the block's v up to this thread.
__device__ __forceinline__ int max_up_to(int v, int* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(v, o, 64);
        v = lane >= o && y > v ? y : v;
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) {
        const int p = part[w];
        v = w < wave && p > v ? p : v;
    }
    return v;
}

// True in all threads of the block of the grid that gets here last, with what the other
// blocks wrote before they came.  Nothing that they read may change before that.
__device__ __forceinline__ bool last_block(int32_t* ticket, int* word) {
    if (gridDim.x == 1) return true;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int n = atomicAdd(ticket, 1);
        if (n == (int)gridDim.x - 1) *ticket = 0;           // for the next launch
        *word = n;
    }
    __syncthreads();
    const bool last = *word == (int)gridDim.x - 1;
    if (last) __threadfence();
    return last;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((uint32_t)tokens + (1u << shift) - 1) >> shift); }

// tokens held by sequence b, within what the table has room for
__device__ __forceinline__ int length_of(const KvPool& p, int64_t b) {
    const int64_t room = p.max_pages << p.page_shift;
    const int n = p.lens[b];
    return n < 0 ? 0 : n > room ? (int)room : n;
}

__device__ __forceinline__ uint32_t count_of(const KvPool& p) {
    const int n = p.state[0];
    return n < 0 ? 0u : n > p.pages ? (uint32_t)p.pages : (uint32_t)n;
}

// What a block holds of the sequences whose items are among its own.
struct Shared {
    uint32_t part[2][2][kWaves];              // of the running sums, in turns
    int mark[kWaves], word;
    int begins[kThreads];                     // item + 1 where a sequence's items begin, 0 elsewhere
    int seq[kThreads], a[kThreads], b[kThreads], c[kThreads];       // of the sequence that begins there
};

// Where, among the block's items c0 .. c0 + 1023, a sequence with items start .. end - 1 begins; -1: none of them is here.
__device__ __forceinline__ int begin_in(uint32_t start, uint32_t end, uint32_t c0) {
    if (start >= end || end <= c0 || start >= c0 + kThreads) return -1;
    return start > c0 ? (int)(start - c0) : 0;
}

__global__ void __launch_bounds__(kThreads) k_kv_plan(KvPool p, KvPlan o) {
    __shared__ Shared lds;
    const int tid = threadIdx.x;
    const uint32_t rows = (uint32_t)o.tokens, c0 = blockIdx.x * kThreads, count = count_of(p);
    const int64_t room = p.max_pages << p.page_shift;
    const bool first = blockIdx.x == 0;
    lds.begins[tid] = 0;
    uint32_t rows_before = 0, pages_before = 0, taken = 0;
    int turn = 0;
    __syncthreads();
    for (int64_t b0 = 0; b0 < p.batch; b0 += kSeqs, turn ^= 1) {
        const int64_t own = b0 + kEach * tid;
        int len[kEach];
        uint32_t n[kEach], start[kEach], need[kEach], first_page[kEach], sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t b = own + e;
            const int q = b < p.batch ? o.q_lens[b] : 0;
            len[e] = b < p.batch ? length_of(p, b) : 0;
            n[e] = q <= 0 ? 0u : (uint32_t)q <= rows ? (uint32_t)q : rows + 1;      // more than fit stay more than fit
            start[e] = sum;
            sum = add_sat(sum, n[e]);
        }
        uint32_t before = add_sat(rows_before, sum_before(sum, lds.part[turn][0]));
        rows_before = add_sat(rows_before, sum);
        sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            start[e] = add_sat(before, start[e]);
            const bool fits = add_sat(start[e], n[e]) <= rows && (int64_t)len[e] + n[e] <= room;
            need[e] = fits ? (uint32_t)(pages_of(len[e] + (int)n[e], p.page_shift) - pages_of(len[e], p.page_shift)) : kMost;
            first_page[e] = sum;
            sum = add_sat(sum, fits ? need[e] : 0u);
        }
        before = add_sat(pages_before, sum_before(sum, lds.part[turn][1]));
        pages_before = add_sat(pages_before, sum);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t b = own + e;
            if (b >= p.batch) break;
            first_page[e] = add_sat(before, first_page[e]);
            const bool served = need[e] == 0 || (need[e] != kMost && add_sat(first_page[e], need[e]) <= count);
            const uint32_t end = add_sat(start[e], n[e]);
            const int after = served ? len[e] + (int)n[e] : len[e];
            taken += served ? need[e] : 0u;
            if (first) {
                o.cu_q[b + 1] = (int)(end < rows ? end : rows);
                o.kv_lens[b] = after;
                o.served[b] = served;
            }
            if (o.advance && gridDim.x == 1) p.lens[b] = after;
            const int at = begin_in(start[e], end, c0);
            if (at >= 0) {
                lds.begins[at] = at + 1;
                lds.seq[at] = (int)b;
                lds.a[at] = len[e] - (int)start[e];
                lds.b[at] = served ? pages_of(len[e], p.page_shift) : -1;
                lds.c[at] = (int)first_page[e];
            }
        }
    }
    if (first && tid == 0) o.cu_q[0] = 0;
    __syncthreads();
    const int at = max_up_to(lds.begins[tid], lds.mark) - 1;
    const uint32_t row = c0 + tid;
    if (row < rows) {
        int position = 0;
        int64_t slot = -1;
        if (at >= 0 && row < rows_before) {
            position = (int)row + lds.a[at];
            const int held = lds.b[at], page = position >> p.page_shift, in = position & ((1 << p.page_shift) - 1);
            if (held >= 0) {
                int32_t* entry = p.table + (int64_t)lds.seq[at] * p.max_pages + page;
                int id;
                if (page < held) {
                    id = *entry;
                } else {
                    id = p.free[count - 1 - (uint32_t)(lds.c[at] + page - held)];
                    if (in == 0) *entry = id;
                }
                if (id >= 0) slot = ((int64_t)id << p.page_shift) + in;
            }
        }
        o.positions[row] = position;
        o.slots[row] = slot;
    }
    if (!o.advance || !last_block(p.state + 1, &lds.word)) return;
    if (gridDim.x > 1)
        for (int64_t b = tid; b < p.batch; b += kThreads) p.lens[b] = o.kv_lens[b];
    sum_before(taken, lds.part[turn][0]);
    if (tid == 0) p.state[0] = (int)(count - taken);
}

// A sequence's pages to give back: low .. low + first - 1, then mid .. mid + slid - 1, then
// high .. ends - 1; what it is left with.
struct Back {
    int low, first, mid, slid, high, ends, len, gone;
    __device__ __forceinline__ uint32_t pages() const { return (uint32_t)(first + slid + (ends - high)); }
};

// Held are pages [0, sink) and [gone, n); of them stay those below ceil(keep / page) that a
// query at position keep or later sees.
__device__ __forceinline__ Back back_of(const KvPool& p, const int32_t* keep, int64_t b) {
    Back r;
    const int len = length_of(p, b), n = pages_of(len, p.page_shift);
    const int k = keep ? keep[b] : len;
    r.len = k < 0 ? 0 : k < len ? k : len;
    const int stay = pages_of(r.len, p.page_shift);
    int sink = 0, gone = 0, slid = 0;
    if (p.window) {
        sink = pages_of(p.sinks, p.page_shift);
        gone = p.gone[b] < sink ? sink : p.gone[b];
        // pages before position keep - window + 1
        slid = r.len >= p.window ? (r.len - p.window + 1) >> p.page_shift : 0;
        slid = slid < stay ? slid : stay;
        slid = slid > gone ? slid : gone;
    }
    r.low = stay;
    r.first = (sink < n ? sink : n) - stay;
    r.first = r.first > 0 ? r.first : 0;
    r.mid = gone;
    r.slid = (slid < n ? slid : n) - gone;
    r.slid = r.slid > 0 ? r.slid : 0;
    r.high = slid > stay ? slid : stay;
    r.ends = n > r.high ? n : r.high;
    r.gone = slid < stay ? slid : stay;
    return r;
}

__global__ void __launch_bounds__(kThreads) k_kv_release(KvPool p, const int32_t* keep) {
    __shared__ Shared lds;
    const int tid = threadIdx.x;
    const uint32_t count = count_of(p), most = (uint32_t)p.pages;
    uint32_t all = 0;
    int turn = 0;
    for (uint32_t c0 = blockIdx.x * kThreads;; c0 += gridDim.x * kThreads) {
        lds.begins[tid] = 0;
        uint32_t before = 0;
        __syncthreads();
        for (int64_t b0 = 0; b0 < p.batch; b0 += kSeqs, turn ^= 1) {
            const int64_t own = b0 + kEach * tid;
            uint32_t n[kEach], start[kEach], sum = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                n[e] = own + e < p.batch ? back_of(p, keep, own + e).pages() : 0u;
                start[e] = sum;
                sum = add_sat(sum, n[e]);
            }
            const uint32_t up = add_sat(before, sum_before(sum, lds.part[turn][0]));
            before = add_sat(before, sum);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                start[e] = add_sat(up, start[e]);
                const int at = begin_in(start[e], add_sat(start[e], n[e]), c0);
                if (at >= 0) {
                    lds.begins[at] = at + 1;
                    lds.seq[at] = (int)(own + e);
                    lds.a[at] = (int)start[e];
                }
            }
        }
        all = before < most ? before : most;
        __syncthreads();
        const int at = max_up_to(lds.begins[tid], lds.mark) - 1;
        const uint32_t item = c0 + tid;
        if (at >= 0 && item < all) {
            const int64_t b = lds.seq[at];
            const Back r = back_of(p, keep, b);
            int i = (int)item - lds.a[at];
            i = i < r.first ? r.low + i : i < r.first + r.slid ? r.mid + i - r.first : r.high + i - r.first - r.slid;
            int32_t* entry = p.table + b * p.max_pages + i;
            const uint32_t to = count + all - 1 - item;
            if (to < most) p.free[to] = *entry;
            *entry = -1;
        }
        if (all <= c0 || all - c0 <= gridDim.x * kThreads) break;       // nothing left for this block
        __syncthreads();
    }
    if (!last_block(p.state + 1, &lds.word)) return;
    __syncthreads();
    for (int64_t b = tid; b < p.batch; b += kThreads) {
        const Back r = back_of(p, keep, b);
        p.lens[b] = r.len;
        if (p.window) p.gone[b] = r.gone;
    }
    if (tid == 0) p.state[0] = (int)(count + all < most ? count + all : most);
}

}  // namespace

const char* launch_kv_plan(const KvPool& p, const KvPlan& o, hipStream_t s) {
    const unsigned blocks = o.tokens > 0 ? (unsigned)((o.tokens + kThreads - 1) / kThreads) : 1;
    k_kv_plan<<<blocks, kThreads, 0, s>>>(p, o);
    return "k_kv_plan";
}

const char* launch_kv_release(const KvPool& p, const int32_t* keep, hipStream_t s) {
    // Usually a few pages of a large pool come back; more than these blocks' items in turns.
    const int64_t most = p.pages < p.batch * p.max_pages ? p.pages : p.batch * p.max_pages, blocks = (most + kThreads - 1) / kThreads;
    k_kv_release<<<(unsigned)(blocks < 64 ? blocks : 64), kThreads, 0, s>>>(p, keep);
    return "k_kv_release";
}

}  // namespace bg
