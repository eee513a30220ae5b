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
// Bound by latency: a step reads 12 bytes a sequence and writes 12 a row.  So: one launch, in
// which each team goes its own way to its items (rows of the step, pages to give back; one to
// a lane): it takes the sums over all sequences itself from the lengths in its cache; leaves a
// mark where a sequence's items begin among its own; and the running maximum of the marks
// gives each item its sequence, without a search.  Running sums go through the vector unit's
// lane shifts.  A team is a wave, which needs no barrier, or for many sequences a block, whose
// 16 waves share the sums.  What others still read (lengths, count) is written when all are
// done: behind the block's barrier, or by the block that comes last, which takes nothing
// from the others and so needs no fence.
// 16 sequences of one new token each: 3.8 us; 300 with 93,000 rows: 6.1 (7.8 by blocks); 2,048 with
// 30,000 rows: 8.7, and 8.2 to take them back (22 and 16 by waves; by blocks with a
// fence in every wave 23.6 and 29).
// Sums saturate, so that no length, however large, passes 32 bits.
#include "bg_device.h"
#include "bg_internal.h"
#include "bg_kv.h"

namespace bg {
namespace {

constexpr int kMaxWaves = 16, kEach = 4;      // waves of a block, sequences of a lane at a time
constexpr uint32_t kMost = 0x7FFFFFFFu;

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return a + b < kMost ? a + b : kMost; }

// f over the wave's lanes up to this one; f commutes and 0 is its neutral element.
template <typename F>
__device__ __forceinline__ uint32_t up_to(uint32_t v, F&& f) {
    auto from = [&](auto CTRL, auto ROWS) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL(), ROWS(), 0xF, true); };
    using std::integral_constant;
    v = f(v, from(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{}));       // 1, 2, 4 and 8 lanes up within 16
    v = f(v, from(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{}));
    v = f(v, from(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{}));
    v = f(v, from(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{}));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));    // lane 15 of 16 to the next 16, in every second
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));    // lane 31 to the upper 32
    return v;
}

// The waves that go through sequences and items together: one, or a block's 16.
template <int WAVES>
struct Team {
    static constexpr int kLanes = 64 * WAVES, kSeqs = kLanes * kEach;
    uint32_t* part;                           // 3 * WAVES words of LDS (WAVES > 1)
    int turn = 0;                             // parts are used in turns: one barrier a sum

    __device__ __forceinline__ int lane() const { return threadIdx.x % kLanes; }
    __device__ __forceinline__ int number() const { return __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes); }       // in the block

    // What a lane wrote to LDS is there for the others.
    __device__ __forceinline__ void sync() {
        if constexpr (WAVES > 1) {
            __syncthreads();
        } else {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    }
    // f over the lanes before this one, and with ALL in v over all of the team.
    template <bool ALL, typename F>
    __device__ __forceinline__ uint32_t before(uint32_t& v, F&& f) {
        const uint32_t x = up_to(v, f), all = __builtin_amdgcn_readlane(x, 63);
        uint32_t r = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x138, 0xF, 0xF, true);       // one lane up
        if constexpr (ALL) v = all;
        if constexpr (WAVES > 1) {
            const int wave = threadIdx.x >> 6;
            uint32_t* const now = part + turn * WAVES;
            turn = turn == 2 ? 0 : turn + 1;
            now[wave] = all;
            __syncthreads();
            uint32_t lower = 0, sum = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const uint32_t y = now[w];
                lower = w < wave ? f(lower, y) : lower;
                sum = f(sum, y);
            }
            r = f(r, lower);
            if constexpr (ALL) v = sum;
        }
        return r;
    }
    __device__ __forceinline__ uint32_t sum_before(uint32_t& v) {
        return before<true>(v, [](uint32_t a, uint32_t b) { return add_sat(a, b); });
    }
    __device__ __forceinline__ uint32_t max_up_to(uint32_t v) {
        auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
        const uint32_t own = v;
        return larger(own, before<false>(v, larger));
    }
};

// Passes when every wave of the launch has read what it reads of the state; true in the
// one block that goes on to write it.
__device__ __forceinline__ bool last_block(int32_t* ticket, int* word) {
    __syncthreads();
    if (gridDim.x == 1) return true;
    if (threadIdx.x == 0) {
        const int n = atomicAdd(ticket, 1);
        if (n == (int)gridDim.x - 1) *ticket = 0;           // for the next launch
        *word = n;
    }
    __syncthreads();
    return *word == (int)gridDim.x - 1;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((uint32_t)tokens + (1u << shift) - 1) >> shift); }

// n tokens of a sequence, within what the table has room for.
__device__ __forceinline__ int length_of(const KvPool& p, int n) {
    const int64_t room = p.max_pages << p.page_shift;
    return n < 0 ? 0 : n > room ? (int)room : n;
}

__device__ __forceinline__ uint32_t count_of(const KvPool& p) {
    const int n = p.state[0];
    return n < 0 ? 0u : n > p.pages ? (uint32_t)p.pages : (uint32_t)n;
}

// Per-sequence words in turns of SEQS, kEach to a lane, asked for two turns ahead.
template <int N, int SEQS>
struct SeqWords {
    const int32_t* from[N];
    int64_t batch;
    bool wide;                                // 16 bytes at a time
    int4_t next[2][N];

    __device__ __forceinline__ SeqWords(const KvPool& p, const int32_t* const (&arrays)[N]) : batch(p.batch) {
        uintptr_t bits = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            from[i] = arrays[i];
            bits |= reinterpret_cast<uintptr_t>(arrays[i]);
        }
        wide = (bits & 15) == 0;
        ask(0, 0);
        ask(1, SEQS);
    }
    __device__ __forceinline__ void ask(int into, int64_t b0) {
        const int64_t own = b0 + kEach * (threadIdx.x % (SEQS / kEach));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int4_t x = {0, 0, 0, 0};
            if (from[i] && wide && own + kEach <= batch) {
                x = *reinterpret_cast<const int4_t*>(from[i] + own);
            } else if (from[i]) {
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (own + e < batch) x[e] = from[i][own + e];
            }
            next[into][i] = x;
        }
    }
    // f(b0, words) for each turn.
    template <typename F>
    __device__ __forceinline__ void turns(F&& f) {
        for (int64_t b0 = 0; b0 < batch; b0 += SEQS) {
            int4_t x[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = next[0][i];
                next[0][i] = next[1][i];
            }
            if (b0 + 2 * SEQS < batch) ask(1, b0 + 2 * SEQS);
            f(b0, x);
        }
    }
};

// Where, among n items from c0 on, a sequence with items start .. end - 1 begins; -1: none of them is here.
__device__ __forceinline__ int begin_in(uint32_t start, uint32_t end, uint32_t c0, uint32_t n) {
    if (start >= end || end <= c0 || start >= c0 + n) return -1;
    return start > c0 ? (int)(start - c0) : 0;
}

struct PlanSeq {
    uint32_t start, n, need, first_page;
    int len, after;
    bool served;
};

// f(b, seq) for the lane's sequences, in turns of all; returns the sum of their rows.
template <int WAVES, typename F>
__device__ __forceinline__ uint32_t plan_walk(const KvPool& p, const KvPlan& o, Team<WAVES>& team, uint32_t count, F&& f) {
    const uint32_t rows = (uint32_t)o.tokens;
    const int64_t room = p.max_pages << p.page_shift;
    uint32_t rows_before = 0, pages_before = 0;
    const int32_t* const arrays[2] = {p.lens, o.q_lens};
    SeqWords<2, Team<WAVES>::kSeqs>(p, arrays).turns([&](int64_t b0, const int4_t (&x)[2]) {
        PlanSeq q[kEach];
        uint32_t sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int asked = x[1][e];
            q[e].len = length_of(p, x[0][e]);
            q[e].n = asked <= 0 ? 0u : (uint32_t)asked <= rows ? (uint32_t)asked : rows + 1;      // more than fit stay more than fit
            q[e].start = sum;
            sum = add_sat(sum, q[e].n);
        }
        uint32_t before = add_sat(rows_before, team.sum_before(sum));
        rows_before = add_sat(rows_before, sum);
        sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            q[e].start = add_sat(before, q[e].start);
            const bool fits = add_sat(q[e].start, q[e].n) <= rows && (int64_t)q[e].len + q[e].n <= room;
            q[e].need = fits ? (uint32_t)(pages_of(q[e].len + (int)q[e].n, p.page_shift) - pages_of(q[e].len, p.page_shift)) : kMost;
            q[e].first_page = sum;
            sum = add_sat(sum, fits ? q[e].need : 0u);
        }
        before = add_sat(pages_before, team.sum_before(sum));
        pages_before = add_sat(pages_before, sum);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            q[e].first_page = add_sat(before, q[e].first_page);
            q[e].served = q[e].need == 0 || (q[e].need != kMost && add_sat(q[e].first_page, q[e].need) <= count);
            q[e].after = q[e].served ? q[e].len + (int)q[e].n : q[e].len;
            const int64_t b = b0 + kEach * team.lane() + e;
            if (b < p.batch) f(e, b, q[e]);
        }
    });
    return rows_before;
}

template <int LANES>
struct PlanLds {
    uint32_t begins[LANES];                   // item + 1 where a sequence's items begin, 0 elsewhere
    int seq[LANES], shift[LANES], held[LANES], fresh[LANES];
};

template <int WAVES>
__global__ void __launch_bounds__(64 * kMaxWaves) k_kv_plan(KvPool p, KvPlan o) {
    constexpr int LANES = 64 * WAVES;
    __shared__ PlanLds<LANES> all_lds[kMaxWaves / WAVES];
    __shared__ uint32_t part[3 * WAVES];
    __shared__ int word;
    Team<WAVES> team{part};
    PlanLds<LANES>& lds = all_lds[team.number()];
    const int lane = team.lane();
    const uint32_t rows = (uint32_t)o.tokens, c0 = (blockIdx.x * (blockDim.x / LANES) + team.number()) * LANES, count = count_of(p);
    const bool first = c0 == 0;               // the team that writes what there is one of per sequence
    lds.begins[lane] = 0;
    team.sync();
    uint32_t taken = 0;
    int after[kEach];                         // of the last turn
    const uint32_t end = plan_walk(p, o, team, count, [&](int e, int64_t b, const PlanSeq& q) {
        taken += q.served ? q.need : 0u;
        after[e] = q.after;
        const uint32_t to = add_sat(q.start, q.n);
        if (first) {
            o.cu_q[b + 1] = (int)(to < rows ? to : rows);
            o.kv_lens[b] = q.after;
            o.served[b] = q.served;
        }
        const int at = begin_in(q.start, to, c0, LANES);
        if (at >= 0) {
            lds.begins[at] = at + 1;
            lds.seq[at] = (int)b;
            lds.shift[at] = q.len - (int)q.start;
            lds.held[at] = q.served ? pages_of(q.len, p.page_shift) : -1;
            lds.fresh[at] = (int)q.first_page;
        }
    });
    if (first && lane == 0) o.cu_q[0] = 0;
    team.sync();
    const int at = (int)team.max_up_to(lds.begins[lane]) - 1;
    const uint32_t row = c0 + lane;
    if (row < rows) {
        int position = 0;
        int64_t slot = -1;
        if (at >= 0 && row < end) {
            position = (int)row + lds.shift[at];
            const int held = lds.held[at], page = position >> p.page_shift, in = position & ((1 << p.page_shift) - 1);
            if (held >= 0) {
                int32_t* entry = p.table + (int64_t)lds.seq[at] * p.max_pages + page;
                int id;
                if (page < held) {
                    id = *entry;
                } else {
                    id = p.free[count - 1 - (uint32_t)(lds.fresh[at] + page - held)];
                    if (in == 0) *entry = id;
                }
                if (id >= 0) slot = ((int64_t)id << p.page_shift) + in;
            }
        }
        o.positions[row] = position;
        o.slots[row] = slot;
    }
    if (!o.advance || !last_block(p.state + 1, &word) || team.number() > 0) return;
    if (p.batch <= Team<WAVES>::kSeqs) {
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (kEach * lane + e < p.batch) p.lens[kEach * lane + e] = after[e];
    } else {
        plan_walk(p, o, team, count, [&](int, int64_t b, const PlanSeq& q) { p.lens[b] = q.after; });
    }
    team.sum_before(taken);
    if (lane == 0) p.state[0] = (int)(count - taken);
}

// A sequence's pages to give back: low .. low + first - 1, then mid .. mid + slid - 1, then
// high .. ends - 1; what it is left with.
struct Back {
    int low, first, mid, slid, high, ends, len, gone;
    __device__ __forceinline__ uint32_t pages() const { return (uint32_t)(first + slid + (ends - high)); }
};

// Held are pages [0, sink) and [gone, n); of them stay those below ceil(keep / page) that a
// query at position keep or later sees.
__device__ __forceinline__ Back back_of(const KvPool& p, bool cut, int held, int keep, int was_gone) {
    Back r;
    const int len = length_of(p, held), n = pages_of(len, p.page_shift), k = cut ? keep : len;
    r.len = k < 0 ? 0 : k < len ? k : len;
    const int stay = pages_of(r.len, p.page_shift);
    int sink = 0, gone = 0, slid = 0;
    if (p.window) {
        sink = pages_of(p.sinks, p.page_shift);
        gone = was_gone < sink ? sink : was_gone;
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

template <int LANES>
struct ReleaseLds {
    uint32_t begins[LANES];
    int seq[LANES], start[LANES];
    Back back[LANES];
};

template <int WAVES>
__global__ void __launch_bounds__(64 * kMaxWaves) k_kv_release(KvPool p, const int32_t* keep) {
    constexpr int LANES = 64 * WAVES;
    __shared__ ReleaseLds<LANES> all_lds[kMaxWaves / WAVES];
    __shared__ uint32_t part[3 * WAVES];
    __shared__ int word;
    Team<WAVES> team{part};
    ReleaseLds<LANES>& lds = all_lds[team.number()];
    const int lane = team.lane();
    const uint32_t count = count_of(p), most = (uint32_t)p.pages, step = gridDim.x * blockDim.x;
    const int32_t* const arrays[3] = {p.lens, keep, p.window ? p.gone : nullptr};
    uint32_t all = 0;
    for (uint32_t c0 = (blockIdx.x * (blockDim.x / LANES) + team.number()) * LANES;; c0 += step) {
        lds.begins[lane] = 0;
        team.sync();
        uint32_t before = 0;
        SeqWords<3, Team<WAVES>::kSeqs>(p, arrays).turns([&](int64_t b0, const int4_t (&x)[3]) {
            const int64_t own = b0 + kEach * lane;
            Back r[kEach];
            uint32_t n[kEach], start[kEach], sum = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                r[e] = back_of(p, keep != nullptr, x[0][e], x[1][e], x[2][e]);      // past the batch: of nothing
                n[e] = r[e].pages();
                start[e] = sum;
                sum = add_sat(sum, n[e]);
            }
            const uint32_t up = add_sat(before, team.sum_before(sum));
            before = add_sat(before, sum);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                start[e] = add_sat(up, start[e]);
                const int at = begin_in(start[e], add_sat(start[e], n[e]), c0, LANES);
                if (at >= 0) {
                    lds.begins[at] = at + 1;
                    lds.seq[at] = (int)(own + e);
                    lds.start[at] = (int)start[e];
                    lds.back[at] = r[e];
                }
            }
        });
        all = before < most ? before : most;
        team.sync();
        const int at = (int)team.max_up_to(lds.begins[lane]) - 1;
        const uint32_t item = c0 + lane;
        if (at >= 0 && item < all) {
            const Back r = lds.back[at];
            int i = (int)item - lds.start[at];
            i = i < r.first ? r.low + i : i < r.first + r.slid ? r.mid + i - r.first : r.high + i - r.first - r.slid;
            int32_t* entry = p.table + (int64_t)lds.seq[at] * p.max_pages + i;
            const uint32_t to = count + all - 1 - item;
            if (to < most) p.free[to] = *entry;
            *entry = -1;
        }
        if (all <= c0 || all - c0 <= step) break;       // nothing left for this team
        team.sync();
    }
    if (!last_block(p.state + 1, &word)) return;
    for (int64_t b = threadIdx.x; b < p.batch; b += blockDim.x) {
        const Back r = back_of(p, keep != nullptr, p.lens[b], keep ? keep[b] : 0, p.window ? p.gone[b] : 0);
        p.lens[b] = r.len;
        if (p.window) p.gone[b] = r.gone;
    }
    if (threadIdx.x == 0) p.state[0] = (int)(count + all < most ? count + all : most);
}

}  // namespace

// A wave's second turn through the sequences costs less than a block's barriers, a third does not.
bool by_waves(const KvPool& p) { return p.batch <= 2 * Team<1>::kSeqs; }

// One block where that takes all rows (no block to wait for), else blocks of four waves, or of 16.
const char* launch_kv_plan(const KvPool& p, const KvPlan& o, hipStream_t s) {
    const int64_t waves = o.tokens > 64 ? (o.tokens + 63) / 64 : 1;
    if (by_waves(p)) {
        const unsigned block = waves <= kMaxWaves ? (unsigned)waves : 4;
        k_kv_plan<1><<<(unsigned)((waves + block - 1) / block), 64 * block, 0, s>>>(p, o);
        return kname("k_kv_plan", 1);
    }
    k_kv_plan<kMaxWaves><<<(unsigned)((waves + kMaxWaves - 1) / kMaxWaves), 64 * kMaxWaves, 0, s>>>(p, o);
    return kname("k_kv_plan", kMaxWaves);
}

// Usually a few pages of each sequence come back; more than these waves' items in turns.
const char* launch_kv_release(const KvPool& p, const int32_t* keep, hipStream_t s) {
    const int64_t most = p.pages < p.batch * p.max_pages ? p.pages : p.batch * p.max_pages;
    const int64_t waves = (most + 63) / 64 < (p.batch + 7) / 8 ? (most + 63) / 64 : (p.batch + 7) / 8;
    if (by_waves(p)) {
        const unsigned block = waves <= kMaxWaves ? (unsigned)waves : kMaxWaves;
        k_kv_release<1><<<(unsigned)((waves + block - 1) / block), 64 * block, 0, s>>>(p, keep);
        return kname("k_kv_release", 1);
    }
    const int64_t blocks = (waves + kMaxWaves - 1) / kMaxWaves;
    k_kv_release<kMaxWaves><<<(unsigned)(blocks < 64 ? blocks : 64), 64 * kMaxWaves, 0, s>>>(p, keep);
    return kname("k_kv_release", kMaxWaves);
}

}  // namespace bg
