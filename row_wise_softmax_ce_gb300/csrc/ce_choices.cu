// ce_choices.cu -- sm_103a kernels of the tokens drawn from a row's softmax, and
// their launchers.
//
//   sample_rows     a token drawn from each row's softmax by a given uniform number
//   verify_drafts   drafted tokens accepted or replaced
//
// Kernels (none uses tensor cores):
//   k_states           every row in steps of 4 KB, a state (m, s) for each step: one
//                      read of the logits, and of the draft rows, in parts of any
//                      number of warps
//   k_sample           sample_rows: a warp per row merges its states, draws a step by
//                      their masses and re-reads that step
//   k_sample_row       states and draw of short rows, a CTA a row
//   k_decide           verify_drafts: a cluster per request merges its rows' states,
//                      finds the first that accepts no draft, and draws its token:
//                      from p, or from max(0, p - q), which reads the two rows once
//                      more
//
// A row is not one CTA's, or one cluster's: rows end together then, and hold their
// share of an SM through the latencies of a merge and a draw (a cluster of warps
// per row, one kernel: sampling 256 x 151936 21.6 us, verification of 64 x 4
// drafts 62 us, of 256 x 7 195). Its states go to memory instead (0.2% of the
// logits), and a kernel that starts as the streaming one ends takes them up.
#include <algorithm>
#include <cstdint>

#include "ce_internal.h"
#include "ce_launch.h"
#include "ce_objectives.cuh"

namespace cerows {

namespace {

// rows that are no distribution, bad drafts, temperatures and ranges
__device__ unsigned long long g_choice_status;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kScan = 8;  // 16-byte loads in flight per thread
constexpr int kStep = 32 * kScan;  // vectors of a step, 4 KB
constexpr int kDrawThreads = 32 * kScan;
constexpr int kRowThreads = 1024;
constexpr int kRowSteps = kRowThreads / 32;  // of a row that k_sample_row takes, at most

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ void count_bad() { atomicAdd(&g_choice_status, 1ull); }

// ---------------------------------------------------------------------------
// Drawing a column. A row is split into segments in column order (a step, 32
// vectors, a vector, a column); a segment's mass is the sum of its weights as a fixed
// point number, rounded down to 2^-36 of the largest weight (2^-60 of the whole
// for weights that add up to at most 1). Fixed point sums are exact: the
// segments' running sums meet without a gap, and a number below the total lies
// in exactly one segment, the same for every warp that looks. f32 running sums
// would move the borders by up to 2^-22 of the row; f64 ones cost as much as
// the rest of the draw (GB300 adds f64 at about two lanes per clock and SM).
using Mass = unsigned long long;

// The numbers 2^-36 and 2^-60 are for weights of at most 1, of which a row has
// at most 2^24, and for those whose sum is at most 1 (to a rounding).
__device__ __forceinline__ Mass mass_of(float w, float unit) { return __float2ull_rd(w * unit); }
constexpr float kUnitWeights = 68719476736.0f;             // 2^36
constexpr float kUnitShares = 1152921504606846976.0f;      // 2^60

// u of the total: u in [0, 1), numbers outside count as the nearest inside, NaN as 0
__device__ __forceinline__ Mass part_of_total(float u, Mass total) {
    u = fminf(fmaxf(u, 0.0f), 0.99999994f);
    return __umul64hi(total, __float2ull_rd(u * 18446744073709551616.0f));
}

__device__ __forceinline__ Mass warp_running_sum(Mass v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Mass p = __shfl_up_sync(kFullMask, v, o);
        if (lane >= o) v += p;
    }
    return v;
}

// The lane whose segment holds t, and t from that segment's start on. `w`: the
// segments' weights in f32, for a t that lies behind the last mass (a segment's
// weights are summed anew and may come to a little less than before): the last
// segment with any mass then, the largest weight if there is none. -1: no
// weight at all.
__device__ __forceinline__ int warp_segment(Mass m, float w, Mass &t) {
    const Mass end = warp_running_sum(m);
    const unsigned hit = __ballot_sync(kFullMask, t < end);
    if (hit) {
        const int at = __ffs(hit) - 1;
        t -= __shfl_sync(kFullMask, end - m, at);
        return at;
    }
    t = ~Mass(0);
    const unsigned some = __ballot_sync(kFullMask, m > 0);
    if (some) return 31 - __clz(some);
    const float top = warp_max(w);
    return top > 0.0f ? __ffs(__ballot_sync(kFullMask, w == top)) - 1 : -1;
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// A row as 16-byte vectors on its own grid: vector q holds columns N q - off ..
// N q - off + N - 1. Vectors [qa, qb) lie in the row; the columns of a partial
// one at either end are loaded one by one, a lane each.
template <typename T>
struct RowGrid {
    static constexpr int N = Vec<T>::kN;
    const T *p;
    int n, off;
    int qa, qb, nq;  // nq vectors in all
    __device__ RowGrid(const T *row, int columns) : p(row), n(columns) {
        off = static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % N);
        qa = off > 0 ? 1 : 0;
        qb = (off + n) / N;
        nq = (off + n + N - 1) / N;
    }
    __device__ int column(int q) const { return N * q - off; }
    __device__ bool whole(int q) const { return q >= qa && q < qb; }
    __device__ bool whole(int q, int end) const { return q >= qa && end <= qb; }
    __device__ uint4 load(int q) const { return ld_stream_u4(reinterpret_cast<const uint4 *>(p - off) + q); }
    // for vectors a lane apart by several: each line is asked for by several loads
    __device__ uint4 load_cached(int q) const { return __ldg(reinterpret_cast<const uint4 *>(p - off) + q); }
    // lane i's column of the partial vector q, -1 if it has none
    __device__ int edge_column(int q, int lane) const {
        const int j = column(q) + lane;
        return lane < N && j >= 0 && j < n ? j : -1;
    }
    __device__ float at(int j) const { return Vec<T>::to_float(p[j]); }
};

// What a column weighs in a draw: 2^((x - m) k), a looked-up draft's column
// (skip) 0; or, kResidual, what its draft row leaves of it, max(0, p - q).
struct Weigh {
    float m, k;        // the largest that may be drawn, and the row's factor
    int skip;          // -1: none
    float c, mq, cq;   // kResidual: -log2 s, the draft row's max and its -log2 s
};

// The weights of a vector's columns, from column j on; x - m first, as the
// row's states take it.
template <typename T, bool kResidual>
__device__ __forceinline__ void weights_of(float (&e)[Vec<T>::kN], const uint4 &x, const uint4 &y, int j, const Weigh &w) {
    const float2 nm = make_float2(-w.m, -w.m), kk = make_float2(w.k, w.k);
#pragma unroll
    for (int i = 0; i < Vec<T>::kN / 2; ++i) {
        const float2 dx = __fadd2_rn(Vec<T>::pair(x, i), nm);
        if (kResidual) {
            // both by the same instructions: rows that are the same leave exactly nothing
            const float2 dy = __fadd2_rn(Vec<T>::pair(y, i), make_float2(-w.mq, -w.mq));
            const float2 p = __ffma2_rn(dx, kk, make_float2(w.c, w.c)), q = __ffma2_rn(dy, kk, make_float2(w.cq, w.cq));
            e[2 * i] = fmaxf(0.0f, ex2_ftz(p.x) - ex2_ftz(q.x));
            e[2 * i + 1] = fmaxf(0.0f, ex2_ftz(p.y) - ex2_ftz(q.y));
        } else {
            const float2 p = __fmul2_rn(dx, kk);
            e[2 * i] = j + 2 * i == w.skip ? 0.0f : ex2_ftz(p.x);
            e[2 * i + 1] = j + 2 * i + 1 == w.skip ? 0.0f : ex2_ftz(p.y);
        }
    }
}
template <int kN>
__device__ __forceinline__ float sum_of(const float (&e)[kN]) {
    float2 s = make_float2(e[0], e[1]);
#pragma unroll
    for (int i = 2; i < kN; i += 2) s = __fadd2_rn(s, make_float2(e[i], e[i + 1]));
    return s.x + s.y;
}

// The columns of a draft row beside a row's: its vectors, or parts of two of
// them where the two rows start at different phases of 16 bytes.
template <typename T>
struct Beside {
    static constexpr int N = Vec<T>::kN;
    const RowGrid<T> &d;
    int by, r;  // columns of vector q start at element r of the draft row's vector q + by
    __device__ Beside(const RowGrid<T> &g, const RowGrid<T> &d_) : d(d_) {
        r = (d.off - g.off + N) % N;
        by = d.off < g.off ? -1 : 0;
        lo = max(g.qa, d.qa - by);
        hi = max(lo, min(g.qb, d.qb - by - (r ? 1 : 0)));
    }
    // the vectors [lo, hi) are whole, the row's and what lies beside them
    int lo, hi;
    __device__ uint4 load(int q) const {
        const uint4 v = d.load(q + by);
        return r == 0 ? v : shift_pair<T>(v, d.load(q + by + 1), r);
    }
};

// N columns of a row from column j on, those outside it -inf, one by one.
template <typename T>
__device__ __noinline__ uint4 columns_from(const T *p, int n, int j) {
    uint4 v = Vec<T>::lowest();
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; i += 2) {
        float2 f = make_float2(-INFINITY, -INFINITY);
        if (j + i >= 0 && j + i < n) f.x = Vec<T>::to_float(p[j + i]);
        if (j + i + 1 >= 0 && j + i + 1 < n) f.y = Vec<T>::to_float(p[j + i + 1]);
        Vec<T>::set_pair(v, i / 2, f);
    }
    return v;
}

// Walking kN segments of one lane: the one that holds t, and t from its start on;
// for a t behind the last mass the last that weighs anything.
template <int kN>
__device__ __forceinline__ int walk(const float (&w)[kN], float unit, Mass &t) {
    int at = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const Mass m = mass_of(w[i], unit);
        if (!found && w[i] > 0.0f) at = i;
        if (!found && t < m) found = true;
        if (!found) t -= m;
    }
    if (!found) t = ~Mass(0);
    return at;
}

// The column of step `step` whose weight holds t, and its logit, by a CTA of
// kScan warps: a warp weighs 32 of the step's vectors, a lane one; every warp
// finds the warp that holds t, and that one the lane and the lane the column. One
// latency, and eight weights a lane, of a request that has the CTA to itself: 1.1
// us. `mine` in that warp only; its column is -1 if nothing weighs anything.
struct Found {
    bool mine;
    int column;
    float x;
};
template <typename T, bool kResidual>
__device__ __forceinline__ Found column_of(const RowGrid<T> &g, const RowGrid<T> &d, int step, const Weigh &w, Mass t,
                                           float *sums) {
    constexpr int N = Vec<T>::kN;
    constexpr float kUnit = kResidual ? kUnitShares : kUnitWeights;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = step * kStep + 32 * warp + lane;
    const Beside<T> beside(g, d);
    uint4 x = Vec<T>::lowest(), y = x;
    if (g.whole(q))
        x = g.load(q);
    else if (q < g.nq)
        x = columns_from(g.p, g.n, g.column(q));
    if (kResidual) {
        if (q >= beside.lo && q < beside.hi)
            y = beside.load(q);
        else if (q < g.nq)
            y = columns_from(d.p, d.n, g.column(q));
    }
    float e[N];
    weights_of<T, kResidual>(e, x, y, g.column(q), w);
    const float mine = sum_of(e), all = warp_sum(mine);
    if (lane == 0) sums[warp] = all;
    __syncthreads();
    float of[kScan];
#pragma unroll
    for (int i = 0; i < kScan; ++i) of[i] = sums[i];
    if (walk(of, kUnit, t) != warp) return Found{false, -1, 0.0f};
    const int l = warp_segment(mass_of(mine, kUnit), mine, t);
    if (l < 0) return Found{true, -1, 0.0f};
    const int at = walk(e, kUnit, t);
    float found = 0.0f;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 xx = Vec<T>::pair(x, i);
        if (2 * i == at) found = xx.x;
        if (2 * i + 1 == at) found = xx.y;
    }
    return Found{true, __shfl_sync(kFullMask, g.column(q) + at, l), __shfl_sync(kFullMask, found, l)};
}

// The first column of step `step` that holds m, by a warp.
template <typename T>
__device__ __forceinline__ int first_of(const RowGrid<T> &g, int step, float m) {
    constexpr int N = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    uint4 x[kScan];
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
        const int q = step * kStep + 32 * u + lane;
        x[u] = g.whole(q) ? g.load(q) : Vec<T>::lowest();
    }
#pragma unroll 1
    for (int u = 0; u < kScan; ++u) {
        const int q = step * kStep + 32 * u + lane;
        if (q < g.nq && !g.whole(q)) x[0] = columns_from(g.p, g.n, g.column(q));
        unsigned at = 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 xx = Vec<T>::pair(x[0], i);
            at |= (xx.x == m ? 1u : 0u) << (2 * i) | (xx.y == m ? 2u : 0u) << (2 * i);
        }
        const unsigned some = __ballot_sync(kFullMask, at != 0);
        if (some) return __shfl_sync(kFullMask, g.column(q) + __ffs(at) - 1, __ffs(some) - 1);
#pragma unroll
        for (int i = 0; i + 1 < kScan; ++i) x[i] = x[i + 1];
    }
    return -1;
}

// One step of a scan: vectors q .. q + kStep - 1 (those below nq) into a state,
// column `skip` (-1: none) left out.
template <typename T>
__device__ __forceinline__ void scan_step(TokState &st, const RowGrid<T> &g, int q, int skip, int lane, float k) {
    constexpr int N = Vec<T>::kN;
    uint4 v[kScan];
    const bool whole = g.whole(q, q + kStep);
    int head = -1, tail = -1;  // of the row's partial vectors, a column a lane
    if (whole) {
#pragma unroll
        for (int u = 0; u < kScan; ++u) v[u] = g.load(q + 32 * u + lane);
    } else {
#pragma unroll
        for (int u = 0; u < kScan; ++u) {
            const int i = q + 32 * u + lane;
            v[u] = g.whole(i) ? g.load(i) : Vec<T>::lowest();
        }
        head = q == 0 && g.qa > 0 ? g.edge_column(0, lane) : -1;
        tail = g.qb < g.nq && g.qb >= max(q, g.qa) && g.qb < q + kStep ? g.edge_column(g.qb, lane) : -1;
        // on their way beside the vectors, no register held
        if (head >= 0) prefetch_l1(g.p + head);
        if (tail >= 0) prefetch_l1(g.p + tail);
    }
    const int skip_q = skip < 0 ? -1 : (skip + g.off) / N;
    if (skip_q >= q && skip_q < q + kStep) {
        const int at = skip + g.off - N * skip_q;
#pragma unroll
        for (int u = 0; u < kScan; ++u)
            if (q + 32 * u + lane == skip_q) {
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    float2 f = Vec<T>::pair(v[u], i);
                    if (2 * i == at) f.x = -INFINITY;
                    if (2 * i + 1 == at) f.y = -INFINITY;
                    Vec<T>::set_pair(v[u], i, f);
                }
            }
    }
    tok_push<T, false, kScan>(st, v, k);
    if (!whole) {
        if (head >= 0 && head != skip) tok_push1<false>(st, g.at(head), k);
        if (tail >= 0 && tail != skip) tok_push1<false>(st, g.at(tail), k);
    }
}

// A row's temperature as its arithmetic takes it; `ok`: 0 or in range.
struct Heat {
    float k, inv_t;
    bool greedy, ok;
    __device__ explicit Heat(float t) {
        greedy = t == 0.0f;
        ok = greedy || (t >= 1e-6f && t <= 1e6f);
        inv_t = 1.0f;
        k = 1.44269504f;
        if (ok && !greedy) {
            // log2(e) / T to a last place: log2(e) in two parts
            inv_t = 1.0f / t;
            k = 1.44269504f * inv_t;
            k += __fmaf_rn(-k, t, 1.44269504f) * inv_t + 1.92596299e-8f * inv_t;
        }
    }
};
__device__ __forceinline__ float temperature_of(const ChoiceArgs &a, int64_t row) {
    return a.temperatures ? a.temperatures[row] : a.temperature;
}

template <typename T>
__device__ __forceinline__ RowGrid<T> target_row(const ChoiceArgs &a, int64_t row) {
    return RowGrid<T>(static_cast<const T *>(a.logits) + row * a.stride, a.vocab);
}
template <typename T>
__device__ __forceinline__ RowGrid<T> draft_row(const ChoiceArgs &a, int64_t row) {
    return RowGrid<T>(static_cast<const T *>(a.draft_logits) + row * a.draft_stride, a.vocab);
}
// Step states of a target row, and of a draft row (behind all target rows').
__device__ __forceinline__ float2 *states_of(const ChoiceArgs &a, int64_t row) { return a.states + row * a.steps; }
__device__ __forceinline__ float2 *draft_states_of(const ChoiceArgs &a, int64_t row) {
    return a.states + (a.rows + row) * a.steps;
}

// A row that emits nothing.
__device__ __forceinline__ void silence(const ChoiceArgs &a, int64_t row) {
    a.tokens[row] = -1;
    if (a.logp) a.logp[row] = 0.0f;
}

// k_states: HBM-bound (591 MB of bf16 rows 87 us, 6.8 TB/s; 78 MB 14 us, as a plain
// read of them). A warp per `unit` steps of a row: (m, s) of each step, its m the
// largest value up to the step's end. Rows [0, rows) are the target's, and, of a
// verification with draft logits, rows [rows, 2 rows) the drafts'; a row in no
// request, and the draft row of a row without a draft, are not read. A row of a
// verification emits nothing until k_decide gives it a token, whatever the offsets
// hold.
template <typename T>
__global__ void __launch_bounds__(kThreads, 8) k_states(ChoiceArgs a, int unit, int units, int64_t warps) {
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t id = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5);
    if (id >= warps) return;
    int64_t row = id / units;
    const int first = static_cast<int>(id - row * units) * unit;
    int skip = -1;
    bool draft = false;
    float temperature = a.temperature;
    if (a.offsets) {
        draft = row >= a.rows;
        if (draft)
            row -= a.rows;
        else if (first == 0 && lane == 0)
            silence(a, row);
        // asked for together: one latency before the row's own
        const int64_t lo = a.offsets[0], hi = a.offsets[a.requests], d = a.drafts[row];
        temperature = temperature_of(a, row);
        const bool drafted = d >= 0 && d < a.vocab && temperature != 0.0f;
        if (row < lo || row >= hi || (draft && !drafted)) return;
        if (!a.draft_logits && drafted) skip = static_cast<int>(d);
    } else {
        temperature = temperature_of(a, row);
    }
    const RowGrid<T> g = draft ? draft_row<T>(a, row) : target_row<T>(a, row);
    const Heat heat(temperature);
    const int n = min(unit, (g.nq + kStep - 1) / kStep - first);
    TokState st = tok_empty();
    float2 mine = make_float2(-INFINITY, 0.0f);
    for (int i = 0; i < n; ++i) {
        scan_step(st, g, (first + i) * kStep, skip, lane, heat.k);
        st = tok_warp_reduce<false>(st, heat.k);
        if (lane == i) mine = make_float2(st.m, st.s);
        st.s = 0.0f;
    }
    // a row of another phase may have a step less: an empty one
    if (lane < unit && first + lane < a.steps)
        (draft ? draft_states_of(a, row) : states_of(a, row))[first + lane] = mine;
}

// A row's step states, by a warp: lane l holds steps l cnt .. l cnt + cnt - 1, the
// first kHeld of them at hand (all of them up to 32 kHeld steps: 262144 f32
// columns, or 524288 of 16 bits).
constexpr int kHeld = 8;
template <bool kShared>
struct StepsOf {
    const float2 *p;
    int n, cnt, first;
    float2 held[kHeld];
    // past L1 where another SM has written them, and may write over them
    __device__ static float2 get(const float2 *at) { return kShared ? *at : __ldcg(at); }
    __device__ StepsOf(const float2 *states, int steps) : p(states), n(steps) {
        cnt = (steps + 31) / 32;
        first = static_cast<int>(threadIdx.x & 31) * cnt;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = i < cnt && first + i < n ? get(p + first + i) : make_float2(-INFINITY, 0.0f);
    }
    // fn(state, i) for each of the lane's steps i, in order
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) const {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < cnt) fn(held[i], i);
        for (int i = kHeld; i < cnt; ++i)
            if (first + i < n) fn(get(p + first + i), i);
    }
    __device__ TokState merged(float k) const {
        float m = -INFINITY, s = 0.0f;
        each([&](float2 v, int) { m = fmaxf(m, v.x); });
        m = warp_max(m);
        const float mm = m == -INFINITY ? 0.0f : m;
        each([&](float2 v, int) { s += v.y * ex2_ftz((v.x - mm) * k); });
        return TokState{m, warp_sum(s), 0.0f};
    }
    // The step that u of all steps' weights falls in, and t from its start on; -1
    // if nothing weighs anything.
    template <typename Weight>
    __device__ __forceinline__ int draw(float unit, float u, Weight weight, Mass &t) const {
        Mass mine = 0;
        each([&](float2 v, int) { mine += mass_of(weight(v), unit); });
        const Mass upto = warp_running_sum(mine), total = __shfl_sync(kFullMask, upto, 31);
        t = part_of_total(u, total);
        if (total == 0) return -1;
        const int l = __ffs(__ballot_sync(kFullMask, t < upto)) - 1;
        Mass rest = t - (upto - mine);  // lane l's
        int at = 0;
        bool found = false;
        each([&](float2 v, int i) {
            const Mass m = mass_of(weight(v), unit);
            if (!found && rest < m) found = true, at = i;
            if (!found) rest -= m;
        });
        t = __shfl_sync(kFullMask, rest, l);
        return __shfl_sync(kFullMask, first + at, l);
    }
};
using Steps = StepsOf<false>;
__device__ __forceinline__ bool is_distribution(const TokState &st) { return isfinite(st.m) && !isnan(st.s); }

// The row's first largest column: the first step that comes to it.
template <typename T, bool kShared>
__device__ __forceinline__ int first_largest(const RowGrid<T> &g, const StepsOf<kShared> &steps, float m) {
    int mine = -1;
    steps.each([&](float2 v, int i) {
        if (mine < 0 && v.x == m) mine = steps.first + i;
    });
    const unsigned some = __ballot_sync(kFullMask, mine >= 0);
    return some ? first_of(g, __shfl_sync(kFullMask, mine, __ffs(some) - 1), m) : -1;
}

// The step that u of a row's own weights falls in.
template <bool kShared>
__device__ __forceinline__ int own_step(const StepsOf<kShared> &steps, const Weigh &w, float u, Mass &t) {
    return steps.draw(kUnitWeights, u, [&](float2 v) { return v.y * ex2_ftz((v.x - w.m) * w.k); }, t);
}

__device__ __forceinline__ float logp_of(float x, const TokState &st, const Heat &heat) {
    return heat.greedy ? 0.0f : (x - st.m) * heat.inv_t - logf(st.s);
}

// A row's token, by a warp. A lane weighs eight vectors that lie side by side, so
// one running sum over the lanes, then the lane's vectors and the vector's columns.
template <typename T, bool kShared>
__device__ __forceinline__ void draw_token(const ChoiceArgs &a, int64_t row, const RowGrid<T> &g, const Heat &heat, float u,
                                           const float2 *states) {
    constexpr int N = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    const StepsOf<kShared> steps(states, a.steps);
    const TokState st = steps.merged(heat.k);
    int column = -1;
    float logp = nan_f();
    if (heat.ok && is_distribution(st)) {
        if (heat.greedy) {
            column = first_largest(g, steps, st.m);
            logp = 0.0f;
        } else {
            const Weigh w{st.m, heat.k, -1, 0.0f, 0.0f, 0.0f};
            Mass t;
            const int q = own_step(steps, w, u, t) * kStep + kScan * lane;
            uint4 x[kScan];
#pragma unroll
            for (int i = 0; i < kScan; ++i) x[i] = g.whole(q + i) ? g.load_cached(q + i) : Vec<T>::lowest();
            if (q < g.qa || q + kScan > g.qb) {
#pragma unroll
                for (int i = 0; i < kScan; ++i)
                    if (q + i < g.nq && !g.whole(q + i)) x[i] = columns_from(g.p, g.n, g.column(q + i));
            }
            float sum[kScan], all = 0.0f, e[N];
            Mass m = 0;
#pragma unroll
            for (int i = 0; i < kScan; ++i) {
                weights_of<T, false>(e, x[i], x[i], 0, w);
                sum[i] = sum_of(e);
                all += sum[i];
                m += mass_of(sum[i], kUnitWeights);
            }
            const int l = warp_segment(m, all, t);
            if (l >= 0) {
                const int at = walk(sum, kUnitWeights, t);
                uint4 v = x[0];
#pragma unroll
                for (int i = 1; i < kScan; ++i)
                    if (i == at) v = x[i];
                weights_of<T, false>(e, v, v, 0, w);
                const int j = walk(e, kUnitWeights, t);
                float xj = 0.0f;
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const float2 xx = Vec<T>::pair(v, i);
                    if (2 * i == j) xj = xx.x;
                    if (2 * i + 1 == j) xj = xx.y;
                }
                column = __shfl_sync(kFullMask, g.column(q + at) + j, l);
                logp = logp_of(__shfl_sync(kFullMask, xj, l), st, heat);
            }
        }
    }
    if (lane == 0) {
        a.tokens[row] = column;
        if (a.logp) a.logp[row] = logp;
        if (column < 0) count_bad();
    }
}

// k_sample: a warp per row, behind k_states. Bound by a row's latencies, over the
// warps resident: a CTA of eight warps per row, as k_decide draws, takes 20.1 us
// for 19.3 (whole calls, 256 x 151936 bf16), 42.3 for 37.1 (1024 x 50257 f32), 18.9
// for 9.1 (2048 x 1076 bf16).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(ChoiceArgs a) {
    const int64_t row = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    const RowGrid<T> g = target_row<T>(a, row);
    const Heat heat(temperature_of(a, row));
    const float u = a.uniforms[row];
    wait_prerequisites();
    draw_token<T, false>(a, row, g, heat, u, states_of(a, row));
}

// k_sample_row: a row of at most 32 steps by one CTA, a warp a step: the states
// stay in shared memory, and one launch does. Taken while the SMs hold the warps,
// 32 each, and short rows somewhat longer (us, on the GPU, k_states and k_sample /
// this, 152 / 600 / 2048 rows: of 1000 f32, one step, 5.3 / 4.1, 5.6 / 4.8, 8.7 /
// 6.9; of 8000 bf16, four, 5.9 / 4.8, 7.8 / 6.3, 14.0 / 12.8; of 16000, eight, 6.3 /
// 5.3, 10.1 / 7.7, 18.8 / 21.4; of 32000, sixteen, 7.7 / 6.5, 13.4 / 13.9, 29.8 /
// 39.6).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_sample_row(ChoiceArgs a) {
    __shared__ float2 states[kRowSteps];
    const int64_t row = blockIdx.x;
    const RowGrid<T> g = target_row<T>(a, row);
    const float u = a.uniforms[row];
    const Heat heat(temperature_of(a, row));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < a.steps) {
        TokState st = tok_empty();
        scan_step(st, g, warp * kStep, -1, lane, heat.k);
        st = tok_warp_reduce<false>(st, heat.k);
        if (lane == 0) states[warp] = make_float2(st.m, st.s);
    }
    __syncthreads();
    if (warp == 0) draw_token<T, true>(a, row, g, heat, u, states);
}

// What becomes of a row: its draft is accepted; or it ends its request, with a
// token that is known (-1, or a greedy row's largest), that comes from p, or that
// comes from what q leaves of p. Of a row that ends its request kOdd: something of
// it is to be counted.
enum Verdict : int { kAccepted = 0, kKnown = 1, kFromOwn = 2, kFromRest = 3, kOdd = 4 };
struct Open {  // of a row whose token is still to be drawn
    Weigh w;
    float m, inv_t, s, u;  // m: the row's max, of w.m's columns and a looked-up draft's
    int step;  // kLookup: where u falls, and t from its start on
    Mass t;
};

// A row's own inputs, asked for before the states are there.
struct RowNumbers {
    int64_t draft;
    float accept, u, xd, yd;
    Heat heat;
    int d;  // the draft, -1: none
};
template <typename T, bool kLookup>
__device__ __forceinline__ RowNumbers row_numbers(const ChoiceArgs &a, int64_t row) {
    RowNumbers r{a.drafts[row], a.uniforms[2 * row], a.uniforms[2 * row + 1], 0.0f, 0.0f, Heat(temperature_of(a, row)), -1};
    r.d = r.draft >= 0 && r.draft < a.vocab ? static_cast<int>(r.draft) : -1;
    if (r.d >= 0) {
        r.xd = target_row<T>(a, row).at(r.d);
        if (!kLookup) r.yd = draft_row<T>(a, row).at(r.d);
    }
    return r;
}

// kLookup: a verification without draft rows.
template <typename T, bool kLookup>
__device__ __forceinline__ int judge(const ChoiceArgs &a, int64_t row, const RowNumbers &r, bool writes, Open *open) {
    const int lane = threadIdx.x & 31;
    const Heat heat = r.heat;
    const bool drafted = r.d >= 0 && !heat.greedy, lookup = kLookup && drafted;
    const Steps steps(states_of(a, row), a.steps);
    TokState q{};
    if (!kLookup && drafted) q = Steps(draft_states_of(a, row), a.steps).merged(heat.k);
    TokState p = steps.merged(heat.k);
    const float others = p.m;
    if (lookup) tok_push1<false>(p, r.xd, heat.k);  // its column is not among the states
    Verdict v = kKnown;
    bool odd = r.draft >= a.vocab;
    int token = -1;
    float logp = 0.0f;
    if (!heat.ok || !is_distribution(p)) {
        odd = true;
        logp = nan_f();
    } else if (heat.greedy) {
        token = first_largest(target_row<T>(a, row), steps, p.m);
        if (token == r.d) v = kAccepted;
    } else {
        Open o{};
        // The columns beside a looked-up draft are weighed by the largest of them: their
        // masses would be too coarse beside a draft that holds nearly all of the row (a
        // rest of 2^-18 of it, or less). Where that one itself weighs nothing beside the
        // draft, as where it is masked, none does.
        const float m = lookup && ex2_ftz((others - p.m) * heat.k) > 0.0f ? others : p.m;
        o.w = Weigh{m, heat.k, lookup ? r.d : -1, -log2f(p.s), q.m, -log2f(q.s)};
        o.m = p.m;
        o.inv_t = heat.inv_t;
        o.s = p.s;
        o.u = r.u;
        const bool from = drafted && (lookup || is_distribution(q));  // else not accepted, the token drawn from p
        odd |= drafted && !from;
        const float pd = ex2_ftz((r.xd - p.m) * heat.k) / p.s, qd = lookup ? 1.0f : ex2_ftz((r.yd - q.m) * heat.k) / q.s;
        if (from && pd > 0.0f && r.accept * qd < pd) {
            v = kAccepted;
        } else {
            v = from && !lookup ? kFromRest : kFromOwn;
            // without draft rows all tokens come from p: the step while the states are at
            // hand, in a row that turns out not to be the request's last as well, and its
            // vectors on their way (32 requests of up to 6 drafts of 50257 f32: 10.9 us
            // for 11.4)
            if (kLookup) {
                o.step = own_step(steps, o.w, r.u, o.t);
                const RowGrid<T> g = target_row<T>(a, row);
                const int q = o.step * kStep + kScan * lane;  // a line a lane
                if (o.step >= 0 && q < g.nq) prefetch_l1(g.p - g.off + g.N * q);
            }
        }
        if (v == kAccepted) {
            token = r.d;
            logp = logp_of(r.xd, p, heat);
        } else if (lane == 0) {
            *open = o;
        }
    }
    if (lane == 0 && writes) {
        if (v == kAccepted || v == kKnown) {
            a.tokens[row] = token;
            if (a.logp) a.logp[row] = logp;
        }
    }
    return odd ? v | kOdd : v;
}

// max(0, p - q) added over the columns of half a step; all of a warp. Two
// exponentials a column, at 16 per clock and SM: 30 million columns (235 rows of
// 128256) take 13 us of them.
template <typename T>
__device__ __forceinline__ float residual_of_vectors(const RowGrid<T> &g, const Beside<T> &beside, int q, int from, int to,
                                                     const Weigh &w) {
    constexpr int kU = kScan / 2;
    const int lane = threadIdx.x & 31;
    uint4 x[kU], y[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int v = q + 32 * u + lane;
        x[u] = v >= from && v < to ? g.load(v) : Vec<T>::lowest();
        y[u] = v >= from && v < to ? beside.load(v) : Vec<T>::lowest();
    }
    float sum = 0.0f, e[Vec<T>::kN];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        weights_of<T, true>(e, x[u], y[u], 0, w);
        sum += sum_of(e);
    }
    return sum;
}
// The half of a step that holds an end of the row, or of the whole vectors beside
// it: what is left of either end a column a lane, at most three vectors, or all of
// a row that is hardly longer.
template <typename T>
__device__ __noinline__ float residual_at_end(const T *p, const T *draft, int n, int q, const Weigh &w) {
    const RowGrid<T> g(p, n), d(draft, n);
    const Beside<T> beside(g, d);
    const int lane = threadIdx.x & 31, end = min(g.nq, q + 32 * (kScan / 2));
    float sum = 0.0f;
    auto columns = [&](int from, int to) {
        for (int j = max(0, g.column(from)) + lane; j < min(n, g.column(to)); j += 32)
            sum += fmaxf(0.0f, ex2_ftz(__fmaf_rn(g.at(j) - w.m, w.k, w.c)) - ex2_ftz(__fmaf_rn(d.at(j) - w.mq, w.k, w.cq)));
    };
    if (q < beside.lo) columns(q, min(end, beside.lo));
    if (end > beside.hi) columns(max(q, beside.hi), end);
    return sum + residual_of_vectors(g, beside, q, beside.lo, min(end, beside.hi), w);
}
template <typename T>
__device__ __forceinline__ float residual_of_half(const RowGrid<T> &g, const RowGrid<T> &d, const Beside<T> &beside, int half,
                                                  const Weigh &w) {
    const int q = half * 32 * (kScan / 2), end = min(g.nq, q + 32 * (kScan / 2));
    return warp_sum(q >= beside.lo && end <= beside.hi ? residual_of_vectors(g, beside, q, q, end, w)
                                                       : residual_at_end(g.p, d.p, g.n, q, w));
}

// k_decide: a cluster per request, behind k_states. Every CTA's warps judge a row
// each, in order, until one accepts no draft (the CTAs of a cluster come to the
// same; the first writes). That row's token is then drawn: from p by the first
// CTA; where it comes from what q leaves of p, the cluster's warps add that up
// over the row's steps first.
template <typename T, bool kLookup>
__global__ void __launch_bounds__(kDrawThreads, 4) k_decide(ChoiceArgs a) {
    constexpr int kRows = kDrawThreads / 32;
    __shared__ int verdicts[kRows];
    __shared__ Open opens[kRows];
    __shared__ float sums[kScan];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int64_t s = cluster_id_x(), lo = a.offsets[0], hi = a.offsets[a.requests];
    const int64_t r0 = a.offsets[s], r1 = a.offsets[s + 1];
    const bool good = r0 >= 0 && r1 >= r0 && r1 <= a.rows, writes = rank == 0;
    // a row outside [lo, hi) has no states: of a table that decreases
    auto has_states = [&](int64_t row) { return good && row < r1 && row >= lo && row < hi; };
    RowNumbers numbers{0, 0.0f, 0.0f, 0.0f, 0.0f, Heat(1.0f), -1};
    if (has_states(r0 + warp)) numbers = row_numbers<T, kLookup>(a, r0 + warp);
    wait_prerequisites();
    int64_t stop = good ? -1 : 0;
    int by = 0, verdict = kAccepted;  // the warp that judged row `stop`, and what it came to
    for (int64_t r = r0; good && r < r1 && stop < 0; r += kRows) {
        const int64_t row = r + warp;
        int v = kKnown;
        if (r > r0) __syncthreads();  // the verdicts before have been read
        if (has_states(row)) {
            if (r > r0) numbers = row_numbers<T, kLookup>(a, row);
            v = judge<T, kLookup>(a, row, numbers, writes, &opens[warp]);
        }
        if (lane == 0) verdicts[warp] = v;
        __syncthreads();
        for (int i = 0; i < kRows && r + i < r1; ++i)
            if (verdicts[i] != kAccepted) {
                stop = r + i;
                verdict = verdicts[i];
                by = i;
                break;
            }
    }
    if (stop < 0) stop = r1;
    if (writes) {
        if (threadIdx.x == 0) {
            a.accepted[s] = good ? stop - r0 : -1;
            if (!good || (verdict & kOdd)) count_bad();
        }
        // rows judged beside it that lie behind it
        const int64_t behind = stop + 1 + threadIdx.x;
        if (good && behind < min(r1, stop - by + kRows)) silence(a, behind);
    }
    verdict &= ~kOdd;
    if (verdict == kAccepted || verdict == kKnown) return;
    const Open o = opens[by];
    const bool rest = !kLookup && verdict == kFromRest;
    const RowGrid<T> g = target_row<T>(a, stop);
    Found f{};
    int step = o.step;
    Mass t = o.t;
    bool own = !rest;
    if (rest) {
        const RowGrid<T> d = draft_row<T>(a, stop);
        const Beside<T> beside(g, d);
        float2 *states = draft_states_of(a, stop);  // the draft row's have served: the steps' sums go over them
        if (C > 1) {  // every CTA has read them
            cluster_arrive();
            cluster_wait();
        }
        float *halves = reinterpret_cast<float *>(states);
        for (int i = static_cast<int>(rank) * kRows + warp; i < 2 * a.steps; i += static_cast<int>(C) * kRows) {
            const float sum = residual_of_half(g, d, beside, i, o.w);
            if (lane == 0) __stcg(halves + i, sum);
        }
        if (C > 1) {
            cluster_arrive_release();
            cluster_wait();
        } else {
            __syncthreads();
        }
        if (!writes) return;
        // steps the halves of which lie behind the row were given sums of 0
        step = Steps(states, a.steps).draw(kUnitShares, o.u, [&](float2 v) { return v.x + v.y; }, t);
        if (step >= 0) {
            f = column_of<T, true>(g, d, step, o.w, t, sums);
        } else {  // nothing left: the two rows are the same, and the draw is from p
            own = true;
        }
    } else if (!writes) {
        return;
    }
    if (own) {
        if (!kLookup) step = own_step(Steps(states_of(a, stop), a.steps), o.w, o.u, t);
        if (step >= 0)
            f = column_of<T, false>(g, g, step, o.w, t, sums);
        else  // nothing but the looked-up draft weighs anything: it is the row's largest
            f = Found{warp == 0, o.w.skip, o.m};
    }
    if (f.mine && lane == 0) {
        a.tokens[stop] = f.column;
        if (a.logp) a.logp[stop] = f.column < 0 ? nan_f() : (f.x - o.m) * o.inv_t - logf(o.s);
    }
}

// ---------------------------------------------------------------------------
// launchers

Launches g_launched;

int elem_size(DType t) { return t == kF32 ? 4 : 2; }

// Steps per warp: as many as let the GPU hold all warps at once, up to four; two
// where that takes more. Measured (us, whole calls, 1 / 2 / 3 / 4 / 6 / 8 / 12
// steps): sample_rows 1 x 32000 bf16 5.7 / 6.3 / 6.9 / 7.6 / 8.8 / 9.9 / 12; 256 x
// 151936 19.2 / 19.1 / 19.4 / 18.7 / 19.2 / 20.2 / 22.3; verify_drafts 32
// requests of up to 6 looked-up drafts of 50257 f32 12.0 / 11.5 / 11.9 / 12.4 /
// 13.5 / 14.9 / 17.7; 256 of up to 7 drafts of 128256 bf16 119.5 / 115.1 / 115.5
// / 115.7 / 116.7 / 115.8 / 118.
int unit_of(int64_t steps, int64_t rows, const DeviceInfo &dev) {
    const int64_t resident = 8 * kWarps * static_cast<int64_t>(dev.sms), unit = (steps * rows + resident - 1) / resident;
    return unit <= 4 ? static_cast<int>(std::max<int64_t>(1, unit)) : 2;
}

template <typename T>
struct Kernels {
    static const void *states() { return reinterpret_cast<const void *>(&k_states<T>); }
    static const void *sample_row() { return reinterpret_cast<const void *>(&k_sample_row<T>); }
    static const void *sample() { return reinterpret_cast<const void *>(&k_sample<T>); }
    static Kernel &decide(bool lookup) {
        static Kernel drawn(reinterpret_cast<const void *>(&k_decide<T, false>), false);
        static Kernel looked_up(reinterpret_cast<const void *>(&k_decide<T, true>), false);
        return lookup ? looked_up : drawn;
    }
};

cudaError_t launch(const void *fn, int64_t ctas, bool dependent, cudaStream_t s, void **args, int threads = kThreads) {
    LaunchConfig l(ctas, threads, 0, dependent, s);
    return cudaLaunchKernelExC(&l.cfg, fn, args);
}
int64_t ctas_of(int64_t warps) { return (warps + kWarps - 1) / kWarps; }

// k_states, a warp per unit of steps of `rows` rows.
cudaError_t launch_states(const void *fn, ChoiceArgs &a, int64_t rows, const DeviceInfo &dev, cudaStream_t s) {
    int unit = unit_of(a.steps, rows, dev);
    int units = (a.steps + unit - 1) / unit;
    int64_t warps = rows * units;
    void *args[] = {&a, &unit, &units, &warps};
    return launch(fn, ctas_of(warps), false, s, args);
}

template <typename T>
cudaError_t sample_as(ChoiceArgs a, const DeviceInfo &dev, cudaStream_t s) {
    void *args[] = {&a};
    if (a.steps <= kRowSteps && a.rows * a.steps <= (a.steps <= 8 ? 56 : 32) * static_cast<int64_t>(dev.sms))
        return launch(Kernels<T>::sample_row(), a.rows, false, s, args, 32 * a.steps);
    if (cudaError_t e = launch_states(Kernels<T>::states(), a, a.rows, dev, s); e != cudaSuccess) return e;
    return launch(Kernels<T>::sample(), ctas_of(a.rows), true, s, args);
}

template <typename T>
cudaError_t verify_as(ChoiceArgs a, const DeviceInfo &dev, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const bool drawn = a.draft_logits != nullptr;
    if (a.rows > 0 && (e = launch_states(Kernels<T>::states(), a, drawn ? 2 * a.rows : a.rows, dev, s))) return e;
    // CTAs per request: three an SM or more (it holds four), with half a step for each
    // of their warps. Measured (us, whole calls, 1 / 2 / 4 / 8): 64 requests of up to 4
    // drafts of 151936 bf16 53.2 / 42.0 / 39.0 / 39.0; 256 of up to 7 of 128256 125 /
    // 116 / 119 / 126.
    int c = 1;
    while (drawn && c < kMaxCluster && c * a.requests < 3 * dev.sms && c * (kDrawThreads / 32) <= a.steps) c *= 2;
    if (a.requests == 0) return cudaSuccess;
    Kernel &k = Kernels<T>::decide(!drawn);
    if ((e = ready(k, dev))) return e;
    void *args[] = {&a};
    LaunchConfig l(a.requests * c, kDrawThreads, c, a.rows > 0, s);
    return cudaLaunchKernelExC(&l.cfg, k.fn, args);
}

}  // namespace

// The scratch: step states of the target rows, then of the draft rows.
int64_t choice_steps(DType t, int64_t vocab) {
    const int N = 16 / elem_size(t);
    return ((vocab + 2 * N - 2) / N + kStep - 1) / kStep;
}
int64_t choice_bytes(DType t, int64_t rows, int64_t vocab, int64_t requests) {
    const int64_t states = 8 * rows * choice_steps(t, vocab);
    return requests < 0 ? states : 2 * states;
}
static void lay_out(DType t, ChoiceArgs &a, void *work) {
    a.steps = static_cast<int>(choice_steps(t, a.vocab));
    a.states = static_cast<float2 *>(work);
}

cudaError_t launch_sample(DType t, const ChoiceArgs &a, void *work, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    ChoiceArgs aa = a;
    lay_out(t, aa, work);
    return t == kF32    ? sample_as<float>(aa, dev, s)
           : t == kBF16 ? sample_as<__nv_bfloat16>(aa, dev, s)
                        : sample_as<__half>(aa, dev, s);
}

cudaError_t launch_verify(DType t, const ChoiceArgs &a, void *work, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    ChoiceArgs aa = a;
    lay_out(t, aa, work);
    return t == kF32    ? verify_as<float>(aa, dev, s)
           : t == kBF16 ? verify_as<__nv_bfloat16>(aa, dev, s)
                        : verify_as<__half>(aa, dev, s);
}

cudaError_t read_choice_status(unsigned long long *out, const DeviceInfo &dev, cudaStream_t s) {
    *out = 0ull;
    if (!g_launched.any(dev)) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_choice_status, sizeof(*out), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

cudaError_t reset_choice_status(const DeviceInfo &dev, cudaStream_t s) {
    if (!g_launched.any(dev)) return cudaSuccess;
    static const unsigned long long zero = 0ull;
    return cudaMemcpyToSymbolAsync(g_choice_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace cerows
