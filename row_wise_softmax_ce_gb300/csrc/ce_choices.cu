// ce_choices.cu -- sm_103a kernels of the choices made from a row's softmax, and
// their launchers.
//
//   sample_rows     a token drawn from each row's softmax by a given uniform number
//   verify_drafts   drafted tokens accepted or replaced
//   route_rows      each row's experts and gates
//   route_grad      the gradient of the gates
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
//   k_route            route_rows: 8 to 32 lanes per row, its columns in shared memory
//   k_zero             its counts
//   k_route_grad       route_grad where only the chosen experts get any
//   k_route_grad_full  where all do
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

// [0] rows that are no distribution, bad drafts, temperatures, ranges and experts;
// [1] bounded waits that gave up
__device__ unsigned long long g_choice_status[2];

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

__device__ __forceinline__ void count_bad() { atomicAdd(&g_choice_status[0], 1ull); }

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
    float m, k;        // the row's
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
    __device__ uint4 load_cached(int q) const {
        const uint4 v = d.load_cached(q + by);
        return r == 0 ? v : shift_pair<T>(v, d.load_cached(q + by + 1), r);
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
// finds the warp that holds t, and that one the lane and the lane the column:
// one latency, and eight weights a lane where a warp alone would take 64 (a
// draw of a step by one warp: 4 us, of a residual 6 us). `mine` in that warp
// only; its column is -1 if nothing weighs anything.
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

// k_states: a warp per `unit` steps of a row: (m, s) of each step, its m the
// largest value up to the step's end. Rows [0, rows) are the target's, and, of a
// verification with draft logits, rows [rows, 2 rows) the drafts'; a row in no
// request, and the draft row of a row without a draft, are not read.
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
        if (draft) row -= a.rows;
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
    float inv_t, s, u;
};

// A row's own inputs, asked for before the states are there.
struct RowNumbers {
    int64_t draft;
    float accept, u, xd, yd;
    Heat heat;
    int d;  // the draft, -1: none
};
template <typename T>
__device__ __forceinline__ RowNumbers row_numbers(const ChoiceArgs &a, int64_t row) {
    RowNumbers r{a.drafts[row], a.uniforms[2 * row], a.uniforms[2 * row + 1], 0.0f, 0.0f, Heat(temperature_of(a, row)), -1};
    r.d = r.draft >= 0 && r.draft < a.vocab ? static_cast<int>(r.draft) : -1;
    if (r.d >= 0) {
        r.xd = target_row<T>(a, row).at(r.d);
        if (a.draft_logits) r.yd = draft_row<T>(a, row).at(r.d);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ int judge(const ChoiceArgs &a, int64_t row, const RowNumbers &r, bool writes, Open *open) {
    const int lane = threadIdx.x & 31;
    const Heat heat = r.heat;
    const bool drafted = r.d >= 0 && !heat.greedy, lookup = drafted && a.draft_logits == nullptr;
    const Steps steps(states_of(a, row), a.steps);
    TokState q{};
    if (drafted && !lookup) q = Steps(draft_states_of(a, row), a.steps).merged(heat.k);
    TokState p = steps.merged(heat.k);
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
        o.w = Weigh{p.m, heat.k, lookup ? r.d : -1, -log2f(p.s), q.m, -log2f(q.s)};
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
template <typename T>
__global__ void __launch_bounds__(kDrawThreads, 4) k_decide(ChoiceArgs a) {
    constexpr int kRows = kDrawThreads / 32;
    __shared__ int verdicts[kRows];
    __shared__ Open opens[kRows];
    __shared__ float sums[kScan];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int64_t s = cluster_id_x(), lo = a.offsets[0], hi = a.offsets[a.requests];
    const int64_t r0 = s < a.requests ? a.offsets[s] : 0, r1 = s < a.requests ? a.offsets[s + 1] : 0;
    const bool good = r0 >= 0 && r1 >= r0 && r1 <= a.rows, writes = rank == 0;
    auto silent = [&](int64_t row) {
        a.tokens[row] = -1;
        if (a.logp) a.logp[row] = 0.0f;
    };
    // a row outside [lo, hi) has no states: of a table that decreases
    auto has_states = [&](int64_t row) { return good && row < r1 && row >= lo && row < hi; };
    RowNumbers numbers{0, 0.0f, 0.0f, 0.0f, 0.0f, Heat(1.0f), -1};
    if (has_states(r0 + warp)) numbers = row_numbers<T>(a, r0 + warp);
    wait_prerequisites();
    if (s == 0 && writes)  // rows in no request
        for (int64_t r = threadIdx.x; r < a.rows; r += kDrawThreads)
            if (r < lo || r >= hi) silent(r);
    if (s >= a.requests) return;
    int64_t stop = good ? -1 : 0;
    int by = 0, verdict = kAccepted;  // the warp that judged row `stop`, and what it came to
    for (int64_t r = r0; good && r < r1 && stop < 0; r += kRows) {
        const int64_t row = r + warp;
        int v = kKnown;
        if (r > r0) __syncthreads();  // the verdicts before have been read
        if (has_states(row)) {
            if (r > r0) numbers = row_numbers<T>(a, row);
            v = judge<T>(a, row, numbers, writes, &opens[warp]);
        } else if (row < r1 && writes && lane == 0) {
            silent(row);
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
        for (int64_t r = stop + 1 + threadIdx.x; good && r < r1; r += kDrawThreads) silent(r);
    }
    verdict &= ~kOdd;
    if (verdict == kAccepted || verdict == kKnown) return;
    const Open o = opens[by];
    const bool rest = verdict == kFromRest;
    const RowGrid<T> g = target_row<T>(a, stop);
    Found f{};
    int step;
    Mass t;
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
        step = own_step(Steps(states_of(a, stop), a.steps), o.w, o.u, t);
        if (step >= 0)
            f = column_of<T, false>(g, g, step, o.w, t, sums);
        else  // nothing but the looked-up draft weighs anything: it is the row's largest
            f = Found{warp == 0, o.w.skip, o.w.m};
    }
    if (f.mine && lane == 0) {
        a.tokens[stop] = f.column;
        if (a.logp) a.logp[stop] = f.column < 0 ? nan_f() : (f.x - o.w.m) * o.inv_t - logf(o.s);
    }
}

// ---------------------------------------------------------------------------
// Routing. L lanes per row (32 / L rows per warp side by side), lane i of a row
// holding columns i V .. i V + V - 1 in registers.
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

// V consecutive columns from j on (those below n), -inf elsewhere, as vectors.
template <typename T, int V>
__device__ __forceinline__ void load_columns(uint4 (&v)[V / Vec<T>::kN], const T *p, int j, int n) {
    constexpr int N = Vec<T>::kN;
    static_assert(V % N == 0, "whole vectors");
    if (j + V <= n && (reinterpret_cast<uintptr_t>(p + j) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < V / N; ++i) v[i] = *reinterpret_cast<const uint4 *>(p + j + N * i);
    } else {
#pragma unroll
        for (int i = 0; i < V / N; ++i)
#pragma unroll
            for (int h = 0; h < N / 2; ++h) {
                const int c = j + N * i + 2 * h;
                Vec<T>::set_pair(v[i], h, make_float2(c < n ? Vec<T>::to_float(p[c]) : -INFINITY,
                                                      c + 1 < n ? Vec<T>::to_float(p[c + 1]) : -INFINITY));
            }
    }
}
template <typename T, int V>
__device__ __forceinline__ void unpack_columns(float (&z)[V], const uint4 (&v)[V / Vec<T>::kN]) {
    constexpr int N = Vec<T>::kN;
#pragma unroll
    for (int i = 0; i < V / N; ++i)
#pragma unroll
        for (int h = 0; h < N / 2; ++h) {
            const float2 f = Vec<T>::pair(v[i], h);
            z[N * i + 2 * h] = f.x;
            z[N * i + 2 * h + 1] = f.y;
        }
}

template <typename T, int V>
__device__ __forceinline__ void store_columns(T *p, int j, int n, const float (&z)[V]) {
    constexpr int N = Vec<T>::kN;
    if (j + V <= n && (reinterpret_cast<uintptr_t>(p + j) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < V / N; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int h = 0; h < N / 2; ++h) Vec<T>::set_pair(v, h, make_float2(z[N * i + 2 * h], z[N * i + 2 * h + 1]));
            *reinterpret_cast<uint4 *>(p + j + N * i) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (j + i < n) p[j + i] = Vec<T>::from_float(z[i]);
    }
}

// The L lanes of a row: their largest value (no NaN among them), their sum.
template <int L>
__device__ __forceinline__ float row_max(float v) {
    if constexpr (L == 32) {
        return warp_max(v);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
template <int L>
__device__ __forceinline__ unsigned row_ballot(bool b) {
    const unsigned all = __ballot_sync(kFullMask, b);
    return L == 32 ? all : (all >> (threadIdx.x & 31 & ~(L - 1))) & ((1u << (L & 31)) - 1u);
}
// a NaN wins
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 1 / x to a last place or two
__device__ __forceinline__ float rcp_of(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp_of(float d) { return ex2_ftz(d * 1.44269504f); }
// 1 / (1 + e^-z) without a difference from 1, for any z
__device__ __forceinline__ float sigmoid(float z) { return rcp_of(1.0f + exp_of(-z)); }

// A score over a factor that those of a row (or of its chosen) have in common,
// `top` the largest of their logits: nothing overflows, and what is next to
// nothing beside 1 is not so beside the others.
__device__ __forceinline__ float relative_score(float z, float top, bool sigmoid_scores) {
    if (!sigmoid_scores) return exp_of(z - top);
    return (z > 0.0f ? 1.0f : exp_of(z - fminf(0.0f, top))) * rcp_of(1.0f + exp_of(-fabsf(z)));
}

// The chosen experts' share of their sum from their logits (-inf: none), over the
// row's lanes.
template <int L>
__device__ __forceinline__ float share_of(float z, bool sigmoid_scores) {
    const float top = row_max<L>(z);
    const float e = z > -INFINITY || isnan(z) ? relative_score(z, top, sigmoid_scores) : 0.0f;
    const float all = row_sum<L>(e);
    return e / (all > 0.0f || isnan(all) ? all : 1.0f);
}

// The counts are zeroed by a kernel that k_route, launched as its programmatic
// dependent, runs beside and waits for before it adds to them (a memset before
// k_route: 4 us more).
__global__ void __launch_bounds__(kRouteThreads) k_zero(unsigned long long *counts, int n) {
    launch_dependents();
    for (int j = threadIdx.x; j < n; j += kRouteThreads) counts[j] = 0;
}

// CTAs of an SM, by the columns a lane holds.
__host__ __device__ constexpr int route_ctas(int v) { return v > 16 ? 3 : 4; }
// Floats of a row in shared memory: its lanes' columns, 16 bytes apart by bank.
__host__ __device__ constexpr int route_row(int lanes, int v) { return lanes * (v + 4); }

// k_route: bound by the instructions of the choice, most of them compares at half
// rate. So as many rows as there are slots share a warp's instructions, and a
// lane keeps the largest of each eight of its columns only: the columns lie in
// shared memory, where the lane that gives one looks for it among eight, takes
// it out and has the largest of the rest. Measured (us, 16384 x 256 bf16, k = 8,
// sigmoid scores with a bias, 4 of 8 groups): this 11.6; a row a warp, with each
// lane's two best columns and the value of its third in registers, 16.0. Counts
// add 1.1 us, and 1.4 more with a CTA per 32 rows than with three an SM.
template <typename T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads, route_ctas(V)) k_route(RouteArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int R = 32 / L, kVecs = V / Vec<T>::kN, kBlocks = V / 8, kLane = V + 4;  // rows of a warp
    const int lane = threadIdx.x & 31, sub = lane & (L - 1), row0 = lane & ~(L - 1), E = a.experts, j0 = sub * V;
    const int per = E / a.groups;
    const bool grouped = a.top_groups < a.groups;
    // groups of whole lanes, a power of two of them
    const int wide = per / V;
    const bool by_lanes = grouped && per % V == 0 && (wide & (wide - 1)) == 0 && wide <= L;
    float *all = reinterpret_cast<float *>(smem);
    float *row_keys = all + ((threadIdx.x >> 5) * R + lane / L) * route_row(L, V), *mine = row_keys + sub * kLane;
    float *bias = all + kRouteWarps * R * route_row(L, V);  // as a row, if there is one
    int *counts = reinterpret_cast<int *>(bias + (a.bias ? route_row(L, V) : 0));  // [experts], if wanted
    if (a.bias || a.counts) {
        if (a.bias)
            for (int j = threadIdx.x; j < L * V; j += kRouteThreads) {
                const float b = j < E ? a.bias[j] : 0.0f;
                bias[j / V * kLane + j % V] = isnan(b) ? -INFINITY : b;
            }
        if (a.counts)
            for (int j = threadIdx.x; j < E; j += kRouteThreads) counts[j] = 0;
        __syncthreads();
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps * R;
    for (int64_t first = (blockIdx.x * int64_t(kRouteWarps) + (threadIdx.x >> 5)) * R; first < a.rows; first += step) {
        const int64_t row = first + lane / L;
        float z[V];
        {
            uint4 raw[kVecs];  // -inf for a padding row or none
#pragma unroll
            for (int i = 0; i < kVecs; ++i) raw[i] = Vec<T>::lowest();
            if (row < a.rows && !(a.weights && a.weights[row] == 0.0f))
                load_columns<T, V>(raw, static_cast<const T *>(a.logits) + row * a.stride, j0, E);
            unpack_columns<T, V>(z, raw);
        }
        float m = max_nan(z[0], z[1], z[2]);
#pragma unroll
        for (int i = 3; i + 1 < V; i += 2) m = max_nan(m, z[i], z[i + 1]);
        m = max_nan(m, z[V - 1], z[V - 1]);
        const bool odd = row_ballot<L>(!(m < INFINITY)) != 0;  // a NaN or +inf
        if (odd) {
            m = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = -INFINITY;
        }
        m = row_max<L>(m);
        float rs = 0.0f;  // softmax: 1 / s, where the scores themselves are asked for
        if (!a.sigmoid && (a.bias || !a.renormalise)) {
            const float mm = m == -INFINITY ? 0.0f : m;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) s += exp_of(z[i] - mm);
            rs = rcp_of(row_sum<L>(s));
        }
        // what the choice goes by, from here on in z: the biased score, or, without a
        // bias, the logit, which orders the experts as their scores do and is exact
        if (a.bias) {
            const float *b = bias + sub * kLane;
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(b + i);
                    z[i] = z[i] > -INFINITY ? sigmoid(z[i]) + f.x : -INFINITY;
                    z[i + 1] = z[i + 1] > -INFINITY ? sigmoid(z[i + 1]) + f.y : -INFINITY;
                    z[i + 2] = z[i + 2] > -INFINITY ? sigmoid(z[i + 2]) + f.z : -INFINITY;
                    z[i + 3] = z[i + 3] > -INFINITY ? sigmoid(z[i + 3]) + f.w : -INFINITY;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(b + i);
                    z[i] = z[i] > -INFINITY ? exp_of(z[i] - m) * rs + f.x : -INFINITY;
                    z[i + 1] = z[i + 1] > -INFINITY ? exp_of(z[i + 1] - m) * rs + f.y : -INFINITY;
                    z[i + 2] = z[i + 2] > -INFINITY ? exp_of(z[i + 2] - m) * rs + f.z : -INFINITY;
                    z[i + 3] = z[i + 3] > -INFINITY ? exp_of(z[i + 3] - m) * rs + f.w : -INFINITY;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(mine + i) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
        auto ranked = [&](float v) { return a.bias || v == -INFINITY ? v : relative_score(v, m, a.sigmoid); };
        bool dropped = false;
        if (by_lanes) {
            float g1 = -INFINITY, g2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                g2 = fmaxf(g2, fminf(g1, z[i]));
                g1 = fmaxf(g1, z[i]);
            }
            g1 = ranked(g1);
            g2 = ranked(g2);
            for (int o = 1; o < wide; o <<= 1) {
                const float o1 = __shfl_xor_sync(kFullMask, g1, o), o2 = __shfl_xor_sync(kFullMask, g2, o);
                g2 = fmaxf(fminf(g1, o1), fmaxf(g2, o2));
                g1 = fmaxf(g1, o1);
            }
            const float rank_by = a.group_top == 2 && g2 > -INFINITY ? g1 + g2 : g1;
            const int own = sub / wide;
            int before = 0;
            for (int g = 0; g < a.groups; ++g) {
                const float o = __shfl_sync(kFullMask, rank_by, row0 + g * wide);
                before += o > rank_by || (o == rank_by && g < own);
            }
            dropped = before >= a.top_groups || own >= a.groups;
        } else if (grouped) {
            __syncwarp();
            auto group_score = [&](int g) {
                float g1 = -INFINITY, g2 = -INFINITY;
                for (int j = g * per; j < g * per + per; ++j) {
                    const float v = row_keys[j / V * kLane + j % V];
                    g2 = fmaxf(g2, fminf(v, g1));
                    g1 = fmaxf(g1, v);
                }
                g1 = ranked(g1);
                g2 = ranked(g2);
                return a.group_top == 2 && g2 > -INFINITY ? g1 + g2 : g1;
            };
            // lane i of the row has groups i, i + L, ..
            constexpr int kMost = kMaxGroups / L;
            float rank_by[kMost];
            int before[kMost];
#pragma unroll
            for (int h = 0; h < kMost; ++h) {
                rank_by[h] = sub + h * L < a.groups ? group_score(sub + h * L) : -INFINITY;
                before[h] = 0;
            }
#pragma unroll
            for (int other = 0; other < kMost; ++other)
                for (int l = 0; l < L && other * L + l < a.groups; ++l) {
                    const float o = __shfl_sync(kFullMask, rank_by[other], row0 + l);
#pragma unroll
                    for (int h = 0; h < kMost; ++h)
                        before[h] += o > rank_by[h] || (o == rank_by[h] && other * L + l < sub + h * L);
                }
            unsigned kept = 0;
#pragma unroll
            for (int h = 0; h < kMost; ++h)
                if (sub + h * L < a.groups && before[h] < a.top_groups) kept |= 1u << (sub + h * L);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) kept |= __shfl_xor_sync(kFullMask, kept, o);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j0 + i >= E || !(kept >> ((j0 + i) / per) & 1u)) z[i] = mine[i] = -INFINITY;
        }
        float top_of[kBlocks], best = -INFINITY;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            float t = z[8 * b];
#pragma unroll
            for (int i = 1; i < 8; ++i) t = fmaxf(t, z[8 * b + i]);
            top_of[b] = t;
            best = fmaxf(best, t);
        }
        if (dropped) best = -INFINITY;
        // the k best, one after another: the largest, the lowest column of equals
        int expert = -1;  // lane i of the row: the i-th
        for (int n = 0; n < a.k; ++n) {
            const float top = row_max<L>(best);
            const int owner = __ffs(row_ballot<L>(best == top)) - 1;
            int j = 0;
            if (sub == owner && top > -INFINITY) {
                int block = kBlocks - 1;
#pragma unroll
                for (int b = kBlocks - 2; b >= 0; --b)
                    if (top_of[b] == top) block = b;
                float4 *at = reinterpret_cast<float4 *>(mine + 8 * block);
                const float4 lo = at[0], hi = at[1];
                float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                int i = 7;
                // the second largest of the eight, which is the largest again if two share it
                float one = v[0], rest = -INFINITY;
#pragma unroll
                for (int h = 1; h < 8; ++h) {
                    rest = fmaxf(rest, fminf(one, v[h]));
                    one = fmaxf(one, v[h]);
                }
#pragma unroll
                for (int h = 6; h >= 0; --h)
                    if (v[h] == top) i = h;
                reinterpret_cast<float *>(at)[i] = -INFINITY;
                best = -INFINITY;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    if (b == block) top_of[b] = rest;
                    best = fmaxf(best, top_of[b]);
                }
                j = j0 + 8 * block + i;
            }
            j = __shfl_sync(kFullMask, j, row0 + owner);
            if (sub == n && top > -INFINITY) expert = j;
        }
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        const float zc = expert >= 0 ? Vec<T>::to_float(p[expert]) : -INFINITY;
        float g = a.renormalise ? share_of<L>(zc, a.sigmoid)
                  : expert < 0  ? 0.0f
                  : a.sigmoid   ? sigmoid(zc)
                                : exp_of(zc - m) * rs;
        g = odd ? nan_f() : g * a.scale;
        if (row < a.rows && sub < a.k) {
            a.chosen[row * a.k + sub] = expert;
            a.gates[row * a.k + sub] = g;
        }
        if (odd && sub == 0) count_bad();
        if (a.counts && expert >= 0) atomicAdd(&counts[expert], 1);
        __syncwarp();  // the row's columns are written anew
    }
    if (a.counts) {
        __syncthreads();
        wait_prerequisites();  // k_zero is done
        for (int j = threadIdx.x; j < E; j += kRouteThreads)
            if (counts[j]) atomicAdd(&a.counts[j], static_cast<unsigned long long>(counts[j]));
    }
}

// The gates' gradient: with G = scale * (gradient of the gates), s the scores, c
// the chosen experts, f the chosen's share of their sum and D = sum of f G:
//   renormalised  softmax: dz_c = f (G - D), 0 elsewhere
//                 sigmoid: dz_c = f (G - D) (1 - s_c), 0 elsewhere
//   otherwise     sigmoid: dz_c = s_c (1 - s_c) G, 0 elsewhere
//                 softmax: dz_j = s_j ([j chosen] G - sum of s_c G_c)
// Only the last needs the whole row (k_route_grad_full); the others read the
// chosen experts' logits and write a row that is 0 but for them.
struct Slot {  // lane i of a row: its i-th expert (-1: none) and G there
    int c;
    float G;
};
__device__ __forceinline__ Slot slot_at(const RouteArgs &a, int64_t row, int sub) {
    Slot x{-1, 0.0f};
    if (row < a.rows && sub < a.k && !(a.weights && a.weights[row] == 0.0f)) {
        const int64_t at = a.chosen[row * a.k + sub];
        x.G = a.gates_grad[row * a.k + sub] * a.scale;
        if (at >= a.experts || at < -1)
            count_bad();
        else
            x.c = static_cast<int>(at);
    }
    return x;
}

// k_route_grad: L lanes per row for its slots. A warp's rows are zeroed and
// filled in shared memory in the gradient's type and written in whole vectors,
// side by side in memory where the gradient is dense.
template <typename T, int L>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad(RouteArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int R = 32 / L, N = Vec<T>::kN;
    const int lane = threadIdx.x & 31, sub = lane & (L - 1), E = a.experts;
    const int pitch = (R * E + N - 1) / N;  // vectors of a warp's rows
    uint4 *vecs = reinterpret_cast<uint4 *>(smem) + (threadIdx.x >> 5) * pitch;
    T *rows = reinterpret_cast<T *>(vecs), *mine = rows + lane / L * E;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps * R;
    for (int64_t first = (blockIdx.x * int64_t(kRouteWarps) + (threadIdx.x >> 5)) * R; first < a.rows; first += step) {
        const int64_t row = first + lane / L;
        const Slot x = slot_at(a, row, sub);
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        const float z = x.c >= 0 ? Vec<T>::to_float(p[x.c]) : -INFINITY;
        for (int i = lane; i < pitch; i += 32) vecs[i] = make_uint4(0, 0, 0, 0);
        float v = 0.0f;
        if (a.renormalise) {
            const float f = share_of<L>(z, a.sigmoid);
            const float D = row_sum<L>(x.c >= 0 ? f * x.G : 0.0f);
            v = f * (x.G - D);
            if (a.sigmoid) v *= sigmoid(-z);
        } else {
            v = sigmoid(z) * sigmoid(-z) * x.G;
        }
        // an expert that a row names twice: its first lane adds up the others', in
        // the order of the slots
        unsigned same = __match_any_sync(kFullMask, x.c >= 0 ? lane / L * E + x.c : -1 - lane);
        const bool leads = __ffs(same) - 1 == lane;
        if (__any_sync(kFullMask, !leads)) {
            float sum = 0.0f;
            for (int i = 0; i < 32; ++i) {
                const float o = __shfl_sync(kFullMask, v, i);
                if (same >> i & 1u) sum += o;
            }
            v = sum;
        }
        __syncwarp();
        if (x.c >= 0 && leads) mine[x.c] = Vec<T>::from_float(v);
        __syncwarp();
        T *to = static_cast<T *>(a.grad) + first * a.grad_stride;
        const int here = static_cast<int>(min(int64_t(R), a.rows - first));  // rows
        if (a.grad_stride == E && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
            const int whole = here * E / N;
            for (int i = lane; i < whole; i += 32) reinterpret_cast<uint4 *>(to)[i] = vecs[i];
            for (int i = whole * N + lane; i < here * E; i += 32) to[i] = rows[i];
        } else {
            for (int r = 0; r < here; ++r)
                for (int i = lane; i < E; i += 32) to[r * a.grad_stride + i] = rows[r * E + i];
        }
        __syncwarp();
    }
}

// k_route_grad_full: lanes as in k_route.
template <typename T, int L, int V>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad_full(RouteArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int R = 32 / L, kRow = L * V;
    const int lane = threadIdx.x & 31, sub = lane & (L - 1), E = a.experts, j0 = sub * V;
    float *mine = reinterpret_cast<float *>(smem) + ((threadIdx.x >> 5) * R + lane / L) * kRow;  // this row's gradient
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps * R;
    for (int64_t first = (blockIdx.x * int64_t(kRouteWarps) + (threadIdx.x >> 5)) * R; first < a.rows; first += step) {
        const int64_t row = first + lane / L;
        const bool live = row < a.rows && !(a.weights && a.weights[row] == 0.0f);
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        uint4 raw[V / Vec<T>::kN];
#pragma unroll
        for (int i = 0; i < V / Vec<T>::kN; ++i) raw[i] = Vec<T>::lowest();
        if (live) load_columns<T, V>(raw, p, j0, E);
        const Slot x = slot_at(a, row, sub);
        const float z = x.c >= 0 ? Vec<T>::to_float(p[x.c]) : -INFINITY;
        float out[V];
        unpack_columns<T, V>(out, raw);
        float m = out[0], s = 0.0f;
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, out[i]);
        m = row_max<L>(m);
        if (m == -INFINITY) m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            out[i] = exp_of(out[i] - m);
            s += out[i];
        }
        s = row_sum<L>(s);
        const float rs = s > 0.0f || isnan(s) ? 1.0f / s : 0.0f;
        const float v = x.c >= 0 ? exp_of(z - m) * rs * x.G : 0.0f;
        const float by = -rs * row_sum<L>(v);
        // v is added to its column through shared memory; a column that a row names
        // twice one after the other, in the order of the slots
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(mine + j0 + i) =
                make_float4(out[i] * by, out[i + 1] * by, out[i + 2] * by, out[i + 3] * by);
        __syncwarp();
        const unsigned same = __match_any_sync(kFullMask, x.c >= 0 ? lane / L * kRow + x.c : -1 - lane);
        if (!__any_sync(kFullMask, (same & (same - 1)) != 0)) {
            if (x.c >= 0) mine[x.c] += v;
        } else {
            for (int i = 0; i < a.k; ++i) {
                if (sub == i && x.c >= 0) mine[x.c] += v;
                __syncwarp();
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 o = *reinterpret_cast<const float4 *>(mine + j0 + i);
            out[i] = o.x, out[i + 1] = o.y, out[i + 2] = o.z, out[i + 3] = o.w;
        }
        __syncwarp();
        if (row < a.rows) store_columns<T, V>(static_cast<T *>(a.grad) + row * a.grad_stride, j0, E, out);
    }
}

// ---------------------------------------------------------------------------
// launchers

Launches g_launched;

int elem_size(DType t) { return t == kF32 ? 4 : 2; }

int64_t capped(int64_t clusters, int64_t cap) {
    clusters = std::min<int64_t>(clusters, int64_t(1) << 20);
    return std::max<int64_t>(1, cap > 0 ? std::min(clusters, cap) : clusters);
}

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
    static Kernel &decide() {
        static Kernel k(reinterpret_cast<const void *>(&k_decide<T>), false);
        return k;
    }
};

cudaError_t launch(const void *fn, int64_t ctas, bool dependent, cudaStream_t s, void **args, int threads = kThreads) {
    LaunchConfig l(ctas, threads, 0, dependent, s);
    return cudaLaunchKernelExC(&l.cfg, fn, args);
}
int64_t ctas_of(int64_t warps) { return (warps + kWarps - 1) / kWarps; }

// A pass of a warp per unit of steps over `rows` rows.
cudaError_t launch_steps(const void *fn, ChoiceArgs &a, int64_t rows, bool dependent, const DeviceInfo &dev, cudaStream_t s) {
    int unit = unit_of(a.steps, rows, dev);
    int units = (a.steps + unit - 1) / unit;
    int64_t warps = rows * units;
    void *args[] = {&a, &unit, &units, &warps};
    return launch(fn, ctas_of(warps), dependent, s, args);
}

template <typename T>
cudaError_t sample_as(ChoiceArgs a, const DeviceInfo &dev, cudaStream_t s) {
    void *args[] = {&a};
    if (a.steps <= kRowSteps && a.rows * a.steps <= (a.steps <= 8 ? 56 : 32) * static_cast<int64_t>(dev.sms))
        return launch(Kernels<T>::sample_row(), a.rows, false, s, args, 32 * a.steps);
    if (cudaError_t e = launch_steps(Kernels<T>::states(), a, a.rows, false, dev, s); e != cudaSuccess) return e;
    return launch(Kernels<T>::sample(), ctas_of(a.rows), true, s, args);
}

template <typename T>
cudaError_t verify_as(ChoiceArgs a, const DeviceInfo &dev, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const bool drawn = a.draft_logits != nullptr;
    if (a.rows > 0 && (e = launch_steps(Kernels<T>::states(), a, drawn ? 2 * a.rows : a.rows, false, dev, s))) return e;
    // CTAs per request: three an SM or more (it holds four), with half a step for each
    // of their warps. Measured (us, whole calls, 1 / 2 / 4 / 8): 64 requests of up to 4
    // drafts of 151936 bf16 53.2 / 42.0 / 39.0 / 39.0; 256 of up to 7 of 128256 125 /
    // 116 / 119 / 126.
    int c = 1;
    while (drawn && c < kMaxCluster && c * a.requests < 3 * dev.sms && c * (kDrawThreads / 32) <= a.steps) c *= 2;
    Kernel &k = Kernels<T>::decide();
    if ((e = ready(k, dev))) return e;
    void *args[] = {&a};
    LaunchConfig l(std::max<int64_t>(1, a.requests) * c, kDrawThreads, c, a.rows > 0, s);
    return cudaLaunchKernelExC(&l.cfg, k.fn, args);
}

template <typename T, int L>
const void *route_kernel_l(int v) {
    return v == 32   ? reinterpret_cast<const void *>(&k_route<T, L, 32>)
           : v == 16 ? reinterpret_cast<const void *>(&k_route<T, L, 16>)
                     : reinterpret_cast<const void *>(&k_route<T, L, 8>);
}
template <typename T>
const void *route_kernel_t(int lanes, int v) {
    return lanes == 32 ? route_kernel_l<T, 32>(v) : lanes == 16 ? route_kernel_l<T, 16>(v) : route_kernel_l<T, 8>(v);
}
const void *route_kernel(DType t, int lanes, int v) {
    return t == kF32    ? route_kernel_t<float>(lanes, v)
           : t == kBF16 ? route_kernel_t<__nv_bfloat16>(lanes, v)
                        : route_kernel_t<__half>(lanes, v);
}
// at eight columns a lane, more where 32 lanes do not hold the row
template <typename T>
const void *route_full_t(int lanes, int v) {
    return v == 32       ? reinterpret_cast<const void *>(&k_route_grad_full<T, 32, 32>)
           : v == 16     ? reinterpret_cast<const void *>(&k_route_grad_full<T, 32, 16>)
           : lanes == 32 ? reinterpret_cast<const void *>(&k_route_grad_full<T, 32, 8>)
           : lanes == 16 ? reinterpret_cast<const void *>(&k_route_grad_full<T, 16, 8>)
                         : reinterpret_cast<const void *>(&k_route_grad_full<T, 8, 8>);
}
const void *route_full_kernel(DType t, int lanes, int v) {
    return t == kF32    ? route_full_t<float>(lanes, v)
           : t == kBF16 ? route_full_t<__nv_bfloat16>(lanes, v)
                        : route_full_t<__half>(lanes, v);
}
template <typename T>
const void *route_grad_t(int lanes) {
    return lanes == 32   ? reinterpret_cast<const void *>(&k_route_grad<T, 32>)
           : lanes == 16 ? reinterpret_cast<const void *>(&k_route_grad<T, 16>)
                         : reinterpret_cast<const void *>(&k_route_grad<T, 8>);
}
const void *route_grad_kernel(DType t, int lanes) {
    return t == kF32    ? route_grad_t<float>(lanes)
           : t == kBF16 ? route_grad_t<__nv_bfloat16>(lanes)
                        : route_grad_t<__half>(lanes);
}

// CTAs of kRouteWarps warps with 32 / lanes rows each, `resident` per SM at most.
cudaError_t launch_route_rows(const void *fn, const RouteArgs &a, int lanes, int resident, int smem, bool dependent,
                              const DeviceInfo &dev, cudaStream_t s) {
    const int per = kRouteWarps * (32 / lanes);
    const int64_t need = (a.rows + per - 1) / per;
    const int64_t ctas = capped(std::min<int64_t>(need, resident * static_cast<int64_t>(dev.sms)), a.grid_cap);
    RouteArgs aa = a;
    void *args[] = {&aa};
    LaunchConfig l(ctas, kRouteThreads, 0, dependent, s, smem);
    return cudaLaunchKernelExC(&l.cfg, fn, args);
}

// As few lanes as hold a row's k slots, and its columns at `most` each.
void route_shape(const RouteArgs &a, int most, int *lanes, int *v) {
    for (*lanes = 8; *lanes < 32 && (*lanes * most < a.experts || *lanes < a.k);) *lanes *= 2;
    for (*v = 8; *lanes * *v < a.experts;) *v *= 2;
}

// Columns of a lane at most: 32, where rows are many and instructions count; 8
// where they are few, a row's latency counts and lanes are to spare. Measured
// (us, bf16, k = 8, sigmoid scores with a bias, 8 / 32 columns): 256 experts in 8
// groups, 32 rows 4.2 / 5.7, 1024 4.4 / 5.9, 2048 5.3 / 6.0, 4096 7.6 / 6.2, 8192
// 13.1 / 7.9, 16384 20.8 / 11.9, 65536 76 / 34; 512 experts, 1024 rows 5.0 / 6.3,
// 4096 8.6 / 7.8, 16384 24 / 18.
int route_most(const RouteArgs &a, const DeviceInfo &dev) {
    int lanes, v;
    route_shape(a, 8, &lanes, &v);
    return a.rows * lanes <= 12 * 32 * static_cast<int64_t>(dev.sms) ? 8 : 32;
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

cudaError_t launch_route(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    if (a.counts) {
        LaunchConfig l(1, kRouteThreads, 0, false, s);
        const cudaError_t e = cudaLaunchKernelEx(&l.cfg, k_zero, a.counts, a.experts);
        if (e != cudaSuccess || a.rows == 0) return e;
    }
    int lanes, v;
    route_shape(a, route_most(a, dev), &lanes, &v);
    const int smem = 4 * ((kRouteWarps * (32 / lanes) + (a.bias ? 1 : 0)) * route_row(lanes, v) +
                          (a.counts ? a.experts : 0));  // at most 45568 bytes
    return launch_route_rows(route_kernel(t, lanes, v), a, lanes, route_ctas(v), smem, a.counts != nullptr, dev, s);
}

cudaError_t launch_route_grad(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    int lanes, v;
    if (!a.sigmoid && !a.renormalise) {
        route_shape(a, 8, &lanes, &v);
        return launch_route_rows(route_full_kernel(t, lanes, v), a, lanes, 8, 4 * kRouteWarps * 32 * v, false, dev, s);
    }
    for (lanes = 8; lanes < a.k;) lanes *= 2;
    const int N = 16 / elem_size(t), smem = 16 * kRouteWarps * ((32 / lanes * a.experts + N - 1) / N);
    const void *fn = route_grad_kernel(t, lanes);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin);
        if (e != cudaSuccess) return e;
    }
    return launch_route_rows(fn, a, lanes, 8, smem, false, dev, s);
}

cudaError_t read_choice_status(unsigned long long out[2], const DeviceInfo &dev, cudaStream_t s) {
    out[0] = out[1] = 0ull;
    if (!g_launched.any(dev)) return cudaSuccess;
    cudaError_t e =
        cudaMemcpyFromSymbolAsync(out, g_choice_status, sizeof(unsigned long long) * 2, 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

cudaError_t reset_choice_status(const DeviceInfo &dev, cudaStream_t s) {
    if (!g_launched.any(dev)) return cudaSuccess;
    static const unsigned long long zero[2] = {0ull, 0ull};
    return cudaMemcpyToSymbolAsync(g_choice_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace cerows
