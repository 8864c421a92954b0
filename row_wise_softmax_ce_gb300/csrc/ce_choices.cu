// ce_choices.cu -- sm_103a kernels of the choices made from a row's softmax, and
// their launchers.
//
//   sample_rows     a token drawn from each row's softmax by a given uniform number
//   verify_drafts   drafted tokens accepted or replaced
//   route_rows      each row's experts and gates
//   route_grad      the gradient of the gates
//
// Kernels (none uses tensor cores):
//   k_states        every row in steps of 4 KB, a state (m, s) for each step: one
//                   read of the logits, and of the draft rows, in parts of any
//                   number of warps
//   k_sample        sample_rows: a warp per row merges its states, draws a step by
//                   their masses and re-reads that step
//   k_decide        verify_drafts: a CTA per request merges its rows' states, finds
//                   the first that accepts no draft and draws from p where the
//                   token comes from p
//   k_residual      the other requests' rows again: what max(0, p - q) leaves of
//                   each step
//   k_replace       their token: a warp per request draws a step and re-reads it
//   k_route         route_rows, a warp per row
//   k_route_grad    route_grad, a warp per row
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
constexpr int kDecideThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ void count_bad() { atomicAdd(&g_choice_status[0], 1ull); }

// ---------------------------------------------------------------------------
// Drawing a column. A row is split into segments in column order (a warp's part,
// a lane's run, a column); a segment's mass is the sum of its weights as a fixed
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

// What a column weighs in a draw.
enum Kind : int {
    kShare = 0,     // 2^((x - m) k)
    kGreedy = 1,    // 1 where x is the row's largest value, else 0
    kResidual = 2,  // max(0, p - q)
    kOthers = 3,    // 2^((x - m) k), the drafted column 0
};
struct Weigh {
    Kind kind;
    float m, k;           // the row's
    float rp, mq, rq;     // kResidual: 1 / s, and the draft row's max and 1 / s
    int skip;             // kOthers: the drafted column
    __device__ float unit() const { return kind == kResidual ? kUnitShares : kUnitWeights; }
    __device__ float residual(float x, float y) const {
        // two rounded products: rows that are the same leave exactly nothing
        return fmaxf(0.0f, __fsub_rn(__fmul_rn(ex2_ftz((x - m) * k), rp), __fmul_rn(ex2_ftz((y - mq) * k), rq)));
    }
    __device__ float operator()(float x, float y, int j) const {
        if (kind == kGreedy) return x == m ? 1.0f : 0.0f;
        if (kind == kResidual) return residual(x, y);
        return kind == kOthers && j == skip ? 0.0f : ex2_ftz((x - m) * k);
    }
};

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
    }
    __device__ bool whole(int q, int end) const { return d.whole(q + by, end + by + (r ? 1 : 0)); }
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

template <typename T>
__device__ __forceinline__ float weight_of(const uint4 &x, const uint4 &y, int j, const Weigh &w) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < Vec<T>::kN / 2; ++i) {
        const float2 xx = Vec<T>::pair(x, i), yy = Vec<T>::pair(y, i);
        sum += w(xx.x, yy.x, j + 2 * i) + w(xx.y, yy.y, j + 2 * i + 1);
    }
    return sum;
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

// The column of step `step` whose weight holds t, and its logit: eight vectors
// next to one another in each lane, so one running sum over the lanes, then the
// lane's vectors and the vector's columns. All of a warp; column -1 if nothing
// weighs anything. kBeside: weights of p and q, else of p alone.
struct Found {
    int column;
    float x;
};
template <typename T, bool kBeside>
__device__ __forceinline__ Found column_of(const RowGrid<T> &g, const RowGrid<T> &d, int step, const Weigh &w, Mass t) {
    constexpr int N = Vec<T>::kN;
    const int lane = threadIdx.x & 31, q = step * kStep + kScan * lane;
    const Beside<T> beside(g, d);
    uint4 x[kScan], y[kBeside ? kScan : 1];
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
        x[u] = Vec<T>::lowest();
        if (g.whole(q + u)) x[u] = g.load_cached(q + u);
        if (kBeside) {
            y[u] = Vec<T>::lowest();
            if (beside.whole(q + u, q + u + 1)) y[u] = beside.load_cached(q + u);
        }
    }
    // partial vectors, and columns that lie in one of the draft row's
#pragma unroll
    for (int u = 0; u < kScan; ++u)
        if (q + u < g.nq) {
            if (!g.whole(q + u)) x[u] = columns_from(g.p, g.n, g.column(q + u));
            if (kBeside && !beside.whole(q + u, q + u + 1)) y[u] = columns_from(d.p, d.n, g.column(q + u));
        }
    float sum[kScan], all = 0.0f;
    Mass m = 0;
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
        sum[u] = weight_of<T>(x[u], kBeside ? y[u] : x[u], g.column(q + u), w);
        all += sum[u];
        m += mass_of(sum[u], w.unit());
    }
    const int l = warp_segment(m, all, t);
    if (l < 0) return Found{-1, 0.0f};
    const int u = walk(sum, w.unit(), t);
    uint4 xu = x[0], yu = y[0];
#pragma unroll
    for (int i = 1; i < kScan; ++i)
        if (i == u) {
            xu = x[i];
            if (kBeside) yu = y[i];
        }
    float e[N], xs[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 xx = Vec<T>::pair(xu, i), yy = Vec<T>::pair(kBeside ? yu : xu, i);
        const int j = g.column(q + u) + 2 * i;
        xs[2 * i] = xx.x, xs[2 * i + 1] = xx.y;
        e[2 * i] = w(xx.x, yy.x, j), e[2 * i + 1] = w(xx.y, yy.y, j + 1);
    }
    const int at = walk(e, w.unit(), t);
    float found = xs[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        if (i == at) found = xs[i];
    return Found{__shfl_sync(kFullMask, g.column(q + u) + at, l), __shfl_sync(kFullMask, found, l)};
}

// One step of a scan: vectors q .. q + kStep - 1 (those below nq) into a state,
// column `skip` (-1: none) left out.
template <typename T>
__device__ __forceinline__ void scan_step(TokState &st, const RowGrid<T> &g, int q, int skip, int lane, float k) {
    constexpr int N = Vec<T>::kN;
    uint4 v[kScan];
    const bool whole = g.whole(q, q + kStep);
    if (whole) {
#pragma unroll
        for (int u = 0; u < kScan; ++u) v[u] = g.load(q + 32 * u + lane);
    } else {
#pragma unroll
        for (int u = 0; u < kScan; ++u) {
            const int i = q + 32 * u + lane;
            v[u] = g.whole(i) ? g.load(i) : Vec<T>::lowest();
        }
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
    if (!whole) {  // the row's partial vectors
        const int head = q == 0 && g.qa > 0 ? g.edge_column(0, lane) : -1;
        const int tail = g.qb < g.nq && g.qb >= max(q, g.qa) && g.qb < q + kStep ? g.edge_column(g.qb, lane) : -1;
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
struct Steps {
    const float2 *p;
    int n, cnt, first;
    float2 held[kHeld];
    __device__ Steps(const float2 *states, int steps) : p(states), n(steps) {
        cnt = (steps + 31) / 32;
        first = static_cast<int>(threadIdx.x & 31) * cnt;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = i < cnt && first + i < n ? p[first + i] : make_float2(-INFINITY, 0.0f);
    }
    // fn(state, i) for each of the lane's steps i, in order
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) const {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) fn(held[i], i);
        for (int i = kHeld; i < cnt; ++i)
            if (first + i < n) fn(p[first + i], i);
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
__device__ __forceinline__ bool is_distribution(const TokState &st) { return isfinite(st.m) && !isnan(st.s); }

// The column that u draws from a row by its own weights (greedy: its first
// largest), without w.skip for kOthers; column -1 if nothing weighs anything.
template <typename T>
__device__ __forceinline__ Found draw_own(const RowGrid<T> &g, const Steps &steps, const Weigh &w, float u) {
    Mass t;
    const int step = steps.draw(kUnitWeights, w.kind == kGreedy ? 0.0f : u, [&](float2 v) {
        return w.kind == kGreedy ? (v.x == w.m ? 1.0f : 0.0f) : v.y * ex2_ftz((v.x - w.m) * w.k);
    }, t);
    return step < 0 ? Found{-1, 0.0f} : column_of<T, false>(g, g, step, w, t);
}

__device__ __forceinline__ float logp_of(float x, const TokState &st, const Heat &heat) {
    return heat.greedy ? 0.0f : (x - st.m) * heat.inv_t - logf(st.s);
}

// k_sample: a warp per row, behind k_states.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(ChoiceArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    const RowGrid<T> g = target_row<T>(a, row);
    const Heat heat(temperature_of(a, row));
    const float u = a.uniforms[row];
    wait_prerequisites();
    const Steps steps(states_of(a, row), a.steps);
    const TokState st = steps.merged(heat.k);
    Found f{-1, 0.0f};
    if (heat.ok && is_distribution(st)) {
        Weigh w{};
        w.kind = heat.greedy ? kGreedy : kShare;
        w.m = st.m;
        w.k = heat.k;
        f = draw_own(g, steps, w, u);
    }
    if (lane == 0) {
        a.tokens[row] = f.column;
        if (a.logp) a.logp[row] = f.column < 0 ? nan_f() : logp_of(f.x, st, heat);
        if (f.column < 0) count_bad();
    }
}

// k_decide: a CTA per request, behind k_states. Its warps judge a row each, in
// order, until one accepts no draft; the token of that row is drawn here where
// it comes from p, and left to k_residual and k_replace where it comes from what
// q leaves of p.
enum Verdict : int { kAccepted = 0, kDrawn = 1, kPending = 2 };

// A row's own inputs, asked for before the states are there.
struct RowNumbers {
    int64_t draft;
    float accept, u, temperature, xd, yd;
    int d;  // the draft, -1: none
};
template <typename T>
__device__ __forceinline__ RowNumbers row_numbers(const ChoiceArgs &a, int64_t row) {
    RowNumbers r{};
    r.draft = a.drafts[row];
    r.accept = a.uniforms[2 * row];
    r.u = a.uniforms[2 * row + 1];
    r.temperature = temperature_of(a, row);
    r.d = r.draft >= 0 && r.draft < a.vocab ? static_cast<int>(r.draft) : -1;
    if (r.d >= 0) {
        r.xd = target_row<T>(a, row).at(r.d);
        if (a.draft_logits) r.yd = draft_row<T>(a, row).at(r.d);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ Verdict judge(const ChoiceArgs &a, int64_t row, const RowNumbers &r) {
    const int lane = threadIdx.x & 31;
    const RowGrid<T> g = target_row<T>(a, row);
    const Heat heat(r.temperature);
    const bool drafted = r.d >= 0 && !heat.greedy, lookup = drafted && a.draft_logits == nullptr;
    const Steps steps(states_of(a, row), a.steps);
    TokState q{};
    if (drafted && !lookup) q = Steps(draft_states_of(a, row), a.steps).merged(heat.k);
    TokState p = steps.merged(heat.k);
    if (lookup) tok_push1<false>(p, r.xd, heat.k);  // its column is not among the states
    Weigh w{};
    w.kind = heat.greedy ? kGreedy : lookup ? kOthers : kShare;
    w.m = p.m;
    w.k = heat.k;
    w.skip = r.d;
    bool odd = r.draft >= a.vocab, accepted = false, drawn = false;
    Found f{-1, 0.0f};
    float logp = 0.0f;
    if (!heat.ok || !is_distribution(p)) {
        odd = true;
        logp = nan_f();
    } else {
        if (drafted) {
            const bool from = lookup || is_distribution(q);  // else not accepted, the token drawn from p
            odd |= !from;
            const float qd = lookup ? 1.0f : ex2_ftz((r.yd - q.m) * heat.k) / q.s;
            accepted = from && r.accept * qd < ex2_ftz((r.xd - p.m) * heat.k) / p.s;
            drawn = from && !lookup && !accepted;
            if (accepted) f = Found{r.d, r.xd};
        }
        if (!accepted && !drawn) {
            f = draw_own(g, steps, w, r.u);
            if (f.column < 0) f = Found{r.d, r.xd};  // nothing but the draft weighs anything
            accepted = heat.greedy && f.column == r.d;
        }
        if (!drawn) logp = logp_of(f.x, p, heat);
    }
    if (lane == 0) {
        a.tokens[row] = f.column;
        if (a.logp) a.logp[row] = logp;
        if (drawn) a.row_states[row] = make_float4(p.m, p.s, q.m, q.s);
        if (odd) count_bad();
    }
    return accepted ? kAccepted : drawn ? kPending : kDrawn;
}

template <typename T>
__global__ void __launch_bounds__(kDecideThreads) k_decide(ChoiceArgs a) {
    constexpr int kRows = kDecideThreads / 32;
    __shared__ int verdicts[kRows];
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t s = blockIdx.x, lo = a.offsets[0], hi = a.offsets[a.requests];
    const int64_t r0 = s < a.requests ? a.offsets[s] : 0, r1 = s < a.requests ? a.offsets[s + 1] : 0;
    const bool good = r0 >= 0 && r1 >= r0 && r1 <= a.rows;
    auto silent = [&](int64_t row) {
        a.tokens[row] = -1;
        if (a.logp) a.logp[row] = 0.0f;
    };
    // a row outside [lo, hi) has no states: of a table that decreases
    auto has_states = [&](int64_t row) { return good && row < r1 && row >= lo && row < hi; };
    RowNumbers numbers{};
    if (has_states(r0 + warp)) numbers = row_numbers<T>(a, r0 + warp);
    wait_prerequisites();
    if (s == 0)  // rows in no request
        for (int64_t r = threadIdx.x; r < a.rows; r += kDecideThreads)
            if (r < lo || r >= hi) silent(r);
    if (s >= a.requests) return;
    Pending pending{-1, 0.0f, 0.0f, 0.0f, 0.0f};
    int64_t stop = good ? -1 : 0;
    for (int64_t r = r0; good && r < r1 && stop < 0; r += kRows) {
        const int64_t row = r + warp;
        Verdict v = kDrawn;
        if (has_states(row)) {
            if (r > r0) numbers = row_numbers<T>(a, row);
            v = judge<T>(a, row, numbers);
        } else if (row < r1 && lane == 0) {
            silent(row);
        }
        if (lane == 0) verdicts[warp] = v;
        __syncthreads();
        for (int i = 0; i < kRows && r + i < r1; ++i)
            if (verdicts[i] != kAccepted) {
                stop = r + i;
                if (verdicts[i] == kPending) {
                    const float4 st = a.row_states[stop];
                    pending = Pending{stop, st.x, st.y, st.z, st.w};
                }
                break;
            }
        __syncthreads();
    }
    if (stop < 0) stop = r1;
    if (threadIdx.x == 0) {
        a.accepted[s] = good ? stop - r0 : -1;
        if (a.pending) a.pending[s] = pending;
        if (!good) count_bad();
    }
    for (int64_t r = stop + 1 + threadIdx.x; good && r < r1; r += kDecideThreads) silent(r);
}

__device__ __forceinline__ Weigh residual_of(const Pending &p, const Heat &heat) {
    Weigh w{};
    w.kind = kResidual;
    w.m = p.m;
    w.k = heat.k;
    w.rp = 1.0f / p.s;
    w.mq = p.mq;
    w.rq = 1.0f / p.sq;
    w.skip = -1;
    return w;
}

// k_residual: a warp per `unit` steps of a pending request's row: the sum of
// max(0, p - q) over each step, over the draft row's states, which have served.
template <typename T>
__global__ void __launch_bounds__(kThreads, 6) k_residual(ChoiceArgs a, int unit, int units, int64_t warps) {
    constexpr int N = Vec<T>::kN, kU = kScan / 2, kHalf = 32 * kU;
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t id = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5);
    wait_prerequisites();
    if (id >= warps) return;
    const int64_t s = id / units;
    const int first = static_cast<int>(id - s * units) * unit;
    const Pending p = a.pending[s];
    if (p.row < 0) return;
    const RowGrid<T> g = target_row<T>(a, p.row), d = draft_row<T>(a, p.row);
    const Beside<T> beside(g, d);
    const Weigh w = residual_of(p, Heat(temperature_of(a, p.row)));
    float mine = 0.0f;
    for (int i = 0; i < unit; ++i) {
        float sum = 0.0f;
        for (int q = (first + i) * kStep; q < min(g.nq, (first + i + 1) * kStep); q += kHalf) {
            const int end = min(g.nq, q + kHalf);
            if (g.whole(q, end) && beside.whole(q, end)) {
                uint4 x[kU], y[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int v = q + 32 * u + lane;
                    x[u] = v < end ? g.load(v) : Vec<T>::lowest();
                    y[u] = v < end ? beside.load(v) : Vec<T>::lowest();
                }
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int h = 0; h < N / 2; ++h) {
                        const float2 xx = Vec<T>::pair(x[u], h), yy = Vec<T>::pair(y[u], h);
                        sum += w.residual(xx.x, yy.x) + w.residual(xx.y, yy.y);
                    }
            } else {
                for (int v = q + lane; v < end; v += 32) {
                    const int j = g.column(v);
                    sum += weight_of<T>(columns_from(g.p, g.n, j), columns_from(d.p, d.n, j), j, w);
                }
            }
        }
        sum = warp_sum(sum);
        if (lane == i) mine = sum;
    }
    if (lane < unit && first + lane < a.steps) draft_states_of(a, p.row)[first + lane].x = mine;
}

// k_replace: a warp per request.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_replace(ChoiceArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t s = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5);
    wait_prerequisites();
    if (s >= a.requests) return;
    const Pending p = a.pending[s];
    if (p.row < 0) return;
    const RowGrid<T> g = target_row<T>(a, p.row), d = draft_row<T>(a, p.row);
    const Heat heat(temperature_of(a, p.row));
    Weigh w = residual_of(p, heat);
    const float u = a.uniforms[2 * p.row + 1];
    const Steps sums(draft_states_of(a, p.row), a.steps);
    Mass t;
    const int step = sums.draw(kUnitShares, u, [&](float2 v) { return v.x; }, t);
    Found f{-1, 0.0f};
    if (step >= 0) f = column_of<T, true>(g, d, step, w, t);
    if (f.column < 0) {  // nothing left: the two rows are the same, and the draw is from p
        w.kind = kShare;
        f = draw_own(g, Steps(states_of(a, p.row), a.steps), w, u);
    }
    if (lane == 0) {
        a.tokens[p.row] = f.column;
        if (a.logp) a.logp[p.row] = f.column < 0 ? nan_f() : logp_of(f.x, TokState{p.m, p.s, 0.0f}, heat);
    }
}

// ---------------------------------------------------------------------------
// Routing. A warp per row; lane l holds columns l V .. l V + V - 1.
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

// V consecutive columns from j on (those below n), -inf elsewhere.
template <typename T, int V>
__device__ __forceinline__ void load_columns(float (&z)[V], const T *p, int j, int n) {
    constexpr int N = Vec<T>::kN;
    if constexpr (V >= N) {
        if (j + V <= n && (reinterpret_cast<uintptr_t>(p + j) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < V / N; ++i) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p + j + N * i);
#pragma unroll
                for (int h = 0; h < N / 2; ++h) {
                    const float2 f = Vec<T>::pair(v, h);
                    z[N * i + 2 * h] = f.x;
                    z[N * i + 2 * h + 1] = f.y;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = j + i < n ? Vec<T>::to_float(p[j + i]) : -INFINITY;
}

__device__ __forceinline__ float exp_of(float d) { return ex2_ftz(d * 1.44269504f); }
// 1 / (1 + e^-z) without a difference from 1, for any z
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// A score over a factor that those of a row (or of its chosen) have in common,
// `top` the largest of their logits: nothing overflows, and what is next to
// nothing beside 1 is not so beside the others.
__device__ __forceinline__ float relative_score(float z, float top, bool sigmoid_scores) {
    if (!sigmoid_scores) return expf(z - top);
    return z > 0.0f ? sigmoid(z) : expf(z - fminf(0.0f, top)) / (1.0f + expf(z));
}

// The chosen experts' share of their sum from their logits (-inf: none), the sum
// over the warp's lanes.
__device__ __forceinline__ float share_of(float z, bool sigmoid_scores) {
    const float top = warp_max(z);
    if (top == -INFINITY) return 0.0f;
    const float e = relative_score(z, top, sigmoid_scores);
    return e / warp_sum(e);
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) k_route(RouteArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    int *counts = reinterpret_cast<int *>(smem);  // [experts], if wanted
    float *mine = reinterpret_cast<float *>(smem + (a.counts ? 4 * ((a.experts + 3) & ~3) : 0)) +
                  (threadIdx.x >> 5) * a.experts;  // this warp's row: what its groups are ranked by
    const int lane = threadIdx.x & 31, E = a.experts, j0 = lane * V;
    const int per = E / a.groups;
    const bool grouped = a.top_groups < a.groups;
    if (a.counts) {
        for (int j = threadIdx.x; j < E; j += kRouteThreads) counts[j] = 0;
        __syncthreads();
    }
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kRouteWarps;
    for (int64_t row = blockIdx.x * int64_t(kRouteWarps) + (threadIdx.x >> 5); row < a.rows; row += warps) {
        int64_t *chosen = a.chosen + row * a.k;
        float *gates = a.gates + row * a.k;
        if (a.weights && a.weights[row] == 0.0f) {
            if (lane < a.k) chosen[lane] = -1, gates[lane] = 0.0f;
            continue;
        }
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        float z[V], by[V];
        load_columns<T, V>(z, p, j0, E);
        bool odd = false;
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            odd |= isnan(z[i]) || z[i] == INFINITY;
            m = fmaxf(m, z[i]);
        }
        if (__any_sync(kFullMask, odd)) {
            if (lane < a.k) chosen[lane] = -1, gates[lane] = nan_f();
            if (lane == 0) count_bad();
            continue;
        }
        m = warp_max(m);
        float rs = 0.0f;
        if (!a.sigmoid) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) s += exp_of(z[i] - m);
            rs = 1.0f / warp_sum(s);
        }
        auto score = [&](float x) { return a.sigmoid ? sigmoid(x) : exp_of(x - m) * rs; };
        // what the choice goes by: the biased score, or, without a bias, the logit,
        // which orders the experts as their scores do and is exact
#pragma unroll
        for (int i = 0; i < V; ++i) {
            by[i] = z[i];
            if (a.bias && j0 + i < E && z[i] > -INFINITY) {
                by[i] = score(z[i]) + a.bias[j0 + i];
                if (isnan(by[i])) by[i] = -INFINITY;
            }
        }
        if (grouped) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j0 + i < E) mine[j0 + i] = a.bias || z[i] == -INFINITY ? by[i] : relative_score(z[i], m, a.sigmoid);
            __syncwarp();
            float best = -INFINITY, second = -INFINITY;
            if (lane < a.groups) {
                for (int i = 0; i < per; ++i) {
                    const float v = mine[lane * per + i];
                    second = fmaxf(second, fminf(v, best));
                    best = fmaxf(best, v);
                }
            }
            const float rank_by = a.group_top == 2 && second > -INFINITY ? best + second : best;
            int before = 0;
            for (int g = 0; g < a.groups; ++g) {
                const float o = __shfl_sync(kFullMask, rank_by, g);
                before += o > rank_by || (o == rank_by && g < lane);
            }
            const unsigned kept = __ballot_sync(kFullMask, lane < a.groups && before < a.top_groups);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j0 + i < E && !(kept >> ((j0 + i) / per) & 1u)) by[i] = -INFINITY;
        }
        // the k best, one after another: the largest, the lowest column of equals
        unsigned taken = 0;
        int expert = -1;  // lane i: the i-th
        for (int n = 0; n < a.k; ++n) {
            float best = -INFINITY;
            int at = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (!(taken >> i & 1u) && by[i] > best) best = by[i], at = i;
            const float top = warp_max(best);
            if (top == -INFINITY) break;
            const int owner = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
            if (lane == owner) taken |= 1u << at;
            const int j = __shfl_sync(kFullMask, j0 + at, owner);
            if (lane == n) expert = j;
        }
        const float zc = expert >= 0 ? Vec<T>::to_float(p[expert]) : -INFINITY;
        float g = a.renormalise ? share_of(zc, a.sigmoid) : expert >= 0 ? score(zc) : 0.0f;
        if (expert < 0) g = 0.0f;
        if (lane < a.k) {
            chosen[lane] = expert;
            gates[lane] = g * a.scale;
        }
        if (a.counts && expert >= 0) atomicAdd(&counts[expert], 1);
    }
    if (a.counts) {
        __syncthreads();
        for (int j = threadIdx.x; j < E; j += kRouteThreads)
            if (counts[j]) atomicAdd(&a.counts[j], static_cast<unsigned long long>(counts[j]));
    }
}

// k_route_grad: with G = scale * (gates' gradient), s the scores, c the chosen
// experts, f the chosen's share of their sum and D = sum of f G:
//   renormalised  softmax: dz_c = f (G - D), 0 elsewhere
//                 sigmoid: dz_c = f (G - D) (1 - s_c), 0 elsewhere
//   otherwise     softmax: dz_j = s_j ([j chosen] G - sum of s_c G_c)
//                 sigmoid: dz_c = s_c (1 - s_c) G, 0 elsewhere
// Only the softmax scores themselves need the whole row; the others read the
// chosen experts' logits.
template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad(RouteArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, E = a.experts, j0 = lane * V;
    float *mine = reinterpret_cast<float *>(smem) + (threadIdx.x >> 5) * E;  // this warp's row of the gradient
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kRouteWarps;
    for (int64_t row = blockIdx.x * int64_t(kRouteWarps) + (threadIdx.x >> 5); row < a.rows; row += warps) {
        T *grad = static_cast<T *>(a.grad) + row * a.grad_stride;
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.0f;
        if (!a.weights || a.weights[row] != 0.0f) {
            const T *p = static_cast<const T *>(a.logits) + row * a.stride;
            int64_t c = lane < a.k ? a.chosen[row * a.k + lane] : -1;
            if (c >= E || c < -1) {
                count_bad();
                c = -1;
            }
            const float z = c >= 0 ? Vec<T>::to_float(p[c]) : -INFINITY;
            const float G = c >= 0 ? a.gates_grad[row * a.k + lane] * a.scale : 0.0f;
            float v = 0.0f;  // the gradient at the chosen expert
            if (a.renormalise) {
                const float f = share_of(z, a.sigmoid);
                const float D = warp_sum(f > 0.0f || isnan(f) ? f * G : 0.0f);
                if (c >= 0) v = f * (G - D);
                if (a.sigmoid && c >= 0) v *= sigmoid(-z);
            } else if (a.sigmoid) {
                if (c >= 0) v = sigmoid(z) * sigmoid(-z) * G;
            } else {
                float x[V];
                load_columns<T, V>(x, p, j0, E);
                float m = -INFINITY, s = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
                m = warp_max(m);
                if (m == -INFINITY) m = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    out[i] = exp_of(x[i] - m);
                    s += out[i];
                }
                s = warp_sum(s);
                const float rs = s > 0.0f || isnan(s) ? 1.0f / s : 0.0f;
                const float sc = c >= 0 ? exp_of(z - m) * rs : 0.0f;
                v = sc * G;
                const float D = warp_sum(v);
#pragma unroll
                for (int i = 0; i < V; ++i) out[i] *= -rs * D;
            }
            // add v to its column: through shared memory, the same column twice one
            // after the other, in the order of the slots
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j0 + i < E) mine[j0 + i] = out[i];
            __syncwarp();
            const unsigned same = __match_any_sync(kFullMask, c >= 0 ? static_cast<int>(c) : -1 - lane);
            const unsigned others = __ballot_sync(kFullMask, (same & (same - 1)) != 0);
            if (others == 0) {
                if (c >= 0) mine[c] += v;
            } else {
                for (int i = 0; i < a.k; ++i) {
                    if (lane == i && c >= 0) mine[c] += v;
                    __syncwarp();
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (j0 + i < E) out[i] = mine[j0 + i];
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (j0 + i < E) grad[j0 + i] = Vec<T>::from_float(out[i]);
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

// Steps per warp: as many as keep the warps at `kWavesOfWarps` times what the GPU
// holds, at most 32 (a lane each).
int unit_of(int64_t steps, int64_t rows, const DeviceInfo &dev) {
    const int64_t resident = 8 * kWarps * static_cast<int64_t>(dev.sms);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(8, steps), steps * rows / resident)));
}

template <typename T>
struct Kernels {
    static const void *states() { return reinterpret_cast<const void *>(&k_states<T>); }
    static const void *sample() { return reinterpret_cast<const void *>(&k_sample<T>); }
    static const void *decide() { return reinterpret_cast<const void *>(&k_decide<T>); }
    static const void *residual() { return reinterpret_cast<const void *>(&k_residual<T>); }
    static const void *replace() { return reinterpret_cast<const void *>(&k_replace<T>); }
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
    if (cudaError_t e = launch_steps(Kernels<T>::states(), a, a.rows, false, dev, s); e != cudaSuccess) return e;
    void *args[] = {&a};
    return launch(Kernels<T>::sample(), ctas_of(a.rows), true, s, args);
}

template <typename T>
cudaError_t verify_as(ChoiceArgs a, const DeviceInfo &dev, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const bool drawn = a.draft_logits != nullptr;
    if (a.rows > 0 && (e = launch_steps(Kernels<T>::states(), a, drawn ? 2 * a.rows : a.rows, false, dev, s))) return e;
    void *args[] = {&a};
    if ((e = launch(Kernels<T>::decide(), std::max<int64_t>(1, a.requests), a.rows > 0, s, args, kDecideThreads))) return e;
    if (!drawn || a.rows == 0 || a.requests == 0) return e;
    if ((e = launch_steps(Kernels<T>::residual(), a, a.requests, true, dev, s))) return e;
    return launch(Kernels<T>::replace(), ctas_of(a.requests), true, s, args);
}

template <typename T>
const void *route_kernel_t(int v, bool grad) {
#define CE_ROUTE(V)                                                           \
    return grad ? reinterpret_cast<const void *>(&k_route_grad<T, V>) : reinterpret_cast<const void *>(&k_route<T, V>)
    switch (v) {
    case 2: CE_ROUTE(2);
    case 4: CE_ROUTE(4);
    case 8: CE_ROUTE(8);
    case 16: CE_ROUTE(16);
    default: CE_ROUTE(32);
    }
#undef CE_ROUTE
}

cudaError_t launch_route_any(DType t, const RouteArgs &a, bool grad, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    int v = 2;
    while (32 * v < a.experts) v *= 2;
    const void *fn = t == kF32    ? route_kernel_t<float>(v, grad)
                     : t == kBF16 ? route_kernel_t<__nv_bfloat16>(v, grad)
                                  : route_kernel_t<__half>(v, grad);
    const int64_t need = (a.rows + kRouteWarps - 1) / kRouteWarps;
    const int64_t ctas = capped(std::min<int64_t>(need, 8 * static_cast<int64_t>(dev.sms)), a.grid_cap);
    const int smem = (a.counts ? 4 * ((a.experts + 3) & ~3) : 0) + 4 * kRouteWarps * a.experts;
    RouteArgs aa = a;
    void *args[] = {&aa};
    LaunchConfig l(ctas, kRouteThreads, 0, false, s, smem);
    return cudaLaunchKernelExC(&l.cfg, fn, args);
}

}  // namespace

// The scratch: step states of the target rows, then of the draft rows, then the
// rows' and the requests' own.
int64_t choice_steps(DType t, int64_t vocab) {
    const int N = 16 / elem_size(t);
    return ((vocab + 2 * N - 2) / N + kStep - 1) / kStep;
}
int64_t choice_bytes(DType t, int64_t rows, int64_t vocab, int64_t requests) {
    const int64_t states = 8 * rows * choice_steps(t, vocab);
    return requests < 0 ? states : 2 * states + 16 * rows + static_cast<int64_t>(sizeof(Pending)) * requests;
}
static void lay_out(DType t, ChoiceArgs &a, void *work) {
    a.steps = static_cast<int>(choice_steps(t, a.vocab));
    a.states = static_cast<float2 *>(work);
    a.row_states = reinterpret_cast<float4 *>(a.states + 2 * a.rows * a.steps);
    a.pending = a.draft_logits ? reinterpret_cast<Pending *>(a.row_states + a.rows) : nullptr;
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
    if (a.counts) {
        const cudaError_t e = cudaMemsetAsync(a.counts, 0, sizeof(unsigned long long) * a.experts, s);
        if (e != cudaSuccess || a.rows == 0) return e;
    }
    return launch_route_any(t, a, false, dev, s);
}

cudaError_t launch_route_grad(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    return launch_route_any(t, a, true, dev, s);
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
