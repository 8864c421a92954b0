// ce_choices.cu -- sm_103a kernels of the choices made from a row's softmax, and
// their launchers.
//
//   sample_rows     a token drawn from each row's softmax by a given uniform number
//   verify_drafts   drafted tokens accepted or replaced
//   route_rows      each row's experts and gates
//   route_grad      the gradient of the gates
//
// Kernels (none uses tensor cores):
//   k_sample        sample_rows: a row over a cluster of CTAs
//   k_verify_rows   verify_drafts: every row by itself, a row over a cluster
//   k_verify_join   its rows into requests: what is emitted ends at the first
//                   draft that is not accepted
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
constexpr int kPartMin = 8192;  // bytes of a row per CTA, at least, when a row is split

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
    __device__ float operator()(float x, float y, int j) const {
        if (kind == kGreedy) return x == m ? 1.0f : 0.0f;
        const float e = ex2_ftz((x - m) * k);
        // two rounded products: rows that are the same leave exactly nothing
        if (kind == kResidual) return fmaxf(0.0f, __fsub_rn(__fmul_rn(e, rp), __fmul_rn(ex2_ftz((y - mq) * k), rq)));
        return kind == kOthers && j == skip ? 0.0f : e;
    }
};

// The weights of the columns [a, b) at p (and q, kResidual only), added in f32.
template <typename T>
__device__ float weight_of_run(const T *p, const T *q, int a, int b, const Weigh &w) {
    constexpr int N = Vec<T>::kN;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p + a) / sizeof(T)) % N);
    const bool same = q == nullptr || ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    float sum = 0.0f;
    auto one = [&](int j) { sum += w(Vec<T>::to_float(p[j]), q ? Vec<T>::to_float(q[j]) : 0.0f, j); };
    int j = a;
    for (const int head = min(b, a + (N - off) % N); j < head; ++j) one(j);
    if (same) {
#pragma unroll 4
        for (; j + N <= b; j += N) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p + j);
            uint4 y = make_uint4(0, 0, 0, 0);
            if (q) y = *reinterpret_cast<const uint4 *>(q + j);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 xx = Vec<T>::pair(x, i), yy = Vec<T>::pair(y, i);
                sum += w(xx.x, yy.x, j + 2 * i) + w(xx.y, yy.y, j + 2 * i + 1);
            }
        }
    }
    for (; j < b; ++j) one(j);
    return sum;
}

// The column of [a, b) whose weight holds t: runs of columns, a lane each, until
// a lane has one. All of a warp; -1 if nothing weighs anything.
template <typename T>
__device__ int column_of(const T *p, const T *q, int a, int b, const Weigh &w, Mass t) {
    const int lane = threadIdx.x & 31;
    while (true) {
        const int n = b - a;
        const int run = n <= 32 ? 1 : ((n + 31) / 32 + 7) & ~7;
        const int lo = min(b, a + lane * run), hi = min(b, lo + run);
        const float sum = weight_of_run(p, q, lo, hi, w);
        const int at = warp_segment(mass_of(sum, w.unit()), sum, t);
        if (at < 0) return -1;
        if (run == 1) return a + at;
        b = min(b, a + (at + 1) * run);
        a += at * run;
    }
}

// ---------------------------------------------------------------------------
// A row over the warps of a cluster: CTA `rank` has `cols` columns, each of its
// warps a quarter of them, in order.
struct Part {
    uint32_t rank, C;
    int warp, lane;
    int c0, n;  // this warp's columns
    __device__ Part(int vocab, int cols) {
        rank = cluster_rank();
        C = cluster_size();
        warp = static_cast<int>(threadIdx.x) >> 5;
        lane = static_cast<int>(threadIdx.x) & 31;
        c0 = min(vocab, static_cast<int>(rank) * cols + warp * (cols / kWarps));
        n = min(vocab, c0 + cols / kWarps) - c0;
    }
    __device__ bool leads() const { return rank == 0 && warp == 0; }
    __device__ int slot() const { return static_cast<int>(rank) * kWarps + warp; }
};

// Exchanges: every warp pushes 16 bytes into its slot in every CTA, and every
// warp reads all of them (ce_objectives.cuh: WarpXchg). Lane l gets slots 2 l
// and 2 l + 1: column order.
struct Meeting {
    WarpXchg<kWarps> &x;
    const Part &part;
    int64_t n = 0;  // exchanges so far
    bool failed = false;
    __device__ void push(float4 v) {
        const int xs = static_cast<int>(n & 1);
        if (part.lane < static_cast<int>(part.C))
            st_async_peer(peer_smem(&x.slot[xs][part.slot()], part.lane), v, peer_smem(&x.bar[xs], part.lane));
    }
    __device__ void collect(float4 &a, float4 &b, const float4 &none) {
        const int xs = static_cast<int>(n & 1), E = kWarps * static_cast<int>(part.C);
        if (!failed)
            failed = __any_sync(kFullMask, !mbar_wait_bounded(&x.bar[xs], static_cast<uint32_t>(n >> 1) & 1u));
        a = 2 * part.lane < E ? x.slot[xs][2 * part.lane] : none;
        b = 2 * part.lane + 1 < E ? x.slot[xs][2 * part.lane + 1] : none;
        __syncwarp();
        // its CTA's other warps may still be reading the slot: nobody pushes to
        // it again before each of them has pushed the next exchange
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&x.bar[xs], 16u * kWarps * part.C);
        ++n;
    }
};

__device__ __forceinline__ float4 as_float4(Mass m) {
    return make_float4(__uint_as_float(static_cast<uint32_t>(m)), __uint_as_float(static_cast<uint32_t>(m >> 32)), 0.0f,
                       0.0f);
}
__device__ __forceinline__ Mass as_mass(const float4 &v) {
    return static_cast<Mass>(__float_as_uint(v.x)) | static_cast<Mass>(__float_as_uint(v.y)) << 32;
}

// The slot among all warps' (masses a and b in lanes' slots 2 l and 2 l + 1)
// that holds u of the total, and t from its start on; -1 if there is no mass.
__device__ __forceinline__ int slot_of(Mass a, Mass b, float u, Mass &t) {
    const Mass end = warp_running_sum(a + b);
    t = part_of_total(u, __shfl_sync(kFullMask, end, 31));
    const unsigned hit = __ballot_sync(kFullMask, t < end);
    if (!hit) return -1;
    const int at = __ffs(hit) - 1;
    const Mass first = __shfl_sync(kFullMask, a, at);
    t -= __shfl_sync(kFullMask, end - a - b, at);
    if (t < first) return 2 * at;
    t -= first;
    return 2 * at + 1;
}

// A row's inputs.
template <typename T>
struct RowIn {
    const T *p, *q;   // the row, and the draft model's (null: none)
    int64_t draft;    // -1: none
    float accept, u;  // the numbers that accept the draft and draw a token
    float T_;         // temperature; 0: greedy
};

// The columns [c0, c0 + n) of a row into a state, without column `skip`.
template <typename T>
__device__ __forceinline__ TokState scan_part(const T *p, const Part &part, int skip, float k) {
    auto nothing = [] {};
    TokState st;
    if (skip >= part.c0 && skip < part.c0 + part.n) {
        st = tok_scan<T, false, kScan, 32, true>(p + part.c0, skip - part.c0, k, part.lane, nothing);
        const TokState r = tok_scan<T, false, kScan, 32, true>(p + skip + 1, part.c0 + part.n - skip - 1, k, part.lane,
                                                               nothing);
        st = tok_merge<false>(st, r, k);
    } else {
        st = tok_scan<T, false, kScan, 32, true>(p + part.c0, part.n, k, part.lane, nothing);
    }
    return tok_warp_reduce<false>(st, k);
}

// One row, by all warps of the cluster: whether its draft was accepted, the same
// in every warp. The token and its log-probability are written by one warp.
template <typename T>
__device__ bool choose_row(const RowIn<T> &in, int vocab, const Part &part, Meeting &meet, int64_t *token, float *logp) {
    const bool greedy = in.T_ == 0.0f;
    if (!greedy && !(in.T_ >= 1e-6f && in.T_ <= 1e6f)) {
        if (part.leads() && part.lane == 0) {
            *token = -1;
            if (logp) *logp = nan_f();
            count_bad();
        }
        return false;
    }
    // log2(e) / T to a last place: log2(e) in two parts
    float k = 1.44269504f, inv_t = 1.0f;
    if (!greedy) {
        inv_t = 1.0f / in.T_;
        k = 1.44269504f * inv_t;
        k += __fmaf_rn(-k, in.T_, 1.44269504f) * inv_t + 1.92596299e-8f * inv_t;
    }
    const bool bad_draft = in.draft >= vocab;
    const int d = in.draft >= 0 && !bad_draft ? static_cast<int>(in.draft) : -1;
    const T *q = d >= 0 && !greedy ? in.q : nullptr;
    const bool lookup = d >= 0 && !greedy && in.q == nullptr;  // a draft that no model drew
    float xd = 0.0f, yd = 0.0f;
    if (d >= 0) {
        xd = Vec<T>::to_float(in.p[d]);
        if (q) yd = Vec<T>::to_float(q[d]);
    }
    const TokState mine = scan_part(in.p, part, lookup ? d : -1, k);
    TokState mine_q = tok_empty();
    if (q) mine_q = scan_part(q, part, -1, k);
    meet.push(make_float4(mine.m, mine.s, mine_q.m, mine_q.s));
    float4 a, b;
    meet.collect(a, b, make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f));
    TokState P = tok_merge<false>(TokState{a.x, a.y, 0.0f}, TokState{b.x, b.y, 0.0f}, k);
    P = tok_warp_reduce<false>(P, k);
    if (lookup) tok_push1<false>(P, xd, k);
    const bool leader = part.leads() && part.lane == 0;
    if (bad_draft && leader) count_bad();
    if (!isfinite(P.m) || isnan(P.s)) {  // no distribution
        if (leader) {
            *token = -1;
            if (logp) *logp = nan_f();
            count_bad();
        }
        return false;
    }
    Weigh w{};
    w.kind = greedy ? kGreedy : lookup ? kOthers : kShare;
    w.m = P.m;
    w.k = k;
    w.skip = d;
    if (d >= 0 && !greedy) {
        const float pd = ex2_ftz((xd - P.m) * k) / P.s;
        float qd = 1.0f;
        bool drawn = true;
        if (q) {
            TokState Q = tok_merge<false>(TokState{a.z, a.w, 0.0f}, TokState{b.z, b.w, 0.0f}, k);
            Q = tok_warp_reduce<false>(Q, k);
            drawn = isfinite(Q.m) && !isnan(Q.s);
            qd = ex2_ftz((yd - Q.m) * k) / Q.s;
            if (drawn) {
                w.kind = kResidual;
                w.rp = 1.0f / P.s;
                w.mq = Q.m;
                w.rq = 1.0f / Q.s;
            } else if (leader) {
                count_bad();  // no distribution: the draft is not accepted, the token drawn from p
            }
        }
        if (drawn && in.accept * qd < pd) {
            if (leader) {
                *token = d;
                if (logp) *logp = (xd - P.m) * inv_t - logf(P.s);
            }
            return true;
        }
    }
    // the masses of the warps' parts
    Mass ma, mb;
    if (w.kind == kResidual) {
        float sum = 0.0f;
        const int run = ((part.n + 31) / 32 + 7) & ~7;
        const int lo = min(part.n, part.lane * run), hi = min(part.n, lo + run);
        sum = weight_of_run(in.p, q, part.c0 + lo, part.c0 + hi, w);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        float4 e, f;
        meet.push(as_float4(mass_of(sum, kUnitShares)));
        meet.collect(e, f, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        ma = as_mass(e);
        mb = as_mass(f);
        // nothing left: the two rows are the same, and the draw is from p
        if (!__any_sync(kFullMask, (ma | mb) != 0)) w.kind = kShare;
    }
    if (w.kind == kGreedy) {
        ma = a.x == P.m;
        mb = b.x == P.m;
    } else if (w.kind != kResidual) {
        ma = mass_of(a.y * ex2_ftz((a.x - P.m) * k), kUnitWeights);
        mb = mass_of(b.y * ex2_ftz((b.x - P.m) * k), kUnitWeights);
    }
    Mass t;
    const int slot = slot_of(ma, mb, greedy ? 0.0f : in.u, t);
    int column = -1;
    if (slot < 0) {
        column = d;  // nothing but the drafted column weighs anything (kOthers)
    } else if (slot == part.slot()) {
        column = column_of(in.p, q, part.c0, part.c0 + part.n, w, t);
    }
    if (slot < 0 ? part.leads() : slot == part.slot()) {
        if (part.lane == 0) {
            *token = column;
            if (logp)
                *logp = greedy ? 0.0f : column < 0 ? nan_f() : (Vec<T>::to_float(in.p[column]) - P.m) * inv_t - logf(P.s);
        }
    }
    if (!greedy || d < 0) return false;
    // a greedy request accepts its draft where it is the row's first largest
    meet.push(make_float4(__int_as_float(slot == part.slot() ? column : -1), 0.0f, 0.0f, 0.0f));
    meet.collect(a, b, make_float4(__int_as_float(-1), 0.0f, 0.0f, 0.0f));
    return __any_sync(kFullMask, __float_as_int(a.x) == d || __float_as_int(b.x) == d);
}

template <typename T>
__device__ __forceinline__ float temperature_of(const ChoiceArgs &a, int64_t row) {
    return a.temperatures ? a.temperatures[row] : a.temperature;
}

// The exchange slots of a cluster exist before a peer pushes, and no CTA leaves
// while a peer may still push to it.
__device__ __forceinline__ void open_meeting(WarpXchg<kWarps> &x) {
    if (threadIdx.x == 0) warp_xchg_init(x, 2, cluster_size());
    __syncthreads();
    cluster_arrive_release();
    cluster_wait();
}
__device__ __forceinline__ void close_meeting(const Meeting &meet) {
    cluster_arrive();
    cluster_wait();
    if (meet.failed && (threadIdx.x & 31) == 0) atomicAdd(&g_choice_status[1], 1ull);
}

// k_sample: a cluster per row.
template <typename T>
__global__ void __launch_bounds__(kThreads, 8) k_sample(ChoiceArgs a, int cols) {
    __shared__ WarpXchg<kWarps> x;
    const Part part(a.vocab, cols);
    open_meeting(x);
    Meeting meet{x, part};
    for (int64_t row = cluster_id_x(); row < a.rows; row += cluster_count_x()) {
        RowIn<T> in{};
        in.p = static_cast<const T *>(a.logits) + row * a.stride;
        in.draft = -1;
        in.u = a.uniforms[row];
        in.T_ = temperature_of<T>(a, row);
        choose_row(in, a.vocab, part, meet, a.tokens + row, a.logp ? a.logp + row : nullptr);
    }
    close_meeting(meet);
}

// k_verify_rows: a cluster per row, each row as if all before it were accepted.
template <typename T>
__global__ void __launch_bounds__(kThreads, 8) k_verify_rows(ChoiceArgs a, int cols) {
    __shared__ WarpXchg<kWarps> x;
    launch_dependents();
    const Part part(a.vocab, cols);
    open_meeting(x);
    Meeting meet{x, part};
    const int64_t first = a.offsets[0], last = a.offsets[a.requests];
    for (int64_t row = cluster_id_x(); row < a.rows; row += cluster_count_x()) {
        if (row < first || row >= last) {
            if (part.leads() && part.lane == 0) {
                a.tokens[row] = -1;
                if (a.logp) a.logp[row] = 0.0f;
                a.accepts[row] = 0;
            }
            continue;
        }
        RowIn<T> in{};
        in.p = static_cast<const T *>(a.logits) + row * a.stride;
        if (a.draft_logits) in.q = static_cast<const T *>(a.draft_logits) + row * a.draft_stride;
        in.draft = a.drafts[row];
        in.accept = a.uniforms[2 * row];
        in.u = a.uniforms[2 * row + 1];
        in.T_ = temperature_of<T>(a, row);
        const bool yes = choose_row(in, a.vocab, part, meet, a.tokens + row, a.logp ? a.logp + row : nullptr);
        if (part.leads() && part.lane == 0) a.accepts[row] = yes;
    }
    close_meeting(meet);
}

// k_verify_join: a warp per request: its accepted drafts, and nothing emitted
// behind the first row that accepts none.
__global__ void __launch_bounds__(kThreads) k_verify_join(ChoiceArgs a) {
    wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t s = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5); s < a.requests; s += warps) {
        const int64_t r0 = a.offsets[s], r1 = a.offsets[s + 1];
        if (r0 < 0 || r1 < r0 || r1 > a.rows) {
            if (lane == 0) {
                a.accepted[s] = -1;
                count_bad();
            }
            continue;
        }
        int64_t n = -1;  // rows before the first that accepts none
        for (int64_t r = r0; r < r1; r += 32) {
            const bool in = r + lane < r1;
            const unsigned stop = __ballot_sync(kFullMask, in && n < 0 && a.accepts[r + lane] == 0);
            const bool over = n >= 0;
            if (n < 0 && stop) n = r - r0 + __ffs(stop) - 1;
            if (in && n >= 0 && (over || r + lane > r0 + n)) {
                a.tokens[r + lane] = -1;
                if (a.logp) a.logp[r + lane] = 0.0f;
            }
        }
        if (lane == 0) a.accepted[s] = n < 0 ? r1 - r0 : n;
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
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

// Columns of a CTA: its warps' parts are multiples of 8.
int cols_of(int64_t vocab, int c) { return static_cast<int>(((vocab + c - 1) / c + 31) & ~int64_t(31)); }

int split_of(DType t, int64_t rows, int64_t vocab, const DeviceInfo &dev) {
    const int64_t fill = 6 * static_cast<int64_t>(dev.sms) / std::max<int64_t>(1, rows);
    const int64_t parts = (vocab * elem_size(t) + kPartMin - 1) / kPartMin;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(fill, parts), kMaxCluster)));
}

template <typename T>
Kernel &sample_kernel() {
    static Kernel k(reinterpret_cast<const void *>(&k_sample<T>), false);
    return k;
}
template <typename T>
Kernel &verify_kernel() {
    static Kernel k(reinterpret_cast<const void *>(&k_verify_rows<T>), false);
    return k;
}

cudaError_t launch_rows(Kernel &k, DType t, const ChoiceArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    if (cudaError_t e = ready(k, dev); e != cudaSuccess) return e;
    const int c = split_of(t, a.rows, a.vocab, dev);
    ChoiceArgs aa = a;
    int cols = cols_of(a.vocab, c);
    void *args[] = {&aa, &cols};
    LaunchConfig l(capped(a.rows, a.grid_cap) * c, kThreads, c, false, s);
    return cudaLaunchKernelExC(&l.cfg, k.fn, args);
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

cudaError_t launch_sample(DType t, const ChoiceArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    Kernel &k = t == kF32    ? sample_kernel<float>()
                : t == kBF16 ? sample_kernel<__nv_bfloat16>()
                             : sample_kernel<__half>();
    return launch_rows(k, t, a, dev, s);
}

cudaError_t launch_verify(DType t, const ChoiceArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    Kernel &k = t == kF32    ? verify_kernel<float>()
                : t == kBF16 ? verify_kernel<__nv_bfloat16>()
                             : verify_kernel<__half>();
    if (a.rows > 0) {
        if (cudaError_t e = launch_rows(k, t, a, dev, s); e != cudaSuccess) return e;
    }
    if (a.requests == 0) return cudaSuccess;
    ChoiceArgs aa = a;
    void *args[] = {&aa};
    const int64_t ctas = std::min<int64_t>((a.requests + kWarps - 1) / kWarps, 8 * static_cast<int64_t>(dev.sms));
    LaunchConfig l(ctas, kThreads, 0, a.rows > 0, s);
    return cudaLaunchKernelExC(&l.cfg, reinterpret_cast<const void *>(&k_verify_join), args);
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
