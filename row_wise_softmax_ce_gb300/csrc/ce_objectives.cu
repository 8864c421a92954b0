// ce_objectives.cu -- sm_103a kernels of the objectives over sampled answers
// and over pairs of answers, and their launchers.
//
//   logp_rows        logp = (x_y - m) / T - log s, H = log s - u / (T s)
//   policy_loss      + the clipped loss of exp(logp - old), the KL term, the
//   policy_step        entropy bonus; its gradient e (a + b log2 e) + [label] c
//   preference_loss  rows -> sequences -> pairs -> loss; the gradient of a
//   preference_step    row is its pair's factor times ([y] - p)
//
// Kernels (all bound by HBM; none uses tensor cores):
//   k_obj_rows       one read of each logit: log-probability, entropy and the
//                    policy's loss of a row, a CTA or a cluster per row
//   k_obj_rows_warp  the same for many short rows, a warp per row
//   k_policy_staged  the policy's loss and gradient, rows held in shared memory
//   k_policy_warp    the same for short rows, held in a warp's registers
//   k_policy_stream  the same for rows too long to hold: read twice
//   k_join           a preference batch's rows into sequences, pairs, the loss
//                    and each row's gradient factor
//   k_pair_grad      the gradient of a preference batch, the rows read again
//   k_weighted_sum   the policy's loss, a fixed-shape tree of f32 pairs
#include <algorithm>
#include <cstdint>

#include "ce_internal.h"
#include "ce_launch.h"
#include "ce_objectives.cuh"

namespace cerows {

namespace {

// [0] rows with a bad label and pairs with a bad range; [1] bounded waits that gave up
__device__ unsigned long long g_objective_status[2];

// Of a forward scan: 128 threads, eight 16-byte loads in flight each, eight
// CTAs per SM. Measured (us; logp 8192 x 128256 bf16 with entropies, 4096 x
// 50257 f32): 64 threads x 8 loads 294, 100; 128 x 4 277, 98; 128 x 6 264, 94;
// 128 x 8 263, 93; 256 x 4 287, 104; 256 x 6 278, 97; the next group loaded
// before the current one is pushed, 128 x 4 271, 94, 256 x 4 274, 96.
constexpr int kScanThreads = 128;
constexpr int kScanUnroll = 8;
constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 4;       // 16-byte loads in flight per thread
constexpr int kRowsMinBytes = 8192;  // bytes of a row per CTA, at least, when a row is split
constexpr int kStagedThreads = 128;

__device__ __forceinline__ bool in_range(int64_t label, int vocab) { return label >= 0 && label < vocab; }

// ---------------------------------------------------------------------------
// k_obj_rows: one CTA per row (looping), or few rows over clusters of C CTAs,
// exactly one row each: every warp scans its part of a contiguous slice of `cols`
// columns and pushes its state into CTA 0's shared memory, whose first warp
// merges them and writes the row. HBM-bound: 7168 rows of 128256 bf16 with
// entropies 256-260 us, 7.1 TB/s; 4096 of 50257 f32, 1/4 masked, 91 us, 6.8 TB/s.
struct RowsXchg {
    float4 slot[kMaxCluster * (kScanThreads / 32)];
    uint64_t bar;
};

// A row that takes no part.
template <int kMode, bool kEnt>
__device__ __forceinline__ void write_dead_row(const ObjArgs &a, int64_t row) {
    a.logp[row] = 0.0f;
    if (kEnt && a.entropy) a.entropy[row] = 0.0f;
    if (kMode == kObjPolicy) a.loss[row] = 0.0f;
    if (kMode == kObjPreference && a.row_state) a.row_state[row] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// A row's label, asked for beside its weight and first used once the row's
// first logits are on their way: not one more latency in a row of few logits.
// volatile keeps the load where it is written.
__device__ __forceinline__ int64_t ld_label(const int64_t *p) {
    int64_t v;
    asm volatile("ld.global.nc.s64 %0, [%1];" : "=l"(v) : "l"(p));
    return v;
}

// A row's numbers beside its logits, and its outputs: one thread's work.
struct RowNumbers {
    float xl = 0.0f, old = 0.0f, ref = 0.0f, adv = 0.0f;
    bool lab_ok = true;
};

template <typename T, int kMode>
__device__ __forceinline__ RowNumbers load_numbers(const ObjArgs &a, int64_t row, const T *p, int64_t label) {
    RowNumbers r;
    if (kMode == kObjPolicy) {
        r.old = a.old_logp[row];
        r.adv = a.adv[row];
        if (a.ref_logp) r.ref = a.ref_logp[row];
    }
    r.lab_ok = in_range(label, a.vocab);
    if (r.lab_ok) r.xl = Vec<T>::to_float(p[label]);
    return r;
}

template <int kMode, bool kEnt>
__device__ __forceinline__ void write_row(const ObjArgs &a, int64_t row, const TokState &st, const RowNumbers &x,
                                          float w) {
    TokRow r;
    if (kMode == kObjPolicy) {
        r = policy_row<kEnt>(a, st, x.xl, x.lab_ok, w, x.adv, x.old, x.ref);
        a.loss[row] = r.loss;
    } else {
        float log_s;
        r = tok_row<kEnt>(st, x.xl, x.lab_ok, a.inv_t, &log_s);
    }
    a.logp[row] = r.logp;
    if (kEnt && a.entropy) a.entropy[row] = r.entropy;
    if (kMode == kObjPreference && a.row_state) a.row_state[row] = make_float4(st.m, 1.0f / st.s, 0.0f, 0.0f);
    if (!x.lab_ok) atomicAdd(&g_objective_status[0], 1ull);
}

template <typename T, int kMode, bool kEnt>
__global__ void __launch_bounds__(kScanThreads, 8) k_obj_rows(ObjArgs a, int cols) {
    constexpr int kW = kScanThreads / 32;
    __shared__ RowsXchg x;
    launch_dependents();
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = static_cast<int>(rank) * cols;
    const int n = max(0, min(a.vocab, c0 + cols) - c0);
    const int64_t G = cluster_count_x();
    int64_t first = 0, last = a.rows;
    if (kMode == kObjPreference) {
        // rows before the first sequence and behind the last take no part
        first = a.offsets[0];
        last = a.offsets[2 * a.pairs];
        if (blockIdx.x == 0 && tid == 0) *a.done = 0;
    }
    if (C > 1) {
        if (rank == 0 && tid == 0) {
            mbar_init(&x.bar, 1);
            fence_mbar_init();
            mbar_arrive_expect_tx(&x.bar, 16u * kW * C);
        }
        cluster_arrive_release();  // CTA 0's barrier exists before a peer pushes: the wait comes before the push
    }
    bool failed = false;
    for (int64_t row = cluster_id_x(); row < a.rows; row += G) {
        int64_t label = 0;
        if (rank == 0 && tid == 0) label = ld_label(a.labels + row);
        const float w = a.weights ? a.weights[row] : 1.0f;
        if (w == 0.0f || (kMode == kObjPreference && (row < first || row >= last))) {
            if (rank == 0 && tid == 0) write_dead_row<kMode, kEnt>(a, row);
            if (C > 1) cluster_wait();
            continue;
        }
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        // the row's numbers, by the thread that writes it. Not before the scan's
        // first loads: its warp would wait for the label before it asked for
        // logits, and the CTA for its warp (8192 x 128256: 300 -> 439 us)
        RowNumbers numbers;
        auto early = [&] {
            if (rank == 0 && tid == 0) numbers = load_numbers<T, kMode>(a, row, p, label);
        };
        TokState st = tok_scan<T, kEnt, kScanUnroll, kScanThreads, true>(p + c0, n, a.k, tid, early);
        st = tok_warp_reduce<kEnt>(st, a.k);
        const float4 mine = make_float4(st.m, st.s, st.u, 0.0f);
        if (C > 1) {
            cluster_wait();  // a cluster has one row
            if (lane == 0) st_async_peer(peer_smem(&x.slot[rank * kW + warp], 0), mine, peer_smem(&x.bar, 0));
            if (rank != 0) return;
            if (warp == 0) failed = !mbar_wait_bounded(&x.bar, 0);
        } else {
            if (lane == 0) x.slot[warp] = mine;
            __syncthreads();
        }
        if (warp == 0) {
            st = tok_empty();
            for (int i = lane; i < kW * static_cast<int>(C); i += 32)
                st = tok_merge<kEnt>(st, TokState{x.slot[i].x, x.slot[i].y, x.slot[i].z}, a.k);
            st = tok_warp_reduce<kEnt>(st, a.k);
            if (tid == 0) write_row<kMode, kEnt>(a, row, st, numbers, w);
        }
        if (row + G < a.rows) __syncthreads();  // the slots are rewritten for the next row
    }
    if (C > 1) {
        // CTA 0 stays while a peer that has not left may still push to it
        if (failed && tid == 0) atomicAdd(&g_objective_status[1], 1ull);
        cluster_arrive();
        cluster_wait();
    }
}

// k_obj_rows_warp: the same for many short rows, a warp per row: no barrier, no
// exchange, four rows per CTA. Bound by a row's latencies over the warps
// resident: 8192 x 2000 f16 policy losses 14.5 us (a CTA per row 31.0).
template <typename T, int kMode, bool kEnt>
__global__ void __launch_bounds__(kScanThreads, 8) k_obj_rows_warp(ObjArgs a) {
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kScanThreads / 32);
    int64_t first = 0, last = a.rows;
    if (kMode == kObjPreference) {
        first = a.offsets[0];
        last = a.offsets[2 * a.pairs];
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    }
    for (int64_t row = blockIdx.x * int64_t(kScanThreads / 32) + (threadIdx.x >> 5); row < a.rows; row += warps) {
        int64_t label = 0;
        if (lane == 0) label = ld_label(a.labels + row);
        const float w = a.weights ? a.weights[row] : 1.0f;
        if (w == 0.0f || (kMode == kObjPreference && (row < first || row >= last))) {
            if (lane == 0) write_dead_row<kMode, kEnt>(a, row);
            continue;
        }
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        RowNumbers numbers;
        auto early = [&] {
            if (lane == 0) numbers = load_numbers<T, kMode>(a, row, p, label);
        };
        TokState st = tok_scan<T, kEnt, kScanUnroll, 32, true>(p, a.vocab, a.k, lane, early);
        st = tok_warp_reduce<kEnt>(st, a.k);
        if (lane == 0) write_row<kMode, kEnt>(a, row, st, numbers, w);
    }
}

// ---------------------------------------------------------------------------
// Writing a slice of a gradient row: columns [0, n) at g from the logits at p
// (coherent loads: g may be p), the label's column `lab` (-1: elsewhere)
// getting c besides, by 16-byte stores: from the same vectors of the logits
// where the two share their phase of 16 bytes, from pairs of vectors otherwise.
template <typename T, bool kB, int kU, int kT>
__device__ __forceinline__ void write_slice(const T *p, T *g, int n, float m, float k, float a, float b, float c,
                                            int lab, int tid) {
    constexpr int N = Vec<T>::kN;
    const int offp = static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % N);
    const int offg = static_cast<int>((reinterpret_cast<uintptr_t>(g) / sizeof(T)) % N);
    auto one = [&](int j) {
        const float x = Vec<T>::to_float(p[j]);
        g[j] = Vec<T>::from_float(j == lab ? tok_label1<kB>(x, m, k, a, b, c) : tok_grad1<kB>(x, m, k, a, b));
    };
    if (offp != offg) {
        // vectors i0 .. i1 - 1 of the gradient's grid, whose logits lie in two
        // whole vectors of the logits' grid inside the slice; the rest, at most
        // three vectors' worth, one by one
        const int headg = (N - offg) % N, lead = offp + headg, r = lead % N;  // r > 0
        const uint4 *pa = reinterpret_cast<const uint4 *>(p - offp) + lead / N;
        const int i0 = lead < N && offp > 0 ? 1 : 0;
        const int i1 = max(i0, (offp + n) / N - lead / N - 1);
        const int first = min(n, headg + N * i0), rest = max(first, min(n, headg + N * i1));
        uint4 *gv = reinterpret_cast<uint4 *>(g + headg);
        for (int i = i0 + tid; i < i1; i += kT) {
            const int j = headg + N * i;
            const uint4 o = tok_grad_vec<T, kB>(shift_pair<T>(__ldcs(pa + i), __ldcs(pa + i + 1), r), m, k, a, b);
            __stcs(gv + i, o);
            if (static_cast<unsigned>(lab - j) < N) one(lab);
        }
        for (int j = tid; j < first + n - rest; j += kT) one(j < first ? j : rest + j - first);
        return;
    }
    const int head = min(n, (N - offp) % N), nvec = (n - head) / N, tail = n - head - N * nvec;
    // the label's logit, read before its vector is written (g may be p), by the
    // thread that owns the vector and so writes both
    const unsigned li = static_cast<unsigned>(lab - head);
    const bool owns = li < static_cast<unsigned>(N * nvec) && static_cast<int>(li / N) % kT == tid;
    const float xl = owns ? Vec<T>::to_float(p[lab]) : 0.0f;
    if (tid < head + tail) one(tid < head ? tid : N * nvec + tid);
    const uint4 *pv = reinterpret_cast<const uint4 *>(p + head);
    uint4 *gv = reinterpret_cast<uint4 *>(g + head);
    int q = tid;
    for (; q + (kU - 1) * kT < nvec; q += kU * kT) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = __ldcs(pv + q + u * kT);
#pragma unroll
        for (int u = 0; u < kU; ++u) __stcs(gv + q + u * kT, tok_grad_vec<T, kB>(v[u], m, k, a, b));
    }
    for (; q < nvec; q += kT) __stcs(gv + q, tok_grad_vec<T, kB>(__ldcs(pv + q), m, k, a, b));
    if (owns) g[lab] = Vec<T>::from_float(tok_label1<kB>(xl, m, k, a, b, c));
}

template <typename T>
__device__ __forceinline__ void zero_slice(T *g, int n, int tid, int nt) {
    constexpr int N = Vec<T>::kN;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) / sizeof(T)) % N);
    const int head = min(n, (N - off) % N), nvec = (n - head) / N;
    const T zero = Vec<T>::from_float(0.0f);
    for (int j = tid; j < head; j += nt) g[j] = zero;
    uint4 *gv = reinterpret_cast<uint4 *>(g + head);
    for (int q = tid; q < nvec; q += nt) __stcs(gv + q, make_uint4(0u, 0u, 0u, 0u));
    for (int j = head + N * nvec + tid; j < n; j += nt) g[j] = zero;
}

// ---------------------------------------------------------------------------
// k_policy_stream: the policy's loss and gradient; the cluster's CTAs read
// their slices twice (state, then gradient), both times by coherent loads: the
// gradient may be written over the logits.
template <typename T, bool kEnt>
__global__ void __launch_bounds__(kRowsThreads, 4) k_policy_stream(ObjArgs a, int cols) {
    __shared__ TokState red[32];
    __shared__ PushXchg xg;
    __shared__ float4 bc;
    launch_dependents();
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int tid = threadIdx.x;
    const int c0 = static_cast<int>(rank) * cols;
    const int n = max(0, min(a.vocab, c0 + cols) - c0);
    const int64_t cid = cluster_id_x(), G = cluster_count_x();
    const int64_t K = cid < a.rows ? (a.rows - 1 - cid) / G + 1 : 0;
    if (tid == 0) push_xchg_init(xg, K, C);
    __syncthreads();
    cluster_arrive();
    bool failed = false;
    int64_t used = 0;
    for (int64_t row = cid; row < a.rows; row += G) {
        const T *p = static_cast<const T *>(a.logits) + row * a.stride + c0;
        T *g = static_cast<T *>(a.grad) + row * a.grad_stride + c0;
        const float w = a.weights ? a.weights[row] : 1.0f;
        if (w == 0.0f) {
            zero_slice(g, n, tid, kRowsThreads);
            if (rank == 0 && tid == 0) {
                a.logp[row] = 0.0f;
                a.loss[row] = 0.0f;
                if (kEnt && a.entropy) a.entropy[row] = 0.0f;
            }
            continue;
        }
        const int64_t label = a.labels[row];
        const bool lab_ok = in_range(label, a.vocab);
        const int lab = lab_ok && label >= c0 && label < c0 + n ? static_cast<int>(label - c0) : -1;
        float xl = 0.0f, old = 0.0f, ref = 0.0f, adv = 0.0f;
        if (tid == 0) {
            if (lab >= 0) xl = Vec<T>::to_float(p[lab]);  // before any CTA of the cluster writes (grad may be logits)
            old = a.old_logp[row];
            adv = a.adv[row];
            if (a.ref_logp) ref = a.ref_logp[row];
        }
        TokState st = tok_scan<T, kEnt, kRowsUnroll, kRowsThreads, false>(p, n, a.k, tid, [] {});
        st = tok_block_reduce_w0<kEnt>(st, red, a.k);
        if (used == 0) cluster_wait();
        if (tid == 0) tok_publish(xg, used, rank, C, st, xl);
        if (tid < 32) {
            const uint32_t owner = lab_ok ? static_cast<uint32_t>(label) / static_cast<uint32_t>(cols) : 0u;
            const TokState s = tok_collect<kEnt>(xg, used, K, C, owner, &xl, a.k, &failed);
            if (tid == 0) {
                const TokRow r = policy_row<kEnt>(a, s, xl, lab_ok, w, adv, old, ref);
                bc = make_float4(r.m, r.a, r.b, r.c);
                if (rank == 0) {
                    a.logp[row] = r.logp;
                    a.loss[row] = r.loss;
                    if (kEnt && a.entropy) a.entropy[row] = r.entropy;
                    if (!lab_ok) atomicAdd(&g_objective_status[0], 1ull);
                }
            }
        }
        ++used;
        __syncthreads();
        const float4 f = bc;
        write_slice<T, kEnt, 4, kRowsThreads>(p, g, n, f.x, a.k, f.y, f.z, f.w, lab, tid);
        __syncthreads();  // bc and red are rewritten for the next row
    }
    if (used == 0) cluster_wait();
    cluster_arrive();
    cluster_wait();
    if (__syncthreads_or(failed) && tid == 0) atomicAdd(&g_objective_status[1], 1ull);
}

// ---------------------------------------------------------------------------
// k_policy_staged: the policy's loss and gradient with each logit read once
// from HBM, rows held in shared memory.
//
// CTA `rank` of a cluster owns columns [c0, c0 + n) of the cluster's rows. A
// slice sits in shared memory on the 16-byte grid of the logits: element i of
// buf holds column c0 - off + i, off = the slice's start modulo 16 bytes. Its
// aligned body arrives by one bulk copy; the at most two partial end vectors
// are loaded by the threads that own them, with -inf outside the slice. Per
// row: one sweep for (m, s, u); the states of the cluster's warps meet by
// pushes; every warp forms the row's factors from the same bits; the gradient
// is written from shared memory; then the copy of the next row that counts
// starts (rows past the grid), its latency hidden behind the SM's other CTAs.
// HBM-bound: 8192 x 50257 bf16 245 us with the loss's sum, 6.7 TB/s of logits
// and gradient; 4096 x 128256 f32 with an entropy bonus 606 us, 6.9 TB/s. A
// reduction over each CTA before the exchange, and one warp forming the
// factors: 256 and 624 us.
struct alignas(16) PolicyHeader {
    WarpXchg<kStagedThreads / 32> xg;
    uint64_t bar;
};
constexpr int kPolicyHeaderBytes = 2176;
static_assert(sizeof(PolicyHeader) <= kPolicyHeaderBytes && kPolicyHeaderBytes % 128 == 0, "staged header");

// A 16-byte vector of grid index q: the slice's columns, -inf elsewhere.
template <typename T>
__device__ __forceinline__ uint4 load_edge(const T *p, int off, int n, int q) {
    constexpr int N = Vec<T>::kN;
    T v[N];
#pragma unroll
    for (int l = 0; l < N; ++l) {
        const int i = N * q + l - off;  // column - c0
        v[l] = i >= 0 && i < n ? p[i] : Vec<T>::from_float(-INFINITY);
    }
    return *reinterpret_cast<const uint4 *>(v);
}

template <typename T, bool kEnt>
__global__ void __launch_bounds__(kStagedThreads, 8) k_policy_staged(ObjArgs a, int cols) {
    constexpr int N = Vec<T>::kN, kU = 4, kT = kStagedThreads;
    extern __shared__ __align__(128) unsigned char smem[];
    launch_dependents();
    PolicyHeader &h = *reinterpret_cast<PolicyHeader *>(smem);
    T *buf = reinterpret_cast<T *>(smem + kPolicyHeaderBytes);
    uint4 *bufv = reinterpret_cast<uint4 *>(buf);
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int tid = threadIdx.x;
    const int c0 = static_cast<int>(rank) * cols;
    const int n = max(0, min(a.vocab, c0 + cols) - c0);
    const int64_t cid = cluster_id_x(), G = cluster_count_x();
    const int64_t K = cid < a.rows ? (a.rows - 1 - cid) / G + 1 : 0;
    const T *logits = static_cast<const T *>(a.logits) + c0;
    auto phase_of = [](const T *p) {
        return static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % Vec<T>::kN);
    };
    auto next_live = [&](int64_t row) {
        if (a.weights)
            while (row < a.rows && a.weights[row] == 0.0f) row += G;
        return row;
    };
    // the bulk copy of the aligned body of `row`'s slice
    uint64_t policy = 0;
    auto issue = [&](int64_t row) {
        const T *p = logits + row * a.stride;
        const int off = phase_of(p);
        const int head = min(n, (N - off) % N);
        const int nvec = (n - head) / N;
        const int qa = (off + head) / N;
        const uint32_t bytes = static_cast<uint32_t>(nvec) * 16u;
        mbar_arrive_expect_tx(&h.bar, bytes);
        if (bytes) bulk_copy_g2s(bufv + qa, p - off + N * qa, bytes, &h.bar, policy);
    };
    int64_t ahead = 0;  // thread 0: the row whose copy is issued next
    if (tid == 0) {
        mbar_init(&h.bar, 1);
        fence_mbar_init();
        warp_xchg_init(h.xg, K, C);
        policy = l2_policy_evict_first();
        ahead = next_live(cid);
        if (ahead < a.rows) {
            issue(ahead);
            ahead = next_live(ahead + G);
        }
    }
    __syncthreads();
    cluster_arrive();  // every CTA's slots exist before a peer pushes: the wait comes before the first push
    bool failed = false, left = false;
    uint32_t parity = 0;
    int64_t used = 0;
    // a row's weight and label are loaded one row ahead, off its critical path
    float w_next = K > 0 && a.weights ? a.weights[cid] : 1.0f;
    int64_t label_next = K > 0 ? a.labels[cid] : 0;
    for (int64_t row = cid; row < a.rows; row += G) {
        const float w = w_next;
        const int64_t label = label_next;
        if (row + G < a.rows) {
            if (a.weights) w_next = a.weights[row + G];
            label_next = a.labels[row + G];
        }
        T *g = static_cast<T *>(a.grad) + row * a.grad_stride + c0;
        if (w == 0.0f) {
            zero_slice(g, n, tid, kT);
            if (rank == 0 && tid == 0) {
                a.logp[row] = 0.0f;
                a.loss[row] = 0.0f;
                if (kEnt && a.entropy) a.entropy[row] = 0.0f;
            }
            continue;
        }
        const T *p = logits + row * a.stride;
        const int off = phase_of(p);
        const int head = min(n, (N - off) % N);
        const int nvec = (n - head) / N;    // whole body vectors
        const int qa = (off + head) / N;    // the first of them (0 or 1)
        const int nq = (off + n + N - 1) / N;  // vectors covering the slice
        const int qe0 = qa == 1 ? 0 : -1, qe1 = qa + nvec < nq ? qa + nvec : -1;  // partial end vectors
        if (qe0 >= 0 && tid == 0) bufv[qe0] = load_edge(p, off, n, qe0);
        if (qe1 >= 0 && (qe1 & (kT - 1)) == tid) bufv[qe1] = load_edge(p, off, n, qe1);
        const float old = a.old_logp[row], adv = a.adv[row], ref = a.ref_logp ? a.ref_logp[row] : 0.0f;
        const bool lab_ok = in_range(label, a.vocab);
        const int lab = lab_ok && label >= c0 && label < c0 + n ? static_cast<int>(label - c0) : -1;
        if (!failed) failed = !mbar_wait_bounded(&h.bar, parity);
        parity ^= 1u;
        TokState st = tok_empty();
        int q = tid;
        for (; q + (kU - 1) * kT < nq; q += kU * kT) {
            uint4 v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) v[u] = bufv[q + u * kT];
            tok_push<T, kEnt, kU>(st, v, a.k);
        }
        for (; q < nq; q += kT) {
            const uint4 v[1] = {bufv[q]};
            tok_push<T, kEnt, 1>(st, v, a.k);
        }
        st = tok_warp_reduce<kEnt>(st, a.k);
        // the label's logit goes with the warp that owns its vector
        const int owner = lab >= 0 ? (off + lab) / N & (kT - 1) : -32;
        float xl = owner == tid ? Vec<T>::to_float(buf[off + lab]) : 0.0f;
        xl = __shfl_sync(kFullMask, xl, owner & 31);
        if (owner / 32 != tid / 32) xl = 0.0f;
        if (used == 0) cluster_wait();
        warp_xchg_push(h.xg, used, rank, C, st, xl);
        st = warp_xchg_collect<kT / 32, kEnt>(h.xg, used, K, C, &xl, a.k, &failed);
        const TokRow r = policy_row<kEnt>(a, st, xl, lab_ok, w, adv, old, ref);
        if (rank == 0 && tid == 0) {
            a.logp[row] = r.logp;
            a.loss[row] = r.loss;
            if (kEnt && a.entropy) a.entropy[row] = r.entropy;
            if (!lab_ok) atomicAdd(&g_objective_status[0], 1ull);
        }
        ++used;
        if (row + G >= a.rows) {
            cluster_arrive();  // nothing more is pushed to or by this CTA
            left = true;
        }
        if (qe0 >= 0 || qe1 >= 0) __syncthreads();  // the edges are read by other threads than their owners
        // the gradient, in 16-byte vectors of its own grid: the logits' own
        // vectors where the two share their phase, shifted ones otherwise
        const float4 f = make_float4(r.m, r.a, r.b, r.c);
        const int offg = phase_of(g);
        const int headg = min(n, (N - offg) % N), nvecg = (n - headg) / N, tailg = n - headg - N * nvecg;
        uint4 *gv = reinterpret_cast<uint4 *>(g + headg);
        const T *src = buf + off;  // column c0
        if (offg == off) {
            const uint4 *bv = bufv + qa;
            int i = tid;
            for (; i + (kU - 1) * kT < nvecg; i += kU * kT) {
                uint4 v[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) v[u] = bv[i + u * kT];
#pragma unroll
                for (int u = 0; u < kU; ++u) __stcs(gv + i + u * kT, tok_grad_vec<T, kEnt>(v[u], f.x, a.k, f.y, f.z));
            }
            for (; i < nvecg; i += kT) __stcs(gv + i, tok_grad_vec<T, kEnt>(bv[i], f.x, a.k, f.y, f.z));
        } else {
            const int lead = off + headg, r = lead % N;
            const uint4 *bv = bufv + lead / N;
#pragma unroll 2
            for (int i = tid; i < nvecg; i += kT)
                __stcs(gv + i, tok_grad_vec<T, kEnt>(shift_pair<T>(bv[i], bv[i + 1], r), f.x, a.k, f.y, f.z));
        }
        if (tid < headg + tailg) {
            const int j = tid < headg ? tid : N * nvecg + tid;
            const float x = Vec<T>::to_float(src[j]);
            g[j] = Vec<T>::from_float(j == lab ? tok_label1<kEnt>(x, f.x, a.k, f.y, f.z, f.w)
                                               : tok_grad1<kEnt>(x, f.x, a.k, f.y, f.z));
        }
        // the label's element of a vector, again, by the thread that wrote it
        const unsigned li = static_cast<unsigned>(lab - headg);
        if (li < static_cast<unsigned>(N * nvecg) && (static_cast<int>(li / N) & (kT - 1)) == tid)
            g[lab] = Vec<T>::from_float(tok_label1<kEnt>(Vec<T>::to_float(src[lab]), f.x, a.k, f.y, f.z, f.w));
        __syncthreads();  // the slice, its edges and the header are free
        if (tid == 0 && ahead < a.rows) {
            fence_proxy_async_smem();
            issue(ahead);
            ahead = next_live(ahead + G);
        }
    }
    if (used == 0) cluster_wait();
    if (!left) cluster_arrive();
    cluster_wait();  // no CTA leaves while a peer may still push to it
    if (__syncthreads_or(failed) && tid == 0) {
        atomicAdd(&g_objective_status[1], 1ull);
        // give a copy still in flight a last bounded chance to land
        (void)mbar_wait_bounded(&h.bar, parity ^ 1u, 10000000ull);
    }
}

// ---------------------------------------------------------------------------
// k_policy_warp: the policy's loss and gradient of short rows, a warp per row
// that it holds in registers (at most kV vectors per lane, and a partial vector
// at either end by single elements). Bound by a row's own latencies (weight and
// label, logits, x[label], the gradient's stores) over the warps resident: 8192
// x 2000 bf16 18.6 us, 3.5 TB/s; a staged CTA per row 36.7 us.
template <typename T, bool kEnt, int kV>
__global__ void __launch_bounds__(kScanThreads, kV > 8 ? 3 : kV > 4 ? 6 : 8) k_policy_warp(ObjArgs a) {
    constexpr int N = Vec<T>::kN;
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kScanThreads / 32);
    for (int64_t row = blockIdx.x * int64_t(kScanThreads / 32) + (threadIdx.x >> 5); row < a.rows; row += warps) {
        const int64_t label = ld_label(a.labels + row);
        const float w = a.weights ? a.weights[row] : 1.0f;
        T *g = static_cast<T *>(a.grad) + row * a.grad_stride;
        if (w == 0.0f) {
            zero_slice(g, a.vocab, lane, 32);
            if (lane == 0) write_dead_row<kObjPolicy, kEnt>(a, row);
            continue;
        }
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % N);
        const int head = min(a.vocab, (N - off) % N), nvec = (a.vocab - head) / N, tail = a.vocab - head - N * nvec;
        const uint4 *pv = reinterpret_cast<const uint4 *>(p + head);
        uint4 v[kV];
#pragma unroll
        for (int u = 0; u < kV; ++u) v[u] = lane + 32 * u < nvec ? __ldcs(pv + lane + 32 * u) : Vec<T>::lowest();
        const int je = lane < head ? lane : lane < head + tail ? N * nvec + lane : -1;  // a single element's column
        float xe = je >= 0 ? Vec<T>::to_float(p[je]) : -INFINITY;
        const RowNumbers x = load_numbers<T, kObjPolicy>(a, row, p, label);
        TokState st = tok_empty();
#pragma unroll
        for (int u = 0; u < kV; u += 4) {
            const uint4 four[4] = {v[u], v[u + 1], v[u + 2], v[u + 3]};
            tok_push<T, kEnt, 4>(st, four, a.k);
        }
        if (je >= 0) tok_push1<kEnt>(st, xe, a.k);
        st = tok_warp_reduce<kEnt>(st, a.k);
        const TokRow r = policy_row<kEnt>(a, st, x.xl, x.lab_ok, w, x.adv, x.old, x.ref);
        if (lane == 0) {
            a.logp[row] = r.logp;
            a.loss[row] = r.loss;
            if (kEnt && a.entropy) a.entropy[row] = r.entropy;
            if (!x.lab_ok) atomicAdd(&g_objective_status[0], 1ull);
        }
        const int lab = x.lab_ok ? static_cast<int>(label) : -1;
        auto one = [&](int j, float xj) {
            g[j] = Vec<T>::from_float(j == lab ? tok_label1<kEnt>(xj, r.m, a.k, r.a, r.b, r.c)
                                               : tok_grad1<kEnt>(xj, r.m, a.k, r.a, r.b));
        };
        const int headg = static_cast<int>((N - (reinterpret_cast<uintptr_t>(g) / sizeof(T)) % N) % N);
        const int by = (headg - (N - off) % N + N) % N;  // the gradient's grid against the logits'
        if (by == 0) {
            uint4 *gv = reinterpret_cast<uint4 *>(g + head);
#pragma unroll
            for (int u = 0; u < kV; ++u)
                if (lane + 32 * u < nvec) __stcs(gv + lane + 32 * u, tok_grad_vec<T, kEnt>(v[u], r.m, a.k, r.a, r.b));
            if (je >= 0) one(je, xe);
            // the label's element of a vector, again, by the lane that wrote it
            const unsigned li = static_cast<unsigned>(lab - head);
            if (li < static_cast<unsigned>(N * nvec) && static_cast<int>(li / N) % 32 == lane) one(lab, x.xl);
        } else {
            // vector q of the gradient's grid from vectors q and q + 1 of the
            // logits', the second the next lane's; what lies before the first
            // and behind the last one by one
            uint4 *gv = reinterpret_cast<uint4 *>(g + head + by);
#pragma unroll
            for (int u = 0; u < kV; ++u) v[u] = tok_grad_vec<T, kEnt>(v[u], r.m, a.k, r.a, r.b);
#pragma unroll
            for (int u = 0; u < kV; ++u) {
                uint4 next = v[u];
                if (lane == 0 && u + 1 < kV) next = v[u + 1 < kV ? u + 1 : u];
                next.x = __shfl_sync(kFullMask, next.x, (lane + 1) & 31);
                next.y = __shfl_sync(kFullMask, next.y, (lane + 1) & 31);
                next.z = __shfl_sync(kFullMask, next.z, (lane + 1) & 31);
                next.w = __shfl_sync(kFullMask, next.w, (lane + 1) & 31);
                if (lane + 32 * u + 1 < nvec) __stcs(gv + lane + 32 * u, shift_pair<T>(v[u], next, by));
            }
            const int whole = max(0, nvec - 1);
            const int before = whole > 0 ? head + by : a.vocab, behind = head + by + N * whole;
            const int singles = whole > 0 ? before + a.vocab - behind : a.vocab;
            for (int i = lane; i < singles; i += 32) {
                const int j = i < before ? i : behind + i - before;
                one(j, Vec<T>::to_float(p[j]));
            }
            const unsigned li = static_cast<unsigned>(lab - head - by);
            if (li < static_cast<unsigned>(N * whole) && static_cast<int>(li / N) % 32 == lane) one(lab, x.xl);
        }
    }
}

// ---------------------------------------------------------------------------
// k_join: one CTA per pair (looping). Half of its threads sum the chosen
// sequence's w logp (and w, for averages), half the rejected's, each in a fixed
// order; one thread forms the pair's loss and the factors dloss / dlogp of the
// two sequences' rows. The CTA that finishes last adds the pairs' losses up,
// again in a fixed order. A chain of latencies, about 5 us behind the rows (f64
// sums and butterflies: 7 us): 24 pairs of 6001 rows.
constexpr int kJoinThreads = 256;

// A sum over rows as an unevaluated pair hi + lo of f32: hi the rounded sum,
// lo the sum of the rounding errors, each exact (two-sum), so the pair carries
// about 48 bits. GB300 adds f64 at about two lanes per clock and SM; an f64
// butterfly over 8 warps alone takes longer than all the rest of such a sum.
// lo means nothing once hi has overflowed or an infinity was added.
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 sum2_add(Sum2 a, Sum2 b) {
    const float s = a.hi + b.hi, bb = s - a.hi;
    return Sum2{s, ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo)};
}
__device__ __forceinline__ Sum2 sum2_mul(float w, float x) {
    const float p = __fmul_rn(w, x);
    return Sum2{p, __fmaf_rn(w, x, -p)};
}
__device__ __forceinline__ double sum2_value(Sum2 v) {
    return isfinite(v.hi) ? static_cast<double>(v.hi) + static_cast<double>(v.lo) : static_cast<double>(v.hi);
}
// over aligned groups of kLanes lanes; every lane gets its group's sum
template <int kLanes = 32>
__device__ __forceinline__ Sum2 sum2_warp(Sum2 v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        v = sum2_add(v, Sum2{__shfl_xor_sync(kFullMask, v.hi, o), __shfl_xor_sync(kFullMask, v.lo, o)});
    return v;
}

// log(1 + exp(x))
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    return (x >= 0.0f ? 1.0f : e) / (1.0f + e);
}

__global__ void __launch_bounds__(kJoinThreads) k_join(JoinArgs j) {
    __shared__ Sum2 part[2][2][kJoinThreads / 64];  // [sequence][sum, count][warp]
    __shared__ float factor[2];
    __shared__ bool last;
    launch_dependents();
    constexpr int kHalf = kJoinThreads / 2;
    const int side = threadIdx.x / kHalf, t = threadIdx.x % kHalf, lane = t & 31, warp = t >> 5;
    const int64_t P = j.pairs;
    // the first pair's range is an input: read while the rows are still being read
    int64_t r0 = 0, r1 = 0;
    auto range = [&](int64_t pair) {
        const int64_t s = side == 0 ? pair : P + pair;
        r0 = j.offsets[s];
        r1 = j.offsets[s + 1];
    };
    if (blockIdx.x < P) range(blockIdx.x);
    wait_prerequisites();
    for (int64_t pair = blockIdx.x; pair < P; pair += gridDim.x) {
        if (pair != blockIdx.x) range(pair);
        const bool ok = r0 >= 0 && r0 <= r1 && r1 <= j.rows;
        Sum2 sum{ok ? 0.0f : nan_f(), 0.0f}, count{0.0f, 0.0f};
        if (ok) {
#pragma unroll 4
            for (int64_t r = r0 + t; r < r1; r += kHalf) {
                const float w = j.weights ? j.weights[r] : 1.0f;
                if (w != 0.0f) sum = sum2_add(sum, sum2_mul(w, j.logp[r]));
                if (j.average) count = sum2_add(count, Sum2{w, 0.0f});
            }
        }
        sum = sum2_warp(sum);
        if (j.average) count = sum2_warp(count);
        if (lane == 0) {
            part[side][0][warp] = sum;
            part[side][1][warp] = count;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            double L[2], per[2];
            for (int q = 0; q < 2; ++q) {
                Sum2 v = part[q][0][0], c = part[q][1][0];
                for (int i = 1; i < kHalf / 32; ++i) v = sum2_add(v, part[q][0][i]), c = sum2_add(c, part[q][1][i]);
                const double n = sum2_value(c);
                per[q] = j.average ? (n != 0.0 ? 1.0 / n : 0.0) : 1.0;
                L[q] = sum2_value(v) * per[q];
                j.seq_logp[q == 0 ? pair : P + pair] = static_cast<float>(L[q]);
            }
            double h = L[0] - L[1];
            if (j.ref_seq) h -= static_cast<double>(j.ref_seq[pair]) - static_cast<double>(j.ref_seq[P + pair]);
            float loss, dh;
            if (j.kind == 2) {
                const double off = h - j.margin - 0.5 / j.beta;
                loss = static_cast<float>(off * off);
                dh = static_cast<float>(2.0 * off);
            } else {
                // f32 from here on, a relative error of |z| 2^-24: exp and log1p of one
                // thread in f64 make a step of 4 pairs x 1000 take 10.9 us, not 9.2
                const float z = static_cast<float>(j.beta * h - j.margin), beta = static_cast<float>(j.beta);
                if (j.kind == 1) {
                    // NaN z: NaN, not the 0 of fmaxf
                    loss = z < 1.0f ? 1.0f - z : z - z;
                    dh = z < 1.0f ? -beta : z - z;
                    if (z == INFINITY) loss = dh = 0.0f;
                } else {
                    const float eps = static_cast<float>(j.smoothing);
                    loss = (1.0f - eps) * softplus(-z);
                    dh = -beta * (1.0f - eps) * sigmoid(-z);
                    if (eps != 0.0f) {
                        loss += eps * softplus(z);
                        dh += beta * eps * sigmoid(z);
                    }
                }
            }
            j.loss_pairs[pair] = loss;
            const double f = static_cast<double>(dh) * j.scale * j.inv_t;
            factor[0] = static_cast<float>(f * per[0]);
            factor[1] = static_cast<float>(-f * per[1]);
        }
        __syncthreads();
        if (!ok && t == 0) atomicAdd(&g_objective_status[0], 1ull);
        if (j.row_state && ok) {
            const float f = factor[side];
            for (int64_t r = r0 + t; r < r1; r += kHalf) {
                const float w = j.weights ? j.weights[r] : 1.0f;
                if (w != 0.0f) j.row_state[r].z = f * w;
            }
        }
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(j.done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    Sum2 sum{0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < P; i += kJoinThreads) sum = sum2_add(sum, Sum2{__ldcg(j.loss_pairs + i), 0.0f});
    sum = sum2_warp(sum);
    if (lane == 0) part[side][0][warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        Sum2 v = part[0][0][0];
        for (int i = 1; i < kJoinThreads / 32; ++i) v = sum2_add(v, part[i / (kHalf / 32)][0][i % (kHalf / 32)]);
        *j.loss = static_cast<float>(sum2_value(v) * j.scale);
    }
}

// ---------------------------------------------------------------------------
// k_pair_grad: factor ([y] - p) of every row, a CTA per part of kPartBytes of
// a row. Rows whose factor is 0 (no weight, or in no sequence) are written as
// zeros without being read. HBM-bound: 1400 rows of 128256 bf16, 3/4 of them
// read, 90-92 us, 6.8-7.0 TB/s. 3000 rows' whole step with 256 threads x 4 vectors in
// flight 293 us, x 1 297, 128 x 4 296, parts of 64 KB 297.
constexpr int kPartBytes = 32768;
constexpr int kPairThreads = 256;
constexpr int kPairUnroll = 4;

template <typename T>
__global__ void __launch_bounds__(kPairThreads) k_pair_grad(ObjArgs a, int parts) {
    constexpr int kCols = kPartBytes / static_cast<int>(sizeof(T));
    wait_prerequisites();
    const int64_t row = blockIdx.x / parts;
    const int c0 = static_cast<int>(blockIdx.x % parts) * kCols;
    const int n = min(a.vocab - c0, kCols);
    T *g = static_cast<T *>(a.grad) + row * a.grad_stride + c0;
    const float4 st = a.row_state[row];
    if (st.z == 0.0f) {
        zero_slice(g, n, threadIdx.x, kPairThreads);
        return;
    }
    const T *p = static_cast<const T *>(a.logits) + row * a.stride + c0;
    const int64_t label = a.labels[row] - c0;
    const int lab = label >= 0 && label < n ? static_cast<int>(label) : -1;
    const bool bad = !isfinite(st.x);
    write_slice<T, false, kPairUnroll, kPairThreads>(p, g, n, st.x, a.k, bad ? nan_f() : -st.z * st.y, 0.0f, st.z, lab,
                                                     threadIdx.x);
}

// ---------------------------------------------------------------------------
// k_weighted_sum: one CTA, or for many rows one cluster, launched as a
// programmatic dependent of the row kernel. Thread g of all sums rows g, g +
// all, ... as f32 pairs; a butterfly over each warp, then over the CTA's warps;
// a cluster's CTAs meet in CTA 0's shared memory. A fixed shape for a number
// of rows: the same bits every run. About 2.5 us behind the row kernel (a
// cluster of f64 butterflies: 4.5 us).
constexpr int kSumCtas = 8;
constexpr int kSumThreads = 512;
constexpr int64_t kSumOneCta = 8192;  // rows up to here: one CTA

// `loss` is written by the grid that this one overlaps until wait_prerequisites:
// not read-only for this kernel's whole life, so neither __restrict__ nor a
// non-coherent load, and read behind the wait only.
__global__ void __launch_bounds__(kSumThreads) k_weighted_sum(const float *loss, const float *__restrict__ weights,
                                                              int64_t rows, double scale, float *out) {
    __shared__ Sum2 warp_part[kSumThreads / 32];
    __shared__ double cta_part[kSumCtas];
    const uint32_t rank = cluster_rank(), C = cluster_size();
    if (C > 1) cluster_arrive();  // every CTA has started before CTA 0's shared memory is written
    wait_prerequisites();         // the row losses are complete and visible
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t all = static_cast<int64_t>(C) * kSumThreads;
    Sum2 s{0.0f, 0.0f};
#pragma unroll 4
    for (int64_t i = static_cast<int64_t>(rank) * kSumThreads + tid; i < rows; i += all)
        s = sum2_add(s, weights ? sum2_mul(weights[i], loss[i]) : Sum2{loss[i], 0.0f});
    s = sum2_warp(s);
    if (lane == 0) warp_part[warp] = s;
    __syncthreads();
    if (C > 1) cluster_wait();
    if (warp == 0) {
        const Sum2 r = sum2_warp<kSumThreads / 32>(warp_part[lane % (kSumThreads / 32)]);
        if (C == 1) {
            if (lane == 0) *out = static_cast<float>(sum2_value(r) * scale);
            return;
        }
        if (lane == 0) st_dsmem_f64(peer_smem(&cta_part[rank], 0), sum2_value(r));
    }
    if (C == 1) return;
    cluster_arrive_release();
    cluster_wait();
    if (rank == 0 && tid == 0) {
        double v = 0.0;
        for (int i = 0; i < kSumCtas; ++i) v += cta_part[i];
        *out = static_cast<float>(v * scale);
    }
}

// ---------------------------------------------------------------------------
// launchers

Launches g_launched;

template <typename T, int kMode, bool kEnt>
Kernel &rows_kernel_m(bool warp) {
    static Kernel row_warp(reinterpret_cast<const void *>(&k_obj_rows_warp<T, kMode, kEnt>), false),
        row_cta(reinterpret_cast<const void *>(&k_obj_rows<T, kMode, kEnt>), false);
    return warp ? row_warp : row_cta;
}

template <typename T>
Kernel &rows_kernel_t(ObjMode mode, bool ent, bool warp) {
    if (mode == kObjPreference) return rows_kernel_m<T, kObjPreference, false>(warp);
    if (mode == kObjPolicy)
        return ent ? rows_kernel_m<T, kObjPolicy, true>(warp) : rows_kernel_m<T, kObjPolicy, false>(warp);
    return ent ? rows_kernel_m<T, kObjLogp, true>(warp) : rows_kernel_m<T, kObjLogp, false>(warp);
}

Kernel &rows_kernel(DType t, ObjMode mode, bool ent, bool warp) {
    return t == kF32    ? rows_kernel_t<float>(mode, ent, warp)
           : t == kBF16 ? rows_kernel_t<__nv_bfloat16>(mode, ent, warp)
                        : rows_kernel_t<__half>(mode, ent, warp);
}

template <typename T, bool kEnt>
Kernel &policy_cluster_m(bool staged) {
    static Kernel once(reinterpret_cast<const void *>(&k_policy_staged<T, kEnt>), true),
        twice(reinterpret_cast<const void *>(&k_policy_stream<T, kEnt>), false);
    return staged ? once : twice;
}

template <typename T>
Kernel &policy_cluster_t(bool ent, bool staged) {
    return ent ? policy_cluster_m<T, true>(staged) : policy_cluster_m<T, false>(staged);
}

Kernel &policy_cluster(DType t, bool ent, bool staged) {
    return t == kF32    ? policy_cluster_t<float>(ent, staged)
           : t == kBF16 ? policy_cluster_t<__nv_bfloat16>(ent, staged)
                        : policy_cluster_t<__half>(ent, staged);
}

template <typename T, int kV>
const void *policy_warp_t(bool ent) {
    return ent ? reinterpret_cast<const void *>(&k_policy_warp<T, true, kV>)
               : reinterpret_cast<const void *>(&k_policy_warp<T, false, kV>);
}

template <int kV>
const void *policy_warp_v(DType t, bool ent) {
    return t == kF32    ? policy_warp_t<float, kV>(ent)
           : t == kBF16 ? policy_warp_t<__nv_bfloat16, kV>(ent)
                        : policy_warp_t<__half, kV>(ent);
}

int elem_size(DType t) { return t == kF32 ? 4 : 2; }

bool wants_entropy(const ObjArgs &a) { return a.entropy != nullptr || a.bonus != 0.0f; }

// CTAs per row of few rows: as many as make at most six CTAs per SM, of at
// least kRowsMinBytes each. Measured (us, rows of 151936 bf16, by CTAs per row
// 1 / 2 / 3 / 4 / 6 / 8 / 12 / 16): 16 rows - / 9.2 / - / 7.6 / 6.3 / 6.3 /
// 6.2 / 6.2; 64 rows - / 14.4 / - / 10.4 / 10.3 / 9.8 / 9.3 / 10.4; 128 rows
// - / 14.9 / - / 12.4 / 12.4 / 12.4 / 14.4 / 14.7; 300 rows 26.5 / 22.7 / 21.0
// / 23.7 / 23.9 / 24.0; 456 rows 30.8 / 28.9 / 32.3 / 29.3 / 31.0 / 31.1; 700
// rows 39.1 / 45.6 / 39.7 / 40.9 / 41.6 / 42.2.
int split_of(DType t, int64_t rows, int64_t vocab, const DeviceInfo &dev) {
    const int64_t fill = 6 * static_cast<int64_t>(dev.sms) / std::max<int64_t>(1, rows);
    const int64_t parts = (vocab * elem_size(t) + kRowsMinBytes - 1) / kRowsMinBytes;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(fill, parts), kMaxCluster)));
}

// The same for a forward pass, whose CTAs hold eight to an SM: between one and
// four waves of whole rows the last wave leaves the GPU half empty, and rows
// in up to four parts of at least 64 KB end closer together. Measured (us,
// rows of 151936 bf16, 1 against 4 CTAs per row): 1024 rows (one wave) 52.0,
// 53.9; 1500 81.8, 74.2; 2000 94.2, 93.7; 3000 137.3, 134.8; 7168 rows of
// 128256 256, 277; rows of 64 KB (2048 x 32000) 26.9, 34.9 (32.2 in two).
int forward_split(DType t, int64_t rows, int64_t vocab, const DeviceInfo &dev) {
    const int64_t wave = 8 * static_cast<int64_t>(dev.sms);
    if (rows <= wave || rows >= 4 * wave) return split_of(t, rows, vocab, dev);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4, vocab * elem_size(t) / 65536)));
}

// Where a warp per row beats a CTA per row. Measured (us, f16 policy losses,
// warp against CTA, rows of 2000 / 4000 / 8000 / 16000 / 32000 / 50257): 300
// rows 6.3, 7.8 / 8.0, 8.1 / 8.3, 8.3 / 14.2, 10.3 / 20.9, 12.4 / 30, 14; 1200
// rows 8.2, 10.3 / 10.3, 10.3 / 12.4, 11.5 / 16.4, 15.0 / 24.7, 19.0; 2400 rows
// 8.3, 14.4 / 12.3, 14.4 / 14.5, 16.1 / 20.5, 21.8 / 31.3, 30.8; 8192 rows
// 14.5, 31.0 / 22.6, 32.6 / 31.3, 33.0 / 46.2, 51.2 / 82.8, 78.4 / 126, 123.
bool forward_warp(DType t, int64_t rows, int64_t vocab, const DeviceInfo &dev) {
    const int64_t bytes = vocab * elem_size(t);
    return bytes <= 8192 || (bytes <= 32768 && rows >= 12 * static_cast<int64_t>(dev.sms));
}

// Rows a warp holds in its registers. Measured (us, policy steps, warp against
// staged CTA): 8192 rows of 1000 bf16 12.4, 33.1, of 2000 18.6, 36.7, of 4000
// 31.0, 44.3, of 2000 f32 28.4, 41.0; 300 rows of 2000 bf16 6.3, 8.2. In 250
// registers, rows of 9 / 12 / 16 KB: 41.1, 43.4 / 45.4, 48.5 / 60.6, 55.8.
constexpr int64_t kWarpStepBytes = 8192;

// Every row kernel loops over rows, so fewer clusters (or CTAs of a warp per
// row) only take more rows each.
int64_t capped(int64_t clusters, const ObjArgs &a) {
    clusters = std::min<int64_t>(clusters, int64_t(1) << 20);
    return std::max<int64_t>(1, a.grid_cap > 0 ? std::min(clusters, a.grid_cap) : clusters);
}
int64_t warp_ctas(const ObjArgs &a) {
    constexpr int kPer = kScanThreads / 32;
    return capped((a.rows + kPer - 1) / kPer, a);
}

int cols_of(int64_t vocab, int c) { return static_cast<int>(((vocab + c - 1) / c + 7) & ~int64_t(7)); }

}  // namespace

cudaError_t launch_obj_rows(DType t, ObjMode mode, const ObjArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    if (forward_warp(t, a.rows, a.vocab, dev)) {
        ObjArgs aa = a;
        void *args[] = {&aa};
        LaunchConfig l(warp_ctas(a), kScanThreads, 0, false, s);
        return cudaLaunchKernelExC(&l.cfg, rows_kernel(t, mode, wants_entropy(a), true).fn, args);
    }
    // a cluster of several CTAs takes one row, no more and no fewer
    const int64_t clusters = capped(a.rows, a);
    const int c = clusters == a.rows ? forward_split(t, a.rows, a.vocab, dev) : 1;
    ObjArgs aa = a;
    int cols = cols_of(a.vocab, c);
    void *args[] = {&aa, &cols};
    Kernel &k = rows_kernel(t, mode, wants_entropy(a), false);
    if (cudaError_t e = ready(k, dev); e != cudaSuccess) return e;
    LaunchConfig l(clusters * c, kScanThreads, c, false, s);
    return cudaLaunchKernelExC(&l.cfg, k.fn, args);
}

// Shared memory of a staged CTA that holds `cols` columns at any phase.
static int64_t staged_smem(DType t, int cols) {
    const int N = 16 / elem_size(t);
    return kPolicyHeaderBytes + 16 * static_cast<int64_t>((cols + 2 * N) / N + 1);
}

// CTAs per row of the staged kernel; 0: the row does not fit a cluster. What
// hides a row's latencies (copy, exchange, write) is the bytes an SM holds, so
// the split that holds most of them, in at most six CTAs. Measured (us, CTAs
// per row: time; CTAs per SM x KB): 4096 x 128256 f32 8: 674; 3 x 64, 9: 724;
// 3 x 57, 10: 613; 4 x 51, 11: 638; 4 x 47, 12: 606; 5 x 43, 14: 660; 5 x 37;
// 8192 x 50257 bf16 1: 273; 2 x 98, 2: 246.2; 4 x 50, 3: 246.3; 6 x 34, 4: 257;
// 8 x 25; 4096 x 32000 bf16 1: 75.8; 3 x 64, 2: 74.7; 6 x 32, 3: 82.0; 8 x 21.
// (Before the warps exchanged their states: 256 threads per CTA 640 at 10, 259
// at 2, 79.9 at 1 against 626, 256, 78; clusters persistent over rows, each
// row's copy issued behind the last one's write, 651 -> 675 at 10, 256 -> 276 at
// 2, 78 -> 91 at 2: the hardware's own scheduling balances better.)
// Those are three vocabularies, and the rule was fitted to them. Where one, two
// or three wide slices just fill an SM it prefers them to five narrow ones, and
// loses (TB/s of logits and gradient, about 1.5 GB of logits, CTAs per SM in
// brackets): f32 57344 6.07 (1) beside 58400 7.02, 114688 5.95 (1) beside 116000
// 7.01, 172000 5.26 (1) beside 173500 6.66, 248320 6.16 (2), 256000 5.68 (3);
// bf16 114688 5.17 (1) beside 116000 6.86, 56000 6.57 (2) beside 57344 6.94,
// 145152 6.64 (3) beside 148000 6.79; 28000 and 28800 f32 6.97 and 7.02, 73600
// and 75000 bf16 6.89 and 6.90 alike.
// With few rows a row is split further, like a forward row.
static int staged_split(DType t, int64_t rows, int64_t vocab, const DeviceInfo &dev) {
    constexpr int64_t kPerSm = 228 * 1024, kReserved = 1024;
    int best = 0;
    int64_t most = 0;
    for (int c = 1; c <= kMaxCluster; ++c) {
        const int64_t smem = staged_smem(t, cols_of(vocab, c));
        if (smem > dev.max_smem_optin) continue;
        const int64_t held = std::min<int64_t>(6, kPerSm / (smem + kReserved)) * (smem - kPolicyHeaderBytes);
        // a tie (within 1/32) goes to the larger split while an SM holds fewer than four CTAs
        const bool few = best != 0 && kPerSm / (staged_smem(t, cols_of(vocab, best)) + kReserved) < 4;
        if (held > most + most / 32 || (few && held >= most - most / 32)) best = c, most = held;
    }
    return best == 0 ? 0 : std::max(best, split_of(t, rows, vocab, dev));
}

cudaError_t launch_policy_grad(DType t, const ObjArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    const bool ent = wants_entropy(a);
    const int64_t clusters = capped(a.rows, a);
    ObjArgs aa = a;
    const int64_t bytes = static_cast<int64_t>(a.vocab) * elem_size(t);
    if (bytes <= kWarpStepBytes) {
        void *args[] = {&aa};
        LaunchConfig l(warp_ctas(a), kScanThreads, 0, false, s);
        return cudaLaunchKernelExC(&l.cfg, bytes <= 2048   ? policy_warp_v<4>(t, ent)
                                           : bytes <= 4096 ? policy_warp_v<8>(t, ent)
                                                           : policy_warp_v<16>(t, ent), args);
    }
    int c = staged_split(t, a.rows, a.vocab, dev);
    const bool staged = c > 0;
    if (!staged) c = kMaxCluster;  // rows too long for the shared memory of a cluster
    int cols = cols_of(a.vocab, c);
    void *args[] = {&aa, &cols};
    const int threads = staged ? kStagedThreads : kRowsThreads;
    Kernel &k = policy_cluster(t, ent, staged);
    if (cudaError_t e = ready(k, dev); e != cudaSuccess) return e;
    LaunchConfig l(clusters * c, threads, c, false, s, staged ? static_cast<int>(staged_smem(t, cols)) : 0);
    return cudaLaunchKernelExC(&l.cfg, k.fn, args);
}

cudaError_t launch_join(const JoinArgs &j, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(j.pairs, 8 * static_cast<int64_t>(dev.sms)));
    JoinArgs jj = j;
    void *args[] = {&jj};
    LaunchConfig l(ctas, kJoinThreads, 0, true, s);
    return cudaLaunchKernelExC(&l.cfg, reinterpret_cast<const void *>(&k_join), args);
}

cudaError_t launch_preference_grad(DType t, const ObjArgs &a, const DeviceInfo &, cudaStream_t s) {
    const int cols = kPartBytes / elem_size(t);
    int parts = (a.vocab + cols - 1) / cols;
    const void *fn = t == kF32    ? reinterpret_cast<const void *>(&k_pair_grad<float>)
                     : t == kBF16 ? reinterpret_cast<const void *>(&k_pair_grad<__nv_bfloat16>)
                                  : reinterpret_cast<const void *>(&k_pair_grad<__half>);
    // at most 2^31 - 1 CTAs in one launch: more parts than that are written by further launches
    const int64_t most = ((int64_t(1) << 31) - 1) / parts;
    for (int64_t r0 = 0; r0 < a.rows; r0 += most) {
        ObjArgs aa = a;
        aa.rows = std::min(most, a.rows - r0);
        aa.logits = static_cast<const char *>(a.logits) + r0 * a.stride * elem_size(t);
        aa.grad = static_cast<char *>(a.grad) + r0 * a.grad_stride * elem_size(t);
        aa.labels = a.labels + r0;
        aa.row_state = a.row_state + r0;
        void *args[] = {&aa, &parts};
        LaunchConfig l(aa.rows * parts, kPairThreads, 0, r0 == 0, s);
        cudaError_t e = cudaLaunchKernelExC(&l.cfg, fn, args);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_weighted_sum(const float *loss, const float *weights, int64_t rows, double scale, float *out,
                                cudaStream_t s) {
    const int ctas = rows > kSumOneCta ? kSumCtas : 1;
    LaunchConfig l(ctas, kSumThreads, ctas > 1 ? ctas : 0, true, s);
    return cudaLaunchKernelEx(&l.cfg, k_weighted_sum, loss, weights, rows, scale, out);
}

cudaError_t read_objective_status(unsigned long long out[2], const DeviceInfo &dev, cudaStream_t s) {
    out[0] = out[1] = 0ull;
    if (!g_launched.any(dev)) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_objective_status, sizeof(unsigned long long) * 2, 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

cudaError_t reset_objective_status(const DeviceInfo &dev, cudaStream_t s) {
    if (!g_launched.any(dev)) return cudaSuccess;
    static const unsigned long long zero[2] = {0ull, 0ull};
    return cudaMemcpyToSymbolAsync(g_objective_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace cerows
