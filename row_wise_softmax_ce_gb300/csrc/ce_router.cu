// ce_router.cu -- sm_103a kernels of the routing of rows to experts, and their
// launchers.
//
//   k_route            route_rows: 4 to 32 lanes per row, its columns in shared memory
//   k_zero             its counts
//   k_route_grad       route_grad where only the chosen experts get any
//   k_route_grad_full  where all do
//
// None uses tensor cores: a row is a few hundred columns, and its choice compares.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ce_internal.h"
#include "ce_launch.h"
#include "ce_objectives.cuh"

namespace cerows {

namespace {

// rows that are no distribution, and bad experts
__device__ unsigned long long g_router_status;

__device__ __forceinline__ void count_bad() { atomicAdd(&g_router_status, 1ull); }

// L lanes per row (32 / L rows per warp side by side), lane i of a row
// holding columns i V .. i V + V - 1 in registers.
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

// V consecutive columns from j on (those below n), -inf elsewhere, as vectors.
template <typename T, int V>
__device__ __forceinline__ void load_columns(uint4 (&v)[V / Vec<T>::kN], const T *p, int j, int n) {
    constexpr int N = Vec<T>::kN;
    static_assert(V % N == 0, "whole vectors");
    const bool vectors = (reinterpret_cast<uintptr_t>(p + j) & 15) == 0;
#pragma unroll
    for (int i = 0; i < V / N; ++i) {
        if (vectors && j + N * i + N <= n) {
            v[i] = *reinterpret_cast<const uint4 *>(p + j + N * i);
        } else {
#pragma unroll
            for (int h = 0; h < N / 2; ++h) {
                const int c = j + N * i + 2 * h;
                Vec<T>::set_pair(v[i], h, make_float2(c < n ? Vec<T>::to_float(p[c]) : -INFINITY,
                                                      c + 1 < n ? Vec<T>::to_float(p[c + 1]) : -INFINITY));
            }
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
    const bool vectors = (reinterpret_cast<uintptr_t>(p + j) & 15) == 0;
#pragma unroll
    for (int i = 0; i < V / N; ++i) {
        if (vectors && j + N * i + N <= n) {
            uint4 v = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int h = 0; h < N / 2; ++h) Vec<T>::set_pair(v, h, make_float2(z[N * i + 2 * h], z[N * i + 2 * h + 1]));
            *reinterpret_cast<uint4 *>(p + j + N * i) = v;
        } else {
#pragma unroll
            for (int h = N * i; h < N * i + N; ++h)
                if (j + h < n) p[j + h] = Vec<T>::from_float(z[h]);
        }
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

// both, two columns at a time
__device__ __forceinline__ float2 exp2_of(float2 d) {
    const float2 t = __fmul2_rn(d, make_float2(1.44269504f, 1.44269504f));
    return make_float2(ex2_ftz(t.x), ex2_ftz(t.y));
}
__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 t = __fmul2_rn(z, make_float2(-1.44269504f, -1.44269504f));
    const float2 s = __fadd2_rn(make_float2(ex2_ftz(t.x), ex2_ftz(t.y)), make_float2(1.0f, 1.0f));
    return make_float2(rcp_of(s.x), rcp_of(s.y));
}

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

// CTAs of an SM, by the columns a lane holds: 80 registers a thread at 32 of them,
// 64 else. Measured (us, with counts, of 2 / 3 / 4 / 5 CTAs): 16384 x 256 bf16, 32 a
// lane, 11.8 / 11.2 / 12.0 / 13.8; 65536 x 64, 16 a lane, 12.7 / 11.3 / 12.1 / 12.3.
__host__ __device__ constexpr int route_ctas(int v) { return v > 16 ? 3 : 4; }
// Words of a row in shared memory: its lanes' columns, 16 bytes apart by bank, the
// rows of a warp 32.
__host__ __device__ constexpr int route_row(int lanes, int v) { return lanes * (v + 4) + (lanes == 8 || lanes == 16 ? 8 : 0); }

// k_route: bound by the instructions of the choice, many of them compares at half
// rate, in waves of a chain of latencies (half of the issue slots are taken). So up
// to eight rows share a warp's instructions, and a lane keeps the
// largest of each eight of its columns only: the columns lie in shared memory,
// where the lane that gives one looks for it among eight, takes it out and has the
// largest of the rest. Measured (us, replayed, 16384 x 256 bf16, k = 8, sigmoid
// scores with a bias, 4 of 8 groups, a tenth of the rows padding): 10.6 without
// counts, 11.6 with them; a row a warp, with each lane's two best columns and the
// value of its third in registers, took 16.0 without counts where the first form of
// this took 11.6. 14592 rows, what three CTAs an SM hold at once, take 8.4 without
// counts, 15000 10.2. Counts take 1.4 us more with a CTA per 32 rows than with three an
// SM. The eight searched by the row's lanes, a column each, take fewer instructions
// in a longer chain: 0.3 us slower here, 6% faster at four times the rows.
template <typename T, int L, int V, int kPer>  // kPer slots a lane
__global__ void __launch_bounds__(kRouteThreads, route_ctas(V)) k_route(RouteArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int R = 32 / L, kVecs = V / Vec<T>::kN, kBlocks = V / 8, kLane = V + 4;  // rows of a warp
    static_assert(kPer * L <= kMaxChosen, "slots");
    const int lane = threadIdx.x & 31, sub = lane & (L - 1), row0 = lane & ~(L - 1), E = a.experts, j0 = sub * V;
    const int per = E / a.groups;
    const bool grouped = a.top_groups < a.groups;
    // groups of whole lanes, a power of two of them
    const int wide = per / V;
    const bool by_lanes = grouped && per % V == 0 && (wide & (wide - 1)) == 0 && wide <= L;
    float *all = reinterpret_cast<float *>(smem);
    float *row_keys = all + ((threadIdx.x >> 5) * R + lane / L) * route_row(L, V), *mine = row_keys + sub * kLane;
    int *slots = reinterpret_cast<int *>(all + kRouteWarps * R * route_row(L, V)) +
                 ((threadIdx.x >> 5) * R + lane / L) * kMaxChosen;  // the row's experts
    float *bias = all + kRouteWarps * R * (route_row(L, V) + kMaxChosen);  // as a row, if there is one
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
        // 0 z adds up to 0 unless something of the warp's is infinite or NaN
        float2 probe = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < V; i += 2) probe = __ffma2_rn(make_float2(z[i], z[i + 1]), make_float2(0.0f, 0.0f), probe);
        const bool plain = !__any_sync(kFullMask, isnan(probe.x + probe.y));
        float m = 0.0f;
        bool odd = false;
        if (!plain || !a.sigmoid || !a.bias) {
            m = max_nan(z[0], z[1], z[2]);
#pragma unroll
            for (int i = 3; i + 1 < V; i += 2) m = max_nan(m, z[i], z[i + 1]);
            m = max_nan(m, z[V - 1], z[V - 1]);
            odd = row_ballot<L>(!(m < INFINITY)) != 0;  // a NaN or +inf
            if (odd) {
                m = -INFINITY;
#pragma unroll
                for (int i = 0; i < V; ++i) z[i] = -INFINITY;
            }
            m = row_max<L>(m);
        }
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
            auto biased = [&](auto score, auto masked) {  // two columns at a time
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(b + i);
                    const float2 lo = __fadd2_rn(score(make_float2(z[i], z[i + 1])), make_float2(f.x, f.y));
                    const float2 hi = __fadd2_rn(score(make_float2(z[i + 2], z[i + 3])), make_float2(f.z, f.w));
                    z[i] = !decltype(masked)::value || z[i] > -INFINITY ? lo.x : -INFINITY;
                    z[i + 1] = !decltype(masked)::value || z[i + 1] > -INFINITY ? lo.y : -INFINITY;
                    z[i + 2] = !decltype(masked)::value || z[i + 2] > -INFINITY ? hi.x : -INFINITY;
                    z[i + 3] = !decltype(masked)::value || z[i + 3] > -INFINITY ? hi.y : -INFINITY;
                }
            };
            if (a.sigmoid) {
                if (plain)
                    biased([](float2 x) { return sigmoid2(x); }, std::false_type());
                else
                    biased([](float2 x) { return sigmoid2(x); }, std::true_type());
            } else {
                biased(
                    [&](float2 x) {
                        const float2 d = exp2_of(__fadd2_rn(x, make_float2(-m, -m)));
                        return __fmul2_rn(d, make_float2(rs, rs));
                    },
                    std::true_type());
            }
        }
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(mine + i) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
        auto ranked = [&](float v) { return a.bias || v == -INFINITY ? v : relative_score(v, m, a.sigmoid); };
        bool dropped = false;
        float top_of[kBlocks];  // the largest of each eight
        if (by_lanes) {
            // the two largest, of pairs, of eights and of the lane's
            float g1 = -INFINITY, g2 = -INFINITY;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
                for (int i = 8 * b; i < 8 * b + 8; i += 2) {
                    const float hi = fmaxf(z[i], z[i + 1]), lo = fminf(z[i], z[i + 1]);
                    if (i == 8 * b) {
                        t1 = hi, t2 = lo;
                    } else {
                        t2 = fmaxf(fmaxf(t2, lo), fminf(t1, hi));
                        t1 = fmaxf(t1, hi);
                    }
                }
                top_of[b] = t1;
                if (b == 0) {
                    g1 = t1, g2 = t2;
                } else {
                    g2 = fmaxf(fmaxf(g2, t2), fminf(g1, t1));
                    g1 = fmaxf(g1, t1);
                }
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
                auto key = [&](int j) { return row_keys[j + (kLane - V) * (j / V)]; };
                float g1 = -INFINITY, g2 = -INFINITY;
                int j = g * per;
                if (per & 1) g1 = key(j++);
#pragma unroll 4
                for (int end = g * per + per; j < end; j += 2) {
                    const float x = key(j), y = key(j + 1);
                    const float hi = fmaxf(x, y), lo = fminf(x, y);
                    g2 = fmaxf(fmaxf(g2, lo), fminf(g1, hi));
                    g1 = fmaxf(g1, hi);
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
            // a lane's columns, from group to group
            __syncwarp();
            int g = j0 / per, left = per - j0 % per;
#pragma unroll
            for (int i = 0; i < V; i += 4) {
#pragma unroll
                for (int h = i; h < i + 4; ++h) {
                    if (g >= a.groups || !(kept >> g & 1u)) z[h] = -INFINITY;
                    if (--left == 0) left = per, ++g;
                }
                *reinterpret_cast<float4 *>(mine + i) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
            }
        }
        if (!by_lanes) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                top_of[b] = z[8 * b];
#pragma unroll
                for (int i = 1; i < 8; ++i) top_of[b] = fmaxf(top_of[b], z[8 * b + i]);
            }
        }
        float best = top_of[0];
#pragma unroll
        for (int b = 1; b < kBlocks; ++b) best = fmaxf(best, top_of[b]);
        if (dropped) best = -INFINITY;
        // the k best, one after another: the largest, the lowest column of equals
#pragma unroll
        for (int h = 0; h < kPer; ++h) slots[sub + h * L] = -1;  // for all k of them
        __syncwarp();
        for (int n = 0; n < a.k; ++n) {
            const float top = row_max<L>(best);
            const int owner = __ffs(row_ballot<L>(best == top)) - 1;
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
                slots[n] = j0 + 8 * block + i;
            }
        }
        __syncwarp();
        // lane i of the row has slots i, i + L, ..
        const T *p = static_cast<const T *>(a.logits) + row * a.stride;
        int expert[kPer];
        float g[kPer], largest = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            expert[h] = slots[sub + h * L];
            g[h] = expert[h] >= 0 ? Vec<T>::to_float(p[expert[h]]) : -INFINITY;
            largest = fmaxf(largest, g[h]);
        }
        if (a.renormalise) largest = row_max<L>(largest);
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            g[h] = expert[h] < 0   ? 0.0f
                   : a.renormalise ? relative_score(g[h], largest, a.sigmoid)
                   : a.sigmoid     ? sigmoid(g[h])
                                   : exp_of(g[h] - m) * rs;
            sum += g[h];
        }
        float by = a.scale;
        if (a.renormalise) {
            sum = row_sum<L>(sum);
            by = sum > 0.0f ? a.scale / sum : 0.0f;
        }
        if (odd) by = nan_f();
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            const int n = sub + h * L;
            if (n < a.k && row < a.rows) {
                a.chosen[row * a.k + n] = expert[h];
                a.gates[row * a.k + n] = g[h] * by;
                if (a.counts && expert[h] >= 0) atomicAdd(&counts[expert[h]], 1);
            }
        }
        if (odd && sub == 0) count_bad();
        __syncwarp();  // the row's columns are written anew
    }
    if (a.counts) {
        __syncthreads();
        wait_prerequisites();  // k_zero is done
        for (int j = threadIdx.x; j < E; j += kRouteThreads)
            if (counts[j]) atomicAdd(&a.counts[j], static_cast<unsigned long long>(static_cast<unsigned>(counts[j])));
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
        if (row_ballot<L>(x.c >= 0) == 0) {  // no experts: zeros, whatever the row holds
#pragma unroll
            for (int i = 0; i < V / Vec<T>::kN; ++i) raw[i] = Vec<T>::lowest();
        }
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

// 8, 16 or 32 columns a lane; 16 lanes have 8 (to 128 columns) or 32 (257 to 512)
template <typename T, int L, int kPer>
const void *route_kernel_l(int v) {
    if constexpr (L != 16)
        if (v == 16) return reinterpret_cast<const void *>(&k_route<T, L, 16, kPer>);
    return v == 32 ? reinterpret_cast<const void *>(&k_route<T, L, 32, kPer>)
                   : reinterpret_cast<const void *>(&k_route<T, L, 8, kPer>);
}
template <typename T>
const void *route_kernel_t(int lanes, int v, int k) {
    if (lanes == 32) return route_kernel_l<T, 32, 1>(v);
    if (lanes == 4) return k <= 4 ? route_kernel_l<T, 4, 1>(v) : route_kernel_l<T, 4, 2>(v);
    if (lanes == 16) return k <= 16 ? route_kernel_l<T, 16, 1>(v) : route_kernel_l<T, 16, 2>(v);
    return k <= 8 ? route_kernel_l<T, 8, 1>(v) : route_kernel_l<T, 8, 4>(v);
}
const void *route_kernel(DType t, int lanes, int v, int k) {
    return t == kF32    ? route_kernel_t<float>(lanes, v, k)
           : t == kBF16 ? route_kernel_t<__nv_bfloat16>(lanes, v, k)
                        : route_kernel_t<__half>(lanes, v, k);
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

// As few lanes, `least` or more, as hold a row's columns at `most` each, and `slots` at one each.
void route_shape(const RouteArgs &a, int least, int most, int slots, int *lanes, int *v) {
    for (*lanes = least; *lanes < 32 && (*lanes * most < a.experts || *lanes < slots);) *lanes *= 2;
    for (*v = 8; *lanes * *v < a.experts;) *v *= 2;
}

// Columns of a lane at most: 32, where rows are many and instructions count; 8
// where they are few, a row's latency counts and lanes are to spare. Measured
// (us, bf16, k = 8, sigmoid scores with a bias, 8 / 32 columns): 256 experts in 8
// groups, 32 rows 3.7 / 5.1, 1024 3.9 / 5.5, 2048 5.0 / 5.4, 4096 7.0 / 5.5, 8192
// 11.9 / 7.0, 16384 18.8 / 10.2, 65536 68 / 30; 512 experts in 8 groups, 1024 rows
// 4.6 / 5.6, 4096 7.8 / 7.2, 16384 21.0 / 16.1; 128 experts, 2048 rows 4.2 / 4.4,
// 4096 5.0 / 4.5.
int route_most(const RouteArgs &a, const DeviceInfo &dev) {
    int lanes, v;
    route_shape(a, 8, 8, 1, &lanes, &v);
    return a.rows * lanes <= 12 * 32 * static_cast<int64_t>(dev.sms) ? 8 : 32;
}

}  // namespace

cudaError_t launch_route(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    if (a.counts) {
        LaunchConfig l(1, kRouteThreads, 0, false, s);
        const cudaError_t e = cudaLaunchKernelEx(&l.cfg, k_zero, a.counts, a.experts);
        if (e != cudaSuccess || a.rows == 0) return e;
    }
    int lanes, v;
    // Four lanes a row, of many rows of up to 128 columns, so that eight share a warp's
    // instructions: for eight slots at most, two a lane, and not where groups would be
    // parts of a lane. Measured (us, bf16, sigmoid scores with a bias, 8 / 4 lanes): 32
    // experts, k = 2, 16384 rows 4.5 / 3.3, 30000 6.1 / 4.1; 64, k = 6, 10000 5.1 / 4.8,
    // 16384 6.0 / 5.0, 30000 8.4 / 6.8; 128, k = 8, 16384 7.4 / 6.7, 30000 10.9 / 9.8.
    const int most = route_most(a, dev);
    route_shape(a, most == 32 && a.k <= 8 ? 4 : 8, most, 1, &lanes, &v);
    if (a.top_groups < a.groups && a.experts / a.groups % v != 0) route_shape(a, 8, most, 1, &lanes, &v);
    const int rows = kRouteWarps * (32 / lanes);
    const int smem = 4 * (rows * (route_row(lanes, v) + kMaxChosen) + (a.bias ? route_row(lanes, v) : 0) +
                          (a.counts ? a.experts : 0));  // at most 46592 bytes
    return launch_route_rows(route_kernel(t, lanes, v, a.k), a, lanes, route_ctas(v), smem, a.counts != nullptr, dev, s);
}

cudaError_t launch_route_grad(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s) {
    g_launched.note(dev);
    int lanes, v;
    if (!a.sigmoid && !a.renormalise) {
        route_shape(a, 8, 8, a.k, &lanes, &v);
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

cudaError_t read_router_status(unsigned long long *out, const DeviceInfo &dev, cudaStream_t s) {
    *out = 0ull;
    if (!g_launched.any(dev)) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_router_status, sizeof(*out), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(s);
}

cudaError_t reset_router_status(const DeviceInfo &dev, cudaStream_t s) {
    if (!g_launched.any(dev)) return cudaSuccess;
    static const unsigned long long zero = 0ull;
    return cudaMemcpyToSymbolAsync(g_router_status, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace cerows
