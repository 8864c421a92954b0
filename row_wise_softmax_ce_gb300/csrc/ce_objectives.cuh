// ce_objectives.cuh -- device-side building blocks of the objectives over
// sampled answers (token log-probabilities, the clipped policy loss, the
// preference loss): 16-byte vectors of f32, bf16 or f16 logits, the online row
// state at a temperature, and the per-row formulas.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ce_device.cuh"
#include "ce_internal.h"

namespace cerows {

// 16 bytes of logits as packed words; kN elements, unpacked two at a time to
// f32 (exact for the 16-bit types), packed with one rounding to nearest.
template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int kN = 4;
    __device__ static float to_float(float x) { return x; }
    __device__ static float from_float(float x) { return x; }
    __device__ static float2 pair(const uint4 &v, int i) {
        return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                      : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ static void set_pair(uint4 &v, int i, float2 p) {
        if (i == 0)
            v.x = __float_as_uint(p.x), v.y = __float_as_uint(p.y);
        else
            v.z = __float_as_uint(p.x), v.w = __float_as_uint(p.y);
    }
    __device__ static uint4 lowest() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    // the larger of the two, lane by lane; a NaN gives way to a number
    __device__ static uint4 vmax(const uint4 &a, const uint4 &b) {
        return make_uint4(m(a.x, b.x), m(a.y, b.y), m(a.z, b.z), m(a.w, b.w));
    }
    __device__ static float hmax(const uint4 &v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }

  private:
    __device__ static uint32_t m(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
};

__device__ __forceinline__ uint32_t &word(uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    __device__ static float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
    __device__ static float2 pair(const uint4 &v, int i) {
        const uint32_t w = word(v, i);
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ static void set_pair(uint4 &v, int i, float2 p) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
        word(v, i) = *reinterpret_cast<const uint32_t *>(&b);
    }
    __device__ static uint4 lowest() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ static uint4 vmax(const uint4 &a, const uint4 &b) {
        return make_uint4(m(a.x, b.x), m(a.y, b.y), m(a.z, b.z), m(a.w, b.w));
    }
    __device__ static float hmax(const uint4 &v) {
        const uint32_t w = m(m(v.x, v.y), m(v.z, v.w));
        return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }

  private:
    __device__ static uint32_t m(uint32_t a, uint32_t b) {
        const __nv_bfloat162 r =
            __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

template <>
struct Vec<__half> {
    static constexpr int kN = 8;
    __device__ static float to_float(__half x) { return __half2float(x); }
    __device__ static __half from_float(float x) { return __float2half_rn(x); }
    __device__ static float2 pair(const uint4 &v, int i) {
        const uint32_t w = word(v, i);
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    __device__ static void set_pair(uint4 &v, int i, float2 p) {
        const __half2 b = __floats2half2_rn(p.x, p.y);
        word(v, i) = *reinterpret_cast<const uint32_t *>(&b);
    }
    __device__ static uint4 lowest() { return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u); }
    __device__ static uint4 vmax(const uint4 &a, const uint4 &b) {
        return make_uint4(m(a.x, b.x), m(a.y, b.y), m(a.z, b.z), m(a.w, b.w));
    }
    __device__ static float hmax(const uint4 &v) {
        const uint32_t w = m(m(v.x, v.y), m(v.z, v.w));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return fmaxf(f.x, f.y);
    }

  private:
    __device__ static uint32_t m(uint32_t a, uint32_t b) {
        const __half2 r = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

// read-only 16 bytes read once: skip L1
__device__ __forceinline__ uint4 ld_stream_u4(const uint4 *p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}

// ---------------------------------------------------------------------------
// Row state at a temperature, k = log2(e) / T: over the columns seen so far,
// m is their max (NaN skipped), s = sum of 2^((x - m) k) = sum of
// exp((x - m) / T), the one at the max included, and u (entropies only) = the
// sum of 2^((x - m) k) (x - m). The subtraction comes first and is not folded
// into one multiply-add with m k: logits may hold the type's lowest value,
// whose product with k overflows, and a row of nothing else is still a
// (uniform) distribution. A NaN makes s NaN; -inf adds exactly 0; +inf makes
// s NaN. A state without a value above -inf has s = 0 (or NaN).
struct TokState {
    float m, s, u;
};

__device__ __forceinline__ TokState tok_empty() { return TokState{-INFINITY, 0.0f, 0.0f}; }

// d = x - m is taken times a weight of 0 where x is -inf (or far below): keep
// it finite there. A NaN d keeps its NaN weight. For a row's sums, which no
// large factor multiplies here; gradient_exponent is the gradient's.
__device__ __forceinline__ float finite_below(float d) { return fmaxf(d, -1.0e30f); }

// move the state to a max m1 >= s.m (m1 above -inf)
template <bool kEnt>
__device__ __forceinline__ void tok_raise(TokState &st, float m1, float k) {
    const float d = st.m - m1;  // -inf from an empty state
    const float f = ex2_ftz(d * k);
    if (kEnt) st.u = f > 0.0f ? fmaf(st.s, d, st.u) * f : 0.0f;
    st.s *= f;
    st.m = m1;
}

// add the columns of one vector, all <= st.m (or NaN); mm = st.m, or 0 while
// nothing above -inf was seen
template <typename T, bool kEnt>
__device__ __forceinline__ void tok_add(float2 &s2, float2 &u2, const uint4 &v, float mm, float k) {
    const float2 nm = make_float2(-mm, -mm), kk = make_float2(k, k);
#pragma unroll
    for (int i = 0; i < Vec<T>::kN / 2; ++i) {
        const float2 d = __fadd2_rn(Vec<T>::pair(v, i), nm);
        const float2 y = __fmul2_rn(d, kk);
        const float2 e = make_float2(ex2_ftz(y.x), ex2_ftz(y.y));
        s2 = __fadd2_rn(s2, e);
        if (kEnt) u2 = __ffma2_rn(e, make_float2(finite_below(d.x), finite_below(d.y)), u2);
    }
}

// push kU vectors
template <typename T, bool kEnt, int kU>
__device__ __forceinline__ void tok_push(TokState &st, const uint4 (&v)[kU], float k) {
    uint4 mx = v[0];
#pragma unroll
    for (int u = 1; u < kU; ++u) mx = Vec<T>::vmax(mx, v[u]);
    const float mv = Vec<T>::hmax(mx);
    if (mv > st.m) tok_raise<kEnt>(st, mv, k);
    const float mm = st.m == -INFINITY ? 0.0f : st.m;
    float2 s2 = make_float2(0.0f, 0.0f), u2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < kU; ++u) tok_add<T, kEnt>(s2, u2, v[u], mm, k);
    st.s += s2.x + s2.y;
    if (kEnt) st.u += u2.x + u2.y;
}

// push one column
template <bool kEnt>
__device__ __forceinline__ void tok_push1(TokState &st, float x, float k) {
    if (x > st.m) tok_raise<kEnt>(st, x, k);
    const float d = x - (st.m == -INFINITY ? 0.0f : st.m);
    const float e = ex2_ftz(d * k);
    st.s += e;
    if (kEnt) st.u = fmaf(e, finite_below(d), st.u);
}

// merge two states
template <bool kEnt>
__device__ __forceinline__ TokState tok_merge(TokState a, TokState b, float k) {
    const float m = fmaxf(a.m, b.m);
    if (m != -INFINITY) {
        tok_raise<kEnt>(a, m, k);
        tok_raise<kEnt>(b, m, k);
    }
    return TokState{m, a.s + b.s, kEnt ? a.u + b.u : 0.0f};
}

// the warp's largest value (no lane holds a NaN)
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Every lane gets the warp's state: the max first, each lane raised to it
// once, then a butterfly of plain sums.
template <bool kEnt>
__device__ __forceinline__ TokState tok_warp_reduce(TokState st, float k) {
    const float m = warp_max(st.m);
    if (m != -INFINITY) tok_raise<kEnt>(st, m, k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        st.s += __shfl_xor_sync(kFullMask, st.s, o);
        if (kEnt) st.u += __shfl_xor_sync(kFullMask, st.u, o);
    }
    return st;
}

// Over the CTA into warp 0 (other warps return garbage). `red` holds >= 32
// states; contains one __syncthreads.
template <bool kEnt>
__device__ __forceinline__ TokState tok_block_reduce_w0(TokState st, TokState *red, float k) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    st = tok_warp_reduce<kEnt>(st, k);
    if (lane == 0) red[warp] = st;
    __syncthreads();
    TokState r = tok_empty();
    if (warp == 0) {
        if (lane < nwarps) r = red[lane];
        r = tok_warp_reduce<kEnt>(r, k);
    }
    return r;
}

// The states of a cluster's CTAs meet as ce_device.cuh's PushXchg does it:
// a slot holds (m, s, u, x[label] or 0).
__device__ __forceinline__ void tok_publish(PushXchg &x, int64_t n, uint32_t rank, uint32_t C, const TokState &st,
                                            float xl) {
    const int xs = static_cast<int>(n & 1);
    const float4 v = make_float4(st.m, st.s, st.u, xl);
    for (uint32_t r = 0; r < C; ++r) st_async_peer(peer_smem(&x.slot[xs][rank], r), v, peer_smem(&x.bar[xs], r));
}

// all of warp 0; *xl = the x[label] published by CTA `owner`. Re-arms the slot
// for exchange n + 2 (at most N in all).
template <bool kEnt>
__device__ __forceinline__ TokState tok_collect(PushXchg &x, int64_t n, int64_t N, uint32_t C, uint32_t owner,
                                                float *xl, float k, bool *failed) {
    const int lane = threadIdx.x & 31;
    const int xs = static_cast<int>(n & 1);
    if (!*failed) *failed = !mbar_wait_bounded(&x.bar[xs], static_cast<uint32_t>(n >> 1) & 1u);
    TokState q = tok_empty();
    float v = 0.0f;
    if (lane < static_cast<int>(C)) {
        const float4 e = *reinterpret_cast<const float4 *>(&x.slot[xs][lane]);
        q = TokState{e.x, e.y, e.z};
        v = e.w;
    }
    *xl = __shfl_sync(kFullMask, v, static_cast<int>(owner));
    const TokState g = tok_warp_reduce<kEnt>(q, k);
    if (lane == 0 && n + 2 < N) mbar_arrive_expect_tx(&x.bar[xs], 16u * C);
    return g;
}

// The same exchange warp by warp, without a reduction over the CTA first: each
// of the kW warps of the cluster's C CTAs pushes its state into slot n % 2 of
// every CTA (lane r into CTA r), and every warp waits for the kW C states of
// its own CTA's slot and merges them: the same bits in every warp, and no CTA
// barrier. Two slots suffice as for PushXchg: a warp pushes exchange n + 2 only
// after all warps have pushed n + 1, which each does only after it has read
// slot n % 2. x[label] comes with the one warp that owns it, 0 with the others.
template <int kW>
struct WarpXchg {
    float4 slot[2][16 * kW];
    uint64_t bar[2];
};

template <int kW>
__device__ __forceinline__ void warp_xchg_init(WarpXchg<kW> &x, int64_t N, uint32_t C) {
    for (int i = 0; i < 2; ++i) mbar_init(&x.bar[i], 1);
    fence_mbar_init();
    for (int i = 0; i < 2; ++i)
        if (i < N) mbar_arrive_expect_tx(&x.bar[i], 16u * kW * C);
}

template <int kW>
__device__ __forceinline__ void warp_xchg_push(WarpXchg<kW> &x, int64_t n, uint32_t rank, uint32_t C,
                                               const TokState &st, float xl) {
    const int xs = static_cast<int>(n & 1), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < static_cast<int>(C))
        st_async_peer(peer_smem(&x.slot[xs][rank * kW + warp], lane), make_float4(st.m, st.s, st.u, xl),
                      peer_smem(&x.bar[xs], lane));
}

template <int kW, bool kEnt>
__device__ __forceinline__ TokState warp_xchg_collect(WarpXchg<kW> &x, int64_t n, int64_t N, uint32_t C, float *xl,
                                                      float k, bool *failed) {
    const int xs = static_cast<int>(n & 1), lane = threadIdx.x & 31, E = kW * static_cast<int>(C);
    if (!*failed) *failed = !mbar_wait_bounded(&x.bar[xs], static_cast<uint32_t>(n >> 1) & 1u);
    TokState st = tok_empty();
    float v = 0.0f;
#pragma unroll
    for (int i = lane; i < 16 * kW; i += 32) {
        if (i >= E) break;
        const float4 e = x.slot[xs][i];
        st = tok_merge<kEnt>(st, TokState{e.x, e.y, e.z}, k);
        v += e.w;
    }
    if (threadIdx.x == 0 && n + 2 < N) mbar_arrive_expect_tx(&x.bar[xs], 16u * kW * C);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    *xl = v;
    return tok_warp_reduce<kEnt>(st, k);
}

// Loads of logits that are read once: past L1, on the read-only path where the
// kernel writes nothing over them (kRead), by coherent loads where a gradient
// may be written over them (in place).
template <bool kRead>
__device__ __forceinline__ uint4 ld_logits(const uint4 *p) {
    return kRead ? ld_stream_u4(p) : __ldcs(p);
}
template <bool kRead, typename T>
__device__ __forceinline__ T ld_logits(const T *p) {
    return kRead ? __ldg(p) : __ldcs(p);
}

// Push the columns [0, n) at p: a scalar head up to the first 16-byte
// boundary, 16-byte vectors kU at a time per thread, a scalar tail. A partial
// group is filled up with -inf (which adds nothing) rather than read vector by
// vector, so a thread's loads never wait for one another. `early` runs once
// the first group's loads are on their way: a load that it waits for costs no
// more than they do.
template <typename T, bool kEnt, int kU, int kT, bool kRead, typename Early>
__device__ __forceinline__ TokState tok_scan(const T *p, int n, float k, int tid, Early early) {
    TokState st = tok_empty();
    constexpr int N = Vec<T>::kN, kStep = kU * kT;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T)) % N);
    const int head = min(n, (N - off) % N);
    const int nvec = (n - head) / N;
    const int tail = n - head - N * nvec;
    const uint4 *pv = reinterpret_cast<const uint4 *>(p + head);
    uint4 v[kU];
    auto load = [&](int q0) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
            v[u] = q0 + u * kT < nvec ? ld_logits<kRead>(pv + q0 + u * kT) : Vec<T>::lowest();
    };
    T ends[2];
    load(tid);
    if (tid < head) ends[0] = ld_logits<kRead>(p + tid);
    if (tid < tail) ends[1] = ld_logits<kRead>(p + head + N * nvec + tid);
    early();
    tok_push<T, kEnt, kU>(st, v, k);
    int q = tid + kStep;
    for (; q + (kU - 1) * kT < nvec; q += kStep) {
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = ld_logits<kRead>(pv + q + u * kT);
        tok_push<T, kEnt, kU>(st, v, k);
    }
    if (q < nvec) {
        load(q);
        tok_push<T, kEnt, kU>(st, v, k);
    }
    if (tid < head) tok_push1<kEnt>(st, Vec<T>::to_float(ends[0]), k);
    if (tid < tail) tok_push1<kEnt>(st, Vec<T>::to_float(ends[1]), k);
    return st;
}

// ---------------------------------------------------------------------------
// What a row's state, its label's logit and its own numbers come to.
struct TokRow {
    float logp, entropy, loss;
    float mean;  // sum of p_j (x_j - m) / T = log s - H, <= 0 (entropies only)
    // gradient: e (a + b y) + [label] c, y = (x - m) k, e = 2^y
    float m, a, b, c;
};

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fffffff); }

// logp = (x_y - m) / T - log s; H = log s - mean, mean = u / (T s). NaN for a bad label and
// for a row that holds a NaN or +inf, or nothing above -inf.
template <bool kEnt>
__device__ __forceinline__ TokRow tok_row(const TokState &g, float xl, bool lab_ok, float inv_t, float *log_s) {
    TokRow r{};
    const bool bad = !isfinite(g.m) || isnan(g.s);
    *log_s = logf(g.s);
    r.m = g.m;
    r.logp = bad || !lab_ok ? nan_f() : (xl - g.m) * inv_t - *log_s;
    if (kEnt) {
        r.mean = g.u * inv_t / g.s;
        r.entropy = bad ? nan_f() : *log_s - r.mean;
    }
    return r;
}

// The clipped policy loss of one row and its gradient's factors:
//   l = max(-A r, -A clamp(r)) + kl (exp(q - logp) - 1 - (q - logp)) - c H
// with r = exp(logp - old). exp(.) - 1 is expm1f: near q = logp the KL term is
// a square of a small number that a difference from 1 would round away.
template <bool kEnt>
__device__ __forceinline__ TokRow policy_row(const ObjArgs &a, const TokState &g, float xl, bool lab_ok, float w,
                                             float adv, float old, float ref) {
    float log_s;
    TokRow r = tok_row<kEnt>(g, xl, lab_ok, a.inv_t, &log_s);
    const float ratio = expf(r.logp - old);
    const float held = isnan(ratio) ? ratio : fminf(fmaxf(ratio, a.clip_lo), a.clip_hi);
    const float plain = -adv * ratio, clipped = -adv * held;
    r.loss = plain < clipped ? clipped : plain;
    float d = plain < clipped ? 0.0f : plain;  // dl / dlogp
    if (a.kl != 0.0f) {
        const float far = ref - r.logp, em1 = expm1f(far);
        r.loss += a.kl * (em1 - far);
        d -= a.kl * em1;
    }
    const float rcp = 1.0f / g.s, f = a.scale * w * a.inv_t;
    r.c = d * f;
    r.a = -d * rcp * f;
    if (kEnt) {
        r.loss -= a.bonus * r.entropy;
        // log p_j + H = (x_j - m) / T - mean. Not entropy - log s for -mean: that
        // returns it with the entropy's rounding, of the size of the whole
        // difference where a row is nearly flat
        r.a -= a.bonus * r.mean * rcp * f;
        r.b = a.bonus * 0.69314718f * rcp * f;  // y ln 2 = (x - m) / T
    }
    return r;
}

// The exponent as the gradient's entropy term takes it: held at -128, where
// 2^y is 0 already, so that a masked column is 0 times a finite number. b y is
// then of a's own order whatever the temperature and the scale; with x - m in
// place of y, b would hold another 1 / T and -inf or the lowest value times it
// overflow.
__device__ __forceinline__ float gradient_exponent(float y) { return fmaxf(y, -128.0f); }

// e (a + b y) over one vector, rounded once to T
template <typename T, bool kB>
__device__ __forceinline__ uint4 tok_grad_vec(const uint4 &v, float m, float k, float a, float b) {
    const float2 nm = make_float2(-m, -m), kk = make_float2(k, k), aa = make_float2(a, a), bb = make_float2(b, b);
    uint4 o;
#pragma unroll
    for (int i = 0; i < Vec<T>::kN / 2; ++i) {
        const float2 d = __fadd2_rn(Vec<T>::pair(v, i), nm);
        const float2 y = __fmul2_rn(d, kk);
        const float2 e = make_float2(ex2_ftz(y.x), ex2_ftz(y.y));
        const float2 c = kB ? __ffma2_rn(make_float2(gradient_exponent(y.x), gradient_exponent(y.y)), bb, aa) : aa;
        Vec<T>::set_pair(o, i, __fmul2_rn(e, c));
    }
    return o;
}

// one element, and the label's: the same bits as the vector's, the one-hot
// term c added in the product's own rounding
template <bool kB>
__device__ __forceinline__ float tok_grad1(float x, float m, float k, float a, float b) {
    const float y = __fmul_rn(x - m, k);
    return __fmul_rn(ex2_ftz(y), kB ? __fmaf_rn(gradient_exponent(y), b, a) : a);
}
template <bool kB>
__device__ __forceinline__ float tok_label1(float x, float m, float k, float a, float b, float c) {
    const float y = __fmul_rn(x - m, k);
    return __fmaf_rn(ex2_ftz(y), kB ? __fmaf_rn(gradient_exponent(y), b, a) : a, c);
}

}  // namespace cerows
