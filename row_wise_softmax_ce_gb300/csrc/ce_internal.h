// ce_internal.h -- launch plans and kernel launchers shared by the C ABI
// (ce_api.cu) and the kernels (ce_kernels.cu). Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace cerows {

enum Path : int {
    kPathAuto = 0,
    kPathStaged = 1,
    kPathStream = 2,
    kPathRetired3 = 3,  // once a ring-of-copies kernel; now refused
    kPathStagedPerRow = 4,
    kPathFlat = 5,
    kPathWarp = 6,  // one warp per row (ce_rows, argmax, slice statistics of many short rows)
    kPathRing = 7,  // argmax through a ring of bulk-copied row chunks (few long rows)
};
enum Op : int { kOpRows = 0, kOpGrad = 1, kOpArgmax = 2, kOpSoftmax = 3, kOpLogSoftmax = 4, kOpCandidates = 5 };
// What the fused two-pass kernels write from a row's (max, exp-sum) state.
enum Mode : int { kModeGrad = 0, kModeSoftmax = 1, kModeLogSoftmax = 2 };

// candidatesInto: a workgroup of 256 threads, each keeping its TOP_EACH = 4
// largest values; a row's candidates are 2048 floats (value, token pairs).
constexpr int kCandThreads = 256;
constexpr int kTopEach = 4;
constexpr int kCandRow = 2 * kCandThreads * kTopEach;
constexpr int kCandMaxCluster = 8;
// Shared memory of the candidates kernel: mbarriers and counters, a ring of
// kCandStages chunks of a row (B blocks of 256 columns on the 16-byte grid of
// the logits: up to 3 floats before the chunk and 1 after), and, for rows
// split over a cluster, the lists CTA 0 pulls from the others. Two chunk
// sizes: 15 blocks keep a split-row CTA at 54 KB (four per SM) for grids of
// many CTAs; 32 blocks (104 KB, two per SM) halve the per-chunk overhead where
// the grid has at most two CTAs per SM (256 decode rows of 151936: 39.1 ->
// about 33 us).
constexpr int kCandChunkSmall = 15;
constexpr int kCandChunkLarge = 32;
constexpr int kCandStages = 3;
constexpr int kCandHeaderBytes = 48;
constexpr int kCandListBytes = kCandThreads * kTopEach * 8;
constexpr int kRingArgmaxSlotBytes = kCandThreads * 8;  // one (value, column) per thread (split rows)
constexpr int cand_stage_floats(int blocks) { return blocks * kCandThreads + 4; }
constexpr int cand_ring_bytes(int blocks) { return kCandHeaderBytes + kCandStages * cand_stage_floats(blocks) * 4; }
constexpr int cand_max_smem_bytes(int blocks) { return cand_ring_bytes(blocks) + kCandListBytes; }
static_assert(kCandStages * 12 <= kCandHeaderBytes && kCandHeaderBytes % 16 == 0 &&
                  cand_stage_floats(kCandChunkSmall) % 4 == 0 && cand_stage_floats(kCandChunkLarge) % 4 == 0 &&
                  4 * (cand_max_smem_bytes(kCandChunkSmall) + 1024) <= 228 * 1024 &&
                  2 * (cand_max_smem_bytes(kCandChunkLarge) + 1024) <= 228 * 1024 && kCandChunkLarge <= 32,
              "candidates smem layout: four small-chunk or two large-chunk CTAs per SM; a 32-bit mark mask");
constexpr int kSplitThreads = 256;

// Per-CTA shared bytes the staged kernel reserves before its row buffer.
constexpr int kStagedHeaderBytes = 2048;
constexpr int kMaxCluster = 16;
// Largest CTA each kernel family is compiled for (its __launch_bounds__).
constexpr int kStagedMaxThreads = 256;
constexpr int kStreamMaxThreads = 256;
struct Plan {
    int path = kPathStream;
    int cluster = 1;       // CTAs per row (a thread-block cluster)
    int threads = 256;     // threads per CTA
    int smem = 0;          // dynamic shared bytes per CTA
    int cols = 0;          // columns per CTA (a multiple of 4)
    int chunk = 0;         // candidates and ring argmax: blocks of 256 columns per ring chunk
    int64_t clusters = 0;  // clusters in the grid (each loops over rows)
};

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    int device = -1;
    int sms = 0;
    int max_smem_optin = 0;  // per block
    int cc_major = 0, cc_minor = 0;
};

// Arguments of one launch; unused pointers are null.
struct Args {
    const float *logits;
    int64_t rows;
    int vocab;
    int64_t stride;
    const int64_t *labels;
    float scale;
    float *grad;
    float *loss;
    float *top;
    float *stats;   // vocab-sharded rows: [rows] float4 (m, t, top, x[label]) of the slice
    int64_t col0;   // vocab-sharded rows: global column of the slice's first column
    const uint64_t *row_at;  // rows given by address (argmaxInto's indirect form), or null
};

// -- the objectives over sampled answers (ce_objectives.cu) ---------------------
enum DType : int { kF32 = 0, kBF16 = 1, kF16 = 2 };
// What a forward kernel writes of a row beside its log-probability.
enum ObjMode : int { kObjLogp = 0, kObjPolicy = 1, kObjPreference = 2 };

// Arguments of one launch; unused pointers are null.
struct ObjArgs {
    const void *logits;
    int64_t rows;
    int vocab;
    int64_t stride;
    const int64_t *labels;
    const float *weights;  // null: every row counts 1; a row of weight 0 is not read
    float k, inv_t;        // log2(e) / T, 1 / T
    float scale;
    float *loss, *logp, *entropy;  // [rows]
    void *grad;
    int64_t grad_stride;
    // policy
    const float *old_logp, *ref_logp, *adv;
    float clip_lo, clip_hi, kl, bonus;
    // preference: sequence s is rows offsets[s] .. offsets[s + 1] - 1
    const int64_t *offsets;
    int64_t pairs;
    float4 *row_state;  // [rows] (m, 1 / s, factor, -)
    uint32_t *done;     // join CTAs that have written their pairs
    int64_t grid_cap;   // at most this many clusters (0: no cap)
};

// The join of a preference batch's rows into sequences, pairs and the loss.
struct JoinArgs {
    const float *logp, *weights;  // [rows]
    int64_t rows;
    const int64_t *offsets;
    int64_t pairs;
    const float *ref_seq;  // [2 pairs] or null
    int kind;
    bool average;
    double beta, smoothing, margin, scale, inv_t;
    float *seq_logp, *loss_pairs, *loss;
    float4 *row_state;  // null: forward only
    uint32_t *done;
};

cudaError_t launch_obj_rows(DType t, ObjMode mode, const ObjArgs &a, const DeviceInfo &dev, cudaStream_t s);
cudaError_t launch_policy_grad(DType t, const ObjArgs &a, const DeviceInfo &dev, cudaStream_t s);
cudaError_t launch_join(const JoinArgs &j, const DeviceInfo &dev, cudaStream_t s);
cudaError_t launch_preference_grad(DType t, const ObjArgs &a, const DeviceInfo &dev, cudaStream_t s);
// *out = scale * sum of weights[i] * loss[i] (weights null: 1), summed as pairs of
// f32 (hi, lo); f64 joins the last parts and applies the scale. Infinite once a
// partial sum passes f32, whatever the scale.
cudaError_t launch_weighted_sum(const float *loss, const float *weights, int64_t rows, double scale, float *out,
                                cudaStream_t s);
// nothing to read or reset on a device that has launched no objective
cudaError_t read_objective_status(unsigned long long out[2], const DeviceInfo &dev, cudaStream_t s);
cudaError_t reset_objective_status(const DeviceInfo &dev, cudaStream_t s);

// -- the choices made from a row's softmax (ce_choices.cu, ce_router.cu) -----------------------
// Arguments of sample_rows and verify_drafts; unused pointers are null.
struct ChoiceArgs {
    const void *logits;
    int64_t rows;
    int vocab;
    int64_t stride;
    float temperature;          // 0: greedy
    const float *temperatures;  // [rows], or null: `temperature` for every row
    const float *uniforms;      // [rows], of a verification [rows, 2]: accept, draw
    int64_t *tokens;            // [rows]
    float *logp;                // [rows] or null
    // verification: request s is rows offsets[s] .. offsets[s + 1] - 1
    const void *draft_logits;  // null: the drafts were not drawn by a model
    int64_t draft_stride;
    const int64_t *drafts;  // [rows], negative: none
    const int64_t *offsets;
    int64_t requests;
    int64_t *accepted;  // [requests]
    // scratch
    int steps;           // of a row
    float2 *states;      // [2 rows, steps] (m, s)
};

constexpr int kMaxExperts = 1024;
constexpr int kMaxChosen = 32;  // experts of a row: its slots in shared memory; of the gradient a lane each
constexpr int kMaxGroups = 32;  // a bit each of what a row keeps

// Arguments of route_rows and route_grad; unused pointers are null.
struct RouteArgs {
    const void *logits;
    int64_t rows;
    int experts;
    int64_t stride;
    int k, groups, top_groups, group_top;
    bool sigmoid, renormalise;
    float scale;
    const float *bias;     // [experts]
    const float *weights;  // [rows], 0: a padding row
    int64_t *chosen;       // [rows, k]
    float *gates;          // [rows, k]
    unsigned long long *counts;  // [experts]
    const float *gates_grad;     // [rows, k]
    void *grad;
    int64_t grad_stride;
    int64_t grid_cap;
};

// bytes of scratch; requests < 0: of a sampling
int64_t choice_bytes(DType t, int64_t rows, int64_t vocab, int64_t requests);
cudaError_t launch_sample(DType t, const ChoiceArgs &a, void *work, const DeviceInfo &dev, cudaStream_t s);
cudaError_t launch_verify(DType t, const ChoiceArgs &a, void *work, const DeviceInfo &dev, cudaStream_t s);
cudaError_t launch_route(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s);
cudaError_t launch_route_grad(DType t, const RouteArgs &a, const DeviceInfo &dev, cudaStream_t s);
// nothing to read or reset on a device that has launched none of them
cudaError_t read_choice_status(unsigned long long *out, const DeviceInfo &dev, cudaStream_t s);
cudaError_t reset_choice_status(const DeviceInfo &dev, cudaStream_t s);
cudaError_t read_router_status(unsigned long long *out, const DeviceInfo &dev, cudaStream_t s);
cudaError_t reset_router_status(const DeviceInfo &dev, cudaStream_t s);

cudaError_t set_kernel_attributes(const DeviceInfo &dev);
cudaError_t max_active_clusters(const Plan &p, Op op, int *n);

cudaError_t launch_rows_stream(const Plan &p, const Args &a, bool stats, cudaStream_t s);
// the two-pass kernels (staged or stream, as p.path says) for kOpGrad,
// kOpSoftmax or kOpLogSoftmax; the output row goes to a.grad
cudaError_t launch_fused(const Plan &p, Op op, const Args &a, cudaStream_t s);
// cand: rows * kCandRow floats
cudaError_t launch_candidates(const Plan &p, const Args &a, float *cand, cudaStream_t s);
// one resident wave on a device of `sms` SMs
cudaError_t launch_split_sum(float *y, const float *parts, int64_t total, int64_t splits, bool add, int sms,
                             cudaStream_t s);
cudaError_t launch_mean(const float *loss, int64_t rows, double *out, cudaStream_t s);
// vocab-sharded rows: combine `shards` slices' statistics; gradient of one slice
cudaError_t launch_stats_combine(const float *stats, int64_t shards, int64_t rows, int64_t vocab_total,
                                 const int64_t *labels, float *loss, float *top, float *combined, int sms,
                                 cudaStream_t s);
cudaError_t launch_grad_from_stats(const Args &a, const float *combined, int sms, cudaStream_t s);
// argmax of few long rows split evenly over `ctas` CTAs; ws: 8 * (ctas + rows) bytes
cudaError_t launch_argmax_flat(const Args &a, int ctas, void *ws, cudaStream_t s);

// a plain read of `bytes` (a multiple of 16, 16-byte aligned) in one resident wave
cudaError_t launch_read_probe(const void *p, int64_t bytes, uint32_t *out, int sms, cudaStream_t s);

cudaError_t read_status(unsigned long long out[2], cudaStream_t s);
cudaError_t reset_status(cudaStream_t s);

}  // namespace cerows
