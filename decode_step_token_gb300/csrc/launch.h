// launch.h -- internal interface between the host code of the C ABI
// (sampler_api.cu) and the translation units that hold the kernels. Not part
// of the public header.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "sampler.h"

namespace dst {

struct SliceHdr;   // defined with the slice kernel
struct SliceBody;

// ---------------------------------------------------------------- slice kernel
// Small batches without history and without probs / logprobs outputs.
struct SliceGeometry {
    int G;           // slices per row
    int W;           // elements per slice
    int units;       // rows x slices, one warp's work each
    int ctas;        // grid
    size_t smem;     // dynamic shared memory per CTA
};

struct SliceWorkspace {
    void* hdr;       // [rows][G] 16-byte slice headers
    void* body;      // [rows][G] slice bodies
    uint32_t* cnt;   // [rows * kSliceCntStride] per row: its arrival counter (alone in a 128-byte line)
                     // and a 256-bin histogram of its truncated units' sketch keys; zero between launches
    unsigned long long* stats;  // may be NULL
};

// Limits and record sizes of the slice kernel (checked against its own
// definitions in slice_kernel.cu).
constexpr int kSliceMaxRows = 256;
constexpr int kSliceMaxSlices = 128;
constexpr size_t kSliceHdrBytes = 16;
constexpr size_t kSliceBodyBytes = 464;
constexpr int kSliceCntStride = 32 + 256;  // 32-bit words between two rows' counters (counter line + histogram)

// True when this library's kernels load on the current device.
bool kernels_loadable();

// Geometry for n_rows x vocab of esize-byte logits on `sms` SMs; false when the
// slice kernel does not take the shape.
bool slice_geometry(int64_t n_rows, int64_t vocab, int esize, int sms, SliceGeometry* g);

// Grant the kernel (every variant) its dynamic shared memory (once per device
// and size).
int slice_prepare(int dtype, size_t smem);

// The slice kernel's variants with the extensions of sampler_sample_ex, for the
// logits' type: the filters alone, or (lp) everything (built in
// slice_kernel_ext.cu).
void* slice_ext_kernel(int dtype, bool lp);

// Enqueue one slice-kernel launch. max_polls bounds each wait on a staging copy.
// ext: the step's extensions (NULL: none). pdl: launched as the programmatic
// dependent of the kernel before it on the stream (it waits for that grid
// before it reads the logits).
int slice_launch(const sampler_args_t* a, const sampler_ext_t* ext, const SliceGeometry& g,
                 const SliceWorkspace& ws, uint32_t max_polls, bool pdl, cudaStream_t stream);

// ---------------------------------------------------------------- LM-head GEMM
constexpr int kLmHeadMaxRows = 256;  // hidden rows of one launch (the MMA's N)

struct LmHeadPlan {
    int NT;              // rows rounded up to 16
    int stages;          // operand stages in shared memory
    uint32_t tmem_cols;  // tensor-memory columns (two accumulators)
    int tiles;           // 128-row weight tiles
    int kchunks;         // 64-wide K stages per tile
    int ctas;            // persistent grid
    size_t smem;
};

bool lm_head_plan(int64_t rows, int64_t vocab, int64_t hidden_dim, int sms, LmHeadPlan* plan);
int lm_head_prepare(size_t smem);
// logits [rows, ldl] bf16 = hidden x weight^T; timeouts counts CTAs whose wait gave up.
int lm_head_launch(const sampler_lm_head_t* g, void* logits, int64_t ldl, int64_t rows, int64_t vocab,
                   const LmHeadPlan& plan, unsigned long long* timeouts, cudaStream_t stream);

// ---------------------------------------------------------------- fork-group kernel
// Everything the slice kernel does not take.
struct GroupGeometry {
    int parts;       // CTAs per cluster
    int slice;       // elements per CTA
    int list_cap, part_cap;
    uint32_t off_list, off_cand, off_cnt, off_stage;
    size_t smem;
};

bool group_geometry(int64_t V, int esize, bool pen, GroupGeometry* g);

// Clusters of the fork-group kernel that fit on the device at once (for the
// given variant and shared memory); 0 on error.
int group_occupancy(int dtype, bool pen, const GroupGeometry& g);

int group_prepare(int dtype, bool pen, size_t smem);

// work: two zeroed counters of the handle (the kernel leaves them zeroed)
int group_launch(const sampler_args_t* a, const GroupGeometry& g, int clusters, uint32_t* work, cudaStream_t stream);

constexpr uint64_t kWaitNs = 2000000000ull;  // a wait inside the kernels below gives up after 2 s

// ---------------------------------------------------------------- scoring and losses
// One row's record: its share of the logits' gradient, with u = (x_v - ref) * c
// d loss / d x_v = 2^u * (k0 + k1 * u) + (v == token ? at_token : 0).
struct RowRecord {
    float c;         // log2(e) / T
    float ref;       // the row's largest logit
    float k0;
    union {
        float k1;
        uint32_t answers;  // pairs (whose k1 is 0): the answers that the row lies in
    };
    float at_token;
    int32_t token;   // -1: the row is written as zeros (left out)
    float inv_s, inv_t;  // 1 / the row's sum of exponentials; 1 / T
};
constexpr size_t kRowRecordBytes = sizeof(RowRecord);

struct RowWorkspace {
    RowRecord* records;  // [rows]
    double* terms;       // [rows] each row's share of the loss (pairs: its logprob)
    double* pair_terms;  // [rows] each pair's share of the loss
    int64_t rows;        // min(the handle's max_rows, SAMPLER_LOSS_MAX_ROWS)
    uint32_t* ticket;    // blocks (or clusters) that have ended; zero between launches
};

enum RowMode : int { kModeScore = 0, kModeScoreGrad = 1, kModePolicy = 2, kModePairs = 3 };

struct LossParams {
    sampler_rows_t rows;
    int mode;
    const float* grad_logprob;  // kModeScoreGrad
    const float* grad_entropy;
    sampler_policy_t policy;    // kModePolicy
    RowWorkspace ws;
    uint64_t wait_ns;           // kWaitNs, or 0: every wait gives up
};

// Clusters that the device holds at once, by the logits' type, gradient, entropy
// and cluster size (1, 2, 4, 8, 16); 0 = not asked yet.
struct RowOccupancy {
    int clusters[2][2][2][5];
};

// Statistics of every row, what the mode makes of them, and (kModeScoreGrad,
// kModePolicy with out_grad) the logits' gradient.
int rows_launch(const LossParams& p, int sms, RowOccupancy* occ, cudaStream_t stream);
// The pairs' loss from the rows' logprobs, and each row's record for pairs_grad_launch.
int pairs_launch(const sampler_rows_t& rows, const sampler_preference_t& pref, const RowWorkspace& ws,
                 cudaStream_t stream);
// dependent: pairs_launch has been called just before on the stream.
int pairs_grad_launch(const sampler_rows_t& rows, const RowWorkspace& ws, bool dependent, cudaStream_t stream);

// ---------------------------------------------------------------- the most likely tokens
// What a part of a row leaves: sums of what is not among its largest, and those.
struct TopPart {
    float ref, s, t;
    int32_t count, bad, failed;  // bad: a NaN or +inf logit; failed: a wait gave up
};
constexpr int kTopUnits = 1024;  // parts of rows that a call may have, where it cuts rows

struct TopWorkspace {
    TopPart* parts;     // [kTopUnits]
    uint64_t* keys;     // [kTopUnits][SAMPLER_MAX_ALTERNATIVES]
    uint32_t* tickets;  // [kTopUnits] parts of a row that are done; zero between launches
};

struct TopParams {
    sampler_rows_t rows;
    sampler_top_t top;
    TopWorkspace ws;
    int parts, part_vecs;  // of a row, worked out by the launch
    uint64_t wait_ns;
};

// Whether a handle has granted the kernels their shared memory, by the logits' type and entropy.
struct TopGrants {
    bool granted[2][2], short_granted[2][2];
};

int top_launch(const TopParams& params, int sms, TopGrants* grants, cudaStream_t stream);

// ---------------------------------------------------------------- distillation
struct DistillParams {
    sampler_rows_t rows;
    sampler_distill_t distill;
    RowWorkspace ws;  // its terms and ticket
    int part_vecs, buffers;  // worked out by the launch
    uint64_t wait_ns;
};

// Clusters that the device holds at once, by the kernel's form, the logits' type, gradient and size of the cluster; 0 = not
// asked yet.
struct DistillOccupancy {
    int clusters[2][2][2][16];
};

int distill_launch(const DistillParams& params, int sms, DistillOccupancy* occ, cudaStream_t stream);

// ---------------------------------------------------------------- 8-bit LM head
int quantize_launch(const sampler_quantize_t& q, int sms, cudaStream_t stream);

// Whether a handle has granted the head's kernels their shared memory, by few or
// many rows and the logits' type.
struct ScaledHeadGrants {
    bool granted[2][2];
};

// dtype: the logits' type
int scaled_head_launch(const sampler_scaled_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows,
                       int64_t vocab, int sms, uint64_t wait_ns, unsigned long long* timeouts,
                       ScaledHeadGrants* grants, cudaStream_t stream);

// ---------------------------------------------------------------- 4-bit LM head
int micro_quantize_launch(const sampler_micro_t& q, int sms, cudaStream_t stream);
int micro_rows_launch(const sampler_micro_rows_t& q, cudaStream_t stream);

// Whether a handle has granted the head's kernels their shared memory, by block size,
// the form of the tiles and the logits' type.
struct MicroHeadGrants {
    bool granted[2][3][2];
};

int micro_head_launch(const sampler_micro_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows, int64_t vocab,
                      int sms, uint64_t wait_ns, unsigned long long* timeouts, MicroHeadGrants* grants,
                      cudaStream_t stream);

}  // namespace dst
