// handle.h -- what a sampler_t points to, shared by the host code of the C ABI
// (sampler_api.cu and train_api.cu). Not part of the public header.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "launch.h"
#include "sampler.h"

struct sampler_s {
    int device;
    int num_sms;
    int64_t max_rows, max_vocab, max_history;
    uint32_t flags;
    uint32_t max_polls;  // of a wait on a staging copy
    uint64_t wait_ns;    // of a wait inside the kernels of scoring, the losses and the 8-bit LM head
    // slice kernel: per-(row, slice) records and per-row arrival counters
    dst::SliceWorkspace slice_ws;
    int slice_rows;
    size_t slice_smem_set[2];  // dynamic shared memory already granted per dtype
    // fork-group kernel
    size_t grp_smem_set[4];
    size_t lmh_smem_set;     // LM-head GEMM
    size_t grp_occ_smem[4];  // shared memory of the cached cluster occupancy below
    int grp_occ[4];          // co-resident clusters of the fork-group kernel
    uint32_t* grp_work;      // the fork-group kernel's chunk counters (zero between launches)
    unsigned long long* stats;  // device counters (diagnostics)
    dst::RowWorkspace row_ws;  // the losses: one record per row, and a launch's ticket
    dst::RowOccupancy row_occ;
    dst::ScaledHeadGrants head_grants;
    dst::MicroHeadGrants micro_grants;
    dst::TopWorkspace top_ws;  // parts of rows of sampler_score_top
    dst::TopGrants top_grants;
    dst::DistillOccupancy distill_occ;
    // staging for sampler_sample_host
    unsigned char* stage_base;
    size_t stage_bytes;
};

namespace dst {

// Restores the calling thread's current device when it goes out of scope.
struct DeviceGuard {
    int prev = -1;
    DeviceGuard() { cudaGetDevice(&prev); }
    ~DeviceGuard()
    {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

// A sampling step's host checks (sampler_args_t and its extensions), and the
// step itself once they have passed, on the handle's device made current. pdl:
// as the programmatic dependent of the kernel enqueued before it, where the
// small-batch kernel takes the step.
int sample_check(sampler_t h, const sampler_args_t* args, const sampler_ext_t* ext);
int sample_launch(sampler_t h, const sampler_args_t* args, const sampler_ext_t* ext, bool pdl, cudaStream_t stream);

}  // namespace dst
