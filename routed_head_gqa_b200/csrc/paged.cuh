// paged.cuh -- arguments of the paged cache's kernels (paged.cu).
#pragma once

#include "common.cuh"

namespace gqe {

constexpr int kPlanMaxSeqs = 16384;  // three prefix sums in shared memory
struct PlanArgs {
    int n_seqs, rows, page_shift, num_pages, max_blocks;
    const int32_t* lengths;   // [n_seqs] cached rows
    const int32_t* new_lens;  // [n_seqs] new rows, -1: the request has ended
    int32_t* free_pages;      // [num_pages] stack
    const int32_t* free_count;
    int32_t* block_table;     // [n_seqs, max_blocks]
    int32_t* lengths_out;
    int32_t* free_count_out;
    int32_t* cu_new;          // [n_seqs + 1]
    int32_t* slots;           // [rows]
    void* status;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream);
struct AppendArgs {
    int64_t rows, k_stride, v_stride, row_bytes;  // strides in bytes
    const char* K_new;
    const char* V_new;
    const int32_t* slots;
    void* K_pages;
    void* V_pages;
    int64_t num_slots;
    void* status;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);

}  // namespace gqe
