// paged.cu -- the paged KV cache of a serving step: block tables and slot maps
// from the requests' lengths (gqe_page_plan), and the step's new K/V rows
// written to their slots (gqe_kv_append).
#include "paged.cuh"

namespace gqe {
namespace {

constexpr uint32_t kWherePlan = 9, kWhereAppend = 10;  // status "where" ids

// ---------------------------------------------------------------------------
// Plan.  With have_b = ceil(l_b / ps) and need_b = ceil((l_b + n_b) / ps) -
// have_b, everything a request takes or gives back is an interval of a prefix
// sum over the requests: its packed rows, the pages it takes off the stack and,
// for an ended one, the pages it puts back.  The sums are over a few thousand
// integers, so every block forms them anew in shared memory (one pass over the
// lengths, from L2) and then writes its share of the rows, pages and requests,
// finding the owner of an index by a search of the prefix: one launch, no
// exchange between blocks, and the same result in every run.  A page taken from
// above the old top of the stack is one given back in this call; it is read from
// the ended request's block table, which no block writes.
// Latency bound: the launch, two dependent rounds of loads and the scan: 3.5 us for
// 8 decodes, 6.3 us for 1000 requests with 230 KB of lengths, pages and slots
// (of which a kernel that does nothing takes 2).
constexpr int kPlanThreads = 512;

struct PlanSums {
    int64_t rows, need, back;
};

__device__ __forceinline__ int find_owner(const int32_t* prefix, int n, int x) {
    int lo = 0, hi = n - 1;  // the last request whose prefix does not exceed x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads)
page_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t prefix[];  // [n + 1] rows, [n + 1] pages taken, [n + 1] pages given back
    __shared__ PlanSums warp_sum[kPlanThreads / 32];
    __shared__ int bad;
    const int n = a.n_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* rows_at = prefix;
    int32_t* need_at = prefix + (n + 1);
    int32_t* back_at = prefix + 2 * (n + 1);
    const int64_t ps = (int64_t)1 << a.page_shift, cap = ps * a.max_blocks;
    if (tid == 0) bad = 0;
    __syncthreads();

    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, n), b1 = min(b0 + per, n);
    PlanSums mine = {0, 0, 0};
    bool wrong = false;
    for (int b = b0; b < b1; ++b) {
        const int64_t l = a.lengths[b], add = a.new_lens[b];
        if (l < 0 || add < -1 || l + (add > 0 ? add : 0) > cap) {
            wrong = true;
            continue;
        }
        const int64_t have = (l + ps - 1) >> a.page_shift;
        if (add < 0) {
            mine.back += have;
        } else {
            mine.rows += add;
            mine.need += ((l + add + ps - 1) >> a.page_shift) - have;
        }
    }
    if (wrong) bad = 1;
    PlanSums run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t r = __shfl_up_sync(0xffffffffu, run.rows, d), p = __shfl_up_sync(0xffffffffu, run.need, d),
                      g = __shfl_up_sync(0xffffffffu, run.back, d);
        if (lane >= d) {
            run.rows += r;
            run.need += p;
            run.back += g;
        }
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    PlanSums at = {run.rows - mine.rows, run.need - mine.need, run.back - mine.back}, total = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const PlanSums s = warp_sum[w];
        if (w < warp) {
            at.rows += s.rows;
            at.need += s.need;
            at.back += s.back;
        }
        total.rows += s.rows;
        total.need += s.need;
        total.back += s.back;
    }
    // Refused as a whole, by every block alike: nothing is taken or given back.
    const int64_t free0 = *a.free_count;
    const bool no_pages = total.need > free0 + total.back;
    const bool refused = bad != 0 || free0 < 0 || free0 + total.back > a.num_pages || total.rows > a.rows || no_pages;
    const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
    if (refused) {
        if (gtid == 0) {
            const bool wrong_args = bad != 0 || free0 < 0 || free0 + total.back > a.num_pages || total.rows > a.rows;
            report_error(a.status, wrong_args ? GQE_ERR_INVALID_ARGUMENT : GQE_ERR_OUT_OF_PAGES, kWherePlan, 0);
            *a.free_count_out = (int32_t)free0;
        }
        for (int b = gtid; b <= n; b += gsize) {
            a.cu_new[b] = 0;
            if (b < n) a.lengths_out[b] = a.lengths[b];
        }
        for (int64_t t = gtid; t < a.rows; t += gsize) a.slots[t] = -1;
        return;
    }
    for (int b = b0; b < b1; ++b) {
        const int l = a.lengths[b], add = a.new_lens[b];
        rows_at[b] = (int)at.rows;
        need_at[b] = (int)at.need;
        back_at[b] = (int)at.back;
        const int have = (int)((l + ps - 1) >> a.page_shift);
        if (add < 0) {
            at.back += have;
        } else {
            at.rows += add;
            at.need += ((l + add + ps - 1) >> a.page_shift) - have;
        }
    }
    if (tid == 0) {
        rows_at[n] = (int)total.rows;
        need_at[n] = (int)total.need;
        back_at[n] = (int)total.back;
    }
    __syncthreads();

    const int count = (int)free0, top = count + (int)total.back, need = (int)total.need;
    auto blocks_of = [&](int b) { return (int)((a.lengths[b] + ps - 1) >> a.page_shift); };
    auto pop = [&](int i) {  // the i-th page taken
        const int x = top - 1 - i;
        if (x < count) return a.free_pages[x];
        const int b = find_owner(back_at, n, x - count);
        return a.block_table[(int64_t)b * a.max_blocks + (x - count - back_at[b])];
    };
    auto check = [&](int page) {
        if ((unsigned)page < (unsigned)a.num_pages) return true;
        report_error(a.status, GQE_ERR_INVALID_ARGUMENT, kWherePlan, 1);
        return false;
    };
    for (int64_t t = gtid; t < a.rows; t += gsize) {
        int slot = -1;
        if (t < rows_at[n]) {
            const int b = find_owner(rows_at, n, (int)t);
            const int pos = a.lengths[b] + ((int)t - rows_at[b]), blk = pos >> a.page_shift, have = blocks_of(b);
            const int page = blk < have ? a.block_table[(int64_t)b * a.max_blocks + blk] : pop(need_at[b] + blk - have);
            if (check(page)) slot = (page << a.page_shift) | (pos & (int)(ps - 1));
        }
        a.slots[t] = slot;
    }
    for (int i = gtid; i < need; i += gsize) {
        const int b = find_owner(need_at, n, i), page = pop(i);
        check(page);
        a.block_table[(int64_t)b * a.max_blocks + blocks_of(b) + (i - need_at[b])] = page;
    }
    for (int j = gtid; j < (int)total.back; j += gsize) {
        const int b = find_owner(back_at, n, j), page = a.block_table[(int64_t)b * a.max_blocks + (j - back_at[b])];
        check(page);  // here, or a later step would blame the request that takes it
        a.free_pages[count + j] = page;
    }
    for (int b = gtid; b <= n; b += gsize) {
        a.cu_new[b] = rows_at[b];
        if (b < n) {
            const int add = a.new_lens[b];
            a.lengths_out[b] = add < 0 ? 0 : a.lengths[b] + add;
        }
    }
    if (gtid == 0) *a.free_count_out = top - need;
}

// ---------------------------------------------------------------------------
// Append: row t of K_new and V_new to row slots[t] of the pages, 16 bytes a
// lane.  lanes (a power of two, at most 32) lanes share a row; each takes every
// lanes-th vector of K and of V, four of each in flight.  HBM bound: each row is
// read once and written once.  16384 rows of 2 x 2 KB: 24 us or 5.6 TB/s (the rate of
// a plain copy: 20.5); 40 rows: 2.2 us, the launch.
constexpr int kAppendThreads = 256;
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const AppendArgs a, int vecs, int lanes) {
    const int sub = threadIdx.x & (lanes - 1);
    const int64_t t = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) / lanes;
    if (t >= a.rows) return;
    const int slot = a.slots[t];
    if (slot < 0) return;  // a row that is not kept
    if (slot >= a.num_slots) {
        if (sub == 0) report_error(a.status, GQE_ERR_INVALID_ARGUMENT, kWhereAppend, (uint32_t)t);
        return;
    }
    const uint4* ks = reinterpret_cast<const uint4*>(a.K_new + t * a.k_stride);
    const uint4* vs = reinterpret_cast<const uint4*>(a.V_new + t * a.v_stride);
    uint4* kd = reinterpret_cast<uint4*>(a.K_pages) + (int64_t)slot * vecs;
    uint4* vd = reinterpret_cast<uint4*>(a.V_pages) + (int64_t)slot * vecs;
    for (int i = sub; i < vecs; i += 4 * lanes) {
        uint4 kr[4], vr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e * lanes < vecs) {
                kr[e] = ld_stream16(ks + i + e * lanes);
                vr[e] = ld_stream16(vs + i + e * lanes);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e * lanes < vecs) {
                kd[i + e * lanes] = kr[e];
                vd[i + e * lanes] = vr[e];
            }
        }
    }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream) {
    // Opting in to more than 48 KB, of static and dynamic together: from well below that,
    // and always to the most a call can need, as the setting outlasts the call and another
    // thread's, were it smaller, would refuse this one's launch.
    constexpr size_t kMost = 3 * (size_t)(kPlanMaxSeqs + 1) * sizeof(int32_t);
    const size_t smem = 3 * (size_t)(a.n_seqs + 1) * sizeof(int32_t);
    if (smem > 32 * 1024) {
        cudaError_t err = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (err != cudaSuccess) return err;
    }
    // one row (or request) per thread, up to a block per SM: a block's scan costs
    // as much as its share of the writes does
    int64_t blocks = ((int64_t)a.rows + a.n_seqs + kPlanThreads - 1) / kPlanThreads;
    if (blocks > 148) blocks = 148;
    page_plan_kernel<<<(unsigned)blocks, kPlanThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
    const int vecs = (int)(a.row_bytes / 16);
    int lanes = 1;
    while (lanes < 32 && lanes < vecs) lanes <<= 1;
    const int64_t blocks = (a.rows * lanes + kAppendThreads - 1) / kAppendThreads;
    kv_append_kernel<<<(unsigned)blocks, kAppendThreads, 0, stream>>>(a, vecs, lanes);
    return cudaGetLastError();
}

}  // namespace gqe
