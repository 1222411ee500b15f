// chunk.cuh -- work units and schedule of the chunk attention over a paged
// cache (gqe_attn_chunk_paged), shared by its kernels.
//
// The step's new tokens are packed: request b owns rows cu_new[b] ..
// cu_new[b+1]-1 and its cache holds lengths[b] rows, the new ones last, so its
// i-th new token sits at position lengths[b] - n_b + i.
//
// Unit.  Every token selects k heads of every KV group, so (request, group,
// WU consecutive new tokens) holds k * WU query rows, row r being token r / k,
// selection r % k: no compaction lists, and a unit's rows differ in position by
// less than WU, which keeps the masked band narrow.  A unit walks its visible
// cache rows in steps of BN: the pages of the first `sinks` keys, then, closed up
// behind them, those from the window's lower edge to the last token, so that a
// few first keys cost a page of a step and not a step.
//
// Schedule.  The lengths live on the device, so the grid cannot be cut on the
// host.  Every CTA instead derives the same split of the whole step: a cost per
// unit (its keys plus a constant for what a unit costs besides), a prefix sum
// over the requests, and part c of P takes the costs [c, c+1) * total / P.  A
// boundary inside a unit splits it between neighbouring parts at a step; its
// parts write partial results (normalised output, log2-sum-exp) that
// chunk_combine_kernel merges in order.  So one long cache, many short ones and
// a mix of decodes and prompt chunks all spread evenly, and a part holds at
// most two partial units: its first (slot 2c) and its last (slot 2c + 1).
// Requests of few query rows (u.few) are split by themselves, so that a kernel
// can treat them in another way: two kinds of units, each over all CTAs.
#pragma once

#include "common.cuh"

namespace gqe {

constexpr int kChunkMaxParts = 512;        // grid limit of the chunk kernels
constexpr uint32_t kWhereChunk = 8;        // status "where" id of the chunk kernels

// One partial unit: what the merge needs to find its rows.
struct __align__(16) ChunkDesc {
    int32_t b, t0, q_nt, rec;  // b: -1 when there is none; q_nt: group << 16 | tokens
    __device__ __forceinline__ int q() const { return q_nt >> 16; }
    __device__ __forceinline__ int nt() const { return q_nt & 0xffff; }
    __device__ __forceinline__ bool same_unit(const ChunkDesc& o) const {
        return b >= 0 && b == o.b && t0 == o.t0 && q_nt == o.q_nt;
    }
};

// A place in the order of units: request, group, unit within both, step.
struct __align__(16) ChunkPlace {
    int b, q, i, s;
};

struct ChunkGeom {
    int T, n_seqs, h, g, k, hpg;
    uint32_t inv_k;   // row / k == row * inv_k >> 16 for a unit's rows
    int W, WU;        // tokens per query tile and per unit
    int BN, bn_shift; // keys per step and their log2
    int align;        // rows that the parts of a unit's key list are aligned to
    float unit_cost[2];  // a unit's fixed cost, in keys, by kind
    float cost_scale; // requests' costs are summed in whole multiples of 1 / cost_scale keys: 32 bits hold a step's
    float per_min;    // 1 / the smallest cost worth a part
    int few_tokens;   // new tokens up to which a request is of the second kind
    int parts;        // CTAs, and parts of either kind at most
    int row_cap, few_cap;  // query rows that the partial records of a unit take, by kind
    int window, sinks;
    int cap;          // rows a block table can hold: page_size * max_blocks
    int page_shift, num_pages, max_blocks;
    const int32_t* cu;
    const int32_t* lengths;
    const int32_t* block_table;
    const int32_t* idx;
    const float* gate;
    void* status;
    ChunkDesc* desc;  // [2 kinds][parts][2]
    ChunkPlace* place;  // [2 kinds][CTAs][2]: where the CTA's work starts, and the first place that is no longer its own
    int32_t* odd;     // [2 kinds][CTAs]: some result of the CTA's units is not finite
    float* part;      // [2 * parts * row_cap + 2 * parts * few_cap][D + 4]
};

struct ChunkItem {
    int b, q;
    int t0, nt;            // first packed token and the number of tokens
    int p0;                // position of token t0
    int lo, hi;            // keys [lo, hi) and, below lo, keys < sinks are seen by some row
    int head, skip;        // list row x is key x for x < head, else key x + skip
    int steps, s0, s1;     // the unit's steps and this part's [s0, s1)
    int rec;               // the unit's first partial record if it is split, else -1
    __device__ __forceinline__ int key(int x) const { return x < head ? x : x + skip; }
};

struct ChunkSeq {
    int t0, n, L;
};

// A request's rows, or none (n = 0) when its entries contradict each other
// (reported): rows outside the packed tensor, a cache shorter than the new
// tokens or longer than the block table.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkGeom& u, int b, int t0, int t1, int L) {
    ChunkSeq s = {t0, (int)((unsigned)t1 - (unsigned)t0), L};  // of any entries, before they are checked
    if (t0 < 0 || t1 < t0 || t1 > u.T || (s.n > 0 && (L < s.n || L > u.cap))) {
        report_error(u.status, GQE_ERR_INVALID_ARGUMENT, kWhereChunk, (uint32_t)b);
        s.n = 0;
    }
    return s;
}
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkGeom& u, int b) {
    return chunk_seq(u, b, u.cu[b], u.cu[b + 1], u.lengths[b]);
}

// 0: many query rows, 1: few.
__device__ __forceinline__ int chunk_kind(const ChunkGeom& u, int n) { return n <= u.few_tokens ? 1 : 0; }

__device__ __forceinline__ int chunk_units(const ChunkGeom& u, int n) { return (n + u.WU - 1) / u.WU; }

// Cost, in keys, of the first i units of a request and group in closed form: unit j
// sees about first + j * WU keys, or the window's span if that is less.  fp32, as
// they only place the boundaries, but every evaluation has to give the same number
// (a request's cost is summed by one and searched by another, and a boundary that
// neither side owns would lose its work), so each product and sum is rounded by
// itself: left to the compiler, copies of the code may contract them differently.
// The prefix sums over requests are in whole numbers, whose intervals tile without
// gaps.
struct ChunkCost {
    float first, span, grow;  // units before `grow` still grow
    __device__ __forceinline__ ChunkCost(const ChunkGeom& u, const ChunkSeq& s)
        : span(0.f), grow(3.4e38f) {
        const float fixed = chunk_kind(u, s.n) ? u.unit_cost[1] : u.unit_cost[0];
        first = (float)(s.L - s.n + min(s.n, u.WU)) + fixed;
        if (u.window) {
            span = (float)u.window + (float)(min(s.n, u.WU) + u.sinks) + fixed;
            grow = ceilf(fmaxf(__fdividef(span - first, (float)u.WU), 0.f));
        }
    }
    __device__ __forceinline__ float operator()(const ChunkGeom& u, int units) const {
        const float i = (float)units, n = fminf(i, grow);
        return __fadd_rn(__fmul_rn(n, __fmaf_rn(0.5f * u.WU, n - 1.f, first)), __fmul_rn(i - n, span));
    }
};
__device__ __forceinline__ uint32_t chunk_cost(const ChunkGeom& u, const ChunkSeq& s) {
    return s.n > 0 ? max(__float2uint_rn(__fmul_rn(__fmul_rn((float)u.g, ChunkCost(u, s)(u, chunk_units(u, s.n))), u.cost_scale)), 1u) : 0;
}

__device__ __forceinline__ void chunk_item(const ChunkGeom& u, const ChunkSeq& s, int b, int q, int i, ChunkItem& it) {
    const int first = i * u.WU;
    it.b = b;
    it.q = q;
    it.t0 = s.t0 + first;
    it.nt = min(u.WU, s.n - first);
    it.p0 = s.L - s.n + first;
    it.hi = it.p0 + it.nt;
    it.lo = it.head = it.skip = 0;
    if (u.window) {
        it.lo = max(0, it.p0 - u.window + 1);
        const int from = it.lo & ~(u.align - 1);
        const int head = (min(u.sinks, it.lo) + u.align - 1) & ~(u.align - 1);
        if (head < from) {  // else the two parts touch: the list is the keys from 0 on
            it.head = head;
            it.skip = from - head;
        }
    }
    it.steps = (it.hi - it.skip + u.BN - 1) >> u.bn_shift;
}

// Whether a row at position p sees key s.
__device__ __forceinline__ bool chunk_sees(const ChunkGeom& u, int p, int s) {
    return s <= p && (u.window == 0 || s > p - u.window || s < u.sinks);
}

// Where a fraction (0 or more, below 1) of request b's work ends (warp-collective,
// the same in every lane).
__device__ __forceinline__ ChunkPlace chunk_place(const ChunkGeom& u, const ChunkSeq& s, int b, float fraction) {
    const int units = chunk_units(u, s.n), lane = threadIdx.x & 31;
    const ChunkCost cost(u, s);
    const float per = cost(u, units);
    ChunkPlace pl;
    pl.b = b;
    fraction *= u.g;
    pl.q = min((int)fraction, u.g - 1);
    const float rest = (fraction - pl.q) * per;
    // the last unit whose prefix does not exceed rest: 32 candidates a round
    int lo = 0, span = units;
    while (span > 1) {
        const int step = (span + 31) >> 5, at = lo + lane * step;
        const unsigned under = __ballot_sync(0xffffffffu, at < lo + span && cost(u, at) <= rest) | 1u;
        const int hit = 31 - __clz(under);
        span = min(step, span - hit * step);
        lo += hit * step;
    }
    pl.i = lo;
    const float before = cost(u, lo), own = cost(u, lo + 1) - before;
    ChunkItem it;
    chunk_item(u, s, b, pl.q, lo, it);
    pl.s = max(0, min((int)(__fdividef(rest - before, own) * it.steps), it.steps - 1));
    return pl;
}

// Shared state of the split: filled by chunk_split, read by the item walk.  An end
// is a request and a fraction of its work; request n_seqs: none.
struct ChunkEnd {
    int b;
    float fraction;
    ChunkSeq seq;
};
struct ChunkSplit {
    uint32_t warp_sum[2][32];
    ChunkEnd end[2][2];  // by kind: this CTA's first place, and the first that is no longer its own
};

// The part that a CTA takes of a kind: opposite ends, so that small amounts of
// both go to different CTAs.
__device__ __forceinline__ int chunk_part(const ChunkGeom& u, int kind, int cta) { return kind ? cta : u.parts - 1 - cta; }

// A CTA's first place and the first place that is no longer its own, of each
// kind.  Called by all kThreads threads of a block.
template <int kThreads>
__device__ __forceinline__ void chunk_split(const ChunkGeom& u, ChunkSplit& sp, int cta) {
    constexpr int nw = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = u.n_seqs <= kThreads ? 1 : (u.n_seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, u.n_seqs), b1 = min(b0 + per, u.n_seqs);
    uint32_t mine[2] = {0, 0};
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const ChunkSeq s = chunk_seq(u, b);
        const uint32_t cost = chunk_cost(u, s);
        if (chunk_kind(u, s.n)) mine[1] += cost; else mine[0] += cost;
    }
    if (tid < 4) sp.end[tid >> 1][tid & 1].b = u.n_seqs;  // overwritten below where the place exists
    uint32_t run[2] = {mine[0], mine[1]};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, run[0], d), y = __shfl_up_sync(0xffffffffu, run[1], d);
        if (lane >= d) {
            run[0] += x;
            run[1] += y;
        }
    }
    if (lane == 31) {
        sp.warp_sum[0][warp] = run[0];
        sp.warp_sum[1][warp] = run[1];
    }
    __syncthreads();
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const uint32_t own = kind ? mine[1] : mine[0];
        if (own == 0) continue;
        uint32_t before = (kind ? run[1] : run[0]) - own, total = 0;
#pragma unroll
        for (int w = 0; w < nw; ++w) {
            if (w < warp) before += sp.warp_sum[kind][w];
            total += sp.warp_sum[kind][w];
        }
        const float want = (float)total * u.per_min;
        const int parts = want < 1.f ? 1 : want > (float)u.parts ? u.parts : (int)want;
        const int c = chunk_part(u, kind, cta);
#pragma unroll 1
        for (int e = 0; e < 2 && c + e < parts; ++e) {  // the last part ends with the step
            const uint32_t x = __umulhi(total, (uint32_t)(__fdividef((float)(c + e), (float)parts) * 4294967296.f));
            if (x < before || x - before >= own) continue;
            uint32_t at = before;
#pragma unroll 1
            for (int b = b0; b < b1; ++b) {
                const ChunkSeq s = chunk_seq(u, b);
                const uint32_t cost = chunk_kind(u, s.n) == kind ? chunk_cost(u, s) : 0;
                if (x - at < cost) {
                    sp.end[kind][e] = {b, __fdividef((float)(x - at), (float)cost), s};
                    break;
                }
                at += cost;
            }
        }
    }
    __syncthreads();
}

// Walks a CTA's items of a kind in order.  Warp-collective: the lanes hold the
// entries of 32 requests, so that a run of short ones costs one round of loads,
// which the first item (whose request the split has left) does not wait for.
struct ChunkWalk {
    ChunkPlace at, to;
    ChunkSeq seq;        // of request at.b
    int t0, t1, L;       // entries of request base + lane
    int kind, base, part;
    __device__ __forceinline__ ChunkWalk(const ChunkGeom& u, const ChunkSplit& sp, int kind, int cta)
        : kind(kind), part(chunk_part(u, kind, cta)) {
        base = sp.end[kind][0].b;
        fetch(u);
#pragma unroll 1
        for (int i = 1; i >= 0; --i) {
            to = at;
            const ChunkEnd e = sp.end[kind][i];
            at = {u.n_seqs, 0, 0, 0};
            if (e.b < u.n_seqs) at = chunk_place(u, e.seq, e.b, e.fraction);
            seq = e.seq;
        }
    }
    // Leaves the places of a fresh walk for the merge (one thread).
    __device__ __forceinline__ void leave(const ChunkGeom& u, int cta) const {
        u.place[2 * (kind * u.parts + cta)] = at;
        u.place[2 * (kind * u.parts + cta) + 1] = to;
    }
    __device__ __forceinline__ void fetch(const ChunkGeom& u) {
        const int b = base + (threadIdx.x & 31);
        t0 = t1 = L = 0;
        if (b < u.n_seqs) {
            t0 = u.cu[b];
            t1 = u.cu[b + 1];
            L = u.lengths[b];
        }
    }
    __device__ __forceinline__ bool next(const ChunkGeom& u, ChunkItem& it) {
        if (at.b >= u.n_seqs) return false;
        if (at.i >= chunk_units(u, seq.n)) {
            at.i = 0;
            if (++at.q >= u.g) {  // the next request that has work of this kind
                at.q = 0;
                int src = at.b - base + 1;
                while (true) {
                    if (src >= 32) {
                        base += 32;
                        if (base >= u.n_seqs || base > to.b) return false;
                        fetch(u);
                        src = 0;
                    }
                    const ChunkSeq s = chunk_seq(u, base + (threadIdx.x & 31), t0, t1, L);
                    const unsigned some = __ballot_sync(0xffffffffu, s.n > 0 && chunk_kind(u, s.n) == kind) >> src;
                    if (some) {
                        src += __ffs(some) - 1;
                        seq = {__shfl_sync(0xffffffffu, s.t0, src), __shfl_sync(0xffffffffu, s.n, src), __shfl_sync(0xffffffffu, s.L, src)};
                        break;
                    }
                    src = 32;
                }
                at.b = base + src;
            }
        }
        if (at.b > to.b || (at.b == to.b && (at.q > to.q || (at.q == to.q && at.i > to.i)))) return false;
        const bool last = at.b == to.b && at.q == to.q && at.i == to.i;
        if (last && at.s >= to.s) return false;
        chunk_item(u, seq, at.b, at.q, at.i, it);
        it.s0 = at.s;
        it.s1 = last ? min(to.s, it.steps) : it.steps;
        it.rec = -1;
        if (it.s0 > 0 || it.s1 < it.steps) {
            const int slot = it.s0 > 0 ? 2 * part : 2 * part + 1;
            it.rec = kind ? 2 * u.parts * u.row_cap + slot * u.few_cap : slot * u.row_cap;
            if ((threadIdx.x & 31) == 0) u.desc[kind * 2 * u.parts + slot] = {it.b, it.t0, it.q << 16 | it.nt, it.rec};
        }
        ++at.i;
        at.s = 0;
        return true;
    }
};

// Whether a CTA has items of a kind.
__device__ __forceinline__ bool chunk_has(const ChunkGeom& u, const ChunkSplit& sp, int kind) {
    return sp.end[kind][0].b < u.n_seqs;
}

// Marks this CTA's descriptors and flags unused (one thread, a block barrier
// before the walks).
__device__ __forceinline__ void chunk_clear(const ChunkGeom& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u.desc[(i >> 1) * 2 * u.parts + 2 * chunk_part(u, i >> 1, blockIdx.x) + (i & 1)].b = -1;
    u.odd[blockIdx.x] = u.odd[u.parts + blockIdx.x] = 0;
}

// Cache row of request b's key s.  A block-table entry outside the page pool is
// reported and read as page 0, as in the paged decode.
__device__ __forceinline__ int64_t chunk_cache_row(const ChunkGeom& u, int b, int s) {
    int pg = u.block_table[(int64_t)b * u.max_blocks + (s >> u.page_shift)];
    if ((unsigned)pg >= (unsigned)u.num_pages) {
        report_error(u.status, GQE_ERR_INVALID_ARGUMENT, kWhereChunk, (uint32_t)b);
        pg = 0;
    }
    return ((int64_t)pg << u.page_shift) + (s & ((1 << u.page_shift) - 1));
}

// The head of a unit's row, or -1 for a selection outside the group (reported).
__device__ __forceinline__ int chunk_head(const ChunkGeom& u, int token, int q, int slot) {
    const int j = u.idx[((int64_t)token * u.g + q) * u.k + slot];
    if (j < q * u.hpg || j >= (q + 1) * u.hpg) {
        report_error(u.status, GQE_ERR_INVALID_ARGUMENT, kWhereChunk, (uint32_t)token);
        return -1;
    }
    return j;
}

// Arguments of a call (host).
struct ChunkArgs {
    const gqe_shape* s;
    const void* Q;
    const void* K_pages;
    const void* V_pages;
    int num_pages, page_shift;
    const int32_t* block_table;
    int max_blocks, n_seqs;
    const int32_t* cu_new;
    const int32_t* lengths;
    int window, sinks;
    const int32_t* idx;
    const float* gate;
    void* O;
    void* scratch;  // chunk_scratch_bytes(s)
    void* status;
    cudaStream_t stream;
};
size_t chunk_scratch_bytes(const gqe_shape* s);
cudaError_t launch_chunk(const ChunkArgs& a);

// How a kernel tiles its units: query rows per tile, tiles per unit, the rows up
// to which a request is of the second kind, keys per step, a unit's fixed cost of
// either kind and the smallest part in keys, blocks per SM.
struct ChunkTiling {
    int rows, tiles, few, keys, unit_keys, few_keys, min_keys, per_sm;
};
ChunkTiling chunk_simt_tiling(int d_h);
cudaError_t launch_chunk_simt(const ChunkGeom& u, const ChunkArgs& a);
ChunkTiling chunk_tc_tiling();
cudaError_t launch_chunk_tc(const ChunkGeom& u, const ChunkArgs& a);

}  // namespace gqe
