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
// keys in steps of BN: the tiles of the first `sinks` keys that lie below the
// window, then the tiles from the window's lower edge to the last token.
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
#pragma once

#include "common.cuh"

namespace gqe {

constexpr int kChunkMaxParts = 512;        // grid limit of the chunk kernels
constexpr uint32_t kWhereChunk = 8;        // status "where" id of the chunk kernels

// One partial unit: what the merge needs to find its rows.
struct ChunkDesc {
    int32_t valid, b, q, t0, nt, s0, s1, steps;
};

struct ChunkGeom {
    int T, n_seqs, h, g, k, hpg;
    int W, WU;        // tokens per query tile and per unit
    int BN;           // keys per step
    int unit_keys;    // a unit's fixed cost, in keys
    int min_cost;     // smallest cost worth a part, in keys
    int row_cap;      // query rows a partial record set holds
    int window, sinks;
    int cap;          // rows a block table can hold: page_size * max_blocks
    int page_shift, num_pages, max_blocks;
    const int32_t* cu;
    const int32_t* lengths;
    const int32_t* block_table;
    const int32_t* idx;
    const float* gate;
    void* status;
    ChunkDesc* desc;  // [2 * parts]
    float* part;      // [2 * parts][row_cap][D + 4]
};

struct ChunkItem {
    int b, q;
    int t0, nt;            // first packed token and the number of tokens
    int p0;                // position of token t0
    int sink_tiles;        // steps 0 .. sink_tiles-1 are tiles 0 ..
    int lo_tile;           // steps sink_tiles .. are tiles lo_tile ..
    int lo, hi;            // keys [lo, hi) and, below lo, keys < sinks are seen by some row
    int steps, s0, s1;     // the unit's steps and this part's [s0, s1)
    __device__ __forceinline__ int tile(int s) const { return s < sink_tiles ? s : lo_tile + (s - sink_tiles); }
};

struct ChunkSeq {
    int t0, n, L;
};

// A request's rows, or none (n = 0) when its entries contradict each other
// (reported): rows outside the packed tensor, a cache shorter than the new
// tokens or longer than the block table.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkGeom& u, int b) {
    ChunkSeq s;
    s.t0 = u.cu[b];
    const int t1 = u.cu[b + 1];
    s.L = u.lengths[b];
    s.n = 0;
    if (s.t0 < 0 || t1 < s.t0 || t1 > u.T) {
        report_error(u.status, GQE_ERR_INVALID_ARGUMENT, kWhereChunk, (uint32_t)b);
        return s;
    }
    const int n = t1 - s.t0;
    if (n > 0 && (s.L < n || s.L > u.cap)) {
        report_error(u.status, GQE_ERR_INVALID_ARGUMENT, kWhereChunk, (uint32_t)b);
        return s;
    }
    s.n = n;
    return s;
}

__device__ __forceinline__ int chunk_units(const ChunkGeom& u, int n) { return (n + u.WU - 1) / u.WU; }

// Cost of the first i units of a request and group, in keys, in closed form:
// unit j sees about first + j * WU keys, or the window's span if that is less.
__device__ __forceinline__ int64_t chunk_cost(const ChunkGeom& u, const ChunkSeq& s, int64_t i) {
    const int64_t first = (int64_t)s.L - s.n + min(s.n, u.WU);
    const int64_t span = u.window ? (int64_t)u.window + u.WU + u.sinks : (int64_t)1 << 40;
    int64_t grow = 0;
    if (first < span) {
        grow = (span - first + u.WU - 1) / u.WU;
        if (grow > i) grow = i;
    }
    return grow * first + u.WU * (grow * (grow - 1) / 2) + (i - grow) * span + i * u.unit_keys;
}

__device__ __forceinline__ void chunk_item(const ChunkGeom& u, const ChunkSeq& s, int b, int q, int i, ChunkItem& it) {
    const int first = i * u.WU;
    it.b = b;
    it.q = q;
    it.t0 = s.t0 + first;
    it.nt = min(u.WU, s.n - first);
    it.p0 = s.L - s.n + first;
    it.hi = it.p0 + it.nt;
    it.lo = u.window ? max(0, it.p0 - u.window + 1) : 0;
    it.lo_tile = it.lo / u.BN;
    it.sink_tiles = min(it.lo_tile, (min(u.sinks, it.lo) + u.BN - 1) / u.BN);
    it.steps = it.sink_tiles + (it.hi + u.BN - 1) / u.BN - it.lo_tile;
}

// Whether a row at position p sees key s.
__device__ __forceinline__ bool chunk_sees(const ChunkGeom& u, int p, int s) {
    return s <= p && (u.window == 0 || s > p - u.window || s < u.sinks);
}

// A place in the order of units: request, group, unit within both, step.
struct ChunkPlace {
    int b, q, i, s;
};

// Where a cost `rest` (within request b's own cost) falls.
__device__ __forceinline__ ChunkPlace chunk_place(const ChunkGeom& u, int b, int64_t rest) {
    const ChunkSeq s = chunk_seq(u, b);
    const int units = chunk_units(u, s.n);
    const int64_t per = chunk_cost(u, s, units);
    ChunkPlace pl;
    pl.b = b;
    pl.q = (int)(rest / per);
    rest -= pl.q * per;
    int lo = 0, hi = units - 1;  // the last unit whose prefix does not exceed rest
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (chunk_cost(u, s, mid) <= rest) lo = mid; else hi = mid - 1;
    }
    pl.i = lo;
    const int64_t before = chunk_cost(u, s, lo), cost = chunk_cost(u, s, lo + 1) - before;
    ChunkItem it;
    chunk_item(u, s, b, pl.q, lo, it);
    pl.s = (int)((rest - before) * it.steps / cost);
    return pl;
}

// Shared state of the split: filled by chunk_split, read by the item walk.
struct ChunkSplit {
    int64_t warp_sum[32];
    ChunkPlace from, to;
    int parts;
};

// This part's first place and the first place that is no longer its own.
// Called by all threads of the block (blockDim.x a multiple of 32, at most 1024).
__device__ __forceinline__ void chunk_split(const ChunkGeom& u, ChunkSplit& sp, int c, int max_parts) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int per = (u.n_seqs + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * per, u.n_seqs), b1 = min(b0 + per, u.n_seqs);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const ChunkSeq s = chunk_seq(u, b);
        if (s.n > 0) mine += u.g * chunk_cost(u, s, chunk_units(u, s.n));
    }
    int64_t run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    if (lane == 31) sp.warp_sum[warp] = run;
    if (tid == 0) {  // overwritten below where the place exists
        sp.from = {u.n_seqs, 0, 0, 0};
        sp.to = {u.n_seqs, 0, 0, 0};
    }
    __syncthreads();
    int64_t before = run - mine, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += sp.warp_sum[w];
        total += sp.warp_sum[w];
    }
    int64_t want = total / u.min_cost;
    const int parts = (int)(want < 1 ? 1 : want > max_parts ? max_parts : want);
    if (tid == 0) sp.parts = parts;
    if (c < parts && total > 0) {
        const int64_t each = total / parts, left = total % parts;
        const int64_t x0 = c * each + c * left / parts, x1 = (c + 1) * each + (c + 1) * left / parts;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t x = e ? x1 : x0;
            if (x < before || x >= before + mine) continue;
            int64_t at = before;
            for (int b = b0; b < b1; ++b) {
                const ChunkSeq s = chunk_seq(u, b);
                const int64_t cost = s.n > 0 ? u.g * chunk_cost(u, s, chunk_units(u, s.n)) : 0;
                if (x < at + cost) {
                    (e ? sp.to : sp.from) = chunk_place(u, b, x - at);
                    break;
                }
                at += cost;
            }
        }
    }
    __syncthreads();
}

// Walks a part's items in order.
struct ChunkWalk {
    ChunkPlace at, to;
    ChunkSeq seq;
    int units, loaded;
    __device__ __forceinline__ explicit ChunkWalk(const ChunkSplit& sp) : at(sp.from), to(sp.to), units(0), loaded(-1) {}
    __device__ __forceinline__ bool next(const ChunkGeom& u, ChunkItem& it) {
        while (true) {
            if (at.b >= u.n_seqs || at.b > to.b) return false;
            if (loaded != at.b) {
                seq = chunk_seq(u, at.b);
                units = chunk_units(u, seq.n);
                loaded = at.b;
            }
            if (at.i >= units) {
                at.i = 0;
                if (units == 0 || ++at.q >= u.g) {
                    at.q = 0;
                    ++at.b;
                }
                continue;
            }
            const bool last = at.b == to.b && at.q == to.q && at.i == to.i;
            if (at.b == to.b && (at.q > to.q || (at.q == to.q && at.i > to.i))) return false;
            if (last && at.s >= to.s) return false;
            chunk_item(u, seq, at.b, at.q, at.i, it);
            it.s0 = at.s;
            it.s1 = last ? min(to.s, it.steps) : it.steps;
            ++at.i;
            at.s = 0;
            return true;
        }
    }
};

__device__ __forceinline__ bool chunk_partial(const ChunkItem& it) { return it.s0 > 0 || it.s1 < it.steps; }
__device__ __forceinline__ int chunk_slot(const ChunkItem& it, int c) { return it.s0 > 0 ? 2 * c : 2 * c + 1; }
__device__ __forceinline__ void chunk_describe(const ChunkGeom& u, const ChunkItem& it, int c) {
    u.desc[chunk_slot(it, c)] = {1, it.b, it.q, it.t0, it.nt, it.s0, it.s1, it.steps};
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

// One row of an item by the formula alone, key by key over the keys the row
// sees (warp-collective; lane holds elements e * 32 + lane).  The tile kernels
// multiply a masked key's weight 0 with its V row, so an infinity or NaN there
// reaches rows that do not see the key; a row whose result is not finite is
// therefore taken again here, where a key that the row does not see is not read.
template <typename T, int D>
__device__ __forceinline__ void chunk_row(const ChunkGeom& u, const ChunkItem& it, int p, const T* q_row, const T* Kp,
                                       const T* Vp, float scale_log2, float (&acc)[D / 32], float& m, float& l) {
    const int lane = threadIdx.x & 31;
    float qv[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        qv[e] = Elem<T>::to_f(q_row[e * 32 + lane]);
        acc[e] = 0.f;
    }
    m = -INFINITY;
    l = 0.f;
    for (int st = it.s0; st < it.s1; ++st) {
        const int k0 = it.tile(st) * u.BN;
        const int k1 = min(k0 + u.BN, p + 1);
        for (int s = k0; s < k1; s += 4) {  // four keys' loads in flight
            float x[4], v[4][D / 32];
            bool on[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                on[j] = s + j < k1 && chunk_sees(u, p, s + j);
                x[j] = 0.f;
                if (on[j]) {
                    const int64_t at = (chunk_cache_row(u, it.b, s + j) * u.g + it.q) * D;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        x[j] = fmaf(qv[e], Elem<T>::to_f(Kp[at + e * 32 + lane]), x[j]);
                        v[j][e] = Elem<T>::to_f(Vp[at + e * 32 + lane]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) x[j] += __shfl_xor_sync(0xffffffffu, x[j], d);
                x[j] *= scale_log2;
                if (!on[j] || x[j] == -INFINITY) continue;  // -inf: weight 0 beside any other key
                const float mx = fmaxf(m, x[j]);
                const float corr = m == -INFINITY ? 0.f : fast_exp2(m - mx), w = fast_exp2(x[j] - mx);
                m = mx;
                l = l * corr + w;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) acc[e] = acc[e] * corr + w * v[j][e];
            }
            if (l != l) {  // a score was NaN: so is the whole row
#pragma unroll
                for (int e = 0; e < D / 32; ++e) acc[e] = l;
                return;
            }
        }
    }
}

// Where a row's result goes: the gated row of O, or the row's partial record.
template <typename T, int D>
__device__ __forceinline__ void chunk_store_row(const ChunkGeom& u, const ChunkItem& it, int c, int r, int token, int head,
                                                const float (&acc)[D / 32], float m, float l, T* O) {
    const int lane = threadIdx.x & 31;
    if (chunk_partial(it)) {
        float* rec = u.part + ((int64_t)chunk_slot(it, c) * u.row_cap + r) * (D + 4);
        const bool none = m == -INFINITY && l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) rec[e * 32 + lane] = acc[e] * inv;
        if (lane == 0) rec[D] = none ? -INFINITY : m + log2f(l);
    } else {
        const float f = u.gate[((int64_t)token * u.g + it.q) * u.k + r % u.k] / l;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            O[((int64_t)token * u.h + head) * D + e * 32 + lane] = Elem<T>::from_f(acc[e] * f);
    }
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

// How a kernel tiles its units: query rows per tile, tiles per unit, keys per
// step, a unit's fixed cost and the smallest part in keys, blocks per SM.
struct ChunkTiling {
    int rows, tiles, keys, unit_keys, min_cost, per_sm;
};
ChunkTiling chunk_simt_tiling();
cudaError_t launch_chunk_simt(const ChunkGeom& u, const ChunkArgs& a, int parts);
ChunkTiling chunk_tc_tiling();
cudaError_t launch_chunk_tc(const ChunkGeom& u, const ChunkArgs& a, int parts);

}  // namespace gqe
