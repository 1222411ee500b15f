// chunk.cu -- host side of the chunk attention (which kernel, its scratch) and the
// merge of the units that the schedule split.  See chunk.cuh.
#include "chunk.cuh"

namespace gqe {
namespace {

// After the tile kernel: block (c, y) of a kind
//  1. takes again the rows of CTA c's whole units whose result is not finite
//     (only if the CTA has flagged one): see chunk_row;
//  2. merges the split unit whose first steps part c holds as its last:
//     O = gate * sum_p 2^(lse_p - M) o_p / sum_p 2^(lse_p - M) over its parts in
//     order (reproducible), one warp per row, rows y apart.
constexpr int kCombineWarps = 8;

// A unit's row from the formula into O.
template <typename T, int D>
__device__ __noinline__ void row_again(const ChunkGeom& u, const ChunkItem& it, int r, int head, const T* Q, const T* Kp,
                                       const T* Vp, float scale_log2, T* O) {
    const int lane = threadIdx.x & 31, token = it.t0 + r / u.k;
    const int64_t row = ((int64_t)token * u.h + head) * D;
    float acc[D / 32], m, l;
    chunk_row<T, D>(u, it, it.p0 + r / u.k, Q + row, Kp, Vp, scale_log2, acc, m, l);
    const float f = u.gate[((int64_t)token * u.g + it.q) * u.k + r % u.k] / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) O[row + e * 32 + lane] = Elem<T>::from_f(acc[e] * f);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kCombineWarps)
chunk_combine_kernel(const ChunkGeom u, const T* __restrict__ Q, const T* __restrict__ Kp, const T* __restrict__ Vp,
                     float scale_log2, T* __restrict__ O) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRec = D + 4, kPer = D / 32, kRows = 4;
    __shared__ int list[kChunkMaxParts];  // the unit's records in order
    __shared__ int count;
    __shared__ ChunkSplit split;
    const int c = blockIdx.x, kind = c < u.parts ? 0 : 1, cta = c - kind * u.parts, end = (kind + 1) * u.parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ChunkDesc d = u.desc[2 * c + 1];
    const bool odd = u.odd[c] != 0;
    if (warp == 0) {
        int n = 1;
        if (lane == 0) list[0] = d.rec;
        for (int p0 = c + 1; p0 < end; p0 += 32) {
            const int p = p0 + lane;
            bool mine = false, other = p >= end;
            ChunkDesc e;
            if (p < end) {
                e = u.desc[2 * p];  // in flight with d
                mine = e.valid && e.q == d.q && e.t0 == d.t0 && e.b == d.b;
                other = e.valid && !mine;
            }
            const unsigned in = __ballot_sync(0xffffffffu, mine), out = __ballot_sync(0xffffffffu, other);
            if (mine) list[n + __popc(in & ((1u << lane) - 1u))] = e.rec;
            n += __popc(in);
            if (out || !d.valid) break;  // a later unit's part: this unit's are all behind
        }
        if (lane == 0) count = n;
    }
    if (odd) {
        chunk_split<32 * kCombineWarps>(u, split, cta);
        ChunkWalk walk(u, split, kind, cta);
        ChunkItem it;
        while (walk.next(u, it, false)) {
            if (it.rec >= 0) continue;
            for (int r = blockIdx.y * kCombineWarps + warp; r < it.nt * u.k; r += gridDim.y * kCombineWarps) {
                const int token = it.t0 + r / u.k, j = u.idx[((int64_t)token * u.g + it.q) * u.k + r % u.k];
                if (j < it.q * u.hpg || j >= (it.q + 1) * u.hpg) continue;
                float check = 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e) check += 0.f * Elem<T>::to_f(O[((int64_t)token * u.h + j) * D + e * 32 + lane]);
                if (__any_sync(0xffffffffu, !(check == 0.f))) row_again<T, D>(u, it, r, j, Q, Kp, Vp, scale_log2, O);
            }
        }
    }
    if (!d.valid) return;
    __syncthreads();
    const int n = count, rows = d.nt * u.k;
    for (int r0 = (blockIdx.y * kCombineWarps + warp) * kRows; r0 < rows; r0 += gridDim.y * kCombineWarps * kRows) {
        // kRows rows at once, so that their loads are in flight together
        int j[kRows];
        float gate[kRows], M[kRows], L[kRows], acc[kRows][kPer];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = min(r0 + i, rows - 1), token = d.t0 + r / u.k;
            const int64_t at = ((int64_t)token * u.g + d.q) * u.k + r % u.k;
            j[i] = u.idx[at];
            gate[i] = u.gate[at];
            M[i] = -INFINITY;
            L[i] = 0.f;
            for (int p = lane; p < n; p += 32) M[i] = fmaxf(M[i], u.part[(int64_t)(list[p] + r) * kRec + D]);
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[i][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], s));
#pragma unroll 2
        for (int p = 0; p < n; ++p) {
            float lse[kRows], v[kRows][kPer];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float* rec = u.part + (int64_t)(list[p] + min(r0 + i, rows - 1)) * kRec;
                lse[i] = rec[D];
#pragma unroll
                for (int e = 0; e < kPer; ++e) v[i][e] = rec[e * 32 + lane];
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (lse[i] == -INFINITY) continue;  // this part holds no key of the row
                const float w = fast_exp2(lse[i] - M[i]);
                L[i] += w;
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[i][e] = fmaf(v[i][e], w, acc[i][e]);
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i, token = d.t0 + r / u.k;
            if (r >= rows || j[i] < d.q * u.hpg || j[i] >= (d.q + 1) * u.hpg) continue;  // no such row
            float check = L[i] * 0.f;
#pragma unroll
            for (int e = 0; e < kPer; ++e) check += acc[i][e] * 0.f;
            if (__any_sync(0xffffffffu, !(check == 0.f))) {
                const ChunkSeq s = chunk_seq(u, d.b);
                ChunkItem it;
                chunk_item(u, s, d.b, d.q, (d.t0 - s.t0) / u.WU, it);
                row_again<T, D>(u, it, r, j[i], Q, Kp, Vp, scale_log2, O);
                continue;
            }
            const float f = gate[i] / L[i];
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                O[((int64_t)token * u.h + j[i]) * D + e * 32 + lane] = Elem<T>::from_f(acc[i][e] * f);
        }
    }
}

int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return sms;
}

size_t a256(size_t n) { return (n + 255) & ~size_t(255); }

bool on_tensor_cores(const gqe_shape* s) { return s->dtype == GQE_BF16 && s->d_h == 128; }

ChunkTiling tiling(const gqe_shape* s) { return on_tensor_cores(s) ? chunk_tc_tiling() : chunk_simt_tiling(); }

int max_parts(const ChunkTiling& t) {
    const int p = t.per_sm * device_sms();
    return p < kChunkMaxParts ? p : kChunkMaxParts;
}

// Query rows of a unit: a step of few tokens cannot fill it.
int row_cap(const gqe_shape* s, const ChunkTiling& t) {
    const int64_t all = (int64_t)s->T * s->k, unit = (int64_t)(t.rows / s->k) * s->k * t.tiles;
    return (int)(all < unit ? all : unit);
}

int few_cap(const gqe_shape* s, const ChunkTiling& t) {
    return (int64_t)s->T * s->k < t.few ? s->T * s->k : t.few;
}

size_t desc_bytes(int parts) { return a256(4 * (size_t)parts * sizeof(ChunkDesc)); }
size_t odd_bytes(int parts) { return a256(2 * (size_t)parts * sizeof(int32_t)); }

ChunkGeom make_geom(const ChunkArgs& a, const ChunkTiling& t, int parts) {
    const gqe_shape& s = *a.s;
    ChunkGeom u;
    u.T = s.T;
    u.n_seqs = a.n_seqs;
    u.h = s.h;
    u.g = s.g;
    u.k = s.k;
    u.hpg = s.h / s.g;
    u.inv_k = (65536 + s.k - 1) / s.k;
    u.W = t.rows / s.k;
    u.WU = t.tiles * u.W;
    u.BN = t.keys;
    u.bn_shift = 0;
    while ((1 << u.bn_shift) < t.keys) ++u.bn_shift;
    u.few_tokens = t.few / s.k;
    u.parts = parts;
    u.row_cap = row_cap(&s, t);
    u.few_cap = few_cap(&s, t);
    u.cap = a.max_blocks << a.page_shift;
    u.window = a.window >= u.cap ? 0 : a.window;
    u.sinks = u.window == 0 ? 0 : a.sinks < u.cap ? a.sinks : u.cap;
    u.page_shift = a.page_shift;
    const int page = 1 << a.page_shift;
    u.align = page < 8 ? 8 : page < t.keys ? page : t.keys;
    // No more than one unit per token, nor than the full ones and one per request.
    int64_t units = (s.T + u.WU - 1) / u.WU + (int64_t)a.n_seqs;
    if (units > s.T) units = s.T;
    u.unit_cost = (float)t.unit_keys;
    u.cost_scale = 1.0f / 16;
    while ((double)units * s.g * ((double)u.cap + u.WU + t.unit_keys) * u.cost_scale + (double)units * s.g > 2.0e9)
        u.cost_scale *= 0.5f;
    u.per_min = 1.0f / (t.min_keys * u.cost_scale);
    u.num_pages = a.num_pages;
    u.max_blocks = a.max_blocks;
    u.cu = a.cu_new;
    u.lengths = a.lengths;
    u.block_table = a.block_table;
    u.idx = a.idx;
    u.gate = a.gate;
    u.status = a.status;
    u.desc = static_cast<ChunkDesc*>(a.scratch);
    u.odd = reinterpret_cast<int32_t*>(static_cast<char*>(a.scratch) + desc_bytes(parts));
    u.part = reinterpret_cast<float*>(static_cast<char*>(a.scratch) + desc_bytes(parts) + odd_bytes(parts));
    return u;
}

template <typename T>
cudaError_t launch_combine(const ChunkGeom& u, const ChunkArgs& a, int kinds, int blocks) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kinds * u.parts, blocks);
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, u, (const T*)a.Q, (const T*)a.K_pages, (const T*)a.V_pages,
                                  1.4426950408889634f / sqrtf((float)a.s->d_h), (T*)a.O);
    };
    switch (a.s->d_h) {
        case 32: return go(chunk_combine_kernel<T, 32>);
        case 64: return go(chunk_combine_kernel<T, 64>);
        default: return go(chunk_combine_kernel<T, 128>);
    }
}

}  // namespace

size_t chunk_scratch_bytes(const gqe_shape* s) {
    const ChunkTiling t = tiling(s);
    const size_t parts = (size_t)max_parts(t), rows = 2 * parts * (row_cap(s, t) + few_cap(s, t));
    return desc_bytes((int)parts) + odd_bytes((int)parts) + a256(rows * (size_t)(s->d_h + 4) * sizeof(float));
}

cudaError_t launch_chunk(const ChunkArgs& a) {
    const ChunkTiling t = tiling(a.s);
    const int parts = max_parts(t);
    const ChunkGeom u = make_geom(a, t, parts);
    const cudaError_t err = on_tensor_cores(a.s) ? launch_chunk_tc(u, a) : launch_chunk_simt(u, a);
    if (err != cudaSuccess) return err;
    const int blocks = (u.row_cap + 4 * kCombineWarps - 1) / (4 * kCombineWarps);  // about four rows a warp
    const int kinds = t.few > 0 ? 2 : 1;
    return a.s->dtype == GQE_BF16 ? launch_combine<__nv_bfloat16>(u, a, kinds, blocks)
                                  : launch_combine<float>(u, a, kinds, blocks);
}

}  // namespace gqe
