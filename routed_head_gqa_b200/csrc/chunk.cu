// chunk.cu -- host side of the chunk attention (which kernel, its scratch) and the
// merge of the units that the schedule split.  See chunk.cuh.
#include "chunk.cuh"

namespace gqe {
namespace {

// Merge of a split unit: O = gate * sum_p 2^(lse_p - M) o_p / sum_p 2^(lse_p - M)
// over its parts in order (reproducible).  Block (c, y) takes the unit whose
// first steps part c holds (its slot 2c + 1), one warp per row, rows y apart.
constexpr int kCombineWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kCombineWarps)
chunk_combine_kernel(const ChunkGeom u, int parts, T* __restrict__ O) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kRec = D + 4, kPer = D / 32;
    __shared__ int16_t list[kChunkMaxParts];  // the unit's slots in order
    __shared__ int count;
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ChunkDesc d = u.desc[2 * c + 1];
    if (!d.valid || d.s1 == d.steps) return;
    if (warp == 0) {
        int n = 1;
        if (lane == 0) list[0] = (int16_t)(2 * c + 1);
        for (int p0 = c + 1; p0 < parts; p0 += 32) {
            const int p = p0 + lane;
            bool mine = false, other = false;
            if (p < parts) {
                const ChunkDesc e = u.desc[2 * p];
                mine = e.valid && e.q == d.q && e.t0 == d.t0 && e.b == d.b;
                other = e.valid && !mine;
            }
            const unsigned in = __ballot_sync(0xffffffffu, mine), out = __ballot_sync(0xffffffffu, other);
            if (mine) list[n + __popc(in & ((1u << lane) - 1u))] = (int16_t)(2 * p);
            n += __popc(in);
            if (out) break;  // a later unit's part: this unit's are all behind
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count, rows = d.nt * u.k;
    for (int r = blockIdx.y * kCombineWarps + warp; r < rows; r += gridDim.y * kCombineWarps) {
        const int token = d.t0 + r / u.k, slot = r % u.k;
        const int j = u.idx[((int64_t)token * u.g + d.q) * u.k + slot];
        if (j < d.q * u.hpg || j >= (d.q + 1) * u.hpg) continue;
        float M = -INFINITY;
        bool nan = false;
        for (int i = lane; i < n; i += 32) {
            const float x = u.part[((int64_t)list[i] * u.row_cap + r) * kRec + D];
            M = fmaxf(M, x);
            nan |= x != x;
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
        if (__any_sync(0xffffffffu, nan)) M = NAN;
        float L = 0.f, acc[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float* rec = u.part + ((int64_t)list[i] * u.row_cap + r) * kRec;
            const float lse = rec[D];
            if (lse == -INFINITY) continue;  // this part holds no key of the row
            const float w = fast_exp2(lse - M);
            L += w;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] = fmaf(rec[e * 32 + lane], w, acc[e]);
        }
        const float f = u.gate[((int64_t)token * u.g + d.q) * u.k + slot] / L;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            O[((int64_t)token * u.h + j) * D + e * 32 + lane] = Elem<T>::from_f(acc[e] * f);
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

ChunkGeom make_geom(const ChunkArgs& a, const ChunkTiling& t, int parts) {
    const gqe_shape& s = *a.s;
    ChunkGeom u;
    u.T = s.T;
    u.n_seqs = a.n_seqs;
    u.h = s.h;
    u.g = s.g;
    u.k = s.k;
    u.hpg = s.h / s.g;
    u.W = t.rows / s.k;
    u.WU = t.tiles * u.W;
    u.BN = t.keys;
    u.unit_keys = t.unit_keys;
    u.min_cost = t.min_cost;
    u.row_cap = row_cap(&s, t);
    u.cap = a.max_blocks << a.page_shift;
    u.window = a.window >= u.cap ? 0 : a.window;
    u.sinks = u.window ? a.sinks : 0;
    u.page_shift = a.page_shift;
    u.num_pages = a.num_pages;
    u.max_blocks = a.max_blocks;
    u.cu = a.cu_new;
    u.lengths = a.lengths;
    u.block_table = a.block_table;
    u.idx = a.idx;
    u.gate = a.gate;
    u.status = a.status;
    u.desc = static_cast<ChunkDesc*>(a.scratch);
    u.part = reinterpret_cast<float*>(static_cast<char*>(a.scratch) + a256(2 * (size_t)parts * sizeof(ChunkDesc)));
    return u;
}

template <typename T>
cudaError_t launch_combine(const ChunkGeom& u, const ChunkArgs& a, int parts, int blocks) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts, blocks);
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (a.s->d_h) {
        case 32: return cudaLaunchKernelEx(&cfg, chunk_combine_kernel<T, 32>, u, parts, (T*)a.O);
        case 64: return cudaLaunchKernelEx(&cfg, chunk_combine_kernel<T, 64>, u, parts, (T*)a.O);
        default: return cudaLaunchKernelEx(&cfg, chunk_combine_kernel<T, 128>, u, parts, (T*)a.O);
    }
}

}  // namespace

size_t chunk_scratch_bytes(const gqe_shape* s) {
    const ChunkTiling t = tiling(s);
    const size_t parts = (size_t)max_parts(t);
    return a256(2 * parts * sizeof(ChunkDesc)) + a256(2 * parts * row_cap(s, t) * (size_t)(s->d_h + 4) * sizeof(float));
}

cudaError_t launch_chunk(const ChunkArgs& a) {
    const ChunkTiling t = tiling(a.s);
    const int parts = max_parts(t);
    const ChunkGeom u = make_geom(a, t, parts);
    const cudaError_t err = on_tensor_cores(a.s) ? launch_chunk_tc(u, a, parts) : launch_chunk_simt(u, a, parts);
    if (err != cudaSuccess) return err;
    const int blocks = (u.row_cap + 4 * kCombineWarps - 1) / (4 * kCombineWarps);  // about four rows a warp
    return a.s->dtype == GQE_BF16 ? launch_combine<__nv_bfloat16>(u, a, parts, blocks)
                                  : launch_combine<float>(u, a, parts, blocks);
}

}  // namespace gqe
