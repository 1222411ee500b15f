// chunk.cu -- host side of the chunk attention (which kernel, its scratch) and the
// merge of the units that the schedule split.  See chunk.cuh.
#include "chunk.cuh"

namespace gqe {
namespace {

// After the tile kernel, block c, of either kind of units:
//  1. takes again the rows of CTA c's whole units whose result is not finite (only
//     if the CTA has flagged one): see chunk_row;
//  2. merges its share of the split units that part c has steps of, its last and its
//     first: O = gate * sum_p 2^(lse_p - M) o_p / sum_p 2^(lse_p - M) over a unit's
//     parts in order (reproducible).  The blocks of a unit's parts take its groups of
//     kRows rows in turn (by the block of its first part alone, 64 prompt units in two
//     to four parts each kept 64 of 148 blocks busy, for 20 us).
// One block per part: with blocks by part and row range, most of them with nothing
// to do, 20 us went by on their starting and leaving.
constexpr int kCombineWarps = 16;
// Rows a warp merges at once: with four, 3 decodes took 19.4 us for 18.3 and 128 windowed
// ones 116 for 112 (registers, code); with one, prompts under a window 212 for 206.
constexpr int kRows = 2;

// The rows of a unit, of a share of its groups of kRows rows, whose result is not
// finite from the formula, a warp each.
template <typename T, int D>
__device__ __noinline__ void unit_again(const ChunkGeom& u, const ChunkItem& it, int share, int shares, int warp, const T* Q,
                                        const T* Kp, const T* Vp, float scale_log2, T* O) {
    const int lane = threadIdx.x & 31;
    for (int r = warp; r < it.nt * u.k; r += kCombineWarps) {
        if (r / kRows % shares != share) continue;
        const int token = it.t0 + r / u.k;
        const int64_t at = ((int64_t)token * u.g + it.q) * u.k + r % u.k;
        const int j = u.idx[at];
        if (j < it.q * u.hpg || j >= (it.q + 1) * u.hpg) continue;
        const int64_t row = ((int64_t)token * u.h + j) * D;
        float check = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) check += 0.f * Elem<T>::to_f(O[row + e * 32 + lane]);
        if (__all_sync(0xffffffffu, check == 0.f)) continue;
        float acc[D / 32], m, l;
        chunk_row<T, D>(u, it, it.p0 + r / u.k, Q + row, Kp, Vp, scale_log2, acc, m, l);
        const float f = u.gate[at] / l;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) O[row + e * 32 + lane] = Elem<T>::from_f(acc[e] * f);
    }
}

// N consecutive elements, N = 4, 2 or 1.
__device__ __forceinline__ void load_lane(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void load_lane(const float* p, float (&f)[2]) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x, f[1] = v.y;
}
__device__ __forceinline__ void load_lane(const float* p, float (&f)[1]) { f[0] = *p; }
__device__ __forceinline__ void store_lane(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_lane(float* p, const float (&f)[2]) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
}
__device__ __forceinline__ void store_lane(float* p, const float (&f)[1]) { *p = f[0]; }
__device__ __forceinline__ void store_lane(__nv_bfloat16* p, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ void store_lane(__nv_bfloat16* p, const float (&f)[2]) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(f[0], f[1]);
}
__device__ __forceinline__ void store_lane(__nv_bfloat16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }

template <typename T, int D>
__global__ void __launch_bounds__(32 * kCombineWarps, 1)
chunk_combine_kernel(const __grid_constant__ ChunkGeom u, const T* __restrict__ Q, const T* __restrict__ Kp, const T* __restrict__ Vp,
                     float scale_log2, T* __restrict__ O) {
    constexpr int kRec = D + 4, kPer = D / 32;
    // The part's last units of many and few rows, and its first unit of many rows (a
    // unit of few is a group for half of the warps at most: the block of its first part
    // merges it alone): the unit, its records in order and this block's share of its groups.
    constexpr int kSets = 3;
    __shared__ int list[kSets][2 * kChunkMaxParts];  // the block's own part at kChunkMaxParts
    __shared__ int from[kSets], count[kSets], share[kSets], shares[kSets];
    __shared__ ChunkDesc desc[kSets];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool odd = false;
    if (warp < kSets) {
        const int kind = warp == 1, first = warp == 2, begin = kind * u.parts, end = begin + u.parts, c = begin + blockIdx.x;
        // The first rounds' loads are in flight together, 32 parts back and ahead.
        const ChunkDesc none = {-1, 0, 0, 0};
        auto at = [&](int p, int last) {
            const bool in = p >= begin && p < end;
            int4 v = make_int4(-1, 0, 0, 0);
            if (in) v = *reinterpret_cast<const int4*>(&u.desc[2 * p + last]);
            return ChunkDesc{v.x, v.y, v.z, v.w};
        };
        const ChunkDesc d = at(c, 1 - first);
        ChunkDesc middle = first ? at(c - 1 - lane, 0) : none, start = first ? at(c - 1 - lane, 1) : none, ahead = at(c + 1 + lane, 0);
        odd = lane == 0 && !first && u.odd[c] != 0;
        int before = 0, after = 1;
        if (first && d.b >= 0) {  // the parts back to the one that has the unit as its last
            for (int p0 = c - 1;;) {
                const unsigned starts = __ballot_sync(0xffffffffu, start.same_unit(d));
                const unsigned in = __ballot_sync(0xffffffffu, start.same_unit(d) || middle.same_unit(d)) &
                                    (starts ? 2u * (starts & -starts) - 1u : 0xffffffffu);
                if (in >> lane & 1)
                    list[warp][kChunkMaxParts - 1 - before - __popc(in & ((1u << lane) - 1u))] = start.same_unit(d) ? start.rec : middle.rec;
                before += __popc(in);
                p0 -= 32;
                if (starts || p0 < begin) break;
                middle = at(p0 - lane, 0);
                start = at(p0 - lane, 1);
            }
        }
        if (d.b >= 0) {
            for (int p0 = c + 1;;) {
                const unsigned in = __ballot_sync(0xffffffffu, ahead.same_unit(d));
                const unsigned out = __ballot_sync(0xffffffffu, ahead.b >= 0 && !ahead.same_unit(d));
                if (in >> lane & 1) list[warp][kChunkMaxParts + after + __popc(in & ((1u << lane) - 1u))] = ahead.rec;
                after += __popc(in);
                p0 += 32;
                if (out || p0 >= end) break;  // a later unit's part: this unit's are all behind
                ahead = at(p0 + lane, 0);
            }
        }
        if (lane == 0) {
            list[warp][kChunkMaxParts] = d.rec;
            from[warp] = kChunkMaxParts - before;
            count[warp] = d.b >= 0 ? before + after : 0;
            share[warp] = before;
            shares[warp] = kind ? 1 : before + after;
            desc[warp] = d;
        }
    }
    if (__syncthreads_or(odd)) {
        for (int kind = 0; kind < 2; ++kind) {
            if (!u.odd[kind * u.parts + blockIdx.x]) continue;  // the same for the whole block
            ChunkWalk walk(u, kind, blockIdx.x);  // the flags are by CTA
            ChunkItem it;
            while (walk.next(u, it, false))
                if (it.rec < 0) unit_again<T, D>(u, it, 0, 1, warp, Q, Kp, Vp, scale_log2, O);
        }
    }
    bool bad = false;
#pragma unroll 1
    for (int set = 0; set < kSets; ++set) {
        const ChunkDesc& d = desc[set];
        const int n = count[set], rows = n ? d.nt() * u.k : 0, every = shares[set];
        const int* recs = list[set] + from[set];
        for (int r0 = (share[set] + every * warp) * kRows; r0 < rows; r0 += every * kCombineWarps * kRows) {
            // kRows rows and two parts at once, all their loads in flight together (with
            // the maxima in a pass of their own, and a row's loads after another's, 45 us
            // for 38 MB of records); lane holds elements kPer * lane ..  The running
            // maximum, sum and row take the parts in order.
            int to[kRows];  // the head
            float gate[kRows], M[kRows], L[kRows], acc[kRows][kPer];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = min(r0 + i, rows - 1), token = r * u.inv_k >> 16;
                const int64_t at = ((int64_t)(d.t0 + token) * u.g + d.q()) * u.k + r - token * u.k;
                to[i] = u.idx[at];  // first used behind the loop, so that the records' loads follow at once
                gate[i] = u.gate[at];
                M[i] = -INFINITY;
                L[i] = 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[i][e] = 0.f;
            }
            for (int p = 0; p < n; p += 2) {
                float lse[2][kRows], v[2][kRows][kPer];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float* rec0 = u.part + (int64_t)recs[min(p + x, n - 1)] * kRec;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        const float* rec = rec0 + min(r0 + i, rows - 1) * kRec;
                        lse[x][i] = p + x < n ? rec[D] : -INFINITY;
                        load_lane(rec + lane * kPer, v[x][i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    // a log-sum-exp of -inf: no key of the row in that part
                    const float m = fmaxf(fmaxf(lse[0][i], lse[1][i]), M[i]), ref = m == -INFINITY ? 0.f : m;
                    const float w = fast_exp2(M[i] - ref), a = fast_exp2(lse[0][i] - ref), b = fast_exp2(lse[1][i] - ref);
                    M[i] = m;
                    L[i] = L[i] * w + a + b;
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        acc[i][e] = acc[i][e] * w + (lse[0][i] == -INFINITY ? 0.f : v[0][i][e] * a) +
                                    (lse[1][i] == -INFINITY ? 0.f : v[1][i][e] * b);
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = r0 + i;
                if (r >= rows || to[i] < d.q() * u.hpg || to[i] >= (d.q() + 1) * u.hpg) continue;
                const int64_t row = (int64_t)(d.t0 + (r * u.inv_k >> 16)) * u.h + to[i];
                const float scale = gate[i] / L[i];
                float check = L[i] * 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    check += acc[i][e] * 0.f;
                    acc[i][e] *= scale;
                }
                if (!(check == 0.f)) bad = true;
                store_lane(O + row * D + lane * kPer, acc[i]);
            }
        }
    }
    if (!__syncthreads_or(bad)) return;
    for (int x = 0; x < kSets; ++x) {
        if (!count[x]) continue;
        const ChunkDesc d = desc[x];
        const ChunkSeq s = chunk_seq(u, d.b);
        ChunkItem it;
        chunk_item(u, s, d.b, d.q(), (d.t0 - s.t0) / u.WU, it);
        unit_again<T, D>(u, it, share[x], shares[x], warp, Q, Kp, Vp, scale_log2, O);
    }
}

int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return sms;
}

size_t a256(size_t n) { return (n + 255) & ~size_t(255); }

bool on_tensor_cores(const gqe_shape* s) { return s->dtype == GQE_BF16; }

ChunkTiling tiling(const gqe_shape* s) { return on_tensor_cores(s) ? chunk_tc_tiling() : chunk_simt_tiling(s->d_h); }

int max_parts(const ChunkTiling& t) {
    const int p = t.per_sm * device_sms();
    return p < kChunkMaxParts ? p : kChunkMaxParts;
}

// Units per group: no more than one per token, nor than the full ones and one per request.
int64_t max_units(const gqe_shape& s, const ChunkTiling& t, int n_seqs) {
    const int64_t full = (s.T + (int64_t)t.tiles * (t.rows / s.k) - 1) / (t.tiles * (t.rows / s.k)) + (int64_t)n_seqs;
    return full < s.T ? full : s.T;
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
size_t place_bytes(int parts) { return a256(4 * (size_t)parts * sizeof(ChunkPlace)); }
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
    const int64_t units = max_units(s, t, a.n_seqs);
    u.unit_cost[0] = (float)t.unit_keys;
    u.unit_cost[1] = (float)t.few_keys;
    u.cost_scale = 1.0f / 16;
    while ((double)units * s.g * ((double)u.cap + u.WU + t.unit_keys + t.few_keys) * u.cost_scale + (double)units * s.g > 2.0e9)
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
    char* at = static_cast<char*>(a.scratch) + desc_bytes(parts);
    u.place = reinterpret_cast<ChunkPlace*>(at);
    u.odd = reinterpret_cast<int32_t*>(at += place_bytes(parts));
    u.part = reinterpret_cast<float*>(at += odd_bytes(parts));
    return u;
}

template <typename T>
cudaError_t launch_combine(const ChunkGeom& u, const ChunkArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(u.parts);
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
    return desc_bytes((int)parts) + place_bytes((int)parts) + odd_bytes((int)parts) + a256(rows * (size_t)(s->d_h + 4) * sizeof(float));
}

cudaError_t launch_chunk(const ChunkArgs& a) {
    const ChunkTiling t = tiling(a.s);
    // No more blocks than a step of this shape can give parts: idle ones cost small steps
    // their starting and leaving.
    const int64_t cap = (int64_t)a.max_blocks << a.page_shift, span = (int64_t)a.window + a.sinks + t.tiles * (t.rows / a.s->k);
    const int64_t keys = (a.window && span < cap ? span : cap) + (t.unit_keys > t.few_keys ? t.unit_keys : t.few_keys);
    const int64_t pieces = max_units(*a.s, t, a.n_seqs) * a.s->g * ((keys + t.min_keys - 1) / t.min_keys);
    const int parts = pieces < max_parts(t) ? (int)pieces : max_parts(t);
    const ChunkGeom u = make_geom(a, t, parts);
    const cudaError_t err = on_tensor_cores(a.s) ? launch_chunk_tc(u, a) : launch_chunk_simt(u, a);
    if (err != cudaSuccess) return err;
    return a.s->dtype == GQE_BF16 ? launch_combine<__nv_bfloat16>(u, a)
                                  : launch_combine<float>(u, a);
}

}  // namespace gqe
