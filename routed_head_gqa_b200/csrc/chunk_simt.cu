// chunk_simt.cu -- routed attention of ragged chunks of new tokens over a paged
// cache on the CUDA cores, for fp32 caches (d_h = 128, 64 or 32).  See chunk.cuh for
// the units and the schedule.
//
// Per unit: up to 64 query rows, 64 keys a step, one pass over the keys with the
// running row maximum and sum (S = Q K^T, P = 2^(S c - m), O += P V, rescaled
// when the maximum grows), all in fp32.  256 threads as 16 x 16: thread (ty, tx)
// holds rows ty + 16 i and keys tx + 16 j of S, and rows ty + 16 i of O, so a row's
// P is written and read by one half warp.  K and V have one buffer each: the copy of
// the next K runs under the softmax and P V, that of the next V under the next S.
//
// Three forms by the unit's rows.  Up to 4 (a decode): run_few, since the 16 x 16
// threads would compute 16 rows (16 decodes, d_h = 128, 146 us against 301).  Up to
// 16: one row per thread.  Above: four.  Bound by the fp32 pipes and shared memory
// (four loads of Q and four of K feed 64 products per thread), 32 heads in 8 groups,
// k = 2: a prompt of 4096 tokens, d_h = 128, 2.56 ms or 27 TFLOP/s; 64 decodes of 1000 to
// 8000 keys 892 us or 2.8 TB/s, of 1000 to 16000 with d_h = 64 745 us or 3.2 TB/s.
#include "chunk.cuh"

namespace gqe {
namespace {

constexpr int kBM = 64, kBN = 64, kThreads = 256;
constexpr int kPStride = kBN + 4;

template <int D>
struct SimtCfg {
    static constexpr int kVec = 16 / sizeof(float);           // elements per 16 bytes
    static constexpr int kKV = D + kVec;                  // K/V row stride: rows 16 bytes apart modulo the banks
    static constexpr int kQ = D + 4;
    static constexpr size_t kSmem = sizeof(float) * (kBM * kQ + kBM * kPStride) + 2 * sizeof(float) * kBN * kKV;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One tile of K or V rows; keys that no row of the unit sees are zeros.
template <int D>
__device__ __forceinline__ void load_tile(const ChunkGeom& u, const ChunkItem& it, int step, const float* pages, float* dst) {
    using C = SimtCfg<D>;
    constexpr int kPer = D / C::kVec;  // 16-byte vectors per row
    for (int v = threadIdx.x; v < kBN * kPer; v += kThreads) {
        const int row = v / kPer, x = (v % kPer) * C::kVec, s = it.key(step * kBN + row);
        const bool on = s < it.hi && (s >= it.lo || s < u.sinks);
        const float* src = pages;
        if (on) src += (chunk_cache_row(u, it.b, s) * u.g + it.q) * D + x;
        cp_async16(dst + row * C::kKV + x, src, on);
    }
}

// N (2 or 4) consecutive elements, to fp32 and back.
__device__ __forceinline__ void load_cols(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void load_cols(const float* p, float (&f)[2]) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x, f[1] = v.y;
}
__device__ __forceinline__ void store_cols(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_cols(float* p, const float (&f)[2]) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
}
struct SimtShared {
    ChunkSplit split;
    ChunkItem item;
    int has;
    int row_j[kBM];
    float wmax[4][kThreads / 32];  // few rows: the warps' maxima, then their sums
};

// The unit's unselected output slots, by the part that holds its first step.
template <int D>
__device__ __forceinline__ void zero_unselected(const ChunkGeom& u, const ChunkItem& it, const SimtShared& sh, float* O) {
    if (it.s0 != 0) return;
    constexpr int kVec = 16 / sizeof(float), kPer = D / kVec;
    for (int v = threadIdx.x; v < it.nt * u.hpg * kPer; v += kThreads) {
        const int x = v % kPer, j = it.q * u.hpg + (v / kPer) % u.hpg, i = v / kPer / u.hpg;
        bool chosen = false;
        for (int r = 0; r < u.k; ++r) chosen |= sh.row_j[i * u.k + r] == j;
        if (!chosen)
            *reinterpret_cast<uint4*>(O + ((int64_t)(it.t0 + i) * u.h + j) * D + x * kVec) = make_uint4(0, 0, 0, 0);
    }
}

template <int D, int NR>
__device__ __forceinline__ void run_item(const ChunkGeom& u, const ChunkItem& it, const SimtShared& sh, const float* Q,
                                         const float* Kp, const float* Vp, float* O, float scale_log2, float* Qs, float* Ps, float* Ks,
                                         float* Vs) {
    using C = SimtCfg<D>;
    constexpr int kVec = C::kVec;
    constexpr int kCols = D / 16, kCW = kCols < 4 ? kCols : 4, kCN = kCols / kCW;  // O columns per thread
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int rows = it.nt * u.k;

    load_tile<D>(u, it, it.s0, Kp, Ks);
    cp_async_commit();
    load_tile<D>(u, it, it.s0, Vp, Vs);
    cp_async_commit();
    // Q rows as fp32 (rows past the unit's, or of a bad selection, as zeros)
    for (int v = tid; v < NR * 16 * (D / kVec); v += kThreads) {
        const int r = v / (D / kVec), x = (v % (D / kVec)) * kVec;
        float f[kVec];
        if (r < rows && sh.row_j[r] >= 0) {
            const int token = it.t0 + r / u.k;
            load_cols(Q + ((int64_t)token * u.h + sh.row_j[r]) * D + x, f);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < kVec; e += 4)
            *reinterpret_cast<float4*>(Qs + r * C::kQ + x + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
    zero_unselected<D>(u, it, sh, O);

    float m[NR], l[NR], acc[NR][kCols];
    int pos[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        const int r = ty + 16 * i;
        pos[i] = r < rows ? it.p0 + r / u.k : -1;  // -1: sees nothing
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[i][e] = 0.f;
    }

    for (int st = it.s0; st < it.s1; ++st) {
        cp_async_wait<1>();  // K of this step
        __syncthreads();
        float s[NR][4];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
        for (int x = 0; x < D; x += kVec) {
            float kf[4][kVec];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_cols(Ks + (tx + 16 * j) * C::kKV + x, kf[j]);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
#pragma unroll
                for (int e = 0; e < kVec; e += 4) {
                    const float4 qf = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * C::kQ + x + e);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(qf.x, kf[j][e], s[i][j]);
                        s[i][j] = fmaf(qf.y, kf[j][e + 1], s[i][j]);
                        s[i][j] = fmaf(qf.z, kf[j][e + 2], s[i][j]);
                        s[i][j] = fmaf(qf.w, kf[j][e + 3], s[i][j]);
                    }
                }
            }
        }
        __syncthreads();  // every thread has read K
        if (st + 1 < it.s1) load_tile<D>(u, it, st + 1, Kp, Ks);
        cp_async_commit();
        int key[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) key[j] = it.key(st * kBN + tx + 16 * j);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = chunk_sees(u, pos[i], key[j]) ? s[i][j] * scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[i], mx);
            const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen so far: every weight 0
            const float corr = fast_exp2(m[i] - ref);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = fast_exp2(s[i][j] - ref);
                sum += w;
                Ps[(ty + 16 * i) * kPStride + tx + 16 * j] = w;
            }
            l[i] = l[i] * corr + sum;  // this thread's keys; summed over the half warp at the end
            m[i] = mn;
#pragma unroll
            for (int e = 0; e < kCols; ++e) acc[i][e] *= corr;
        }
        __syncwarp();
        cp_async_wait<1>();  // V of this step
        __syncthreads();
#pragma unroll 2
        for (int key = 0; key < kBN; key += 4) {
            float4 pf[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) pf[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * kPStride + key);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                float vf[kCN][kCW];
#pragma unroll
                for (int cn = 0; cn < kCN; ++cn)
                    load_cols(Vs + (key + kk) * C::kKV + cn * 16 * kCW + tx * kCW, vf[cn]);
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const float w = kk == 0 ? pf[i].x : kk == 1 ? pf[i].y : kk == 2 ? pf[i].z : pf[i].w;
#pragma unroll
                    for (int e = 0; e < kCols; ++e) acc[i][e] = fmaf(w, vf[e / kCW][e % kCW], acc[i][e]);
                }
            }
        }
        __syncthreads();  // every thread has read V
        if (st + 1 < it.s1) load_tile<D>(u, it, st + 1, Vp, Vs);
        cp_async_commit();
    }

    const bool partial = it.rec >= 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        float sum = l[i];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const int r = ty + 16 * i;
        const int j = r < rows ? sh.row_j[r] : -1;
        const bool none = m[i] == -INFINITY && sum == 0.f;
        const float inv = none && partial ? 0.f : 1.f / sum;
        float check = 0.f;
#pragma unroll
        for (int e = 0; e < kCols; ++e) check += acc[i][e] * 0.f;  // 0, or NaN when a value is not finite
        if (j >= 0 && !(check + sum * 0.f == 0.f)) u.odd[blockIdx.x] = 1;
        if (j >= 0) {
            const int token = it.t0 + r / u.k;
            float* rec = partial ? u.part + (int64_t)(it.rec + r) * (D + 4) : nullptr;
            float* o = O + ((int64_t)token * u.h + j) * D;
            const float f = partial ? inv : u.gate[((int64_t)token * u.g + it.q) * u.k + r % u.k] * inv;
#pragma unroll
            for (int cn = 0; cn < kCN; ++cn) {
                float out[kCW];
#pragma unroll
                for (int e = 0; e < kCW; ++e) out[e] = acc[i][cn * kCW + e] * f;
                const int col = cn * 16 * kCW + tx * kCW;
                if (partial)
                    store_cols(rec + col, out);
                else
                    store_cols(o + col, out);
            }
            if (partial && tx == 0) rec[D] = none ? -INFINITY : m[i] + log2f(sum);
        }
    }
}

// Few rows (a decode): the 16 x 16 threads over rows and keys would compute 16 rows
// for 1 to 4.  Scores: four threads a key, a quarter of the head each.  P V: a thread
// per element of the head and kThreads / D groups of keys, joined at the end.  The
// running maximum is the tile's for all threads, from shared memory.
template <int D, int R>
__device__ __forceinline__ void run_few(const ChunkGeom& u, const ChunkItem& it, SimtShared& sh, const float* Q, const float* Kp,
                                        const float* Vp, float* O, float scale_log2, float* Qs, float* Ps, float* Ks, float* Vs) {
    using C = SimtCfg<D>;
    constexpr int kVec = C::kVec, kGroups = kThreads / D, kKeys = kBN / kGroups, kQuarter = D / 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, key = tid >> 2, part = tid & 3;
    const int col = tid % D, grp = tid / D;
    const int rows = it.nt * u.k;
    load_tile<D>(u, it, it.s0, Kp, Ks);
    cp_async_commit();
    load_tile<D>(u, it, it.s0, Vp, Vs);
    cp_async_commit();
    for (int x = tid; x < R * D; x += kThreads) {
        const int r = x / D, c = x % D;
        float q = 0.f;
        if (r < rows && sh.row_j[r] >= 0) q = Q[((int64_t)(it.t0 + r / u.k) * u.h + sh.row_j[r]) * D + c];
        Qs[r * C::kQ + c] = q;
    }
    zero_unselected<D>(u, it, sh, O);
    float m[R], l[R], acc[R];
    int pos[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = acc[r] = 0.f;
        pos[r] = r < rows ? it.p0 + r / u.k : -1;
    }
    for (int st = it.s0; st < it.s1; ++st) {
        cp_async_wait<1>();
        __syncthreads();
        float s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = 0.f;
#pragma unroll
        for (int x = 0; x < kQuarter; x += kVec) {
            // quarters interleaved by 16 bytes, so that four threads read 64 adjacent ones
            const int at = x * 4 + part * kVec;
            float kf[kVec];
            load_cols(Ks + key * C::kKV + at, kf);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < kVec; ++e) s[r] = fmaf(Qs[r * C::kQ + at + e], kf[e], s[r]);
        }
        const int abs_key = it.key(st * kBN + key);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
            s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
            s[r] = chunk_sees(u, pos[r], abs_key) ? s[r] * scale_log2 : -INFINITY;
            float mx = s[r];
#pragma unroll
            for (int d = 16; d >= 4; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            if (lane == 0) sh.wmax[r][warp] = mx;
        }
        __syncthreads();  // K read, maxima written
        if (st + 1 < it.s1) load_tile<D>(u, it, st + 1, Kp, Ks);
        cp_async_commit();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mx = m[r];
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) mx = fmaxf(mx, sh.wmax[r][w]);
            const float ref = mx == -INFINITY ? 0.f : mx, corr = fast_exp2(m[r] - ref);
            m[r] = mx;
            const float w = fast_exp2(s[r] - ref);
            l[r] = l[r] * corr + (part == 0 ? w : 0.f);  // this thread's keys; summed at the end
            acc[r] *= corr;
            if (part == 0) Ps[r * kPStride + key] = w;
        }
        cp_async_wait<1>();
        __syncthreads();  // V here, P written
#pragma unroll
        for (int k0 = 0; k0 < kKeys; k0 += 4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = Vs[(grp * kKeys + k0 + e) * C::kKV + col];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 w = *reinterpret_cast<const float4*>(Ps + r * kPStride + grp * kKeys + k0);
                acc[r] = fmaf(w.x, v[0], acc[r]);
                acc[r] = fmaf(w.y, v[1], acc[r]);
                acc[r] = fmaf(w.z, v[2], acc[r]);
                acc[r] = fmaf(w.w, v[3], acc[r]);
            }
        }
        __syncthreads();  // V and P read
        if (st + 1 < it.s1) load_tile<D>(u, it, st + 1, Vp, Vs);
        cp_async_commit();
    }
    // join the groups of keys (in the tile of P) and the threads' sums
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = l[r];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) sh.wmax[r][warp] = sum;
        Ps[r * kThreads + tid] = acc[r];
    }
    __syncthreads();
    const bool partial = it.rec >= 0;
    for (int x = tid; x < rows * D; x += kThreads) {
        const int r = x / D, c = x % D, j = sh.row_j[r];
        if (j < 0) continue;
        float sum = 0.f, o = 0.f, mr = -INFINITY;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sum += sh.wmax[r][w];
#pragma unroll
        for (int g2 = 0; g2 < kGroups; ++g2) o += Ps[r * kThreads + g2 * D + c];
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i == r) mr = m[i];
        const bool none = mr == -INFINITY && sum == 0.f;
        const int token = it.t0 + r / u.k;
        if (!(o * 0.f + sum * 0.f == 0.f)) u.odd[blockIdx.x] = 1;
        if (partial) {
            float* rec = u.part + (int64_t)(it.rec + r) * (D + 4);
            rec[c] = none ? 0.f : o / sum;
            if (c == 0) rec[D] = none ? -INFINITY : mr + log2f(sum);
        } else {
            O[((int64_t)token * u.h + j) * D + c] =
                o * (u.gate[((int64_t)token * u.g + it.q) * u.k + r % u.k] / sum);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 128 ? 1 : 2)
chunk_simt_kernel(const __grid_constant__ ChunkGeom u, const float* __restrict__ Q, const float* __restrict__ Kp, const float* __restrict__ Vp,
                  float* __restrict__ O, float scale_log2) {
    using C = SimtCfg<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ SimtShared sh;
    float* Qs = reinterpret_cast<float*>(smem);
    float* Ps = Qs + kBM * C::kQ;
    float* Ks = Ps + kBM * kPStride;
    float* Vs = Ks + kBN * C::kKV;
    const int tid = threadIdx.x;

    if (tid == 0) chunk_clear(u);
    chunk_split<kThreads>(u, sh.split, blockIdx.x);
    if (!chunk_has(u, sh.split, 0)) return;
    ChunkWalk walk(u, sh.split, 0, blockIdx.x);
    if (tid == 0) walk.leave(u, blockIdx.x);
    while (true) {
        if (tid < 32) {
            ChunkItem it;
            const bool has = walk.next(u, it);
            if (tid == 0) {
                sh.has = has;
                sh.item = it;
            }
        }
        __syncthreads();
        if (!sh.has) break;
        const ChunkItem it = sh.item;
        const int rows = it.nt * u.k;
        for (int r = tid; r < rows; r += kThreads) sh.row_j[r] = chunk_head(u, it.t0 + r / u.k, it.q, r % u.k);
        __syncthreads();
        if (rows <= 2)
            run_few<D, 2>(u, it, sh, Q, Kp, Vp, O, scale_log2, Qs, Ps, Ks, Vs);
        else if (rows <= 4)
            run_few<D, 4>(u, it, sh, Q, Kp, Vp, O, scale_log2, Qs, Ps, Ks, Vs);
        else if (rows <= 16)
            run_item<D, 1>(u, it, sh, Q, Kp, Vp, O, scale_log2, Qs, Ps, Ks, Vs);
        else
            run_item<D, 4>(u, it, sh, Q, Kp, Vp, O, scale_log2, Qs, Ps, Ks, Vs);
        __syncthreads();  // the item, its row table and tiles may be overwritten
    }
    cp_async_wait<0>();
}

template <int D>
cudaError_t launch_typed(const ChunkGeom& u, const ChunkArgs& a) {
    const size_t smem = SimtCfg<D>::kSmem;
    cudaError_t err = cudaFuncSetAttribute(chunk_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    const float scale_log2 = 1.4426950408889634f / sqrtf((float)D);
    chunk_simt_kernel<D><<<u.parts, kThreads, smem, a.stream>>>(u, (const float*)a.Q, (const float*)a.K_pages,
                                                                 (const float*)a.V_pages, (float*)a.O, scale_log2);
    return cudaGetLastError();
}

}  // namespace

// Two blocks per SM where their shared memory allows it (64 decodes, d_h = 64: 189 us, one
// block 286; d_h = 32: 138 and 220).  A unit's fixed cost is set to one step and the smallest
// part to one: with none, 3 or 6 steps, 64 decodes (d_h = 128) take 911, 899 and 909 us for
// 892 and a prompt of 4096 tokens 2.81, 2.50 and 2.59 ms for 2.56; with parts of two or four,
// a step of five short chunks (d_h = 32) takes 28 and 35 us for 18.5.
ChunkTiling chunk_simt_tiling(int d_h) { return {kBM, 1, 0, kBN, kBN, 0, kBN, d_h == 128 ? 1 : 2}; }

cudaError_t launch_chunk_simt(const ChunkGeom& u, const ChunkArgs& a) {
    switch (a.s->d_h) {
        case 32: return launch_typed<32>(u, a);
        case 64: return launch_typed<64>(u, a);
        case 128: return launch_typed<128>(u, a);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gqe
