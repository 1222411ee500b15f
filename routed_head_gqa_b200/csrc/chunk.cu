// chunk.cu -- host side of the chunk attention (which kernel, its scratch) and the
// merge of the units that the schedule split.  See chunk.cuh.
#include "chunk.cuh"

namespace gqe {
namespace {

// After the tile kernel, block c merges its share of the split units that part c has
// steps of, of either kind, its last and its first: O = gate * sum_p 2^(lse_p - M) o_p /
// sum_p 2^(lse_p - M) over a unit's parts in order (reproducible).  The blocks of a
// unit's parts take its groups of kRows rows in turn (by the block of its first part
// alone, 64 prompt units in two to four parts each kept 64 of 148 blocks busy, for 20 us).
// One block per part: with blocks by part and row range, most of them with nothing
// to do, 20 us went by on their starting and leaving.
//
// Only where the tile kernel has flagged a result that is not finite: it multiplies a
// hidden key's weight 0 with its V row, so that an infinity or NaN there reaches rows of
// the unit that do not see the key.  Such spoilt rows are taken again by the formula,
// spread over all blocks (take_again); the merge leaves them out.  What is not finite
// otherwise stays: it comes from what the row sees.
constexpr int kCombineWarps = 16;
// Rows a warp merges at once: with four, 3 decodes took 19.4 us for 18.3 and 128 windowed
// ones 116 for 112 (registers, code); with one, prompts under a window 212 for 206.
constexpr int kRows = 2;

// N consecutive elements, N = 4, 2 or 1.
__device__ __forceinline__ void load_lane(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void load_lane(const __nv_bfloat16* p, float (&f)[2]) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void load_lane(const __nv_bfloat16* p, float (&f)[1]) { f[0] = __bfloat162float(*p); }
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

// A unit's band: the keys that some of its rows see and others do not, at most 255
// behind its first token and as many at the window's lower edge.  A bit for each whose V
// row holds an infinity or NaN, and for each whose K row holds a NaN.
constexpr int kBandSide = 256;
struct Spoilt {
    uint32_t v[kCombineWarps], k[kCombineWarps];  // the lower edge, then the later tokens
};
static_assert(32 * kCombineWarps == 2 * kBandSide, "a word for each warp");

__device__ __forceinline__ int band_key(const ChunkItem& it, int x) { return x < kBandSide ? it.lo + x : it.p0 + 1 + x - kBandSide; }

// As chunk_cache_row, for a key that the tile kernel has looked up (and reported).
__device__ __forceinline__ int seen_row(const ChunkGeom& u, int b, int s) {
    const int pg = u.block_table[(int64_t)b * u.max_blocks + (s >> u.page_shift)];
    return ((unsigned)pg < (unsigned)u.num_pages ? pg << u.page_shift : 0) + (s & ((1 << u.page_shift) - 1));
}

// Fills sp (called by the whole block); whether any V row is marked.
template <typename T, int D>
__device__ __noinline__ bool find_spoilt(const ChunkGeom& u, const ChunkItem& it, const T* Kp, const T* Vp, Spoilt& sp) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool low = 32 * warp < kBandSide;
    const int n = !low ? it.nt - 1 : u.window ? min(it.hi - 1 - u.window, it.p0) - it.lo + 1 : 0;
    const int first = 32 * warp, end = min(n - first % kBandSide, 32);  // this warp's word
    uint32_t words[2];  // of V and K
    const int own = lane < end ? seen_row(u, it.b, band_key(it, first + lane)) : 0;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const T* pages = (which ? Kp : Vp) + it.q * D + lane * kPer;
        uint32_t word = 0;
#pragma unroll 1
        for (int i = 0; i < end; i += 4) {  // four keys' loads in flight
            float v[4][kPer];
#pragma unroll
            for (int j = 0; j < 4; ++j) load_lane(pages + (int64_t)__shfl_sync(0xffffffffu, own, i + j) * (u.g * D), v[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float sum = 0.f;  // NaN if a value is, or an infinity of V
#pragma unroll
                for (int e = 0; e < kPer; ++e) sum += v[j][e] != v[j][e] || !which ? v[j][e] * 0.f : 0.f;
                if (__any_sync(0xffffffffu, sum != sum)) word |= 1u << (i + j);
            }
        }
        word = end > 0 ? word & 0xffffffffu >> (32 - end) : 0;
        if (which) words[1] = word; else words[0] = word;
    }
    uint32_t v_word = words[0], k_word = words[1];
    if (low) v_word &= ~(uint32_t)((1ull << min(max(u.sinks - it.lo - first, 0), 32)) - 1);  // every row sees the first keys
    __syncthreads();  // the words of the unit before have been read
    if (lane == 0) {
        sp.v[warp] = v_word;
        sp.k[warp] = k_word;
    }
    return __syncthreads_or(v_word != 0);
}

// Whether the row at position p has a spoilt element: of a value that is not finite in a
// key that it does not see, and not NaN in one that it sees, which makes the result NaN
// anyway, as a score of NaN does for the whole row.  Warp-collective.
template <typename T, int D>
__device__ __noinline__ bool row_spoilt(const ChunkGeom& u, const ChunkItem& it, int p, const T* Vp, const Spoilt& sp) {
    constexpr int kPer = D / 32;
    constexpr uint32_t kAll = (1u << kPer) - 1u;
    const int lane = threadIdx.x & 31;
    bool whole = false;
    if (lane < kCombineWarps)
#pragma unroll 1
        for (uint32_t w = sp.k[lane]; w; w &= w - 1) whole |= chunk_sees(u, p, band_key(it, 32 * lane + __ffs(w) - 1));
    if (__any_sync(0xffffffffu, whole)) return false;
    uint32_t spoilt = 0, nan = 0;
#pragma unroll 1
    for (int word = 0; word < kCombineWarps; ++word)
#pragma unroll 1
        for (uint32_t w = sp.v[word]; w; w &= w - 1) {
            const int s = band_key(it, 32 * word + __ffs(w) - 1);
            const bool sees = chunk_sees(u, p, s);
            if (!sees && __all_sync(0xffffffffu, spoilt == kAll)) continue;
            float v[kPer];
            load_lane(Vp + ((int64_t)seen_row(u, it.b, s) * u.g + it.q) * D + lane * kPer, v);
            uint32_t hit = 0;
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (v[e] != v[e] || (!sees && !(v[e] * 0.f == 0.f))) hit |= 1u << e;
            if (sees) nan |= hit; else spoilt |= hit;
            if (sees && __all_sync(0xffffffffu, nan == kAll)) return false;
        }
    return __any_sync(0xffffffffu, spoilt & ~nan);
}

// What the warps of a block found of a row, over their shares of its keys.
template <int D>
struct RowParts {
    float m[kCombineWarps], l[kCombineWarps], acc[kCombineWarps][D];
};

// The row of Q and O at `row`, at position p, by the formula alone, key by key over the
// keys that it sees, every 16th 32 of them by a warp.  Called by the whole block.
template <typename T, int D>
__device__ __noinline__ void row_again(const ChunkGeom& u, const ChunkItem& it, int p, int64_t row, float gate,
                                       const T* Q, const T* Kp, const T* Vp, float scale_log2, T* O, RowParts<D>& sh) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float qv[kPer], acc[kPer], m = -INFINITY, l = 0.f;
    load_lane(Q + row * D + lane * kPer, qv);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    const int end = p + 1 - it.skip;  // of the unit's key list
#pragma unroll 1
    for (int x0 = 32 * warp; x0 < end; x0 += 32 * kCombineWarps) {
        // a lane per key: its row, or -1 (a key that the row does not see is neither
        // looked up nor used)
        const int s = it.key(x0 + lane), own = chunk_sees(u, p, s) ? seen_row(u, it.b, s) : -1;
#pragma unroll 1
        for (int i = 0; i < min(32, end - x0); i += 4) {  // four keys' loads in flight
            float x[4], v[4][kPer];
            bool on[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at_row = __shfl_sync(0xffffffffu, own, i + j);
                const int64_t at = ((int64_t)max(at_row, 0) * u.g + it.q) * D + lane * kPer;
                float k[kPer];
                load_lane(Kp + at, k);
                load_lane(Vp + at, v[j]);
                on[j] = at_row >= 0;
                x[j] = 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e) x[j] = fmaf(qv[e], k[e], x[j]);
            }
            float mx = m;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) x[j] += __shfl_xor_sync(0xffffffffu, x[j], d);
                x[j] = on[j] ? x[j] * scale_log2 : -INFINITY;
                mx = fmaxf(mx, x[j]);
            }
            const float corr = m == -INFINITY ? 0.f : fast_exp2(m - mx);
            m = mx;
            l *= corr;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] *= corr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (x[j] == -INFINITY) continue;  // weight 0 beside any other key
                const float w = fast_exp2(x[j] - m);
                l += w;
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, v[j][e], acc[e]);
            }
        }
        if (l != l) break;  // a score was NaN: so is the whole row
    }
    __syncthreads();  // the row before has been read
    if (lane == 0) {
        sh.m[warp] = m;
        sh.l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) sh.acc[warp][lane * kPer + e] = acc[e];
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= D) return;
    float M = -INFINITY, L = 0.f, sum = 0.f;
#pragma unroll 1
    for (int w = 0; w < kCombineWarps; ++w) M = fmaxf(M, sh.m[w]);
#pragma unroll 1
    for (int w = 0; w < kCombineWarps; ++w) {
        // no key with a weight: 0 (its sum is 0, or NaN for a NaN score)
        const float f = sh.m[w] == -INFINITY ? 0.f : fast_exp2(sh.m[w] - M);
        L += sh.l[w] * f;
        sum += sh.acc[w][e] * f;
    }
    O[row * D + e] = Elem<T>::from_f(sum * __fdividef(gate, L));
}

// Takes the spoilt rows of the whole step again, by all blocks: each goes through the
// flagged CTAs' units, by the places that they left (its own split of the step might
// place a border one step off, as the compiler is free to round the costs in another way
// in another kernel), and takes every gridDim.x-th row.  A prompt of 2048 tokens behind
// 12000 keys (0.24 ms): NaN in a value that all rows see, 1.4 ms; in the last new one, which
// spoils the 510 rows of a unit of each group, 3.0; decodes have nothing to take again.
// (A warp for each row that is not finite, over its whole cache: 184 and 139 ms.)
template <typename T, int D>
__device__ __forceinline__ void take_again(const ChunkGeom& u, const T* Q, const T* Kp, const T* Vp, float scale_log2, T* O, Spoilt& sp,
                                           RowParts<D>& sh) {
    int turn = 0;  // the block that the next row falls to
    unsigned odd = 0;  // of 32 flags, those behind the last
#pragma unroll 1
    for (int base = -32;;) {
        while (!odd && (base += 32) < 2 * u.parts) {
            const int mine = base + (threadIdx.x & 31);
            odd = __ballot_sync(0xffffffffu, mine < 2 * u.parts && u.odd[mine] != 0);
        }
        if (!odd) break;
        const int flag = base + __ffs(odd) - 1;
        odd &= odd - 1;
        const int kind = flag >= u.parts, first = kind * u.parts, part = chunk_part(u, kind, flag - first);
        const ChunkPlace at = u.place[2 * flag], to = u.place[2 * flag + 1];
        ChunkPlace x = at;
        // a unit that goes on from the part before comes with that one, if it is flagged
        if (x.s > 0 && u.odd[first + chunk_part(u, kind, part - 1)]) ++x.i;
#pragma unroll 1
        for (; x.b < u.n_seqs && x.b <= to.b; ++x.b, x.q = x.i = 0) {
            const int t0 = u.cu[x.b], t1 = u.cu[x.b + 1], L = u.lengths[x.b];
            const ChunkSeq s = {t0, (int)((unsigned)t1 - (unsigned)t0), L};
            // no work, one row a unit, or entries that contradict each other (as chunk_seq, which has reported them)
            if (t0 < 0 || t1 < t0 || t1 > u.T || s.n < 2 || L < s.n || L > u.cap || chunk_kind(u, s.n) != kind) continue;
#pragma unroll 1
            for (; x.q < u.g; ++x.q, x.i = 0)
#pragma unroll 1
                for (; x.i * u.WU < s.n; ++x.i) {
                    if (x.b == to.b && (x.q > to.q || (x.q == to.q && (x.i > to.i || (x.i == to.i && to.s == 0))))) break;
                    ChunkItem it;
                    chunk_item(u, s, x.b, x.q, x.i, it);
                    if (!find_spoilt<T, D>(u, it, Kp, Vp, sp)) continue;
                    const int rows = it.nt * u.k;
#pragma unroll 1
                    for (int r = ((int)blockIdx.x >= turn ? 0 : (int)gridDim.x) + blockIdx.x - turn; r < rows; r += gridDim.x) {
                        const int token = r * u.inv_k >> 16, t = it.t0 + token;
                        const int64_t pick = ((int64_t)t * u.g + it.q) * u.k + r - token * u.k;
                        const int j = u.idx[pick];
                        if (j < it.q * u.hpg || j >= (it.q + 1) * u.hpg) continue;
                        if (row_spoilt<T, D>(u, it, it.p0 + token, Vp, sp))  // the same in every warp
                            row_again<T, D>(u, it, it.p0 + token, (int64_t)t * u.h + j, u.gate[pick], Q, Kp, Vp, scale_log2, O, sh);
                    }
                    turn = (turn + rows) % gridDim.x;
                }
        }
    }
}

// The split units that a block merges a share of (see the kernel): each with its records
// in order, from list[.][from], and this block's share of its groups of kRows rows.
constexpr int kSets = 3;
struct MergeSets {
    int list[kSets][2 * kChunkMaxParts];
    int from[kSets], count[kSets], share[kSets], shares[kSets];
    ChunkDesc desc[kSets];
};

// Merges a set, without the spoilt rows of a unit that has some (sp, it; else null).
template <typename T, int D>
__device__ __forceinline__ void merge_set(const ChunkGeom& u, const MergeSets& sets, int set, T* O, const ChunkItem* it, const T* Vp,
                                          const Spoilt* sp) {
    constexpr int kRec = D + 4, kPer = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const ChunkDesc& d = sets.desc[set];
    const int n = sets.count[set], rows = n ? d.nt() * u.k : 0, every = sets.shares[set];
    const int* recs = sets.list[set] + sets.from[set];
    for (int r0 = (sets.share[set] + every * warp) * kRows; r0 < rows; r0 += every * kCombineWarps * kRows) {
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
            const int r = r0 + i, token = r * u.inv_k >> 16;
            if (r >= rows || to[i] < d.q() * u.hpg || to[i] >= (d.q() + 1) * u.hpg) continue;
            if (sp && row_spoilt<T, D>(u, *it, it->p0 + token, Vp, *sp)) continue;
            const int64_t row = (int64_t)(d.t0 + token) * u.h + to[i];
            const float scale = gate[i] / L[i];
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[i][e] *= scale;
            store_lane(O + row * D + lane * kPer, acc[i]);
        }
    }
}

// The merge of a step that has flags.  The code of this and what it calls is kept small:
// that it is there costs each step about a microsecond (3 decodes 17.9 us, without it 16.4;
// with eight keys in flight and a merge of its own here 18.7).
template <typename T, int D>
__device__ __forceinline__ void merge_odd(const ChunkGeom& u, const MergeSets& sets, const T* Q, const T* Kp, const T* Vp, float scale_log2,
                                          T* O, Spoilt& sp, RowParts<D>& sh) {
#pragma unroll 1
    for (int set = 0; set < kSets; ++set) {
        if (!sets.count[set]) continue;  // the same for the whole block
        const ChunkDesc d = sets.desc[set];
        const int kind = set == 1;
        bool odd = false;  // a flagged CTA has steps of the unit
#pragma unroll 1
        for (int p = threadIdx.x; p < u.parts; p += 32 * kCombineWarps) {
            const ChunkDesc* own = u.desc + 2 * (kind * u.parts + p);
            odd |= u.odd[kind * u.parts + chunk_part(u, kind, p)] && (own[0].same_unit(d) || own[1].same_unit(d));
        }
        ChunkItem it;
        const ChunkSeq s = {u.cu[d.b], u.cu[d.b + 1] - u.cu[d.b], u.lengths[d.b]};
        chunk_item(u, s, d.b, d.q(), (d.t0 - s.t0) / u.WU, it);
        const bool spoilt = __syncthreads_or(odd) && find_spoilt<T, D>(u, it, Kp, Vp, sp);
        merge_set<T, D>(u, sets, set, O, &it, Vp, spoilt ? &sp : nullptr);
    }
    take_again<T, D>(u, Q, Kp, Vp, scale_log2, O, sp, sh);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kCombineWarps, 1)
chunk_combine_kernel(const __grid_constant__ ChunkGeom u, const T* __restrict__ Q, const T* __restrict__ Kp, const T* __restrict__ Vp,
                     float scale_log2, T* __restrict__ O) {
    // The part's last units of many and few rows, and its first unit of many rows (a
    // unit of few is a group for half of the warps at most: the block of its first part
    // merges it alone).
    __shared__ MergeSets sets;
    __shared__ Spoilt spoilt;
    __shared__ RowParts<D> row_parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // every CTA's flags, looked at behind the lists below
    static_assert(2 * kChunkMaxParts <= 2 * 32 * kCombineWarps, "two flags a thread");
    const int odd0 = tid < 2 * u.parts ? u.odd[tid] : 0;
    const int odd1 = tid + 32 * kCombineWarps < 2 * u.parts ? u.odd[tid + 32 * kCombineWarps] : 0;
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
        int before = 0, after = 1;
        if (first && d.b >= 0) {  // the parts back to the one that has the unit as its last
            for (int p0 = c - 1;;) {
                const unsigned starts = __ballot_sync(0xffffffffu, start.same_unit(d));
                const unsigned in = __ballot_sync(0xffffffffu, start.same_unit(d) || middle.same_unit(d)) &
                                    (starts ? 2u * (starts & -starts) - 1u : 0xffffffffu);
                if (in >> lane & 1)
                    sets.list[warp][kChunkMaxParts - 1 - before - __popc(in & ((1u << lane) - 1u))] = start.same_unit(d) ? start.rec : middle.rec;
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
                if (in >> lane & 1) sets.list[warp][kChunkMaxParts + after + __popc(in & ((1u << lane) - 1u))] = ahead.rec;
                after += __popc(in);
                p0 += 32;
                if (out || p0 >= end) break;  // a later unit's part: this unit's are all behind
                ahead = at(p0 + lane, 0);
            }
        }
        if (lane == 0) {
            sets.list[warp][kChunkMaxParts] = d.rec;
            sets.from[warp] = kChunkMaxParts - before;
            sets.count[warp] = d.b >= 0 ? before + after : 0;
            sets.share[warp] = before;
            sets.shares[warp] = kind ? 1 : before + after;
            sets.desc[warp] = d;
        }
    }
    if (__syncthreads_or(odd0 | odd1)) {  // the same for every block
        merge_odd<T, D>(u, sets, Q, Kp, Vp, scale_log2, O, spoilt, row_parts);
        return;
    }
#pragma unroll 1
    for (int set = 0; set < kSets; ++set) merge_set<T, D>(u, sets, set, O, nullptr, nullptr, nullptr);
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
