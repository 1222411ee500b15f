// chunk_tc.cu -- routed attention of ragged chunks of new tokens over a paged
// cache on the sm_100a tensor cores (bf16, d_h = 128, 64 or 32), with an optional sliding
// window.  See chunk.cuh for the units, the schedule and the masks.
//
// A unit has up to two query tiles of 128 rows (W = floor(128 / k) tokens of k
// rows each) over one stream of 128-key K/V tiles.  A unit of at most 16 rows (a
// decode, or a few tokens of it) is turned around: the keys take the 128 lanes,
// S^T = K Q^T is 128 x 16 and O^T += V^T P 128 x 16, so that all threads share
// the exponentials of a step (as one row per thread, k threads would work and
// 128 - k would wait: 3500 clocks a step, 1.8 times what the step's K/V take from
// HBM) and the MMAs shrink with the rows.  Its two warpgroups take every other
// step, each with its own maximum, sum and O^T, merged at the end of the item.
//
// Roles (384 threads, with small pages 512; one persistent CTA per SM):
//   warp 0      K/V tiles by TMA, a box per page (of at most 128 rows), lane by lane;
//               pages that no row of the unit sees are loaded from outside the pool,
//               which the TMA fills with zeros.
//   warps 12-15 in its place, small pages: 16-byte asynchronous copies, a quarter of
//               the rows each (one warp had so few in flight that 64 decodes on
//               4-row pages ran at 1.3 TB/s, four at 3.6)
//   warp 1      MMA issuer (one thread): S_t = Q_t K^T
//   warp 2      walks the part's items (a ring of 4) and tables their rows of Q and O;
//               gathers Q of the units of few rows by 16-byte asynchronous copies
//   warp 3      MMA issuer (one thread): O_t += P_t V.  Before it, the whole warp
//               zeroes the tile's V rows that no row of the unit sees (past the
//               last token, outside the window): their weight is 0, but 0 times
//               what an unused row holds may be NaN.
//   warps 4-7   softmax and epilogue of query tile 0, a row per thread (few rows: the
//               even steps, a key per thread); before them the copies of its rows of
//               Q, under the epilogue of the unit before (copied by warp 2, a prompt's
//               256 rows held each unit up for 9600 clocks), and the zero rows of the
//               unselected heads as bulk copies of 2 d_h bytes from shared memory
//               (issued by warp 2 instead, prompts under a window took 257 us for 209)
//   warps 8-11  the same for query tile 1 (few rows: the odd steps)
// A CTA runs its units of one kind and then those of the other; what the kinds use
// differently (Q tiles and stages, the stages of the epilogue and the hand-over of few
// rows) changes hands at kind_done, kind_done_v and x_free.
//
// TMEM: one S buffer [0,128) that the tiles take in turn, P_0 [128,192) and P_1
// [192,256) (bf16 pairs), O_0 [256,384), O_1 [384,512).  The softmax copies S to
// registers and hands the buffer back at once, so the next S runs under it.  Few
// rows: S^T_t [64 t, 64 t + 16), O^T_t the first 16 columns of O_t, P in shared
// memory as the second operand.
//
// Bounds and figures (d_h = 128, 32 heads in 8 groups, k = 2).  Decodes: HBM; 64 of
// 1000 to 16000 keys, 64-row pages, 2.5 GB, 389 us or 6.46 TB/s (a plain copy: 6.55);
// 128 under a window of 1024, nine steps each, 112 us or 4.8 TB/s (a unit's end
// costs its groups about 2.5 us, under which the stages fill and then wait).  Prompts:
// the exponentials and the S -> P -> O chain of a step, 3200 clocks of which the
// products take 2048, and 12000 a unit (its first S and its epilogue overlap no
// products): two chunks of 4096 tokens behind 12000 to 28000 keys, 1.64 to 1.66 ms or
// 930 TFLOP/s at the power cap.  Narrow heads move half or a quarter of the bytes in the
// same chain of waits: the 64 decodes with d_h = 64, 281 us or 4.0 TB/s, d_h = 32, 241 us.
//
// Rounding: P is rounded to bf16 for the second product (half a step, 2^-8 of
// each weight, the same size as the output's own rounding); the row sums take
// the unrounded weights, and everything else is fp32.
#include <atomic>
#include <climits>

#include "chunk.cuh"
#include "exp2_fma.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace gqe {
namespace {

using namespace sm100;
using bf16 = __nv_bfloat16;

constexpr int kBM = 128, kBN = 128, kQT = 2;
constexpr int kFew = 16;                   // query rows up to which a unit is turned around
constexpr int kItems = 4;                  // items in flight between the walk and the other roles
constexpr uint32_t kPart = 8 * 64 * 2;     // 64 elements of 8 rows, a swizzle atom
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: p <= 2^8 between rescales
constexpr uint32_t kWhereChunkTc = 11;     // status "where" id of this kernel
// Threads and register split (setmaxnreg): 4 control warps and, for gathered
// pages, 4 that copy rows; 8 softmax warps.
template <bool kGather>
struct Split {
    static constexpr int kThreads = kGather ? 512 : 384;
    static constexpr int kRegsLaunch = kGather ? 128 : 168;
    static constexpr int kRegsCtl = kGather ? 56 : 72, kRegsSoftmax = kGather ? 200 : 216;
    static_assert((kThreads - 256) * kRegsCtl + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "more registers than the launch has");
};

// kH: a head in 64-element parts, two (d_h = 128) or one (d_h = 64, or 32 in one
// padded with zeros).
template <int kH>
struct Smem {
    // A Q, K or V tile: groups of 8 rows, the kH parts of a group one after the other,
    // so that one box fetches both parts of a page (a box per page and part held 16-row
    // pages at 5.8 TB/s).
    static constexpr uint32_t kTile = kBM / 8 * kH * kPart;
    static constexpr int kStages = 4 / kH;         // K and V tiles in flight, each
    // Q_0, the K stages, the V stages, Q_1.  Few rows, whose Q is small, have Q_0 and
    // Q_1 as one more stage.
    uint8_t tile[2 * kStages + 2][kTile];
    uint8_t qf[2][kH * kFew * 128];      // few rows: Q, for two items
    uint8_t p[kQT][kFew * 256];          // few rows: P_t [16 rows][128 keys] bf16, two 64-key halves
    float x[kFew][128];                  // few rows: O^T_1 on its way to warpgroup 0
    __device__ __forceinline__ uint8_t* q(int t) { return tile[t ? 2 * kStages + 1 : 0]; }
    __device__ __forceinline__ uint8_t* k(bool few, int st) { return tile[st + (few ? 0 : 1)]; }
    __device__ __forceinline__ uint8_t* v(int st) { return tile[kStages + 1 + st]; }
    // Many rows: 64 bytes of each of a softmax warp's 32 rows on their way out, in a
    // half of the group's own p and of x.
    __device__ __forceinline__ uint4* stage(int t, int w) {
        return reinterpret_cast<uint4*>(w < 2 ? p[t] + w * 2048 : reinterpret_cast<uint8_t*>(x) + t * 4096 + (w - 2) * 2048);
    }
    float x_ml[2][kFew];                 //   with its maxima and sums
    uint4 zero[16];                     // a row of zeros, for the unselected output slots
    float4 wmax[kQT][2][kFew];           // few rows: the four warps' maxima of a step
    float4 wsum[kQT][kFew];              //   and their sums at the end
    ChunkItem item[kItems];
    int32_t has[kItems];                 // 0: no more items of the kind
    int32_t row[kItems][kQT][kBM];       // each query row's row of Q and O seen as [T * h, d_h], -1: none
    int32_t kv_row[4][kBN / 4];          // cache rows being copied (gathered pages)
    ChunkSplit split;
    // barriers, in the order of kBarCounts
    uint64_t item_full[kItems], rows_full[kItems], item_free[kItems];
    // by kind: the many rows' kStages stages, the few's one more
    uint64_t kv_full_k[2 * kStages + 1], kv_full_v[2 * kStages + 1], kv_empty_k[2 * kStages + 1], kv_empty_v[2 * kStages + 1];
    uint64_t s_full[kQT], p_empty[kQT], o_full[kQT], q_full[kQT], q_empty[kQT], p_full[kQT], o_empty[kQT], st_free[kQT], vote[kQT], qm_full[kQT];
    uint64_t x_full, x_free, s_free, mma_drain, mma_drain2, kind_done, kind_done_v;
    uint32_t tmem_base;
    int32_t abort_flag;
};

// Arrivals that complete a barrier: the readers of an item (warps 0, 1, 3, the
// eight softmax warps, and for gathered pages the four that copy in warp 0's place),
// the 128 threads of those, the four warps of a warpgroup, or one.
template <int kH, bool kGather>
__device__ __forceinline__ uint32_t bar_count(int i) {
    constexpr int kS = 2 * Smem<kH>::kStages + 1, kFree = 2 * kItems, kLoads = 3 * kItems, kOnes = kLoads + 2 * kS,
                  kWarps = kOnes + 2 * kS + 5 * kQT, kTail = kWarps + 5 * kQT + 3;
    return i < kFree ? 1 : i < kLoads ? (kGather ? 14 : 11) : i < kOnes ? (kGather ? 128 : 1) : i < kWarps ? 1 : i < kTail ? 4 : 1;
}
template <int kH>
constexpr int bar_total() { return 3 * kItems + 8 * Smem<kH>::kStages + 4 + 10 * kQT + 7; }

// Place in the ring of K/V stages, and the parity of its round.  The two kinds of
// units have rings of their own, kStages or one more, with barriers of their own.
template <int kStages>
struct Ring {
    int st;
    uint32_t phase;
    bool few;
    __device__ __forceinline__ explicit Ring(bool few) : st(0), phase(0), few(few) {}
    __device__ __forceinline__ int bar() const { return few ? kStages + st : st; }
    __device__ __forceinline__ int size() const { return kStages + (few ? 1 : 0); }
    __device__ __forceinline__ void next() {
        if (++st == size()) {
            st = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void prev() {
        if (--st < 0) {
            st = size() - 1;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void turn() {  // to the other kind
        st = 0;
        phase = 0;
        few = !few;
    }
};

struct Params {
    const bf16* Q;
    bf16* O;
    float scale_log2;
    const bf16* K;  // gathered pages only
    const bf16* V;
    int d;          // d_h
};

__device__ __forceinline__ void tma_load_5d(const CUtensorMap* map, uint64_t* bar, void* dst, int c0, int c1, int c2, int c3,
                                            int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

template <class S>
__device__ __forceinline__ bool aborted(S& sm) { return *((volatile int32_t*)&sm.abort_flag) != 0; }
// Bounded wait of at most kWaitTimeoutNs, in few instructions: the roles wait in
// some fifty places, and a kernel that outgrows the instruction cache (253 KB with
// mbar_wait and the error report at each of them) pays for it at every change of
// phase, 1.7 times the time of the steps around a unit's ends.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u64 t0, t;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u64 t0, %%globaltimer;\n"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE;\n\t"
        "mov.u64 t, %%globaltimer;\n\tsub.u64 t, t, t0;\n\tsetp.lt.u64 q, t, %4;\n\t"
        "@q bra AGAIN;\n"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs), "l"(kWaitTimeoutNs)
        : "memory");
    return ok != 0;
}
// A wait that ran out: every role stops at its next item, and the kernel reports
// the place when it ends.
template <class S>
__device__ __forceinline__ void fail(S& sm, int32_t detail) { *((volatile int32_t*)&sm.abort_flag) = detail; }
// The whole warp waits; false if the wait ran out for any lane.
template <class S>
__device__ __forceinline__ bool warp_wait(S& sm, uint64_t* bar, uint32_t parity, int32_t detail) {
    if (__all_sync(0xffffffffu, bar_wait(bar, parity))) return true;
    fail(sm, detail);
    return false;
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void ld_wait_bind(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void ld_bind(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Steps of the item that query tile t takes part in: the first ones, up to its
// own last token (none when the unit has no token for the tile).  Few rows: every
// other step, from step t on.
__device__ __forceinline__ int tile_steps(const ChunkGeom& u, const ChunkItem& it, int t, bool few) {
    if (few) return (it.s1 - it.s0 + 1 - t) >> 1;
    if (it.nt <= t * u.W) return 0;
    const int hi = it.p0 + min(it.nt, (t + 1) * u.W);
    const int end = min(it.s1, (hi - it.skip + kBN - 1) / kBN);
    return max(0, end - it.s0);
}

// Bits 0 .. n-1 of a word (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
    uint32_t m;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(m) : "r"(max(n, 0)));
    return m;
}

// S_t = Q_t K(it)^T: eight K steps of 16 over 128-byte swizzled tiles; a step
// moves the descriptors' start address only (d_h = 64: four).
template <int kH>
__device__ __forceinline__ void issue_s(uint32_t tmem, uint32_t dhi, uint32_t q_lo, uint32_t k_lo) {
    constexpr uint32_t idesc = idesc_bf16_f32(kBM, kBN, false, false);
#pragma unroll
    for (int kk = 0; kk < 4 * kH; ++kk) {
        const uint32_t off = (uint32_t)(((kk >> 2) * kPart + (kk & 3) * 32) >> 4);
        umma_ss(tmem + kColS, smem_desc_join(q_lo + off, dhi), smem_desc_join(k_lo + off, dhi), idesc, kk > 0 ? 1u : 0u);
    }
}
// O_t += P_t V(it), P_t from TMEM, V as an MN-major operand.
template <int kH>
__device__ __forceinline__ void issue_pv(uint32_t tmem, uint32_t dhi, int t, uint32_t v_lo, bool first) {
    constexpr uint32_t idesc = idesc_bf16_f32(kBM, 64 * kH, false, true);
#pragma unroll
    for (int kk = 0; kk < kBN / 16; ++kk)
        umma_ts(tmem + kColO + t * 128, tmem + kColP + 64 * t + kk * 8, smem_desc_join(v_lo + (uint32_t)((kk * 2 * kH * kPart) >> 4), dhi),
                idesc, first && kk == 0 ? 0u : 1u);
}

// Few rows: S^T_t = K(it) Q^T, and O^T_t += V(it)^T P_t with V as an MN-major
// operand of M = 128 elements of the head (d_h = 64: the part twice, its leading
// byte offset 0) and P_t from shared memory.
template <int kH>
__device__ __forceinline__ void issue_st(uint32_t tmem, uint32_t dhi, int t, uint32_t q_lo, uint32_t k_lo) {
    constexpr uint32_t idesc = idesc_bf16_f32(kBN, kFew, false, false);
#pragma unroll
    for (int kk = 0; kk < 4 * kH; ++kk) {
        const uint32_t off = (uint32_t)(((kk >> 2) * kPart + (kk & 3) * 32) >> 4);
        umma_ss(tmem + kColS + 64 * t, smem_desc_join(k_lo + off, dhi), smem_desc_join(q_lo + off, dhi), idesc, kk > 0 ? 1u : 0u);
    }
}
template <int kH>
__device__ __forceinline__ void issue_pvt(uint32_t tmem, uint32_t dhi, uint32_t p_hi, int t, uint32_t v_lo, uint32_t p_lo, bool first) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, kFew, true, false);
#pragma unroll
    for (int kk = 0; kk < kBN / 16; ++kk)
        umma_ss(tmem + kColO + t * 128, smem_desc_join(v_lo + (uint32_t)((kk * 2 * kH * kPart) >> 4), dhi),
                smem_desc_join(p_lo + (uint32_t)(((kk >> 2) * kFew * 128 + (kk & 3) * 32) >> 4), p_hi), idesc,
                first && kk == 0 ? 0u : 1u);
}

__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Softmax, epilogue and merge of an item of at most NR rows (few rows), for the
// warpgroup of tile t.  Each thread holds one key of a step, then one element of
// the head.  Returns false when a wait ran out.
template <int NR, int kH>
__device__ __forceinline__ bool few_item(const ChunkGeom& u, const Params& p, Smem<kH>& sm, const ChunkItem& it, int slot, int t,
                                         uint32_t tmem, uint32_t& ctile, uint32_t& o_it, uint32_t& votes, uint32_t& swaps) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = warp & 3, col = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + kColS + 64 * t, o_addr = tmem + lane_off + kColO + 128 * t;
    const int rows = it.nt * u.k, steps = it.s1 - it.s0, n = tile_steps(u, it, t, true);
    const int d = kH == 2 ? 128 : p.d;
    const bool partial = it.rec >= 0;
    // gate of row `lane`, in flight until the epilogue
    float gate = 0.f;
    if (t == 0 && !partial && lane < rows) {
        const int token = lane * u.inv_k >> 16;
        gate = u.gate[((int64_t)(it.t0 + token) * u.g + it.q) * u.k + lane - token * u.k];
    }
    float m[NR], l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    // the four warps of the group have written what the others read next
    auto meet = [&]() {
        warp_arrive(&sm.vote[t]);
        const bool ok = warp_wait(sm, &sm.vote[t], votes & 1, 46);
        ++votes;
        return ok;
    };
#pragma unroll 1
    for (int i = 0; i < n; ++i, ++ctile) {
        if (!warp_wait(sm, &sm.s_full[t], ctile & 1, 47)) return false;
        tc_fence_after();
        uint32_t s[16];
        tmem_ld16(s_addr, s);
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < 16; ++r) asm volatile("" : "+r"(s[r]));
        tc_fence_before();
        warp_arrive(&sm.st_free[t]);
        const int x0 = (it.s0 + 2 * i + t) * kBN, key = it.key(x0 + col);
        const bool need_mask = x0 + it.skip + kBN - 1 > it.p0 || (u.window && x0 + it.skip <= it.hi - 1 - u.window);
        float x[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) x[r] = __uint_as_float(s[r]) * p.scale_log2;
        if (need_mask) {
            int pos = it.p0, left = u.k;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                if (!chunk_sees(u, pos, key)) x[r] = -INFINITY;
                if (--left == 0) {
                    left = u.k;
                    ++pos;
                }
            }
        }
        float* mine = reinterpret_cast<float*>(sm.wmax[t][votes & 1]) + wq;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float y = warp_max(x[r]);
            if (lane == 0) mine[4 * r] = y;
        }
        const float4* all = sm.wmax[t][votes & 1];
        if (!meet()) return false;
        // Lazy rescaling as for many rows; the same for every thread of the group.
        float alpha[NR];
        bool rescale = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float4 w = all[r];
            const float mx = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
            alpha[r] = 1.f;
            if (mx > m[r] + kRescaleThreshold || m[r] == -INFINITY) {
                if (m[r] != -INFINITY) {
                    alpha[r] = fast_exp2(m[r] - mx);
                    rescale |= r < rows;
                }
                m[r] = mx;
            }
        }
        // P_t and O^T_t: free once the group's previous product has completed
        if (ctile > 0 && !warp_wait(sm, &sm.p_empty[t], (ctile - 1) & 1, 48)) return false;
        if (rescale) {
            tc_fence_after();
            uint32_t o[16];
            tmem_ld16(o_addr, o);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < 16; ++r) asm volatile("" : "+r"(o[r]));
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
                l[r] *= alpha[r];
            }
            tmem_st16(o_addr, o);
            tmem_st_wait();
        }
        uint8_t* pt = sm.p[t] + (wq >> 1) * (kFew * 128);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float w = fast_exp2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
            l[r] += w;
            *reinterpret_cast<bf16*>(pt + r * 128 + (((col & 63) * 2) ^ ((r & 7) << 4))) = __float2bfloat16_rn(w);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&sm.p_full[t]);
    }
    uint32_t o[16];
    if (n > 0) {
        if (!warp_wait(sm, &sm.o_full[t], o_it & 1, 49)) return false;
        ++o_it;
        tc_fence_after();
        tmem_ld16(o_addr, o);
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < 16; ++r) asm volatile("" : "+r"(o[r]));
        tc_fence_before();
        warp_arrive(&sm.o_empty[t]);
        float* mine = reinterpret_cast<float*>(sm.wsum[t]) + wq;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float y = warp_sum(l[r]);
            if (lane == 0) mine[4 * r] = y;
        }
        if (!meet()) return false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float4 w = sm.wsum[t][r];
            l[r] = (w.x + w.y) + (w.z + w.w);
        }
    }
    if (steps > 1) {  // both groups took part: group 1 hands its state to group 0
        if (t == 1) {
            if (!warp_wait(sm, &sm.x_free, swaps & 1, 50)) return false;
            ++swaps;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                sm.x[r][col] = __uint_as_float(o[r]);
                if (col == 0) {
                    sm.x_ml[0][r] = m[r];
                    sm.x_ml[1][r] = l[r];
                }
            }
            warp_arrive(&sm.x_full);
            return true;
        }
        if (!warp_wait(sm, &sm.x_full, swaps & 1, 51)) return false;
        ++swaps;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float m1 = sm.x_ml[0][r], mx = fmaxf(m[r], m1), ref = mx == -INFINITY ? 0.f : mx;
            const float a = fast_exp2(m[r] - ref), b = fast_exp2(m1 - ref);  // 0 where a group saw no key
            o[r] = __float_as_uint(__uint_as_float(o[r]) * a + sm.x[r][col] * b);
            l[r] = l[r] * a + sm.x_ml[1][r] * b;
            m[r] = mx;
        }
        warp_arrive(&sm.x_free);
    } else if (t == 1) {
        return true;
    }
    float check = 0.f;  // stays 0, or NaN when a value is not finite
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int out = r < rows ? sm.row[slot][0][r] : -1;
        const float gm = __shfl_sync(0xffffffffu, gate, r);
        if (out < 0 || col >= d) continue;
        const float v = __uint_as_float(o[r]);
        check += v * 0.f + l[r] * 0.f;
        if (partial) {
            const bool none = m[r] == -INFINITY && l[r] == 0.f;
            float* rec = u.part + (int64_t)(it.rec + r) * (d + 4);
            rec[col] = none ? 0.f : v / l[r];
            if (col == 0) rec[d] = none ? -INFINITY : m[r] + log2f(l[r]);
        } else {
            p.O[(int64_t)out * d + col] = __float2bfloat16_rn(v * (gm / l[r]));
        }
    }
    if (!(check == 0.f)) u.odd[u.parts + blockIdx.x] = 1;
    return true;
}

// Copies rows of 64 kH elements (of which d exist, the others zeros) to a 128-byte
// swizzled tile, 16 bytes a lane, whole rows of adjacent lanes.  at: the rows'
// indexes in shared memory, -1 for a row of zeros.
template <int kH, int kUnroll>
__device__ __forceinline__ void copy_rows(uint32_t tile, const bf16* base, int64_t stride, const int32_t* at, int rows, int d) {
    constexpr int kPer = 4 / kH;  // rows a copy
    const int lane = threadIdx.x & 31, sub = lane / (8 * kH), c = lane % (8 * kH);
    const uint32_t dst = tile + (c >> 3) * kPart + sub * 128;
    const bool in = kH == 2 || c * 8 < d;
    const bf16* src = base + c * 8;
#pragma unroll kUnroll
    for (int r = 0; r < rows; r += kPer) {
        const int from = at[r + sub];
        const bool on = from >= 0 && in;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (r >> 3) * kH * kPart + (r & 7) * 128 + (((c & 7) ^ ((r + sub) & 7)) << 4)),
                     "l"(on ? src + from * stride : base), "r"(on ? 16 : 0)
                     : "memory");
    }
}

// kGather: small pages, fetched row by row.
template <int kH, bool kGather>
__global__ void __launch_bounds__(Split<kGather>::kThreads, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                const __grid_constant__ ChunkGeom u, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    using S = Smem<kH>;
    S& sm = *smem_align1024<S>(smem_raw);
    constexpr int kBars = bar_total<kH>();
    constexpr uint32_t kTileBytes = S::kTile;
    constexpr int kStages = S::kStages;
    const int d = kH == 2 ? 128 : p.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    static_assert(kBars <= 96, "one barrier per thread of warps 1 to 3");
    if (warp >= 1 && warp <= 3) {
        if (tid - 32 < kBars) mbar_init(&sm.item_full[0] + (tid - 32), bar_count<kH, kGather>(tid - 32));
        fence_barrier_init();
    }
    if (tid == 96) sm.abort_flag = 0;
    if (warp == 4 && lane < 16) {
        sm.zero[lane] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // Launched as a programmatic dependent of the kernel before it: the set-up
    // above overlaps its tail; nothing it writes is read before this wait.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Blocks of the merge may take their places as this kernel's leave.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 96) chunk_clear(u);
    tc_fence_before();
    chunk_split<Split<kGather>::kThreads>(u, sm.split, blockIdx.x);  // with block barriers
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // The kinds of units this CTA has, in the order in which it runs them: every
    // other CTA begins with the few-row ones, whose K/V stream from HBM while the
    // others keep the tensor cores busy.
    const bool has_many = chunk_has(u, sm.split, 0), has_few = chunk_has(u, sm.split, 1);
    if (!has_many && !has_few) {
        if (warp == 0) tmem_dealloc(tmem, kTmemCols);
        return;
    }
    const int phases = has_many && has_few ? 2 : 1;
    const bool few_first = has_few && (!has_many || (blockIdx.x & 1));

    if (kGather && warp == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<kGather>::kRegsCtl));
    } else if (kGather ? warp >= 12 : warp == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<kGather>::kRegsCtl));
        // ------------------------------------------------------------ K/V tiles
        // (gathered: a quarter of the rows a warp; one warp has so few 16-byte copies in
        // flight that 64 decodes ran at 1.3 TB/s)
        const int quarter = kGather ? warp - 12 : 0;
        const int shift = u.page_shift;
        const int box_rows = shift >= 7 ? kBN : 1 << shift;
        const int boxes = kBN / box_rows;  // per tile
        Ring<kStages> ring(few_first);
        int issued = 0;       // steps of this kind
        bool k_pending = false, turned = false;
        bool ok = true;
        if (!kGather && lane == 0) {
            tma_prefetch_desc(&mapK);
            tma_prefetch_desc(&mapV);
        }
#pragma unroll 1
        for (int ui = 0, ends = 0; ok && !aborted(sm); ++ui) {
            const int slot = ui % kItems;
            if (!warp_wait(sm, &sm.item_full[slot], (ui / kItems) & 1, 1)) break;
            if (!sm.has[slot]) {
                warp_arrive(&sm.item_free[slot]);
                if (++ends == phases) break;
                ring.turn();
                issued = 0;
                turned = true;
                continue;
            }
            const ChunkItem it = sm.item[slot];
#pragma unroll 1
            for (int s = it.s0; s < it.s1; ++s, ++issued, ring.next()) {
                const int b = ring.bar(), x0 = s * kBN;
                const uint32_t par = ring.phase ^ 1;
                int page = 0, in_page = 0;
                if constexpr (kGather) {
                    const int key = it.key(x0 + quarter * 32 + lane);
                    const bool on = key < it.hi && (key >= it.lo || key < u.sinks);
                    __syncwarp();
                    sm.kv_row[quarter][lane] = on ? (int)chunk_cache_row(u, it.b, key) : -1;
                    __syncwarp();
                } else if (lane < boxes) {
                    const int key = it.key(x0 + lane * box_rows);
                    const bool on = key < it.hi && (key + box_rows > it.lo || key < u.sinks);
                    page = u.num_pages;  // outside the pool: zeros
                    in_page = key & ((1 << shift) - 1);
                    if (on) page = (int)(chunk_cache_row(u, it.b, key) >> shift);
                }
                auto load = [&](const CUtensorMap* map, const bf16* pages, uint64_t* bar, uint8_t* dst) {
                    if constexpr (kGather) {
                        copy_rows<kH, 4>(smem_u32(dst) + quarter * 4 * kH * kPart, pages + (int64_t)it.q * d, (int64_t)u.g * d,
                                         sm.kv_row[quarter], kBN / 4, d);
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
                    } else {
                        if (lane == 0) mbar_arrive_expect_tx(bar, kTileBytes);
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_5d(map, bar, dst + lane * (box_rows >> 3) * kH * kPart, 0, 0, 0, it.q,
                                        (page << (shift - 3)) + (in_page >> 3));
                    }
                };
                // the second kind's stages lie in the first's memory
                if (turned && !warp_wait(sm, &sm.kind_done, 0, 4)) { ok = false; break; }
                if (!warp_wait(sm, &sm.kv_empty_k[b], par, 2)) { ok = false; break; }
                load(&mapK, p.K, &sm.kv_full_k[b], sm.k(ring.few, ring.st));
                k_pending = true;
                if (turned && !warp_wait(sm, &sm.kind_done_v, 0, 5)) { ok = false; break; }
                if (!warp_wait(sm, &sm.kv_empty_v[b], par, 3)) { ok = false; break; }
                load(&mapV, p.V, &sm.kv_full_v[b], sm.v(ring.st));
                k_pending = false;
            }
            warp_arrive(&sm.item_free[slot]);
        }
        // Drain: every issued load lands before the CTA may exit.
        if (k_pending) bar_wait(&sm.kv_full_k[ring.bar()], ring.phase);
#pragma unroll 1
        for (int back = min(issued, ring.size()); back > 0; --back) {
            ring.prev();
            bar_wait(&sm.kv_full_k[ring.bar()], ring.phase);
            bar_wait(&sm.kv_full_v[ring.bar()], ring.phase);
        }
    } else if (warp == 1) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<kGather>::kRegsCtl));
        // ------------------------------------------------------------ MMA issuer: S
        if (lane == 0) {
            const uint32_t dhi = smem_desc_hi(kH * kPart, kSwizzle128B);
            const uint32_t q_lo0 = smem_desc_lo(smem_u32(sm.q(0)), 16), q_lo1 = smem_desc_lo(smem_u32(sm.q(1)), 16);
            const uint32_t qf_lo = smem_desc_lo(smem_u32(sm.qf[0]), 16);
            Ring<kStages> ring(few_first);
            uint32_t s_cnt = 0, st_cnt[kQT] = {0, 0};
            bool ok = true;
            // the S buffer is free: its last reader of either form is done
            auto s_buffer = [&]() { return s_cnt == 0 || bar_wait(&sm.s_free, (s_cnt - 1) & 1); };
            auto st_buffer = [&](int t) { return st_cnt[t] == 0 || bar_wait(&sm.st_free[t], (st_cnt[t] - 1) & 1); };
            bool few = few_first;
            uint32_t q_use[kQT] = {0, 0}, qm_use[kQT] = {0, 0}, few_it = 0;  // fills of the Q buffers so far; few-row items
    #pragma unroll 1
        for (int ui = 0, ends = 0; ok && !aborted(sm); ++ui) {
                const int slot = ui % kItems;
                if (!bar_wait(&sm.item_full[slot], (ui / kItems) & 1)) { fail(sm, 10); break; }
                if (!sm.has[slot]) {
                    mbar_arrive(&sm.item_free[slot]);
                    if (++ends == phases) break;
                    umma_commit(&sm.kind_done);  // the first kind's S have read their Q and K
                    few = !few;
                    ring.turn();
                    continue;
                }
                const int n = sm.item[slot].s1 - sm.item[slot].s0;
                const int n0 = tile_steps(u, sm.item[slot], 0, few), n1 = tile_steps(u, sm.item[slot], 1, few);
                const int tiles = sm.item[slot].nt > u.W ? 2 : 1;
                mbar_arrive(&sm.item_free[slot]);
                // Q: few rows, the buffers in turn, filled by warp 2; many, one per tile,
                // filled by the tile's softmax warps
                const int qb = few ? few_it++ & 1 : 0;
                const uint32_t q_lo = qf_lo + qb * (sizeof(sm.qf[0]) >> 4);
                for (int t = 0; t < kQT && ok; ++t) {
                    if (few ? t != qb : (t ? tiles < 2 || n1 == 0 : n0 == 0)) continue;
                    if (few) {
                        ok = bar_wait(&sm.q_full[t], (t ? q_use[1] : q_use[0]) & 1);
                        if (t) ++q_use[1]; else ++q_use[0];
                    } else {
                        ok = bar_wait(&sm.qm_full[t], (t ? qm_use[1] : qm_use[0]) & 1);
                        if (t) ++qm_use[1]; else ++qm_use[0];
                    }
                }
                if (!ok) { fail(sm, 11); break; }
                if (few ? !s_buffer() : !(st_buffer(0) && st_buffer(1))) { fail(sm, 14); break; }
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i, ring.next()) {
                    const uint32_t k_lo = smem_desc_lo(smem_u32(sm.k(few, ring.st)), 16);
                    if (!bar_wait(&sm.kv_full_k[ring.bar()], ring.phase)) { fail(sm, 12); ok = false; break; }
                    if (kGather) fence_proxy_async_smem();  // rows written by plain copies
                    if (few) {
                        const int t = i & 1;
                        if (!st_buffer(t)) { fail(sm, 15); ok = false; break; }
                        tc_fence_after();
                        issue_st<kH>(tmem, dhi, t, q_lo, k_lo);
                        umma_commit(&sm.s_full[t]);
                        if (t) ++st_cnt[1]; else ++st_cnt[0];
                    }
#pragma unroll 1
                    for (int t = 0; t < kQT && !few; ++t) {
                        if (i >= (t ? n1 : n0)) continue;
                        if (!s_buffer()) { fail(sm, 13); ok = false; break; }
                        tc_fence_after();
                        issue_s<kH>(tmem, dhi, t ? q_lo1 : q_lo0, k_lo);
                        umma_commit(&sm.s_full[t]);
                        ++s_cnt;
                    }
                    if (!ok) break;
                    umma_commit(&sm.kv_empty_k[ring.bar()]);
                }
                if (!ok) break;
                if (few) umma_commit(&sm.q_empty[qb]);
            }
            umma_commit(&sm.mma_drain);  // all issued MMAs complete before TMEM is released
            bar_wait(&sm.mma_drain, 0);
        }
    } else if (warp == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<kGather>::kRegsCtl));
        // ------------------------------------------------------------ items, row tables, Q
        // this lane's rows 4 lane .. 4 lane + 3 of a tile: token within the tile
        // (negative: none), selection
        int tok[4], sel[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = lane * 4 + e;
            const int token = r * u.inv_k >> 16;
            tok[e] = r < u.W * u.k ? token : INT_MIN / 2;
            sel[e] = r - token * u.k;
        }
        uint32_t ui = 0, few_it = 0;
        bool ok = true;
#pragma unroll 1
        for (int phase = 0; phase < phases && ok; ++phase) {
            const bool few = (phase == 0) == few_first;
            ChunkWalk walk(u, sm.split, few, blockIdx.x);
            if (lane == 0) walk.leave(u, blockIdx.x);
#pragma unroll 1
            for (; !aborted(sm); ++ui) {
                const int slot = ui % kItems;
                if (!warp_wait(sm, &sm.item_free[slot], ((ui / kItems) & 1) ^ 1, 20)) { ok = false; break; }
                ChunkItem it;
                const bool has = walk.next(u, it);  // the same in every lane
                if (!has) {  // every barrier of the ring sees every entry
                    if (lane == 0) {
                        sm.has[slot] = 0;
                        mbar_arrive(&sm.item_full[slot]);
                        mbar_arrive(&sm.rows_full[slot]);
                    }
                    ++ui;
                    break;
                }
                int row[kQT][4];  // the lane's rows of Q
#pragma unroll
                for (int t = 0; t < kQT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int off = tok[e] + t * u.W;
                        row[t][e] = off >= 0 && off < it.nt ? u.idx[((int64_t)(it.t0 + off) * u.g + it.q) * u.k + sel[e]] : -1;
                    }
                if (lane == 0) {
                    sm.has[slot] = 1;
                    sm.item[slot] = it;
                    mbar_arrive(&sm.item_full[slot]);
                }
                __syncwarp();
#pragma unroll
                for (int t = 0; t < kQT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int off = tok[e] + t * u.W, j = row[t][e];
                        const bool there = off >= 0 && off < it.nt, good = there && j >= it.q * u.hpg && j < (it.q + 1) * u.hpg;
                        if (there && !good) report_error(u.status, GQE_ERR_INVALID_ARGUMENT, kWhereChunk, (uint32_t)(it.t0 + off));
                        sm.row[slot][t][lane * 4 + e] = good ? (it.t0 + off) * u.h + j : -1;
                    }
                warp_arrive(&sm.rows_full[slot]);
                if (!few) continue;  // the softmax warps copy the tiles
                const int buf = few_it & 1;
                if (!warp_wait(sm, &sm.q_empty[buf], ((few_it >> 1) & 1) ^ 1, 21)) { ok = false; break; }
                ++few_it;
                copy_rows<kH, 4>(smem_u32(sm.qf[buf]), p.Q, d, sm.row[slot][0], kFew, d);
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();  // from the generic to the tensor cores' view
                warp_arrive(&sm.q_full[buf]);
            }
        }
    } else if (warp == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<kGather>::kRegsCtl));
        // ------------------------------------------------------------ MMA issuer: O += P V
        const uint32_t dhi = smem_desc_hi(kH * kPart, kSwizzle128B);
        const uint32_t p_hi = smem_desc_hi(kPart, kSwizzle128B);
        const uint32_t v_lo0 = smem_desc_lo(smem_u32(sm.v(0)), kH == 2 ? kPart : 0);
        const uint32_t p_lo0 = smem_desc_lo(smem_u32(sm.p[0]), 16), p_lo1 = smem_desc_lo(smem_u32(sm.p[1]), 16);
        const int page = 1 << u.page_shift;
        Ring<kStages> ring(few_first);
        uint32_t c[kQT] = {0, 0}, o_cnt[kQT] = {0, 0};
        bool ok = true;
        bool few = few_first;
#pragma unroll 1
        for (int ui = 0, ends = 0; ok && !aborted(sm); ++ui) {
            const int slot = ui % kItems;
            if (!warp_wait(sm, &sm.item_full[slot], (ui / kItems) & 1, 30)) break;
            if (!sm.has[slot]) {
                warp_arrive(&sm.item_free[slot]);
                if (++ends == phases) break;
                if (lane == 0) umma_commit(&sm.kind_done_v);  // its O have read their V
                __syncwarp();
                few = !few;
                ring.turn();
                continue;
            }
            const ChunkItem it = sm.item[slot];
            warp_arrive(&sm.item_free[slot]);
            const int n = it.s1 - it.s0, n0 = tile_steps(u, it, 0, few), n1 = tile_steps(u, it, 1, few);
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i, ring.next()) {
                const int st = ring.st;
                if (!warp_wait(sm, &sm.kv_full_v[ring.bar()], ring.phase, 31)) { ok = false; break; }
                if (kGather) fence_proxy_async_smem();
                // Rows of loaded pages that no row of the unit sees: past the last
                // token, and between the first `sinks` keys and the window.
                const int x0 = (it.s0 + i) * kBN, x1 = x0 + kBN;  // of the key list
                if (x1 > it.hi - it.skip || (u.window && x0 < it.lo - it.skip)) {
                    uint8_t* v = sm.v(st);
                    auto zero = [&](int a, int b) {
                        a = max(a, x0);
                        b = min(b, x1);
#pragma unroll 1
                        for (int x = lane; x < (b - a) * 8 * kH; x += 32) {
                            const int r = a - x0 + x / (8 * kH);
                            *reinterpret_cast<uint4*>(v + ((r >> 3) * kH + (kH == 2 && (x & 8) ? 1 : 0)) * kPart + (r & 7) * 128 +
                                                      (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    };
                    zero(it.hi - it.skip, ((it.hi + page - 1) & ~(page - 1)) - it.skip);
                    if (u.window) {
                        zero(u.sinks, it.head);
                        zero(max(it.head + it.skip, u.sinks) - it.skip, it.lo - it.skip);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll 1
                for (int t = 0; t < kQT; ++t) {
                    const int j = few ? i >> 1 : i;  // the group's own step
                    if (few ? (i & 1) != t : i >= (t ? n1 : n0)) continue;
                    if (!warp_wait(sm, &sm.p_full[t], c[t] & 1, 32)) { ok = false; break; }
                    if (j == 0 && !warp_wait(sm, &sm.o_empty[t], (o_cnt[t] & 1) ^ 1, 33)) { ok = false; break; }
                    if (lane == 0) {
                        tc_fence_after();
                        const uint32_t v_lo = v_lo0 + st * (kTileBytes >> 4);
                        if (few)
                            issue_pvt<kH>(tmem, dhi, p_hi, t, v_lo, t ? p_lo1 : p_lo0, j == 0);
                        else
                            issue_pv<kH>(tmem, dhi, t, v_lo, j == 0);
                        umma_commit(&sm.p_empty[t]);
                        if (j == (t ? n1 : n0) - 1) umma_commit(&sm.o_full[t]);
                    }
                    ++c[t];
                    if (j == 0) ++o_cnt[t];
                }
                if (!ok) break;
                if (lane == 0) umma_commit(&sm.kv_empty_v[ring.bar()]);
                __syncwarp();
            }
        }
        if (lane == 0) {
            umma_commit(&sm.mma_drain2);
            bar_wait(&sm.mma_drain2, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Split<kGather>::kRegsSoftmax));
        // ------------------------------------------------------------ softmax + epilogue (tile t)
        const int t = (warp - 4) >> 2;     // query tile of this warpgroup
        const int wq = warp & 3;           // TMEM lane quarter of this warp
        const int r = wq * 32 + lane;      // query row owned by this thread
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + kColS;
        const uint32_t p_addr = tmem + lane_off + kColP + 64 * t;
        const uint32_t o_addr = tmem + lane_off + kColO + t * 128;
        const int off = t * u.W + (r * u.inv_k >> 16);  // this row's token within the unit, and its selection
        const int sel = r - (r * u.inv_k >> 16) * u.k;
        const bool in_tile = r < u.W * u.k;
        const uint64_t C2 = pk2(p.scale_log2, p.scale_log2);
        uint32_t ctile = 0, o_it = 0, votes = 0, swaps = 0;
        uint32_t ui = 0;
        // The next item of the kind, or null at its end (or after a failure).
        auto take = [&]() -> const ChunkItem* {
            if (aborted(sm) || !warp_wait(sm, &sm.item_full[ui % kItems], (ui / kItems) & 1, 40)) return nullptr;
            if (sm.has[ui % kItems]) return &sm.item[ui % kItems];
            warp_arrive(&sm.item_free[ui++ % kItems]);
            return nullptr;
        };
        auto done = [&]() { warp_arrive(&sm.item_free[ui++ % kItems]); };
        // The unselected output slots of the tile's tokens, by the part that holds
        // the unit's first step: a bulk copy of a row of zeros each, the k threads of
        // a token taking its slots in turn.
        auto zero_fill = [&](const ChunkItem& it, int toks) {
            if (it.s0 != 0 || r >= toks * u.k) return;  // k of hpg heads or all, of which some may be none
            const int32_t* rows = sm.row[ui % kItems][t] + (r - sel);
            const int first = (it.t0 + off) * u.h + it.q * u.hpg;
            bf16* o = p.O + (int64_t)first * d;
            int turn = 0;
#pragma unroll 1
            for (int a0 = 0; a0 < u.hpg; a0 += 32) {
                uint32_t free = low_bits(u.hpg - a0);
#pragma unroll 1
                for (int a = 0; a < u.k; ++a) {
                    const int j = rows[a] - first - a0;
                    if (j >= 0 && j < 32) free &= ~(1u << j);
                }
#pragma unroll 1
                for (; free; free &= free - 1) {
                    if (turn == sel)
                        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                         o + (int64_t)(a0 + __ffs(free) - 1) * d),
                                     "r"(smem_u32(sm.zero)), "r"(d * 2)
                                     : "memory");
                    if (++turn == u.k) turn = 0;
                }
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int phase = 0; phase < phases; ++phase) {
        if ((phase == 0) == few_first) {
            // x is free for group 1's first hand-over once group 0 has no stage in it
            if (t == 0) warp_arrive(&sm.x_free);
            while (const ChunkItem* next = take()) {
                const ChunkItem it = *next;
                const int slot = ui % kItems;
                if (!warp_wait(sm, &sm.rows_full[slot], (ui / kItems) & 1, 41)) break;
                if (t == 0) zero_fill(it, it.nt);
                if (!(it.nt * u.k <= 4 ? few_item<4, kH>(u, p, sm, it, slot, t, tmem, ctile, o_it, votes, swaps)
                                       : few_item<16, kH>(u, p, sm, it, slot, t, tmem, ctile, o_it, votes, swaps)))
                    break;
                done();
            }
            if (phase + 1 == phases) continue;
            // The few-row items' products have read the stage that lies in the Q tiles, and
            // group 0 has read what group 1 handed over, where the epilogue's stages lie.
            if (!aborted(sm)) warp_wait(sm, t ? &sm.kind_done_v : &sm.kind_done, 0, 53);
            if (!aborted(sm)) warp_wait(sm, &sm.x_free, swaps & 1, 52);
            continue;
        }
        // This warp's rows of an item's Q tile, in flight until q_ready.
        auto load_q = [&](int slot) {
            copy_rows<kH, 4>(smem_u32(sm.q(t)) + wq * 4 * kH * kPart, p.Q, d, sm.row[slot][t] + wq * 32, 32, d);
        };
        auto q_ready = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();  // from the generic to the tensor cores' view
            warp_arrive(&sm.qm_full[t]);
        };
        bool loaded = false;  // the next item's Q tile is on its way already
        while (const ChunkItem* next = take()) {
            const ChunkItem& it = *next;  // read again where it is used: registers are short in the loop
            const int slot = ui % kItems;
            const int n = tile_steps(u, it, t, false);
            const int toks = min(it.nt - t * u.W, u.W);  // of this tile; 0 or less: none
            // Every item's rows_full phase is waited for in turn, as a later one may
            // complete before a waiter of the same parity looks.
            if (!warp_wait(sm, &sm.rows_full[slot], (ui / kItems) & 1, 41)) break;
            if (toks <= 0) {
                done();
                continue;
            }
            // A tile without steps in this part (only a CTA's first unit has such) has no Q
            // either: nobody would wait before the next unit's came.
            if (n > 0) {
                if (!loaded) load_q(slot);
                q_ready();
            }
            loaded = false;
            const bool partial = it.rec >= 0;
            const bool mine = in_tile && off < it.nt;
            const int token = it.t0 + off;
            const float gate = mine ? u.gate[((int64_t)token * u.g + it.q) * u.k + sel] : 0.f;
            zero_fill(it, toks);
            const int out_row = mine ? sm.row[slot][t][r] : -1;
            const bool live = wq * 32 < toks * u.k;  // some row of this warp is a query row
            // Keys this row sees: [low, pos] and those below u.sinks.  A padding row
            // sees all (its result is dropped).
            const int pos = mine ? it.p0 + off : INT_MAX - 1;
            const int low = mine ? pos - u.window + 1 : 0;
            const int pos_first = it.p0 + t * u.W, low_last = u.window ? pos_first + toks - u.window : INT_MIN;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            const int x_first = it.s0 * kBN, skip = it.skip;
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++ctile) {
                if (!warp_wait(sm, &sm.s_full[t], ctile & 1, 42)) { ok = false; break; }
                if (!live) {  // no query row: hand both buffers on, P no sooner than the slot is free
                    if (lane == 0) mbar_arrive(&sm.s_free);
                    if (ctile > 0 && !warp_wait(sm, &sm.p_empty[t], (ctile - 1) & 1, 45)) { ok = false; break; }
                    if (lane == 0) mbar_arrive(&sm.p_full[t]);
                    continue;
                }
                tc_fence_after();
                uint32_t s[4][32];
                const int x0 = x_first + i * kBN, kv0 = x0 + skip;  // of the key list; its key behind the first ones
                const bool need_mask = kv0 + kBN - 1 > pos_first || kv0 < low_last;
                uint64_t sum2[4];
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) tmem_ld32(s_addr + cb * 32, s[cb]);
                ld_wait_bind(s[0]);
                ld_bind(s[1]);
                ld_bind(s[2]);
                ld_bind(s[3]);
                tc_fence_before();
                warp_arrive(&sm.s_free);
                // Hide what a row does not see: per 32 keys a bit each, applied where some
                // of the warp's rows need it.
                if (need_mask) {
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        const int k0 = kv0 + cb * 32, head = it.head - x0 - cb * 32;
                        uint32_t see = low_bits(pos + 1 - k0);
                        if (u.window) {
                            see &= ~low_bits(low - k0) | low_bits(u.sinks - k0);
                            if (head > 0) see = (see & ~low_bits(head)) | low_bits(min(head, u.sinks - x0 - cb * 32));
                        }
                        if (__any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see & (1u << e))) s[cb][e] = __float_as_uint(-INFINITY);
                        }
                    }
                }
                // The exponentials are taken against the running max while the step's row
                // max is formed alongside: unless some row of the warp grew its max by
                // more than the threshold, P is final; else O_t and the row's sum are
                // rescaled and the exponentials taken once more.  An item's first step
                // forms the max beforehand.
                if (i == 0) {
                    float mq[4];
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        float a0 = __uint_as_float(s[cb][0]);
#pragma unroll
                        for (int e = 1; e < 31; e += 2)
                            a0 = fmax3(a0, __uint_as_float(s[cb][e]), __uint_as_float(s[cb][e + 1]));
                        mq[cb] = fmaxf(a0, __uint_as_float(s[cb][31]));
                    }
                    m = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * p.scale_log2;
                }
                bool slot_ok = true, slot_free = false;
#pragma unroll 1
                while (true) {
                    const float ref = m == -INFINITY ? 0.f : m;  // no key seen so far: weights of 0
                    const uint64_t NM2 = pk2(-ref, -ref);
                    float mq[4];
                    uint32_t pk[2][16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum2[e] = 0;
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        float a0 = __uint_as_float(s[cb][0]);
#pragma unroll
                        for (int e = 1; e < 31; e += 2)
                            a0 = fmax3(a0, __uint_as_float(s[cb][e]), __uint_as_float(s[cb][e + 1]));
                        mq[cb] = fmaxf(a0, __uint_as_float(s[cb][31]));
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            up2(ffma2(pk2(__uint_as_float(s[cb][2 * e]), __uint_as_float(s[cb][2 * e + 1])), C2, NM2), x0, x1);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            sum2[e & 3] = fadd2(sum2[e & 3], pk2(p0, p1));
                            pk[cb & 1][e] = pack_bf16x2(p0, p1);
                        }
                        // The first two chunks wait in registers for the tile's P slot: free
                        // once its previous P.V has completed (and with it O_t so far).
                        if (cb == 1) {
                            if (!slot_free) {
                                slot_free = true;
                                if (ctile > 0 && !__all_sync(0xffffffffu, bar_wait(&sm.p_empty[t], (ctile - 1) & 1))) slot_ok = false;
                                tc_fence_after();
                            }
                            tmem_st16(p_addr, pk[0]);
                            tmem_st16(p_addr + 16, pk[1]);
                        } else if (cb > 1) {
                            tmem_st16(p_addr + cb * 16, pk[cb & 1]);
                        }
                    }
                    const float mx = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * p.scale_log2;
                    // A row whose max was still -inf has weights taken against 0: right only
                    // if it still sees nothing.
                    const bool grown = m == -INFINITY ? mx != -INFINITY : mx > m + kRescaleThreshold;
                    if (__all_sync(0xffffffffu, !grown)) break;
                    const float alpha = grown && m != -INFINITY ? fast_exp2(m - mx) : 1.0f;  // -inf: O_t's row is 0
                    if (grown) m = mx;
                    l *= alpha;
                    if (i > 0) {
#pragma unroll 1
                        for (int cb = 0; cb < 2 * kH; ++cb) {
                            uint32_t o[32];
                            tmem_ld32(o_addr + cb * 32, o);
                            ld_wait_bind(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(o_addr + cb * 32, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                            tmem_st16(o_addr + cb * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
                        }
                    }
                }
                float sa, sb;
                up2(fadd2(fadd2(sum2[0], sum2[1]), fadd2(sum2[2], sum2[3])), sa, sb);
                l += sa + sb;
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&sm.p_full[t]);
                if (!slot_ok) {
                    if (lane == 0) fail(sm, 43);
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
            // The tile's last S is done: its Q buffer takes the next item's rows while
            // this one's epilogue runs.
            {
                const int ns = (ui + 1) % kItems;
                if (!warp_wait(sm, &sm.item_full[ns], ((ui + 1) / kItems) & 1, 54)) break;
                if (sm.has[ns] && sm.item[ns].nt > t * u.W) {
                    if (!warp_wait(sm, &sm.rows_full[ns], ((ui + 1) / kItems) & 1, 55)) break;
                    load_q(ns);
                    loaded = true;
                }
            }
            // Epilogue: O_t / l, gated, as the bf16 row of O, or the row's partial
            // record (o, log2-sum-exp); none of this part's keys seen: -inf.  A row per
            // thread would store 16 bytes to each of 32 lines at a time, so 64 bytes of
            // each row at a time go through shared memory and out as whole sectors.
            const int rec_row = it.rec + t * u.W * u.k + wq * 32;
            if (n == 0) {
                if (partial && mine) u.part[(int64_t)(rec_row + lane) * (d + 4) + d] = -INFINITY;
                done();
                continue;
            }
            if (!warp_wait(sm, &sm.o_full[t], o_it & 1, 44)) break;
            ++o_it;
            if (!live) {
                warp_arrive(&sm.o_empty[t]);
                done();
                continue;
            }
            tc_fence_after();
            uint32_t o[2 * kH][32];
#pragma unroll
            for (int cb = 0; cb < 2 * kH; ++cb) tmem_ld32(o_addr + cb * 32, o[cb]);
            ld_wait_bind(o[0]);
#pragma unroll
            for (int cb = 1; cb < 2 * kH; ++cb) ld_bind(o[cb]);
            tc_fence_before();
            warp_arrive(&sm.o_empty[t]);
            const bool none = m == -INFINITY && l == 0.f;
            const float f = partial ? (none ? 0.f : 1.f / l) : gate / l;
            float check[4] = {l * 0.f, 0.f, 0.f, 0.f};  // stays 0, or NaN when a value is not finite
#pragma unroll
            for (int cb = 0; cb < 2 * kH; ++cb)
#pragma unroll
                for (int e = 0; e < 32; ++e) check[e & 3] = fmaf(__uint_as_float(o[cb][e]), 0.f, check[e & 3]);
            if (out_row >= 0) {
                if (!((check[0] + check[1]) + (check[2] + check[3]) == 0.f)) u.odd[blockIdx.x] = 1;
                if (partial) u.part[(int64_t)(rec_row + lane) * (d + 4) + d] = none ? -INFINITY : m + log2f(l);
            }
            uint4* stage = sm.stage(t, wq);
            // This lane's 16 bytes of four of the warp's rows: 8 e + lane / 4.
            uint4* to[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 8 * e + (lane >> 2), there = __shfl_sync(0xffffffffu, out_row, row);
                to[e] = there < 0 ? nullptr
                        : partial ? reinterpret_cast<uint4*>(u.part + (int64_t)(rec_row + row) * (d + 4)) + (lane & 3)
                                  : reinterpret_cast<uint4*>(p.O + (int64_t)there * d) + (lane & 3);
            }
            // Writes 64 bytes (piece cb) of every row of the warp.
            auto flush = [&](const uint4 (&v)[4], int cb) {
#pragma unroll
                for (int c = 0; c < 4; ++c) stage[lane * 4 + (c ^ ((lane >> 1) & 3))] = v[c];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 8 * e + (lane >> 2);
                    if (to[e]) to[e][cb * 4] = stage[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
                }
                __syncwarp();
            };
            if (partial) {
#pragma unroll
                for (int cb = 0; cb < 4 * kH; ++cb) {
                    if (kH == 1 && cb * 16 >= d) break;
                    uint4 v[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t* w = &o[cb >> 1][(cb & 1) * 16 + 4 * c];
                        v[c] = make_uint4(__float_as_uint(__uint_as_float(w[0]) * f), __float_as_uint(__uint_as_float(w[1]) * f),
                                          __float_as_uint(__uint_as_float(w[2]) * f), __float_as_uint(__uint_as_float(w[3]) * f));
                    }
                    flush(v, cb);
                }
            } else {
#pragma unroll
                for (int cb = 0; cb < 2 * kH; ++cb) {
                    if (kH == 1 && cb * 32 >= d) break;
                    uint4 v[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t* w = &o[cb][8 * c];
                        v[c].x = pack_bf16x2(__uint_as_float(w[0]) * f, __uint_as_float(w[1]) * f);
                        v[c].y = pack_bf16x2(__uint_as_float(w[2]) * f, __uint_as_float(w[3]) * f);
                        v[c].z = pack_bf16x2(__uint_as_float(w[4]) * f, __uint_as_float(w[5]) * f);
                        v[c].w = pack_bf16x2(__uint_as_float(w[6]) * f, __uint_as_float(w[7]) * f);
                    }
                    flush(v, cb);
                }
            }
            done();
        }
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the zero rows are out
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (tid == 0 && sm.abort_flag != 0)
        report_error(u.status, GQE_ERR_DEVICE_TIMEOUT, kWhereChunkTc, (uint32_t)sm.abort_flag);
}

}  // namespace

// A unit's fixed cost is set to five steps of many rows and one of few, and the smallest
// part to two steps.  With 2, 4 or 8 steps for many rows, a step of 28 decodes and 4 chunks
// takes 139.7, 139.2 and 140.2 us for 139.4 and prompts under a window 203 to 204 each; with
// none or three for few, 64 decodes take 391 and 385 us for 389, but 3 decodes 19.0 and 18.7
// for 17.9.  Parts of one step or four: 3 decodes 17.2 and 19.4 us, and 64-element heads under
// a window 22.6 each for 22.2.
ChunkTiling chunk_tc_tiling() { return {kBM, kQT, kFew, kBN, 5 * kBN, kBN, 2 * kBN, 1}; }

namespace {

// The setmaxnreg split draws on the registers of the launch: a property of the
// compiled kernels, checked once per process.
template <int kH, bool kGather>
bool registers_suffice() {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, chunk_tc_kernel<kH, kGather>) == cudaSuccess && f.numRegs >= Split<kGather>::kRegsLaunch;
}

template <int kH, bool kGather>
cudaError_t launch_typed(const ChunkGeom& u, const ChunkArgs& a, const CUtensorMap& mapK, const CUtensorMap& mapV) {
    static std::atomic<int> state{0};
    if (state.load(std::memory_order_acquire) == 0)
        state.store(registers_suffice<kH, kGather>() ? 1 : -1, std::memory_order_release);
    if (state.load(std::memory_order_acquire) != 1) return cudaErrorNotSupported;
    Params p;
    p.Q = (const bf16*)a.Q;
    p.O = (bf16*)a.O;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)a.s->d_h);
    p.K = (const bf16*)a.K_pages;
    p.V = (const bf16*)a.V_pages;
    p.d = a.s->d_h;
    const size_t smem = sizeof(Smem<kH>) + 1024;
    auto kern = chunk_tc_kernel<kH, kGather>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(u.parts);
    cfg.blockDim = dim3(Split<kGather>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, mapK, mapV, u, p);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkGeom& u, const ChunkArgs& a) {
    const gqe_shape& s = *a.s;
    const int page = 1 << a.page_shift;
    // A box per page of the TMA, or for smaller pages copies, row by row.  64 decodes of
    // 1000 to 8000 keys, pages of 8 rows: d_h = 128, 213 us by boxes and 315 by copies;
    // d_h = 64, whose boxes are half as large, 207 and 186.  16 rows: boxes, 189 and 165.
    const bool gather = page < (s.d_h == 128 ? 8 : 16);
    CUtensorMap mapK{}, mapV{};
    if (!gather) {
        const uint64_t row_bytes = (uint64_t)s.d_h * 2;
        const int parts = s.d_h == 128 ? 2 : 1;
        // 64 elements, 8 rows, parts, groups, 8-row groups of the pool
        const uint64_t dims[5] = {(uint64_t)(s.d_h / parts), 8, (uint64_t)parts, (uint64_t)s.g, (uint64_t)a.num_pages * page / 8};
        const uint64_t strides[4] = {s.g * row_bytes, 128, row_bytes, 8 * s.g * row_bytes};
        const uint32_t box[5] = {64, 8, (uint32_t)parts, 1, (uint32_t)(page < kBN ? page : kBN) / 8};
        if (!make_bf16_map(&mapK, a.K_pages, 5, dims, strides, box)) return cudaErrorInvalidValue;
        if (!make_bf16_map(&mapV, a.V_pages, 5, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (s.d_h == 128) return gather ? launch_typed<2, true>(u, a, mapK, mapV) : launch_typed<2, false>(u, a, mapK, mapV);
    return gather ? launch_typed<1, true>(u, a, mapK, mapV) : launch_typed<1, false>(u, a, mapK, mapV);
}

}  // namespace gqe
