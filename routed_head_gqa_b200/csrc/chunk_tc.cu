// chunk_tc.cu -- routed attention of ragged chunks of new tokens over a paged
// cache on the sm_100a tensor cores (bf16, d_h = 128), with an optional sliding
// window.  See chunk.cuh for the units, the schedule and the masks.
//
// A unit has up to two query tiles of 128 rows (W = floor(128 / k) tokens of k
// rows each) over one stream of 128-key K/V tiles; a decode has one tile of k
// rows, and only the warp that holds them works on its softmax.
//
// Roles (384 threads, one persistent CTA per SM):
//   warp 0      K/V tiles by TMA: one box per page (of at most 128 rows) and
//               64-column half, lane by lane; pages of fewer than 8 rows by
//               tile::gather4.  Pages that no row of the unit sees are loaded
//               from outside the pool, which the TMA fills with zeros.
//   warp 1      MMA issuer (one thread): S_t = Q_t K^T
//   warp 2      walks the part's items (a ring of 4), gathers the routed rows of Q
//   warp 3      MMA issuer (one thread): O_t += P_t V.  Before it, the whole warp
//               zeroes the tile's V rows that no row of the unit sees (past the
//               last token, outside the window): their weight is 0, but 0 times
//               what an unused row holds may be NaN.
//   warps 4-7   softmax, epilogue and zero fill of query tile 0, a row per thread
//   warps 8-11  the same for query tile 1
// TMEM: one S buffer [0,128) that the tiles take in turn, P_0 [128,192) and P_1
// [192,256) (bf16 pairs), O_0 [256,384), O_1 [384,512).  The softmax copies S to
// registers and hands the buffer back at once, so the next S runs under it.
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

constexpr int kD = 128, kBM = 128, kBN = 128, kQT = 2, kThreads = 384;
constexpr int kItems = 4;                  // items in flight between the walk and the other roles
constexpr uint32_t kHalf = 128 * 64 * 2;   // one [128][64] bf16 box, 16 KB
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: p <= 2^8 between rescales
constexpr uint32_t kWhereChunkTc = 11;     // status "where" id of this kernel
// Register split (setmaxnreg): 4 control warps at 88, 8 softmax warps at 208.
constexpr int kRegsLaunch = 168, kRegsCtl = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsCtl + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split exceeds the launch");

struct Smem {
    uint8_t q[kQT][kTileBytes];
    uint8_t k[2][kTileBytes];
    uint8_t v[2][kTileBytes];
    ChunkItem item[kItems];
    int32_t has[kItems];                 // 0: no more items
    int32_t row_j[kItems][kQT][kBM];     // head of each query row, -1: none
    ChunkSplit split;
    uint64_t item_full[kItems], item_free[kItems], rows_full[kItems];
    uint64_t kv_full_k[2], kv_full_v[2], kv_empty_k[2], kv_empty_v[2];
    uint64_t s_full[kQT], p_full[kQT], p_empty[kQT], o_full[kQT], o_empty[kQT];
    uint64_t s_free, q_full, q_empty, mma_drain, mma_drain2;
    uint32_t tmem_base;
    int32_t abort_flag;
};

struct Params {
    const bf16* Q;
    const bf16* K;
    const bf16* V;
    bf16* O;
    float scale_log2;
    int q_rows;   // rows of Q seen as [T * h, 128]
    int kv_rows;  // rows of K seen as [num_pages * page_size * g, 128] (gathered pages only)
};

__device__ __forceinline__ bool aborted(Smem& sm) { return *((volatile int32_t*)&sm.abort_flag) != 0; }
__device__ __forceinline__ void fail(Smem& sm, const ChunkGeom& u, uint32_t detail) {
    atomicExch(&sm.abort_flag, 1);
    report_error(u.status, GQE_ERR_DEVICE_TIMEOUT, kWhereChunkTc, detail);
}
// The whole warp waits; false (reported once) if the wait ran out for any lane.
__device__ __forceinline__ bool warp_wait(Smem& sm, const ChunkGeom& u, uint64_t* bar, uint32_t parity, uint32_t detail) {
    if (__all_sync(0xffffffffu, mbar_wait(bar, parity))) return true;
    if ((threadIdx.x & 31) == 0) fail(sm, u, detail);
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
// own last token (none when the unit has no token for the tile).
__device__ __forceinline__ int tile_steps(const ChunkGeom& u, const ChunkItem& it, int t) {
    if (it.nt <= t * u.W) return 0;
    const int hi = it.p0 + min(it.nt, (t + 1) * u.W);
    const int end = min(it.s1, it.sink_tiles + (hi + kBN - 1) / kBN - it.lo_tile);
    return max(0, end - it.s0);
}

// Bits 0 .. n-1 of a word (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// S_t = Q_t K(it)^T: eight K steps of 16 over 128-byte swizzled tiles; a step
// moves the descriptors' start address only.
__device__ __forceinline__ void issue_s(uint32_t tmem, uint32_t dhi, uint32_t q_lo, uint32_t k_lo) {
    constexpr uint32_t idesc = idesc_bf16_f32(kBM, kBN, false, false);
#pragma unroll
    for (int kk = 0; kk < kD / 16; ++kk) {
        const uint32_t off = (uint32_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
        umma_ss(tmem + kColS, smem_desc_join(q_lo + off, dhi), smem_desc_join(k_lo + off, dhi), idesc, kk > 0 ? 1u : 0u);
    }
}
// O_t += P_t V(it), P_t from TMEM, V as an MN-major operand.
__device__ __forceinline__ void issue_pv(uint32_t tmem, uint32_t dhi, int t, uint32_t v_lo, bool first) {
    constexpr uint32_t idesc = idesc_bf16_f32(kBM, kD, false, true);
#pragma unroll
    for (int kk = 0; kk < kBN / 16; ++kk)
        umma_ts(tmem + kColO + t * 128, tmem + kColP + 64 * t + kk * 8, smem_desc_join(v_lo + (uint32_t)((kk * 2048) >> 4), dhi),
                idesc, first && kk == 0 ? 0u : 1u);
}

// kGather: pages of fewer than 8 rows, fetched row by row.
template <bool kGather>
__global__ void __launch_bounds__(kThreads, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ ChunkGeom u, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *smem_align1024<Smem>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.kv_full_k[i], 1);
            mbar_init(&sm.kv_full_v[i], 1);
            mbar_init(&sm.kv_empty_k[i], 1);
            mbar_init(&sm.kv_empty_v[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.rows_full[i], 1);
            mbar_init(&sm.item_free[i], 11);  // warps 0, 1, 3 and the eight softmax warps
        }
        for (int t = 0; t < kQT; ++t) {
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.p_full[t], 4);   // one arrive per warp of the tile's warpgroup
            mbar_init(&sm.p_empty[t], 1);
            mbar_init(&sm.o_full[t], 1);
            mbar_init(&sm.o_empty[t], 4);
        }
        mbar_init(&sm.s_free, 4);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.mma_drain, 1);
        mbar_init(&sm.mma_drain2, 1);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // Launched as a programmatic dependent of the kernel before it: the set-up
    // above overlaps its tail; nothing it writes is read before this wait.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    chunk_split(u, sm.split, blockIdx.x, gridDim.x);  // with block barriers
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        // ------------------------------------------------------------ K/V tiles
        const int shift = u.page_shift;
        const int box_rows = shift >= 7 ? kBN : 1 << shift;
        const int boxes = kBN / box_rows;  // per tile and half
        uint32_t kv_it = 0;
        bool k_pending = false;
        bool ok = true;
        if (lane == 0) {
            tma_prefetch_desc(&mapK);
            tma_prefetch_desc(&mapV);
        }
        for (uint32_t ui = 0; ok && !aborted(sm); ++ui) {
            const int slot = ui % kItems;
            if (!warp_wait(sm, u, &sm.item_full[slot], (ui / kItems) & 1, 1)) break;
            if (!sm.has[slot]) break;
            const ChunkItem it = sm.item[slot];
            for (int s = it.s0; s < it.s1; ++s, ++kv_it) {
                const int st = kv_it & 1, kv0 = it.tile(s) * kBN;
                const uint32_t par = ((kv_it >> 1) & 1) ^ 1;
                int page = 0, in_page = 0, row[4];
                if constexpr (kGather) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = kv0 + lane * 4 + e;
                        const bool on = key < it.hi && (key >= it.lo || key < u.sinks);
                        row[e] = on ? (int)(chunk_cache_row(u, it.b, key) * u.g + it.q) : p.kv_rows;
                    }
                } else if (lane < 2 * boxes) {
                    const int key = kv0 + (lane >> 1) * box_rows;
                    const bool on = key < it.hi && (key + box_rows > it.lo || key < u.sinks);
                    page = u.num_pages;  // outside the pool: zeros
                    in_page = key & ((1 << shift) - 1);
                    if (on) page = (int)(chunk_cache_row(u, it.b, key) >> shift);
                }
                auto load = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* dst) {
                    if constexpr (kGather) {
                        tma_gather4_2d(map, bar, dst + lane * 512, 0, row[0], row[1], row[2], row[3]);
                        tma_gather4_2d(map, bar, dst + kHalf + lane * 512, 64, row[0], row[1], row[2], row[3]);
                    } else if (lane < 2 * boxes) {
                        const int half = lane & 1;
                        tma_load_4d(map, bar, dst + half * kHalf + (lane >> 1) * box_rows * 128, half * 64, it.q, in_page, page);
                    }
                };
                if (!warp_wait(sm, u, &sm.kv_empty_k[st], par, 2)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full_k[st], kTileBytes);
                __syncwarp();
                load(&mapK, &sm.kv_full_k[st], sm.k[st]);
                k_pending = true;
                if (!warp_wait(sm, u, &sm.kv_empty_v[st], par, 3)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full_v[st], kTileBytes);
                __syncwarp();
                load(&mapV, &sm.kv_full_v[st], sm.v[st]);
                k_pending = false;
            }
            warp_arrive(&sm.item_free[slot]);
        }
        // Drain: every issued load lands before the CTA may exit.
        if (k_pending) mbar_wait(&sm.kv_full_k[kv_it & 1], (kv_it >> 1) & 1);
        for (uint32_t back = 1; back <= 2 && back <= kv_it; ++back) {
            const uint32_t i = kv_it - back;
            mbar_wait(&sm.kv_full_k[i & 1], (i >> 1) & 1);
            mbar_wait(&sm.kv_full_v[i & 1], (i >> 1) & 1);
        }
    } else if (warp == 1) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        // ------------------------------------------------------------ MMA issuer: S
        if (lane == 0) {
            const uint32_t dhi = smem_desc_hi(1024, kSwizzle128B);
            const uint32_t q_lo0 = smem_desc_lo(smem_u32(sm.q[0]), 16), q_lo1 = smem_desc_lo(smem_u32(sm.q[1]), 16);
            const uint32_t k_lo0 = smem_desc_lo(smem_u32(sm.k[0]), 16), k_lo1 = smem_desc_lo(smem_u32(sm.k[1]), 16);
            uint32_t kv_it = 0, s_cnt = 0;
            bool ok = true;
            for (uint32_t ui = 0; ok && !aborted(sm); ++ui) {
                const int slot = ui % kItems;
                if (!mbar_wait(&sm.item_full[slot], (ui / kItems) & 1)) { fail(sm, u, 10); break; }
                if (!sm.has[slot]) break;
                const int n = sm.item[slot].s1 - sm.item[slot].s0;
                const int n0 = tile_steps(u, sm.item[slot], 0), n1 = tile_steps(u, sm.item[slot], 1);
                mbar_arrive(&sm.item_free[slot]);
                if (!mbar_wait(&sm.q_full, ui & 1)) { fail(sm, u, 11); break; }
                for (int i = 0; i < n && ok; ++i, ++kv_it) {
                    if (!mbar_wait(&sm.kv_full_k[kv_it & 1], (kv_it >> 1) & 1)) { fail(sm, u, 12); ok = false; break; }
                    for (int t = 0; t < kQT; ++t) {
                        if (i >= (t ? n1 : n0)) continue;
                        if (s_cnt > 0 && !mbar_wait(&sm.s_free, (s_cnt - 1) & 1)) { fail(sm, u, 13); ok = false; break; }
                        tc_fence_after();
                        issue_s(tmem, dhi, t ? q_lo1 : q_lo0, (kv_it & 1) ? k_lo1 : k_lo0);
                        umma_commit(&sm.s_full[t]);
                        ++s_cnt;
                    }
                    if (!ok) break;
                    umma_commit(&sm.kv_empty_k[kv_it & 1]);
                }
                if (ok) umma_commit(&sm.q_empty);
            }
            umma_commit(&sm.mma_drain);  // all issued MMAs complete before TMEM is released
            mbar_wait(&sm.mma_drain, 0);
        }
    } else if (warp == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        // ------------------------------------------------------------ items, row tables, Q
        ChunkWalk walk(sm.split);
        if (lane == 0) {
            tma_prefetch_desc(&mapQ);
            u.desc[2 * blockIdx.x].valid = u.desc[2 * blockIdx.x + 1].valid = 0;
        }
        const int tile_rows = u.W * u.k;
        int64_t armed = -1;
        for (uint32_t ui = 0; !aborted(sm); ++ui) {
            const int slot = ui % kItems;
            if (!warp_wait(sm, u, &sm.item_free[slot], ((ui / kItems) & 1) ^ 1, 20)) break;
            ChunkItem it;
            const bool has = walk.next(u, it);  // the same in every lane
            if (lane == 0) {
                sm.has[slot] = has;
                if (has) {
                    sm.item[slot] = it;
                    if (chunk_partial(it)) chunk_describe(u, it, blockIdx.x);
                }
                mbar_arrive(&sm.item_full[slot]);
            }
            if (!has) break;
            const int tiles = it.nt > u.W ? 2 : 1;
            int row[kQT][4];  // this lane's rows 4 lane .. 4 lane + 3 of each tile, as rows of Q
#pragma unroll
            for (int t = 0; t < kQT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = lane * 4 + e, off = t * u.W + r / u.k;
                    int j = -1;
                    if (r < tile_rows && off < it.nt) j = chunk_head(u, it.t0 + off, it.q, r % u.k);
                    sm.row_j[slot][t][r] = j;
                    row[t][e] = j >= 0 ? (it.t0 + off) * u.h + j : p.q_rows;  // outside: zeros
                }
            warp_arrive(&sm.rows_full[slot]);
            if (!warp_wait(sm, u, &sm.q_empty, (ui & 1) ^ 1, 21)) break;
            if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, tiles * kTileBytes);
            __syncwarp();
#pragma unroll
            for (int t = 0; t < kQT; ++t)
                if (t < tiles) {
                    uint8_t* dst = sm.q[t] + lane * 512;
                    tma_gather4_2d(&mapQ, &sm.q_full, dst, 0, row[t][0], row[t][1], row[t][2], row[t][3]);
                    tma_gather4_2d(&mapQ, &sm.q_full, dst + kHalf, 64, row[t][0], row[t][1], row[t][2], row[t][3]);
                }
            armed = ui;
        }
        if (armed >= 0) mbar_wait(&sm.q_full, armed & 1);  // the last Q loads land before the CTA may exit
    } else if (warp == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        // ------------------------------------------------------------ MMA issuer: O += P V
        const uint32_t dhi = smem_desc_hi(1024, kSwizzle128B);
        const uint32_t v_lo0 = smem_desc_lo(smem_u32(sm.v[0]), kHalf), v_lo1 = smem_desc_lo(smem_u32(sm.v[1]), kHalf);
        const int page = 1 << u.page_shift;
        uint32_t kv_it = 0, c[kQT] = {0, 0}, o_cnt[kQT] = {0, 0};
        bool ok = true;
        for (uint32_t ui = 0; ok && !aborted(sm); ++ui) {
            const int slot = ui % kItems;
            if (!warp_wait(sm, u, &sm.item_full[slot], (ui / kItems) & 1, 30)) break;
            if (!sm.has[slot]) break;
            const ChunkItem it = sm.item[slot];
            warp_arrive(&sm.item_free[slot]);
            const int n = it.s1 - it.s0, n0 = tile_steps(u, it, 0), n1 = tile_steps(u, it, 1);
            for (int i = 0; i < n && ok; ++i, ++kv_it) {
                if (!warp_wait(sm, u, &sm.kv_full_v[kv_it & 1], (kv_it >> 1) & 1, 31)) { ok = false; break; }
                // Rows of loaded pages that no row of the unit sees: past the last
                // token, and between the first `sinks` keys and the window.
                const int kv0 = it.tile(it.s0 + i) * kBN, kv1 = kv0 + kBN;
                if (kv1 > it.hi || kv0 < it.lo) {
                    uint8_t* v = sm.v[kv_it & 1];
                    auto zero = [&](int a, int b) {
                        a = max(a, kv0);
                        b = min(b, kv1);
                        for (int x = lane; x < (b - a) * 16; x += 32)
                            *reinterpret_cast<uint4*>(v + ((x & 8) ? kHalf : 0) + (a - kv0 + (x >> 4)) * 128 + (x & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    };
                    zero(it.hi, (it.hi + page - 1) & ~(page - 1));
                    if (u.window) {
                        zero(u.sinks, min(it.lo, (u.sinks + page - 1) & ~(page - 1)));
                        zero(max(u.sinks, it.lo & ~(page - 1)), it.lo);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                for (int t = 0; t < kQT; ++t) {
                    if (i >= (t ? n1 : n0)) continue;
                    if (!warp_wait(sm, u, &sm.p_full[t], c[t] & 1, 32)) { ok = false; break; }
                    if (i == 0 && !warp_wait(sm, u, &sm.o_empty[t], (o_cnt[t] & 1) ^ 1, 33)) { ok = false; break; }
                    if (lane == 0) {
                        tc_fence_after();
                        issue_pv(tmem, dhi, t, (kv_it & 1) ? v_lo1 : v_lo0, i == 0);
                        umma_commit(&sm.p_empty[t]);
                        if (i == (t ? n1 : n0) - 1) umma_commit(&sm.o_full[t]);
                    }
                    ++c[t];
                    if (i == 0) ++o_cnt[t];
                }
                if (!ok) break;
                if (lane == 0) umma_commit(&sm.kv_empty_v[kv_it & 1]);
                __syncwarp();
            }
        }
        if (lane == 0) {
            umma_commit(&sm.mma_drain2);
            mbar_wait(&sm.mma_drain2, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ softmax + epilogue (tile t)
        const int t = (warp - 4) >> 2;     // query tile of this warpgroup
        const int wq = warp & 3;           // TMEM lane quarter of this warp
        const int r = wq * 32 + lane;      // query row owned by this thread
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t s_addr = tmem + lane_off + kColS;
        const uint32_t p_addr = tmem + lane_off + kColP + 64 * t;
        const uint32_t o_addr = tmem + lane_off + kColO + t * 128;
        const int off = t * u.W + r / u.k;  // this row's token within the unit, and its selection
        const int sel = r % u.k;
        const bool in_tile = r < u.W * u.k;
        const uint64_t C2 = pk2(p.scale_log2, p.scale_log2);
        uint32_t ctile = 0, o_it = 0;
        for (uint32_t ui = 0; !aborted(sm); ++ui) {
            const int slot = ui % kItems;
            if (!warp_wait(sm, u, &sm.item_full[slot], (ui / kItems) & 1, 40)) break;
            if (!sm.has[slot]) break;
            const ChunkItem it = sm.item[slot];
            const int n = tile_steps(u, it, t);
            const int toks = min(it.nt - t * u.W, u.W);  // of this tile; 0 or less: none
            if (toks <= 0) {
                warp_arrive(&sm.item_free[slot]);
                continue;
            }
            const bool partial = chunk_partial(it);
            const bool mine = in_tile && off < it.nt;
            const int token = it.t0 + off;
            const float gate = mine ? u.gate[((int64_t)token * u.g + it.q) * u.k + sel] : 0.f;
            if (!warp_wait(sm, u, &sm.rows_full[slot], (ui / kItems) & 1, 41)) break;
            // The unselected output slots of the tile's tokens, by the part that
            // holds the unit's first step.
            if (it.s0 == 0 && u.k < u.hpg) {
                for (int x = wq * 32 + lane; x < toks * u.hpg * 16; x += 128) {
                    const int j = it.q * u.hpg + (x >> 4) % u.hpg, tok = (x >> 4) / u.hpg;
                    bool chosen = false;
                    for (int a = 0; a < u.k; ++a) chosen |= sm.row_j[slot][t][tok * u.k + a] == j;
                    if (!chosen)
                        *reinterpret_cast<uint4*>(p.O + ((int64_t)(it.t0 + t * u.W + tok) * u.h + j) * kD + (x & 15) * 8) =
                            make_uint4(0, 0, 0, 0);
                }
            }
            const int head = mine ? sm.row_j[slot][t][r] : -1;
            const bool live = wq * 32 < toks * u.k;  // some row of this warp is a query row
            // Keys this row sees: [low, pos] and those below u.sinks.  A padding row
            // sees all (its result is dropped).
            const int pos = mine ? it.p0 + off : INT_MAX - 1;
            const int low = mine && u.window ? pos - u.window + 1 : INT_MIN;
            const int pos_first = it.p0 + t * u.W, low_last = u.window ? pos_first + toks - u.window : INT_MIN;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int i = 0; i < n; ++i, ++ctile) {
                if (!warp_wait(sm, u, &sm.s_full[t], ctile & 1, 42)) { ok = false; break; }
                if (!live) {  // no query row: hand both buffers on, P no sooner than the slot is free
                    if (lane == 0) mbar_arrive(&sm.s_free);
                    if (ctile > 0 && !warp_wait(sm, u, &sm.p_empty[t], (ctile - 1) & 1, 45)) { ok = false; break; }
                    if (lane == 0) mbar_arrive(&sm.p_full[t]);
                    continue;
                }
                tc_fence_after();
                uint32_t s[4][32];
                const int kv0 = it.tile(it.s0 + i) * kBN;
                const bool need_mask = kv0 + kBN - 1 > pos_first || (kv0 < low_last && kv0 + kBN > u.sinks);
                uint64_t sum2[4] = {0, 0, 0, 0};
                float m_use = m;
                bool done = false, slot_ok = true;
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) tmem_ld32(s_addr + cb * 32, s[cb]);
                ld_wait_bind(s[0]);
                ld_bind(s[1]);
                ld_bind(s[2]);
                ld_bind(s[3]);
                tc_fence_before();
                warp_arrive(&sm.s_free);
                // P slot of this tile: free once the tile's previous P.V has
                // completed (which also completes O_t up to the previous step).
                auto wait_slot = [&]() {
                    if (ctile > 0 && !__all_sync(0xffffffffu, mbar_wait(&sm.p_empty[t], (ctile - 1) & 1))) slot_ok = false;
                    tc_fence_after();
                };
                // On an unmasked step after the first, the exponentials are taken
                // against the running max while the step's row max is formed
                // alongside: unless some row of the warp grew its max by more than
                // the threshold, P is final.
                if (!need_mask && i > 0) {
                    const uint64_t NM2 = pk2(-m, -m);
                    float mq[4];
                    uint32_t pk[4][16];
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
                            pk[cb][e] = pack_bf16x2(p0, p1);
                        }
                        // the first two chunks wait in registers for the slot
                        if (cb == 1) {
                            wait_slot();
                            tmem_st16(p_addr, pk[0]);
                            tmem_st16(p_addr + 16, pk[1]);
                        } else if (cb > 1) {
                            tmem_st16(p_addr + cb * 16, pk[cb]);
                        }
                    }
                    const float mx = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * p.scale_log2;
                    done = __all_sync(0xffffffffu, mx <= m + kRescaleThreshold);
                    if (!done) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum2[e] = 0;
                    }
                }
                if (!done) {
                    if (need_mask) {
#pragma unroll
                        for (int cb = 0; cb < 4; ++cb) {
                            const int k0 = kv0 + cb * 32;
                            const uint32_t see = low_bits(pos + 1 - k0) & (~low_bits(low < k0 ? 0 : low - k0) | low_bits(u.sinks - k0));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see & (1u << e))) s[cb][e] = __float_as_uint(-INFINITY);
                        }
                    }
                    float mq[4];
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        float a0 = __uint_as_float(s[cb][0]);
#pragma unroll
                        for (int e = 1; e < 31; e += 2)
                            a0 = fmax3(a0, __uint_as_float(s[cb][e]), __uint_as_float(s[cb][e + 1]));
                        mq[cb] = fmaxf(a0, __uint_as_float(s[cb][31]));
                    }
                    const float mx = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * p.scale_log2;
                    // Lazy rescaling: keep the running max unless it grows by more
                    // than the threshold.  A row that has seen no key so far has
                    // weights 0 only, and O_t rows of 0: nothing to rescale.
                    bool rescale = false;
                    if (mx > m + kRescaleThreshold || m == -INFINITY) {
                        m_use = mx;
                        rescale = m != -INFINITY;
                    }
                    wait_slot();
                    if (__any_sync(0xffffffffu, rescale)) {
                        const float alpha = rescale ? fast_exp2(m - m_use) : 1.0f;
#pragma unroll 1
                        for (int cb = 0; cb < 4; ++cb) {
                            uint32_t o[32];
                            tmem_ld32(o_addr + cb * 32, o);
                            ld_wait_bind(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(o_addr + cb * 32, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                            tmem_st16(o_addr + cb * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
                        }
                        l *= alpha;
                    }
                    const float ref = m_use == -INFINITY ? 0.f : m_use;
                    const uint64_t NM2 = pk2(-ref, -ref);
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            up2(ffma2(pk2(__uint_as_float(s[cb][2 * e]), __uint_as_float(s[cb][2 * e + 1])), C2, NM2), x0, x1);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            sum2[e & 3] = fadd2(sum2[e & 3], pk2(p0, p1));
                            pk[e] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(p_addr + cb * 16, pk);
                    }
                }
                float sa, sb;
                up2(fadd2(fadd2(sum2[0], sum2[1]), fadd2(sum2[2], sum2[3])), sa, sb);
                l += sa + sb;
                m = m_use;
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&sm.p_full[t]);
                if (!slot_ok) {
                    if (lane == 0) fail(sm, u, 43);
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
            // Epilogue: O_t / l, gated, as the bf16 row of O, or the row's partial
            // record (o, log2-sum-exp); none of this part's keys seen: -inf.
            float* rec = u.part + ((int64_t)chunk_slot(it, blockIdx.x) * u.row_cap + t * u.W * u.k + r) * (kD + 4);
            if (n == 0) {
                if (partial && mine) rec[kD] = -INFINITY;
                warp_arrive(&sm.item_free[slot]);
                continue;
            }
            if (!warp_wait(sm, u, &sm.o_full[t], o_it & 1, 44)) break;
            ++o_it;
            if (!live) {
                warp_arrive(&sm.o_empty[t]);
                warp_arrive(&sm.item_free[slot]);
                continue;
            }
            tc_fence_after();
            uint32_t o[4][32];
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) tmem_ld32(o_addr + cb * 32, o[cb]);
            ld_wait_bind(o[0]);
            ld_bind(o[1]);
            ld_bind(o[2]);
            ld_bind(o[3]);
            tc_fence_before();
            warp_arrive(&sm.o_empty[t]);
            const bool none = m == -INFINITY && l == 0.f;
            const float f = partial ? (none ? 0.f : 1.f / l) : gate / l;
            float check[4] = {l * 0.f, 0.f, 0.f, 0.f};  // stays 0, or NaN when a value is not finite
#pragma unroll
            for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                for (int e = 0; e < 32; ++e) check[e & 3] = fmaf(__uint_as_float(o[cb][e]), 0.f, check[e & 3]);
            const bool redo = head >= 0 && !((check[0] + check[1]) + (check[2] + check[3]) == 0.f);
            if (head >= 0 && !redo) {
                if (partial) {
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            reinterpret_cast<float4*>(rec + cb * 32)[v] =
                                make_float4(__uint_as_float(o[cb][4 * v]) * f, __uint_as_float(o[cb][4 * v + 1]) * f,
                                            __uint_as_float(o[cb][4 * v + 2]) * f, __uint_as_float(o[cb][4 * v + 3]) * f);
                    rec[kD] = none ? -INFINITY : m + log2f(l);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.O + ((int64_t)token * u.h + head) * kD);
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint4 pk;
                            pk.x = pack_bf16x2(__uint_as_float(o[cb][8 * v + 0]) * f, __uint_as_float(o[cb][8 * v + 1]) * f);
                            pk.y = pack_bf16x2(__uint_as_float(o[cb][8 * v + 2]) * f, __uint_as_float(o[cb][8 * v + 3]) * f);
                            pk.z = pack_bf16x2(__uint_as_float(o[cb][8 * v + 4]) * f, __uint_as_float(o[cb][8 * v + 5]) * f);
                            pk.w = pack_bf16x2(__uint_as_float(o[cb][8 * v + 6]) * f, __uint_as_float(o[cb][8 * v + 7]) * f);
                            dst[cb * 4 + v] = pk;
                        }
                }
            }
            for (unsigned again = __ballot_sync(0xffffffffu, redo); again; again &= again - 1) {
                const int src = __ffs(again) - 1;
                const int jj = __shfl_sync(0xffffffffu, head, src), tok = __shfl_sync(0xffffffffu, token, src);
                const int pp = __shfl_sync(0xffffffffu, pos, src);
                float a2[kD / 32], m2, l2;
                chunk_row<bf16, kD>(u, it, pp, p.Q + ((int64_t)tok * u.h + jj) * kD, p.K, p.V, p.scale_log2, a2, m2, l2);
                chunk_store_row<bf16, kD>(u, it, blockIdx.x, t * u.W * u.k + wq * 32 + src, tok, jj, a2, m2, l2, p.O);
            }
            warp_arrive(&sm.item_free[slot]);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

ChunkTiling chunk_tc_tiling() { return {kBM, kQT, kBN, 2 * kBN, 4 * kBN, 1}; }

cudaError_t launch_chunk_tc(const ChunkGeom& u, const ChunkArgs& a, int parts) {
    const gqe_shape& s = *a.s;
    // The setmaxnreg split needs exactly kRegsLaunch registers per thread at
    // launch (a property of the compiled kernels: checked once per process).
    static std::atomic<int> regs_checked{0};
    if (regs_checked.load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes fa, fb;
        cudaError_t e = cudaFuncGetAttributes(&fa, chunk_tc_kernel<false>);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fb, chunk_tc_kernel<true>);
        if (e != cudaSuccess) return e;
        regs_checked.store(fa.numRegs == kRegsLaunch && fb.numRegs == kRegsLaunch ? 1 : -1, std::memory_order_release);
    }
    if (regs_checked.load(std::memory_order_acquire) != 1) return cudaErrorNotSupported;

    const int page = 1 << a.page_shift;
    const bool gather = page < 8;
    const int64_t q_rows = (int64_t)s.T * s.h, kv_rows = (int64_t)a.num_pages * page * s.g;
    if (q_rows >= ((int64_t)1 << 31) - 1 || (gather && kv_rows >= ((int64_t)1 << 31) - 1)) return cudaErrorNotSupported;
    CUtensorMap mapK, mapV, mapQ;
    const uint64_t row_bytes = kD * 2;
    const uint32_t row_box[2] = {64, 1};
    if (gather) {
        const uint64_t dims[2] = {(uint64_t)kD, (uint64_t)kv_rows};
        if (!make_bf16_map(&mapK, a.K_pages, 2, dims, &row_bytes, row_box)) return cudaErrorInvalidValue;
        if (!make_bf16_map(&mapV, a.V_pages, 2, dims, &row_bytes, row_box)) return cudaErrorInvalidValue;
    } else {
        const uint64_t dims[4] = {(uint64_t)kD, (uint64_t)s.g, (uint64_t)page, (uint64_t)a.num_pages};
        const uint64_t strides[3] = {row_bytes, s.g * row_bytes, (uint64_t)page * s.g * row_bytes};
        const uint32_t box[4] = {64, 1, (uint32_t)(page < kBN ? page : kBN), 1};
        if (!make_bf16_map(&mapK, a.K_pages, 4, dims, strides, box)) return cudaErrorInvalidValue;
        if (!make_bf16_map(&mapV, a.V_pages, 4, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const uint64_t qdims[2] = {(uint64_t)kD, (uint64_t)q_rows};
    if (!make_bf16_map(&mapQ, a.Q, 2, qdims, &row_bytes, row_box)) return cudaErrorInvalidValue;

    Params p;
    p.Q = (const bf16*)a.Q;
    p.K = (const bf16*)a.K_pages;
    p.V = (const bf16*)a.V_pages;
    p.O = (bf16*)a.O;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)kD);
    p.q_rows = (int)q_rows;
    p.kv_rows = (int)kv_rows;
    const size_t smem = sizeof(Smem) + 1024;
    auto kern = gather ? chunk_tc_kernel<true> : chunk_tc_kernel<false>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, mapK, mapV, mapQ, u, p);
}

}  // namespace gqe
