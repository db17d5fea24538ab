// linear_tiles.cu - the product with an epilogue for many rows, where the tensor cores bound it.
//
// gemm.cuh's kernels keep a weight tile in front of the tensor core and bring the rows to it: right where the
// weights are most of the bytes.  With thousands of rows both operands are large, every byte of either is
// read by many tiles, and the order of the tiles decides what the L2 holds.  Here:
//
//   tiles       a CTA pair (.cta_group::2) forms 256 rows of x by 256 rows of w (gated: 128 gates and their
//               128 ups, the gates from one CTA of the pair and the ups from the other), each CTA bringing
//               128 rows of each: 64 KB a k-block for 2 x 256 x 256 x 128 (8 bits) operations;
//   order       tiles go to the pairs in turn, row tiles fastest within groups of `group` of them, so that
//               the tiles in flight are nearly a square and share what they read, kept in the L2 as long as
//               it can (evict_last; without it 3 % slower);
//   rows        of x lie along the accumulator's lanes: a thread of the epilogue has one row, its scale in a
//               register, and neighbouring columns, with a gate and its up both its own;
//   epilogue    eight warps a CTA, while the next tile's sums go into the accumulator's other half (2 x 256
//               columns of TMEM): residual in by TMA before the sums are ready, outputs out by TMA, both
//               through the same swizzled 4 KB of shared memory a warp and 32 x 128 bytes of outputs.
//
// Bound by the tensor cores and, over many calls, by the board's power: 2080 rows 4096 -> 2 x 14336 in 8 bits
// 164 us at first (3.0 PFLOP/s, 80 % of the tensor pipe's cycles; the ninth row tile has 32 rows of 256) and 177
// to 181 call after call; 8192 rows 14336 -> 4096 324 to 328 us (2.9 to 3.0 PFLOP/s).  Tiles of 128 columns take 1.75
// times as long (the pair's operands then cost the shared memory more than the tensor core's time).
#include <algorithm>
#include <mutex>

#include "../../include/eagle_tree.h"
#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.cuh"

namespace eagle {
namespace {

constexpr int kTile = 256;      // rows of x and of w that a pair's tile has
constexpr int kHalf = 128;      // rows of each that a CTA brings
constexpr int kStages = 5;
constexpr uint32_t kOperandBytes = kHalf * 128;          // 16 KB
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kEpilogueWarps = 8, kEpilogueThreads = kEpilogueWarps * 32;
constexpr int kThreads = 64 + kEpilogueThreads;          // warp 0: copies, warp 1: MMAs, then the epilogue
constexpr uint32_t kSlotBytes = 32 * 128;                // outputs that one copy takes: 32 rows of 128 bytes
constexpr uint32_t kFull = 0xffffffffu;

struct TileArgs {
    int32_t rows, M, num_kb;
    int32_t row_tiles, col_tiles, group;
    LinearEpilogue ep;
    const __nv_bfloat16 *bias;
    int32_t out_bf16, residual_tma;
    int32_t *status;
};

struct TileCtl {
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t res[kEpilogueWarps][2];  // a warp's slots: the residual is in
    uint64_t drain;                   // used only when unwinding after a timeout
    uint32_t tmem_base;
    int32_t abort;
    float scale[kTile];               // of the tile's rows of w
    uint16_t bias[kTile];
};

constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * 2 * kSlotBytes + sizeof(TileCtl);
static_assert(kSmem <= 232448, "227 KB");
__device__ __forceinline__ void tile_of(const TileArgs &a, int32_t u, int32_t &rt, int32_t &ct) {
    const int32_t per = a.group * a.col_tiles, g = u / per, first = g * a.group;
    const int32_t gr = min(a.group, a.row_tiles - first), in = u - g * per;
    ct = in / gr;
    rt = first + in - ct * gr;
}

// kSplit: a cluster of two pairs forms one tile, each from its half of K, and each finishes half of the tile's
// columns.
// kLong: the tensor core's accumulator truncates, so a long sum of bf16 products is too small by a part that
// grows with its length (14336 products 1.7e-5, more than an fp32 output should lose): the sums of kSegment
// k-blocks at a time are added up, rounded to nearest, in the accumulator's other half (2.1e-6; up to 4096 products in
// one go 4.4e-6).  The products wait meanwhile: 2080 rows 14336 -> 4096 in bf16 157 us, 142 with bf16 out.  Segments of
// half the length lose half as much and cost as much again; the sums in registers do not fit beside 10 warps.
// 8-bit products, mostly multiples of the accumulator's step, lose 1.0e-6 of 14336 and are left whole.
constexpr int kSegment = 32;
template <bool kFp8, bool kGated, bool kSplit, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tiles_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_r,
                        const TileArgs a) {
    constexpr int32_t BK = kFp8 ? 128 : 64;
    constexpr int32_t kCols = kGated ? kHalf : kTile;  // outputs of a tile's row
    constexpr uint32_t kTmemCols = kSplit && !kLong ? kTile : 2 * kTile;
    constexpr uint32_t kSums = kLong ? kTile : 0;  // where the epilogue finds the sums, in an accumulator
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint8_t *slots = ring + kStages * kStageBytes;
    TileCtl *ctl = reinterpret_cast<TileCtl *>(slots + kEpilogueWarps * 2 * kSlotBytes);
    volatile int32_t *abort_flag = &ctl->abort;

    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // workers: pairs, or the clusters that share a tile; `part` of the tile's K is this pair's
    constexpr int32_t split = kSplit ? 2 : 1;
    const int32_t rank = blockIdx.x & 1;
    const int32_t pairs = static_cast<int32_t>(gridDim.x >> 1) / split, pair = static_cast<int32_t>(blockIdx.x >> 1) / split;
    const int32_t part = kSplit ? static_cast<int32_t>(blockIdx.x >> 1) - pair * split : 0;
    const uint32_t leader = 2u * part;  // cluster rank of this pair's even CTA
    const int32_t units = a.row_tiles * a.col_tiles;
    const int32_t kb_begin = kSplit ? a.num_kb * part / split : 0, kb_end = kSplit ? a.num_kb * (part + 1) / split : a.num_kb;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->acc_full[i], 1);
            mbar_init(&ctl->acc_empty[i], 2 * kEpilogueWarps);  // both CTAs' epilogue warps
            for (int w = 0; w < kEpilogueWarps; ++w) mbar_init(&ctl->res[w][i], 1);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmap_x);
        prefetch_tensormap(&tmap_w);
    }
    if (warp == 1) {
        tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;

    uint32_t issued = 0, issued_parity = 0;  // the copying thread's, for unwinding

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = policy_evict_last();
            // both CTAs' copies count on the even CTA's barrier, which expects the bytes of both
            auto load_w = [&](int s, int32_t kb, int32_t ct) {
                const int32_t y = kGated ? rank * a.M + ct * kHalf : ct * kTile + rank * kHalf;
                tma_load_2d_pair(ring + s * kStageBytes + kOperandBytes, &tmap_w, peer_addr(&ctl->full[s], leader), kb * BK, y, keep);
            };
            auto load_x = [&](int s, int32_t kb, int32_t rt) {
                tma_load_2d_pair(ring + s * kStageBytes, &tmap_x, peer_addr(&ctl->full[s], leader), kb * BK, rt * kTile + rank * kHalf, keep);
            };
            auto expect = [&](int s) {
                if (rank == 0) mbar_arrive_expect_tx(&ctl->full[s], 2 * kStageBytes);
            };
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            pdl_wait();  // x, and w where a caller has just quantised it, come from kernels before
            for (int32_t u = pair; u < units && ok; u += pairs) {
                int32_t rt, ct;
                tile_of(a, u, rt, ct);
                for (int32_t kb = kb_begin; kb < kb_end; ++kb) {
                    if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag)) {
                        *abort_flag = 1;
                        latch(a.status, kDevTimeout);
                        ok = false;
                        break;
                    }
                    expect(static_cast<int>(stage));
                    load_w(static_cast<int>(stage), kb, ct);
                    load_x(static_cast<int>(stage), kb, rt);
                    issued |= 1u << stage;
                    issued_parity = phase ? (issued_parity | (1u << stage)) : (issued_parity & ~(1u << stage));
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = kFp8 ? idesc_e4m3_f32(kTile, kTile) : idesc_bf16_f32(kTile, kTile);
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            const int32_t segments = kLong ? (kb_end - kb_begin + kSegment - 1) / kSegment : 1;
            for (int32_t u = pair, seg = 0; u < units && ok; seg = seg + 1 < segments ? seg + 1 : 0, u += seg == 0 ? pairs : 0) {
                const int32_t kb0 = kb_begin + seg * kSegment, kb1 = kLong ? min(kb_end, kb0 + kSegment) : kb_end;
                if (!mbar_wait(&ctl->acc_empty[acc], acc_phase ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * kTile;
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&ctl->full[stage], phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t x0 = smem_u32(ring + stage * kStageBytes), w0 = x0 + kOperandBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of the 128 an MMA
                        const uint64_t dx = sw128_kmajor_desc(x0 + kk * 32), dw = sw128_kmajor_desc(w0 + kk * 32);
                        if (kFp8)
                            mma_f8_ss_pair(d_tmem, dx, dw, idesc, kb > kb0 || kk > 0);
                        else
                            mma_bf16_ss_pair(d_tmem, dx, dw, idesc, kb > kb0 || kk > 0);
                    }
                    mma_commit_pair_mc(&ctl->empty[stage], static_cast<uint16_t>(3u << leader));  // the stage is free in both CTAs
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair_mc(&ctl->acc_full[acc], static_cast<uint16_t>(3u << leader));  // each CTA drains its own 128 rows
                if (!kLong) acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok) {
                *abort_flag = 1;
                latch(a.status, kDevTimeout);
            }
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: warps 2..9, TMEM lane quarter = warp % 4, columns in two halves ----------------
        pdl_wait();
        const int32_t ew = warp - 2, q = warp & 3, side = ew >> 2, et = threadIdx.x - 64;
        // this CTA's outputs of a row (all of the tile's, or its half), and those of one warp
        constexpr int32_t slice = kCols / split, span = slice / 2;
        const int32_t chunk_cols = a.out_bf16 ? min(span, 64) : 32, chunks = span / chunk_cols;
        const int32_t row_bytes = a.out_bf16 ? 2 * chunk_cols : 128;
        uint8_t *const slot0 = slots + ew * 2 * kSlotBytes;
        uint32_t acc = 0, acc_phase = 0, res_phase = 0;
        // chunks of all tiles so far: the slots take turns, also from one tile to the next where a tile is one chunk,
        // so that a slot's last copy is never the newest
        int32_t turn = 0;
        // kSplit: the pairs' sums of a CTA's columns meet in its shared memory, where the copies are over: from
        // the other pair [accumulator columns of the slice / 4][128 rows][4].  The two cluster barriers are met
        // by every thread of the cluster (the other warps', behind their work).
        constexpr int32_t half_slice = kTile / split / 2;
        auto exchange = [&](bool skip) {
            __syncwarp();
            cluster_sync();  // every CTA's copies and products are over
            if (!__any_sync(kFull, skip)) {
                const uint32_t t_row = tmem_base + kSums + (static_cast<uint32_t>(q * 32) << 16);
                const int32_t to = part ^ 1;
                const uint32_t at = peer_addr(ring, 2u * to + rank) + static_cast<uint32_t>(side * half_slice * 512 + (q * 32 + lane) * 16);
                const int32_t col = kGated ? side * kHalf + to * half_slice : (2 * to + side) * half_slice;
                for (int32_t c = 0; c < half_slice; c += 32) {
                    uint32_t r[32];
                    __syncwarp();
                    tmem_ld_32(t_row + col + c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) st_peer_v4(at + static_cast<uint32_t>(c + 4 * i) * 512, r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
            }
            __syncwarp();
            cluster_sync();  // every part is here
        };
        // the other pair's sums of columns c .. c + 31 of the slice, added (a sum of two: in either order the same)
        auto add_parts = [&](uint32_t (&r)[32], int32_t c) {
            const float4 *src = reinterpret_cast<const float4 *>(ring + c * 512) + q * 32 + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 x = src[i * 128];
                const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) r[4 * i + k] = __float_as_uint(__uint_as_float(r[4 * i + k]) + y[k]);
            }
        };
        for (int32_t u = pair; u < units; u += pairs) {
            int32_t rt, ct;
            tile_of(a, u, rt, ct);
            const int32_t row0 = rt * kTile + rank * kHalf + q * 32, row = row0 + lane, first = part * slice + side * span;
            const int32_t col0 = ct * kCols + first;
            if (a.residual_tma && lane == 0) {
                bulk_wait_read<0>();  // the slots' last outputs are on their way
                for (int32_t c = 0; c < chunks; ++c) {
                    mbar_arrive_expect_tx(&ctl->res[ew][c], 32 * row_bytes);
                    tma_load_2d(slot0 + ((turn + c) & 1) * kSlotBytes, &tmap_r, &ctl->res[ew][c], col0 + c * chunk_cols, row0, policy_evict_first());
                }
            }
            // the columns' scales and biases: a thread each
            float cs = 1.0f;
            uint16_t cb = 0;
            {
                const int32_t o = kGated ? ct * kHalf + (et & (kHalf - 1)) : ct * kTile + et;
                const int32_t wr = kGated && et >= kHalf ? a.M + o : o;
                if (o < a.M) {
                    if (kFp8) cs = a.ep.w_scale[wr];
                    if (a.bias) cb = reinterpret_cast<const uint16_t *>(a.bias)[wr];
                }
            }
            const float rs = kFp8 ? (row < a.rows ? a.ep.x_scale[row] : 0.0f) : 1.0f;
            bool got = true;
            if constexpr (kLong) {
                named_barrier_sync(1, kEpilogueThreads);  // all are done with the last tile's sums
                const uint32_t from = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + side * kHalf;
                for (int32_t kb = kb_begin; kb < kb_end; kb += kSegment) {
                    got = got && mbar_wait(&ctl->acc_full[0], acc_phase, abort_flag);
                    got = __all_sync(kFull, got);
                    if (!got) break;
                    tc_fence_after();
                    for (int32_t c = 0; c < kHalf; c += 32) {
                        uint32_t r[32], s[32];
                        tmem_ld_32(from + c, r);
                        if (kb > kb_begin) {
                            tmem_ld_32(from + kSums + c, s);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(s[j]));
                        } else {
                            tmem_wait_ld();
                        }
                        tmem_st_32(from + kSums + c, r);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(peer_addr(&ctl->acc_empty[0], leader));
                    acc_phase ^= 1u;
                }
            } else {
                got = mbar_wait(&ctl->acc_full[acc], acc_phase, abort_flag);
            }
            if (!got) {
                *abort_flag = 1;
                latch(a.status, kDevTimeout);
            }
            if constexpr (kSplit && kLong) named_barrier_sync(1, kEpilogueThreads);  // sums that other warps send
            if constexpr (kSplit) {
                tc_fence_after();
                exchange(!got || *abort_flag);
            }
            // all threads give up together, and all are done with the last tile's columns
            if (named_barrier_or(1, kEpilogueThreads, !got || *abort_flag)) {
                if (a.residual_tma && lane == 0)  // let the copies land
                    for (int32_t c = 0; c < chunks; ++c) mbar_wait(&ctl->res[ew][c], res_phase, nullptr);
                break;
            }
            ctl->scale[et] = cs;
            ctl->bias[et] = cb;
            named_barrier_sync(1, kEpilogueThreads);
            tc_fence_after();
            const uint32_t t_row = tmem_base + kSums + (static_cast<uint32_t>(q * 32) << 16) + acc * kTile;
            for (int32_t c = 0; c < chunks; ++c, ++turn) {
                uint8_t *const slot = slot0 + (turn & 1) * kSlotBytes, *const mine = slot + lane * row_bytes;
                if (a.residual_tma) {
                    if (!mbar_wait(&ctl->res[ew][c], res_phase, abort_flag)) {
                        *abort_flag = 1;
                        latch(a.status, kDevTimeout);
                    }
                } else {
                    if (lane == 0) bulk_wait_read<1>();  // the slot's last outputs are on their way
                    __syncwarp();
                }
                for (int32_t p = 0; p < chunk_cols / 32; ++p) {
                    const int32_t at = first + c * chunk_cols + p * 32;  // column of the tile
                    uint32_t r[32], r2[32];
                    __syncwarp();
                    tmem_ld_32(t_row + at, r);
                    if (kGated) tmem_ld_32(t_row + kHalf + at, r2);
                    tmem_wait_ld();
                    if (!kLong && c == chunks - 1 && p == chunk_cols / 32 - 1) {  // the sums are out of the accumulator
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(peer_addr(&ctl->acc_empty[acc], leader));
                    }
                    if constexpr (kSplit) {
                        add_parts(r, at - part * slice);
                        if (kGated) add_parts(r2, slice + at - part * slice);
                    }
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float s = kFp8 ? rs * ctl->scale[at + j] : 1.0f, b = __uint_as_float(static_cast<uint32_t>(ctl->bias[at + j]) << 16);
                        v[j] = kFp8 ? fmaf(__uint_as_float(r[j]), s, b) : __uint_as_float(r[j]) + b;
                    }
                    if constexpr (kGated) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float s = kFp8 ? rs * ctl->scale[kHalf + at + j] : 1.0f;
                            const float b = __uint_as_float(static_cast<uint32_t>(ctl->bias[kHalf + at + j]) << 16);
                            const float up = kFp8 ? fmaf(__uint_as_float(r2[j]), s, b) : __uint_as_float(r2[j]) + b;
                            v[j] = silu(v[j]) * up;
                        }
                    } else if (a.ep.act != kActNone) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = activation(a.ep.act, v[j]);
                    }
                    if (a.out_bf16) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // 8 outputs, a swizzled 16-byte piece of the lane's row
                            const int32_t turn = row_bytes == 128 ? lane & 7 : (lane >> 1) & 3;
                            uint4 *piece = reinterpret_cast<uint4 *>(mine + (((p * 4 + i) ^ turn) << 4));
                            if (a.residual_tma) {
                                const uint4 x = *piece;
                                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    v[8 * i + 2 * k] = __fadd_rn(v[8 * i + 2 * k], __uint_as_float(xw[k] << 16));
                                    v[8 * i + 2 * k + 1] = __fadd_rn(v[8 * i + 2 * k + 1], __uint_as_float(xw[k] & 0xffff0000u));
                                }
                            }
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 two = __floats2bfloat162_rn(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
                                w[k] = *reinterpret_cast<const uint32_t *>(&two);
                            }
                            *piece = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        if (a.ep.residual && row < a.rows) {
                            const __nv_bfloat16 *res = a.ep.residual + static_cast<int64_t>(row) * a.ep.ldr + col0 + c * 32;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (col0 + c * 32 + j < a.M) v[j] = __fadd_rn(v[j], __bfloat162float(res[j]));
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4 *>(mine + ((i ^ (lane & 7)) << 4)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && row0 < a.rows && col0 + c * chunk_cols < a.M) tma_store_2d(&tmap_y, slot, col0 + c * chunk_cols, row0);
                if (lane == 0) bulk_commit();
            }
            res_phase ^= 1u;
            if (!kLong) {
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
        if (lane == 0) bulk_wait_all();  // before the slots go away
    }

    if (kSplit && warp < 2) {  // the epilogue's two cluster barriers
        cluster_sync();
        cluster_sync();
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) {
        // let every copy and MMA that this CTA started land before its memory goes to another
        if (warp == 0 && lane == 0) {
            if (rank == 1) {
                // this CTA's copies count on the other's barriers: give them a bounded time to land
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 200000ull) {
                }
            } else {
                for (int s = 0; s < kStages; ++s)
                    if ((issued >> s) & 1u) mbar_wait(&ctl->full[s], (issued_parity >> s) & 1u, nullptr);
            }
        }
        if (warp == 1 && lane == 0 && rank == 0) {
            mma_commit_pair_mc(&ctl->drain, static_cast<uint16_t>(1u << leader));
            mbar_wait(&ctl->drain, 0, nullptr);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    __syncwarp();
    cluster_sync();  // neither CTA leaves before the other is done with its memory and barriers
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const TileArgs);
template <bool kSplit>
Kernel kernel_of(bool fp8, bool gated, bool lng) {
    if (fp8) return gated ? linear_tiles_kernel<true, true, kSplit, false> : linear_tiles_kernel<true, false, kSplit, false>;
    if (lng) return gated ? linear_tiles_kernel<false, true, kSplit, true> : linear_tiles_kernel<false, false, kSplit, true>;
    return gated ? linear_tiles_kernel<false, true, kSplit, false> : linear_tiles_kernel<false, false, kSplit, false>;
}

// Clusters of 4 CTAs that fit on a device at once; 0 where that is not known: tiles are not shared then.
std::mutex g_mu;
int32_t g_clusters[64];

int32_t count_clusters() {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(128);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel_of<true>(true, false, false), &cfg) == cudaSuccess) return n;
    cudaGetLastError();
    return 0;
}

}  // namespace

cudaError_t prepare_linear_tiles() {
    for (int i = 0; i < 16; ++i) {
        const Kernel k = i < 8 ? kernel_of<false>(i & 1, i & 2, i & 4) : kernel_of<true>(i & 1, i & 2, i & 4);
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
        if (e != cudaSuccess) return e;
    }
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_mu);
    g_clusters[dev] = count_clusters();
    return cudaSuccess;
}

bool launch_linear_tiles(bool fp8, const LinearEpilogue &ep, const void *w, int64_t ldw, int32_t M, int32_t K, const void *x,
                         int64_t ldx, int32_t rows, const void *bias, void *out, int64_t ldo, bool out_bf16, int32_t *status,
                         int32_t pairs, cudaStream_t st, cudaError_t *err) {
    const bool gated = ep.act == kActSwiglu;
    const int32_t es = fp8 ? 1 : 2, box = 128 / es, cols = gated ? kHalf : kTile;
    TileArgs a{};
    a.rows = rows;
    a.M = M;
    a.num_kb = (K + box - 1) / box;
    a.row_tiles = (rows + kTile - 1) / kTile;
    a.col_tiles = (M + cols - 1) / cols;
    // even groups of at most 12 row tiles: over 5 to 40 row tiles of four products (4096 and 14336 -> 4096, 4096 -> 2 x
    // 14336 and 32000) in both types within 1 % of the best of groups of 3 to 40 nearly everywhere, where fixed groups
    // of 4 cost up to 5 %, one group of all up to 4 %; 5 % are left at 9 row tiles, 14336 -> 4096 (groups of 3), and
    // at 40 of bf16 (4)
    const int32_t groups = (a.row_tiles + 11) / 12;
    a.group = (a.row_tiles + groups - 1) / groups;
    a.ep = ep;
    a.bias = static_cast<const __nv_bfloat16 *>(bias);
    a.out_bf16 = out_bf16;
    a.residual_tma = ep.residual && out_bf16;
    a.status = status;
    int dev = 0;
    *err = cudaGetDevice(&dev);
    if (*err != cudaSuccess) return true;
    const int64_t units = static_cast<int64_t>(a.row_tiles) * a.col_tiles;
    // Fewer tiles than pairs: two pairs to a tile, where the clusters fit on the device at once (36 of 4 CTAs on 152
    // SMs) and each half is long enough (512 rows, 4096 x 4096: 15.3 -> 14.2 us in 8 bits, 24 -> 19 in bf16)
    const int32_t split = units <= g_clusters[dev] && a.num_kb >= 8 ? 2 : 1;
    const int32_t span = cols / split / 2, chunk = out_bf16 ? std::min(span, 64) : 32;
    CUtensorMap mx, mw, my, mr{};
    if (!encode_swizzled_rows(&mx, es, x, K, rows, ldx, box, kHalf) ||
        !encode_swizzled_rows(&mw, es, w, K, gated ? int64_t{2} * M : M, ldw, box, kHalf))
        return false;
    // outputs, or a residual, that a tensor map does not take
    if (!encode_swizzled_rows(&my, out_bf16 ? 2 : 4, out, M, rows, ldo, chunk, 32)) return false;
    if (a.residual_tma && !encode_swizzled_rows(&mr, 2, ep.residual, M, rows, ep.ldr, chunk, 32)) return false;
    const unsigned cluster = 2u * static_cast<unsigned>(split);
    const dim3 grid(split > 1 ? cluster * static_cast<unsigned>(units) : 2u * static_cast<unsigned>(units < pairs ? units : pairs));
    const bool lng = !out_bf16 && a.num_kb > 2 * kSegment * split;  // 8-bit products are summed exactly enough
    *err = launch_pdl_cluster(split > 1 ? kernel_of<true>(fp8, gated, lng) : kernel_of<false>(fp8, gated, lng), grid, dim3(kThreads),
                              cluster, kSmem, st, mx, mw, my, mr, a);
    return true;
}

}  // namespace eagle
