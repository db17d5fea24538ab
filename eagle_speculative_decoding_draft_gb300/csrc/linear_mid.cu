// linear_mid.cu - the product with an epilogue for 17 to 128 rows, where the weights' bytes bound it and the
// rows are too many for linear_few.cu's registers.
//
// As in gemm.cuh a tile of 128 rows of w (gated: 64 gates and their ups) is the MMA's M and the rows of x are
// its N, so the tensor core does no more than the rows ask for.  But a tile's K is split over a cluster of up
// to 8 CTAs, two CTAs fit an SM, and each has one part of one tile: all of a small matrix is under way at once,
// one CTA's beginning and end fall into the other's copies, and the parts' sums meet through the cluster's
// shared memory, each CTA finishing its share of the rows.  No partial sum goes through memory.  Bound by the
// memory and, towards 128 rows, by what the SMs take from the L2 (a row of x goes to every tile): 61 rows,
// 4096 -> 2 x 11008 in 8 bits 19.8 us (0.68 of the measured copy rate; 25.9 through gemm.cuh's stream), 4096 ->
// 4096 8.7 us, 9.2 with a residual (13.8).  Two epilogue warps an accumulator quarter: a warp alone on its scheduler
// takes twice as long over a share (128 rows, 4096 -> 4096: 13.4 -> 11.4 us).
#include <algorithm>
#include <type_traits>

#include "../../include/eagle_tree.h"
#include "gemm.cuh"

namespace eagle {
namespace {

constexpr int kMidStages = 6;  // at most
constexpr size_t kMidSmem = 113 * 1024;
// K-blocks (of 128 bytes: 64 bf16 or 128 8-bit products) that an accumulator sums in one go where fp32 goes out; the
// segments are added up rounded to nearest.  The tensor core adds 16 products (32 in 8 bits) to what it has and
// truncates, so a sum is too small by a part that grows with its length: of bf16 products 1.0e-6 (norm-wise,
// measured) for 1024 of them, 2.1e-6 for 2048, 4.4e-6 for 4096, 1.7e-5 for 14336; of 8-bit ones, mostly multiples
// of the accumulator's step, 2.2e-7 for 4096 and 1.0e-6 for 14336.
__host__ __device__ constexpr int32_t segment_of(bool fp8) { return fp8 ? 32 : 16; }
constexpr int kMidThreads = 64 + 256;  // warp 0: copies, warp 1: MMAs, then two warps an accumulator quarter

struct MidCtl {
    uint64_t full[kMidStages], empty[kMidStages], acc_full, acc_empty, drain;
    uint32_t tmem_base;
    int32_t abort;
};

struct MidArgs {
    LinearArgs l;      // M, rows, n_tile, num_kb, stages, bias, out, ldo, out_bf16, ep, status
    int32_t split;     // CTAs of a cluster
    int32_t tmem_cols;
};

__device__ __forceinline__ void tmem_ld_4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// A cluster of a.split CTAs a (tile, chunk of n_tile rows): blockIdx.x / split the tile, blockIdx.y the chunk.
// kLong (fp32 out): segment_of k-blocks are summed at a time, in an accumulator beside the one for their sums
// (61 rows, 14336 -> 4096 in bf16 24.0 -> 24.2 us; with everything in one accumulator 7.9e-6 lost where a CTA has
// all 14336 products, 1.0e-6 so).
template <class Op, bool kLong>
__global__ void __launch_bounds__(kMidThreads, 2)
    linear_mid_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x, const MidArgs m) {
    constexpr int32_t BK = k_block<Op>(), kSegment = segment_of(Op::kFp8);
    const LinearArgs &a = m.l;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const int32_t stages = a.stages, n = a.n_tile, S = m.split;
    const uint32_t stage_bytes = kABytes + static_cast<uint32_t>(n) * 128u;
    MidCtl *ctl = reinterpret_cast<MidCtl *>(ring + static_cast<size_t>(stages) * stage_bytes);
    volatile int32_t *abort_flag = &ctl->abort;
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t tile = static_cast<int32_t>(blockIdx.x) / S, part = static_cast<int32_t>(blockIdx.x) - tile * S;
    const int32_t row0 = static_cast<int32_t>(blockIdx.y) * n;
    const int32_t kb_begin = a.num_kb * part / S, kb_end = a.num_kb * (part + 1) / S;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmap_w);
        prefetch_tensormap(&tmap_x);
        for (int s = 0; s < stages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->acc_full, 1);
        mbar_init(&ctl->acc_empty, kMidThreads / 32 - 2);  // the epilogue's warps
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, static_cast<uint32_t>(m.tmem_cols));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // behind the allocation: a kernel that begins beside this one and takes all of the SM's tensor memory would
    // wait for this grid's end, and a CTA that has none yet for that kernel's
    pdl_launch_dependents();
    const uint32_t tmem_base = ctl->tmem_base;
    uint32_t issued = 0, issued_parity = 0;  // the copying thread's, for unwinding

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
            pdl_wait();
            uint32_t stage = 0, phase = 0;
            for (int32_t kb = kb_begin; kb < kb_end; ++kb) {
                if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag)) {
                    *abort_flag = 1;
                    latch(a.status, kDevTimeout);
                    break;
                }
                mbar_arrive_expect_tx(&ctl->full[stage], stage_bytes);
                uint8_t *dst = ring + static_cast<size_t>(stage) * stage_bytes;
                if constexpr (Op::kGated) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tma_load_3d(dst + i * (kABytes / 4), &tmap_w, &ctl->full[stage], kb * BK, tile * (BM / 2) + 16 * i, 0, pol_w);
                } else {
                    tma_load_2d(dst, &tmap_w, &ctl->full[stage], kb * BK, tile * BM, pol_w);
                }
                tma_load_2d(dst + kABytes, &tmap_x, &ctl->full[stage], kb * BK, row0, pol_x);
                issued |= 1u << stage;
                issued_parity = phase ? (issued_parity | (1u << stage)) : (issued_parity & ~(1u << stage));
                if (++stage == static_cast<uint32_t>(stages)) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = Op::kFp8 ? idesc_e4m3_f32(BM, static_cast<uint32_t>(n)) : idesc_bf16_f32(BM, static_cast<uint32_t>(n));
            uint32_t stage = 0, phase = 0, acc_phase = 0;
            int32_t held = 0;  // k-blocks in the accumulator
            bool ok = true;
            for (int32_t kb = kb_begin; kb < kb_end; ++kb, ++held) {
                if (kLong && held == kSegment) {  // they join the sums
                    mma_commit(&ctl->acc_full);
                    ok = mbar_wait(&ctl->acc_empty, acc_phase, abort_flag);
                    acc_phase ^= 1u;
                    held = 0;
                }
                ok = ok && mbar_wait(&ctl->full[stage], phase, abort_flag);
                if (!ok) {
                    *abort_flag = 1;
                    latch(a.status, kDevTimeout);
                    break;
                }
                tc_fence_after();
                const uint32_t w0 = smem_u32(ring) + stage * stage_bytes, x0 = w0 + kABytes;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t dw = sw128_kmajor_desc(w0 + kk * 32), dx = sw128_kmajor_desc(x0 + kk * 32);
                    if (Op::kFp8)
                        mma_f8_ss(tmem_base, dw, dx, idesc, held > 0 || kk > 0);
                    else
                        mma_bf16_ss(tmem_base, dw, dx, idesc, held > 0 || kk > 0);
                }
                mma_commit(&ctl->empty[stage]);
                if (++stage == static_cast<uint32_t>(stages)) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok) mma_commit(&ctl->acc_full);
        }
        __syncwarp();
    } else {
        pdl_wait();
        if constexpr (!kLong) {
            if (!mbar_wait(&ctl->acc_full, 0, abort_flag)) {
                *abort_flag = 1;
                latch(a.status, kDevTimeout);
            }
            __syncwarp();
            tc_fence_after();
        } else {
            const uint32_t lanes = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            uint32_t phase = 0;
            for (int32_t kb = kb_begin; kb < kb_end; kb += kSegment, phase ^= 1u) {
                const bool got = mbar_wait(&ctl->acc_full, phase, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    *abort_flag = 1;
                    latch(a.status, kDevTimeout);
                    break;
                }
                tc_fence_after();
                for (int32_t c = 32 * ((warp - 2) >> 2); c < n; c += 64) {  // this warp's columns, as below
                    uint32_t r[32];
                    tmem_ld_32(lanes + static_cast<uint32_t>(c), r);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 2 && kb > kb_begin; ++h) {
                        uint32_t s[16];
                        tmem_ld_16(lanes + static_cast<uint32_t>(n + c + 16 * h), s);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[16 * h + i] = __float_as_uint(__uint_as_float(r[16 * h + i]) + __uint_as_float(s[i]));
                    }
                    tmem_st_32(lanes + static_cast<uint32_t>(n + c), r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->acc_empty);
            }
            named_barrier_sync(1, kMidThreads - 64);  // sums that other warps of the quarter have stored
            tc_fence_after();
        }
    }
    // The parts' sums: CTA `to` of the cluster finishes rows to * share .. of the chunk, and finds those that
    // the others send it, from each [rows / 4][128 rows of w][4], where its copies are over.
    const int32_t share = n / S;
    const int32_t q = warp & 3, turn = (warp - 2) >> 2, ml = q * 32 + lane;
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (kLong ? static_cast<uint32_t>(n) : 0u);
    const bool fine = !__any_sync(0xffffffffu, *abort_flag != 0);
    if (S > 1) {
        cluster_sync();
        if (warp >= 2 && fine) {
            for (int32_t c = 32 * turn; c < n; c += 64) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld_32(t_row + static_cast<uint32_t>(c), r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // a share is a multiple of 4 rows
                    const int32_t to = (c + 4 * i) / share, at = c + 4 * i - to * share;
                    if (to != part)
                        st_peer_v4(peer_addr(ring, static_cast<uint32_t>(to)) +
                                       static_cast<uint32_t>(((part < to ? part : part - 1) * share + at) * 512 + ml * 16),
                                   r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
            }
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp >= 2 && fine) {
        const Column col = column_of<Op>(a, tile, ml);
        const int32_t end = min(a.rows - row0, n);  // rows of the chunk
        auto rows = [&](auto count) {  // as many at a time
            constexpr int C = decltype(count)::value;
            for (int32_t c = C * turn; c < share; c += 2 * C) {
                const int32_t n0 = part * share + c;
                if (n0 >= end) break;
                uint32_t r[C];
                __syncwarp();
                if constexpr (C == 16)
                    tmem_ld_16(t_row + static_cast<uint32_t>(n0), r);
                else if constexpr (C == 8)
                    tmem_ld_8(t_row + static_cast<uint32_t>(n0), r);
                else
                    tmem_ld_4(t_row + static_cast<uint32_t>(n0), r);
                tmem_wait_ld();
                float v[C];
                for (int32_t from = 0; from < S; ++from) {  // in their order
                    const float4 *src = reinterpret_cast<const float4 *>(ring + ((from < part ? from : from - 1) * share + c) * 512) + ml;
#pragma unroll
                    for (int k = 0; k < C; k += 4) {
                        float4 x = make_float4(__uint_as_float(r[k]), __uint_as_float(r[k + 1]), __uint_as_float(r[k + 2]),
                                               __uint_as_float(r[k + 3]));
                        if (from != part) x = src[k / 4 * 128];
                        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[k + j] = from == 0 ? y[j] : v[k + j] + y[j];
                    }
                }
                finish<Op>(a, col, row0 + n0, v);
                store_rows<Op>(a, col, row0, n0, end, v);
            }
        };
        if (share % 32 == 0)
            rows(std::integral_constant<int, 16>{});
        else if (share % 16 == 0)
            rows(std::integral_constant<int, 8>{});
        else
            rows(std::integral_constant<int, 4>{});
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) {
        // let every copy and MMA that this CTA started land before its memory goes to another
        if (warp == 0 && lane == 0)
            for (int s = 0; s < stages; ++s)
                if ((issued >> s) & 1u) mbar_wait(&ctl->full[s], (issued_parity >> s) & 1u, nullptr);
        if (warp == 1 && lane == 0) {
            mma_commit(&ctl->drain);
            mbar_wait(&ctl->drain, 0, nullptr);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, static_cast<uint32_t>(m.tmem_cols));
    }
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const MidArgs);
template <bool kLong>
Kernel kernel_of(bool fp8, bool gated) {
    if (fp8) return gated ? linear_mid_kernel<EpilogueOp<true, true>, kLong> : linear_mid_kernel<EpilogueOp<true, false>, kLong>;
    return gated ? linear_mid_kernel<EpilogueOp<false, true>, kLong> : linear_mid_kernel<EpilogueOp<false, false>, kLong>;
}

}  // namespace

cudaError_t prepare_linear_mid() {
    for (int i = 0; i < 8; ++i) {
        const Kernel k = i < 4 ? kernel_of<false>(i & 1, i & 2) : kernel_of<true>(i & 1, i & 2);
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kMidSmem));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

bool launch_linear_mid(bool fp8, const LinearEpilogue &ep, const void *w, int64_t ldw, int32_t M, int32_t K, const void *x,
                       int64_t ldx, int32_t rows, const void *bias, void *out, int64_t ldo, bool out_bf16, int32_t *status,
                       int32_t sms, cudaStream_t st, cudaError_t *err) {
    const bool gated = ep.act == kActSwiglu;
    const int32_t es = fp8 ? 1 : 2, box = 128 / es, cols = gated ? BM / 2 : BM;
    MidArgs m{};
    LinearArgs &a = m.l;
    a.M = M;
    a.K = K;
    a.rows = rows;
    const int32_t chunks = (rows + 127) / 128;
    a.n_tile = ((rows + chunks - 1) / chunks + 31) / 32 * 32;  // shares of 4 rows at least
    a.num_kb = (K + box - 1) / box;
    a.num_tiles = (M + cols - 1) / cols;
    const size_t stage = kABytes + static_cast<size_t>(a.n_tile) * 128;
    a.stages = static_cast<int32_t>(std::min<size_t>(kMidStages, (kMidSmem - 1024 - sizeof(MidCtl)) / stage));
    a.bias = static_cast<const __nv_bfloat16 *>(bias);
    a.out = out;
    a.ldo = ldo;
    a.out_bf16 = out_bf16;
    a.ep = ep;
    a.status = status;
    // as many parts as two CTAs an SM leave room for at once (61 rows, 4096 -> 4096 in 8 bits: 15.7, 11.4, 9.1 and
    // 9.5 us with 1, 2, 4 and 8; 4096 -> 6144: 16.1, 11.7, 10.3 and, in two waves, 16.4; 4096 -> 2 x 11008: 19.9 with
    // one, 26 with two), of at least two k-blocks, and of eight where eight parts exchange the sums of more than 32 rows
    // (1024 -> 1024 in bf16, 61 and 128 rows: 5.9 and 8.2 us with four, 6.5 and 9.3 with eight)
    const int32_t most = a.n_tile > 32 && a.num_kb < 64 ? 4 : 8;
    m.split = 1;
    while (m.split < most && static_cast<int64_t>(a.num_tiles) * chunks * m.split <= sms && a.num_kb >= 4 * m.split) m.split *= 2;
    const bool lng = !out_bf16 && (a.num_kb + m.split - 1) / m.split > segment_of(fp8);
    m.tmem_cols = 32;
    while (m.tmem_cols < a.n_tile * (lng ? 2 : 1)) m.tmem_cols *= 2;
    CUtensorMap mw, mx;
    if (gated ? !encode_gated_rows(&mw, es, w, K, M, ldw, 16) : !encode_swizzled_rows(&mw, es, w, K, M, ldw, box, BM)) return false;
    if (!encode_swizzled_rows(&mx, es, x, K, rows, ldx, box, a.n_tile)) return false;
    const size_t smem = 1024 + a.stages * stage + sizeof(MidCtl);
    const dim3 grid(static_cast<unsigned>(a.num_tiles * m.split), static_cast<unsigned>(chunks));
    *err = launch_pdl_cluster(lng ? kernel_of<true>(fp8, gated) : kernel_of<false>(fp8, gated), grid, dim3(kMidThreads),
                              static_cast<unsigned>(m.split), smem, st, mw, mx, m);
    return true;
}

}  // namespace eagle
