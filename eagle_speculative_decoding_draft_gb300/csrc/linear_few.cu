// linear_few.cu - the product with an epilogue for up to 16 rows, where the weights' bytes bound it and a
// call is short.
//
// A weight is used for 16 products at most: what counts is that the memory is busy from the first
// microsecond to the last.  So there is no ring, no tensor map and no accumulator to set up: a block has 16
// rows of w (gated: 8 gates and their ups, which the instruction then leaves in one thread), its warps share
// out K in pieces of 128 bytes, and every lane has up to four pieces' loads in flight straight into the
// registers from which mma.sync (m16n8, 32 bytes of K) takes them.  Both operands leave K in the same order, so which element a lane's register holds does
// not matter as long as it is the same one in w and in x: 16 neighbouring bytes a lane are two instructions'
// operands.  The warps' sums meet in shared memory, where the epilogue takes them; nothing is cut between
// blocks.  Bound by the memory: one row, 4096 -> 2 x 14336 in bf16 34 us, 1.0 of the measured copy rate, in
// 8 bits 20.2 us (0.86); 4096 -> 4096 in 8 bits 4.4 us (0.56: the call's own latency), against 10.6 through the
// ring of gemm.cuh.
#include <type_traits>

#include "../../include/eagle_tree.h"
#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.cuh"

namespace eagle {
namespace {

constexpr int kRows = 16;  // of w, or gates

struct FewArgs {
    int32_t rows, M, k_bytes;
    const uint8_t *w, *x;
    int64_t ldw, ldx;  // bytes
    LinearEpilogue ep;
    const __nv_bfloat16 *bias;
    void *out;
    int64_t ldo;
    int32_t out_bf16;
};

// Bytes off .. off + 15 of a row of `n`; those behind its end are 0 and are not read.
template <int kSize>
__device__ __forceinline__ uint4 tail16(const uint8_t *row, int32_t off, int32_t n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; i += kSize)
        if (off + i < n) {
            const uint32_t v = kSize == 1 ? row[off + i] : *reinterpret_cast<const uint16_t *>(row + off + i);
            w[i >> 2] |= v << (8 * (i & 3));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int kSize, bool kStream, bool kTail>
__device__ __forceinline__ uint4 load16(const uint8_t *row, int32_t off, int32_t n) {
    if (!kTail || off + 16 <= n) {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + off);
        return kStream ? __ldcs(p) : __ldg(p);
    }
    return tail16<kSize>(row, off, n);
}

template <bool kFp8>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (kFp8)
        asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kBlocks blocks of 8 rows of x.  kLong (bf16 operands, fp32 out, more than kSegment products a warp): mma.sync truncates
// what it adds up, as tcgen05 does (3.8e-6 of 14336 products over 4 warps, norm-wise; 1.1e-5 of 40000), so the sums
// go to the warp's place in shared memory every kSegment products and are added there, rounded to nearest (1.0e-6).
constexpr int kSegment = 1024;
template <bool kFp8, bool kGated, int kBlocks, int kWarps, bool kLong = false>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) linear_few_kernel(const FewArgs a) {
    constexpr int kThreads = 32 * kWarps, kSize = kFp8 ? 1 : 2;
    constexpr int kOut = kGated ? kRows / 2 : kRows;  // the instruction's rows 0-7 and 8-15: gates and their ups
    constexpr int kAhead = kBlocks == 1 ? 4 : 2;      // pieces in flight a lane: what 128 registers hold
    __shared__ float sums[kWarps][kRows][8 * kBlocks + 1];
    pdl_launch_dependents();
    pdl_wait();
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int32_t o0 = blockIdx.x * kOut;
    const uint8_t *w[2], *x[kBlocks];
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows behind the last one are computed and not stored
        w[h] = a.w + (kGated ? static_cast<int64_t>(h) * a.M + min(o0 + g, a.M - 1) : min(o0 + g + 8 * h, a.M - 1)) * a.ldw;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) x[b] = a.x + static_cast<int64_t>(min(8 * b + g, a.rows - 1)) * a.ldx;
    float acc[kBlocks][4] = {};
    // N pieces of 128 bytes, kWarps of them apart; kTail: some bytes may lie behind the rows' end
    auto pieces = [&](int32_t at, auto n, auto tail) {
        constexpr int N = decltype(n)::value;
        constexpr bool kTail = decltype(tail)::value;
        uint4 wq[N][2][2], xq[N][2][kBlocks];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t off = at + i * kWarps * 128 + h * 64 + t * 16;
#pragma unroll
                for (int r = 0; r < 2; ++r) wq[i][h][r] = load16<kSize, true, kTail>(w[r], off, a.k_bytes);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) xq[i][h][b] = load16<kSize, false, kTail>(x[b], off, a.k_bytes);
            }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const uint4 &u = wq[i][h][0], &v = wq[i][h][1], &y = xq[i][h][b];
                    mma<kFp8>(acc[b], u.x, v.x, u.y, v.y, y.x, y.y);
                    mma<kFp8>(acc[b], u.z, v.z, u.w, v.w, y.z, y.w);
                }
    };
    bool some = false;
    auto put = [&] {  // every thread has places of its own
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &s = sums[warp][g + 8 * (i >> 1)][8 * b + 2 * t + (i & 1)];
                s = kLong && some ? s + acc[b][i] : acc[b][i];
                if (kLong) acc[b][i] = 0.0f;
            }
        some = true;
    };
    int32_t at = warp * 128;
    [[maybe_unused]] int32_t held = 0;  // products a row that acc has
    for (; at + (kAhead - 1) * kWarps * 128 + 128 <= a.k_bytes; at += kAhead * kWarps * 128) {
        pieces(at, std::integral_constant<int, kAhead>{}, std::false_type{});
        if (kLong && (held += kAhead * 128 / kSize) >= kSegment) {
            put();
            held = 0;
        }
    }
    for (; at < a.k_bytes; at += kWarps * 128) pieces(at, std::integral_constant<int, 1>{}, std::true_type{});
    put();
    __syncthreads();
    for (int32_t i = threadIdx.x; i < kOut * 8 * kBlocks; i += kThreads) {
        const int32_t m = i % kOut, n = i / kOut, o = o0 + m;
        if (n >= a.rows || o >= a.M) continue;
        float z[2] = {};
#pragma unroll
        for (int p = 0; p < (kGated ? 2 : 1); ++p) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += sums[k][p * kOut + m][n];
            const int32_t wr = p * a.M + o;
            const float bias = a.bias ? __bfloat162float(a.bias[wr]) : 0.0f;
            z[p] = kFp8 ? fmaf(s, a.ep.x_scale[n] * a.ep.w_scale[wr], bias) : s + bias;
        }
        float y = kGated ? silu(z[0]) * z[1] : activation(a.ep.act, z[0]);
        if (a.ep.residual) y = __fadd_rn(y, __bfloat162float(a.ep.residual[static_cast<int64_t>(n) * a.ep.ldr + o]));
        if (a.out_bf16)
            static_cast<__nv_bfloat16 *>(a.out)[static_cast<int64_t>(n) * a.ldo + o] = __float2bfloat16_rn(y);
        else
            static_cast<float *>(a.out)[static_cast<int64_t>(n) * a.ldo + o] = y;
    }
}

}  // namespace

cudaError_t launch_linear_few(bool fp8, const LinearEpilogue &ep, const void *w, int64_t ldw, int32_t M, int32_t K, const void *x,
                              int64_t ldx, int32_t rows, const void *bias, void *out, int64_t ldo, bool out_bf16,
                              int32_t sms, cudaStream_t st) {
    const int32_t es = fp8 ? 1 : 2;
    const bool gated = ep.act == kActSwiglu, two = rows > 8;
    const FewArgs a{rows, M, K * es, static_cast<const uint8_t *>(w), static_cast<const uint8_t *>(x), ldw * es, ldx * es, ep,
                    static_cast<const __nv_bfloat16 *>(bias), out, ldo, out_bf16};
    const int32_t outs = gated ? kRows / 2 : kRows;
    const dim3 grid(static_cast<unsigned>((M + outs - 1) / outs));
    // more blocks than two an SM: smaller ones, whose beginnings and ends fall between the others' loads (32000 rows
    // of 4096 8-bit weights 25.7 -> 22.7 us; but 4096 rows, one wave of larger ones, 5.3 against 3.8)
    const bool wide = static_cast<int64_t>(grid.x) <= 2 * sms;
    auto go = [&](auto eight, auto four) {
        return wide ? launch_pdl(eight, grid, dim3(256), 0, st, a) : launch_pdl(four, grid, dim3(128), 0, st, a);
    };
#define FEW(F, G, N) go(linear_few_kernel<F, G, N, 8>, linear_few_kernel<F, G, N, 4>)
#define LONG(G, N) go(linear_few_kernel<false, G, N, 8, true>, linear_few_kernel<false, G, N, 4, true>)
    if (fp8) {
        if (gated) return two ? FEW(true, true, 2) : FEW(true, true, 1);
        return two ? FEW(true, false, 2) : FEW(true, false, 1);
    }
    if (!out_bf16 && K > (wide ? 8 : 4) * kSegment) {
        if (gated) return two ? LONG(true, 2) : LONG(true, 1);
        return two ? LONG(false, 2) : LONG(false, 1);
    }
    if (gated) return two ? FEW(false, true, 2) : FEW(false, true, 1);
    return two ? FEW(false, false, 2) : FEW(false, false, 1);
#undef LONG
#undef FEW
}

}  // namespace eagle
