// norm.cu - the rows that go into a product: the residual's addition and the root-mean-square norm, in bf16
// or in 8 bits with one scale a row, and rows quantised as they are.
//
//   h = x + residual,  y = w h / sqrt(mean(h^2) + eps)
//   s = max(max |y| / 448, 2^-100),  c = y / s rounded to the nearest e4m3 value, ties to even
//
// A row is read once and stays in registers.  Its norm is one factor r = 1 / sqrt(...), so the largest |y| is
// r max |w h|, and one reduction over the row finds the sum of squares and that maximum together.  Bound by the
// memory: 16382 rows of 8192 with their residual (1.07 GB) in 152 us, 1.04 of the measured copy rate; 2080 rows
// of 14336 quantised (89 MB) in 15.1 us, 0.87, with the quotients two at a time (one at a time 19.3); 512 rows of 4096
// with their residual to 8 bits 4.1 us (0.53: a launch's beginning and end).
#include <cuda_fp8.h>

#include "../../include/eagle_tree.h"
#include "common.cuh"
#include "kernels.cuh"

namespace eagle {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr float kTop = 448.0f;            // the largest e4m3 value
constexpr float kLeast = 7.888609e-31f;   // 2^-100
constexpr int32_t kMaxCols = 32768;

struct RowArgs {
    int32_t rows, n;
    int64_t ldx, ldr, lds, ldy;
    const __nv_bfloat16 *x, *residual, *w;
    __nv_bfloat16 *sum;
    void *y;       // bf16 or e4m3
    float *scale;  // [rows], 8-bit rows
    float eps;
};

__device__ __forceinline__ void unpack8(const uint4 &q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Elements e .. e + 7 of a row of n; those behind its end are 0 and are not read.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p, int32_t e, int32_t n) {
    if (e + 8 <= n) return *reinterpret_cast<const uint4 *>(p + e);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (e + i < n) w[i >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[e + i])) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int32_t e, int32_t n, const uint4 &q) {
    if (e + 8 <= n) {
        *reinterpret_cast<uint4 *>(p + e) = q;
        return;
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (e + i < n) p[e + i] = __ushort_as_bfloat16(static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1))));
}

// The scale of a row whose largest magnitude is `amax`; NaN where that is none or infinite.
__device__ __forceinline__ float row_scale(float amax) {
    return amax <= 3.4028235e38f ? fmaxf(__fdiv_rn(amax, kTop), kLeast) : __int_as_float(0x7fffffff);
}
__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// The codes of two values: their quotients by the scale, to the nearest fp32 value, then to the nearest code.  A
// quotient is a product with the reciprocal, corrected once (P. Markstein, IBM J. Res. Dev. 34, 1990), two at a
// time: bf16 values over a bf16 maximum often lie on a tie between two codes, where the last bit decides.
struct Quotient {
    uint64_t inv2, minus2;
    __device__ __forceinline__ Quotient(float s, float inv) : inv2(pack_2(inv, inv)), minus2(pack_2(-s, -s)) {}
    __device__ __forceinline__ uint32_t codes(uint64_t v) const {
        const uint64_t q = mul_2(v, inv2);
        const float2 c = unpack_2(fma_2(fma_2(q, minus2, v), inv2, q));
        return e4m3_pair(c.x, c.y);
    }
};
// Codes e .. e + 7 of a row of n.
__device__ __forceinline__ void store_codes(uint8_t *y, int32_t e, int32_t n, const uint32_t (&w)[2]) {
    if (e + 8 <= n) {
        *reinterpret_cast<uint2 *>(y + e) = make_uint2(w[0], w[1]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (e + k < n) y[e + k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
}

// A row a blockDim.x threads (blockDim.y rows a block, where a row is one warp's), V pieces of 8 elements a
// thread, blockDim.x pieces apart.
template <int V>
constexpr int max_threads() { return V < 4 ? 1024 : 512; }  // 64 registers a thread, or 128

template <int V, bool kFp8>
__global__ void __launch_bounds__(max_threads<V>()) norm_kernel(const RowArgs a) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    pdl_launch_dependents();
    pdl_wait();
    const int32_t row = static_cast<int32_t>(blockIdx.x * blockDim.y + threadIdx.y), t = threadIdx.x, T = blockDim.x;
    if (row >= a.rows) return;  // whole warps, and only where a row is a warp's
    const __nv_bfloat16 *x = a.x + row * a.ldx, *res = a.residual ? a.residual + row * a.ldr : nullptr;
    uint4 xq[V], rq[V], wq[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = (t + i * T) * 8;
        xq[i] = load8(x, e, a.n);
        if (res) rq[i] = load8(res, e, a.n);
        if (V < 8) wq[i] = load8(a.w, e, a.n);
    }
    float h[V][8];
    float ss = 0.0f;
    uint32_t top = 0;  // bits of the largest |w h|: a NaN's are above an infinity's, and those above all others
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = (t + i * T) * 8;
        unpack8(xq[i], h[i]);
        if (res) {
            float r[8];
            unpack8(rq[i], r);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] += r[k];
            if (a.sum && e < a.n) store8(a.sum + row * a.lds, e, a.n, pack8(h[i]));
        }
        float w[8];
        unpack8(V < 8 ? wq[i] : load8(a.w, e, a.n), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ss = fmaf(h[i][k], h[i][k], ss);
            h[i][k] *= w[k];
        }
        if (kFp8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(h[i][k]) & 0x7fffffffu);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    if (kFp8) top = __reduce_max_sync(kFull, top);
    if (T > 32) {
        if ((t & 31) == 0) {
            s_sum[t >> 5] = ss;
            s_max[t >> 5] = top;
        }
        __syncthreads();
        // every warp adds up the warps' sums the same way
        const int32_t lane = t & 31, warps = T >> 5;
        ss = lane < warps ? s_sum[lane] : 0.0f;
        top = lane < warps ? s_max[lane] : 0u;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        if (kFp8) top = __reduce_max_sync(kFull, top);
    }
    const float r = rsqrtf(ss / static_cast<float>(a.n) + a.eps);
    if constexpr (kFp8) {
        // two factors: with an eps near 0, r / s passes fp32 where the row is nothing and s its least value
        const float s = row_scale(__uint_as_float(top) * r), inv = __frcp_rn(s);
        if (t == 0) a.scale[row] = s;
        const uint64_t r2 = pack_2(r, r);
        const Quotient by(s, inv);
        uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t e = (t + i * T) * 8;
            if (e >= a.n) break;
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 8; k += 2) w[k >> 2] |= by.codes(mul_2(pack_2(h[i][k], h[i][k + 1]), r2)) << (8 * (k & 3));
            store_codes(y, e, a.n, w);
        }
    } else {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t e = (t + i * T) * 8;
            if (e >= a.n) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] *= r;
            store8(y, e, a.n, pack8(h[i]));
        }
    }
}

// Rows as they are, by the same threads.  The magnitudes of bf16 values rank as whole numbers do, two to a
// word.
template <int V>
__global__ void __launch_bounds__(max_threads<V>()) quantize_kernel(const RowArgs a) {
    __shared__ uint32_t s_max[32];
    pdl_launch_dependents();
    pdl_wait();
    const int32_t row = static_cast<int32_t>(blockIdx.x * blockDim.y + threadIdx.y), t = threadIdx.x, T = blockDim.x;
    if (row >= a.rows) return;  // whole warps, and only where a row is a warp's
    const __nv_bfloat16 *x = a.x + row * a.ldx;
    uint4 xq[V];
#pragma unroll
    for (int i = 0; i < V; ++i) xq[i] = load8(x, (t + i * T) * 8, a.n);
    uint32_t two = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t w[4] = {xq[i].x, xq[i].y, xq[i].z, xq[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) two = __vmaxu2(two, w[k] & 0x7fff7fffu);
    }
    uint32_t top = __reduce_max_sync(kFull, max(two << 16, two & 0xffff0000u));
    if (T > 32) {
        if ((t & 31) == 0) s_max[t >> 5] = top;
        __syncthreads();
        top = __reduce_max_sync(kFull, (t & 31) < (T >> 5) ? s_max[t & 31] : 0u);
    }
    const float s = row_scale(__uint_as_float(top));
    if (t == 0) a.scale[row] = s;
    const Quotient by(s, __frcp_rn(s));
    uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t e = (t + i * T) * 8;
        if (e >= a.n) break;
        const uint32_t w[4] = {xq[i].x, xq[i].y, xq[i].z, xq[i].w};
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k >> 1] |= by.codes(pack_2(w[k] << 16, w[k] & 0xffff0000u)) << (16 * (k & 1));
        store_codes(y, e, a.n, c);
    }
}

template <int V>
cudaError_t launch_rows_v(const RowArgs &a, bool norm, bool fp8, dim3 grid, dim3 block, cudaStream_t st) {
    if (!norm) return launch_pdl(quantize_kernel<V>, grid, block, 0, st, a);
    if (fp8) return launch_pdl(norm_kernel<V, true>, grid, block, 0, st, a);
    return launch_pdl(norm_kernel<V, false>, grid, block, 0, st, a);
}

cudaError_t launch_rows(const RowArgs &a, bool norm, bool fp8, cudaStream_t st) {
    const int32_t pieces = (a.n + 7) / 8;
    // few rows: as many threads a row as it has pieces, up to 1024; many: four pieces a thread, so that an SM holds
    // several rows at once (2080 rows of 14336 quantised with 1, 2, 4 and 8: 17.9, 18.1, 15.7 and 16.4 us; 16382
    // rows of 8192 normed in bf16: 163, 159, 153 and 163)
    int32_t V = 1;
    dim3 block, grid;
    if (pieces <= 128) {  // a warp a row
        while (32 * V < pieces) V *= 2;
        block = dim3(32, 4);
        grid = dim3(static_cast<unsigned>((a.rows + 3) / 4));
    } else {
        while (pieces > (V < 4 ? 1024 : 512) * V) V *= 2;
        if (a.rows >= 512)
            while (V < 4 && pieces > 128 * V) V *= 2;
        block = dim3(static_cast<unsigned>(((pieces + V - 1) / V + 31) / 32 * 32));
        grid = dim3(static_cast<unsigned>(a.rows));
    }
    if (V == 1) return launch_rows_v<1>(a, norm, fp8, grid, block, st);
    if (V == 2) return launch_rows_v<2>(a, norm, fp8, grid, block, st);
    if (V == 4) return launch_rows_v<4>(a, norm, fp8, grid, block, st);
    return launch_rows_v<8>(a, norm, fp8, grid, block, st);
}

bool off(const void *p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; }

}  // namespace

cudaError_t launch_quantize_rows(const void *x, int64_t ldx, int32_t rows, int32_t n, void *y, int64_t ldy, float *scale,
                                 cudaStream_t st) {
    RowArgs a{};
    a.rows = rows;
    a.n = n;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.ldx = ldx;
    a.y = y;
    a.ldy = ldy;
    a.scale = scale;
    return launch_rows(a, false, true, st);
}

cudaError_t launch_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w, float eps,
                            int32_t rows, int32_t n, void *sum, int64_t lds, void *y, int64_t ldy, float *scale,
                            cudaStream_t st) {
    RowArgs a{};
    a.rows = rows;
    a.n = n;
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.ldx = ldx;
    a.residual = static_cast<const __nv_bfloat16 *>(residual);
    a.ldr = ldr;
    a.w = static_cast<const __nv_bfloat16 *>(w);
    a.eps = eps;
    a.sum = static_cast<__nv_bfloat16 *>(sum);
    a.lds = lds;
    a.y = y;
    a.ldy = ldy;
    a.scale = scale;
    return launch_rows(a, true, scale != nullptr, st);
}

}  // namespace eagle

extern "C" {

eagle_status eagle_rms_norm(const void *d_x, int64_t ldx, const void *d_residual, int64_t ldr, const void *d_weight,
                            float eps, int32_t rows, int32_t cols, void *d_sum, int64_t lds, eagle_dtype y_dtype,
                            void *d_y, int64_t ldy, float *d_scale, eagle_stream_t stream) {
    using namespace eagle;
    NvtxRange nvtx_range("eagle_rms_norm");
    if (rows < 0 || cols < 1 || !(eps >= 0.0f)) return EAGLE_ERR_INVALID_ARG;
    if (y_dtype != EAGLE_BF16 && y_dtype != EAGLE_E4M3) return EAGLE_ERR_INVALID_ARG;
    const bool fp8 = y_dtype == EAGLE_E4M3;
    if (ldx < cols || ldx % 8 || ldy < cols || ldy % (fp8 ? 16 : 8)) return EAGLE_ERR_INVALID_ARG;
    if (d_residual && (ldr < cols || ldr % 8)) return EAGLE_ERR_INVALID_ARG;
    if (d_sum && (!d_residual || lds < cols || lds % 8)) return EAGLE_ERR_INVALID_ARG;
    if (fp8 != (d_scale != nullptr)) return EAGLE_ERR_INVALID_ARG;
    if (cols > kMaxCols) return EAGLE_ERR_UNSUPPORTED;
    if (rows == 0) return EAGLE_OK;
    if (!d_x || !d_weight || !d_y) return EAGLE_ERR_INVALID_ARG;
    if (off(d_x, 16) || off(d_residual, 16) || off(d_weight, 16) || off(d_sum, 16) || off(d_y, 16) || off(d_scale, 4))
        return EAGLE_ERR_INVALID_ARG;
    return launch_rms_norm(d_x, ldx, d_residual, ldr, d_weight, eps, rows, cols, d_sum, lds, d_y, ldy, d_scale,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}

eagle_status eagle_quantize_rows(const void *d_x, int64_t ldx, int32_t rows, int32_t cols, void *d_y, int64_t ldy,
                                 float *d_scale, eagle_stream_t stream) {
    using namespace eagle;
    NvtxRange nvtx_range("eagle_quantize_rows");
    if (rows < 0 || cols < 1 || ldx < cols || ldx % 8 || ldy < cols || ldy % 16) return EAGLE_ERR_INVALID_ARG;
    if (cols > kMaxCols) return EAGLE_ERR_UNSUPPORTED;
    if (rows == 0) return EAGLE_OK;
    if (!d_x || !d_y || !d_scale || off(d_x, 16) || off(d_y, 16) || off(d_scale, 4)) return EAGLE_ERR_INVALID_ARG;
    return launch_quantize_rows(d_x, ldx, rows, cols, d_y, ldy, d_scale, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}

}  // extern "C"
