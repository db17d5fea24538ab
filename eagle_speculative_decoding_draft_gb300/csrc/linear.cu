// linear.cu - the streamed-weight product with an epilogue: the kernels of gemm.cuh's forms for bf16 and for
// 8-bit (e4m3) operands, plain and gated, and their entry point.
//
// A draft layer's products are followed by what is small next to them: the operands' scales, a bias, an
// activation, the residual's addition.  Done on the accumulator they cost no pass over memory.
#include <mutex>

#include "../../include/eagle_tree.h"
#include "gemm.cuh"

namespace eagle {
namespace {

// Latches the waits that run out in calls without a status word of the caller's.
__device__ int32_t g_status;

template <class Op>
cudaError_t prepare_form() {
    cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<0, Op>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kMaxDynSmem));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(linear_tc_kernel<1, Op>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kMaxDynSmem));
}

}  // namespace

// SMs of the current device, 0 where they cannot be read or are more than the tickets count.
int32_t linear_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms <= static_cast<int>(kLinearTicketBytes / 4) ? sms : 0;
}

size_t linear_workspace(int32_t rows, int32_t sms) {
    return kLinearTicketBytes + linear_partials_bytes(sms, linear_n_tile(rows < kLinearMaxRows ? rows : kLinearMaxRows));
}

cudaError_t prepare_linear_forms(int32_t **status_word) {
    static std::mutex mu;
    static int32_t *words[64] = {};  // null: not prepared yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    *status_word = words[dev];
    if (*status_word) return cudaSuccess;
    e = prepare_kernels();
    if (e == cudaSuccess) e = prepare_form<EpilogueOp<false, false>>();
    if (e == cudaSuccess) e = prepare_form<EpilogueOp<true, false>>();
    if (e == cudaSuccess) e = prepare_form<EpilogueOp<false, true>>();
    if (e == cudaSuccess) e = prepare_form<EpilogueOp<true, true>>();
    if (e == cudaSuccess) e = prepare_linear_mid();
    if (e == cudaSuccess) e = prepare_linear_tiles();
    void *word = nullptr;
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&word, g_status);
    if (e == cudaSuccess) *status_word = words[dev] = static_cast<int32_t *>(word);
    return e;
}

cudaError_t launch_linear_form(const LinearPlan &p, const LinearArgs &a, cudaStream_t st) {
    switch (p.form) {
        case 1: return launch_form<EpilogueOp<false, false>>(p, a, st);
        case 2: return launch_form<EpilogueOp<true, false>>(p, a, st);
        case 3: return launch_form<EpilogueOp<false, true>>(p, a, st);
        case 4: return launch_form<EpilogueOp<true, true>>(p, a, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_linear(bool fp8, const LinearEpilogue &ep, const void *w, int64_t ldw, int32_t M, int32_t K, const void *x,
                          int64_t ldx, int32_t rows, const void *bias, void *y, int64_t ldy, bool y_bf16, void *ws, int32_t *status,
                          int32_t sms, cudaStream_t st) {
    if (rows <= kLinearFewRows) return launch_linear_few(fp8, ep, w, ldw, M, K, x, ldx, rows, bias, y, ldy, y_bf16, sms, st);
    int32_t *own = nullptr;
    cudaError_t e = prepare_linear_forms(&own);
    if (e != cudaSuccess) return e;
    if (!status) status = own;
    // Over 128 rows the tensor cores bound the product, or nearly so: whole tiles of both operands (256 rows,
    // 4096 -> 2 x 11008 in 8 bits: 30 us, and 43 with the weights past 128 rows at a time; 128 rows: 29 and 22).  But
    // where tiles of 128 rows of either leave room for four parts of K each, those are quicker still (256 rows, 4096
    // -> 4096 in 8 bits: 12.2 us against 13.1, 14336 -> 4096 21.8 against 25.4, in bf16 34 against 42; 1024 rows,
    // 14336 -> 1024: 20 against 24; but 384 rows, 4096 -> 4096, three parts' room: 15.5 against 14.2).
    // Outputs that no bulk store takes go through linear_mid.cu in chunks of 128 rows, or through the weights' stream
    // where there is a workspace for it, the weights have more tiles than the device SMs and the rows eight chunks
    // (2080 and 8192 rows, 4096 -> 31999: 390 and 1430 us in chunks, 290 and 1020 in the stream, in bf16 700 and 2610,
    // 460 and 1750; but 2080 rows, 4096 -> 4095: 38 and 64, 1024 -> 1001 9 and 23; 600 rows, 4096 -> 31999: 115 and
    // 112, 4096 -> 2 x 14335: 91 and 105).
    const int32_t cols = ep.act == kActSwiglu ? 64 : 128;
    const int64_t w_tiles = (M + cols - 1) / cols, small = w_tiles * ((rows + 127) / 128);
    const bool mid = rows <= kLinearMidRows || (2 * small <= sms && static_cast<int64_t>(K) * (fp8 ? 1 : 2) >= 1024);
    if (!mid) {
        const int32_t pairs = linear_pair_workers(sms);
        if (pairs > 0 && launch_linear_tiles(fp8, ep, w, ldw, M, K, x, ldx, rows, bias, y, ldy, y_bf16, status, pairs, st, &e)) return e;
    }
    const bool stream = ws && w_tiles > sms && rows > 1024 && (fp8 || y_bf16 || K <= 4096);  // (it has no parts for long sums)
    if (!stream)
        return launch_linear_mid(fp8, ep, w, ldw, M, K, x, ldx, rows, bias, y, ldy, y_bf16, status, sms, st, &e) ? e : cudaErrorInvalidValue;
    LinearPlan p;
    if (!plan_linear(&p, fp8, ep, w, ldw, M, K, x, ldx, rows, bias, y, ldy, y_bf16,
                     reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kLinearTicketBytes), static_cast<int32_t *>(ws), status, sms))
        return cudaErrorInvalidValue;
    return launch_linear_bf16(p, st);
}

}  // namespace eagle

extern "C" {

size_t eagle_linear_epilogue_workspace_bytes(int32_t rows) {
    const int32_t sms = eagle::linear_sms();
    if (rows < 1 || rows > eagle::kLinearMaxLaunchRows || sms < 1) return 0;
    return eagle::linear_workspace(rows, sms);
}

eagle_status eagle_linear(const eagle_linear_args *l, void *d_ws, size_t ws_bytes, int32_t *d_status,
                          eagle_stream_t stream) {
    using namespace eagle;
    NvtxRange nvtx_range("eagle_linear");
    if (!l || l->rows < 0 || l->rows > kLinearMaxLaunchRows || l->in_features < 1 || l->out_features < 1)
        return EAGLE_ERR_INVALID_ARG;
    if (l->dtype != EAGLE_BF16 && l->dtype != EAGLE_E4M3) return EAGLE_ERR_INVALID_ARG;
    if (l->y_dtype != EAGLE_BF16 && l->y_dtype != EAGLE_F32) return EAGLE_ERR_INVALID_ARG;
    if (l->act < EAGLE_ACT_NONE || l->act > EAGLE_ACT_SWIGLU) return EAGLE_ERR_INVALID_ARG;
    if (l->rows == 0) return EAGLE_OK;
    const bool fp8 = l->dtype == EAGLE_E4M3;
    const int32_t M = l->out_features, K = l->in_features, step = fp8 ? 16 : 8;
    if (M > (1 << 28) || K > (1 << 28)) return EAGLE_ERR_INVALID_ARG;
    auto off = [](const void *p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; };
    if (!l->w || !l->x || !l->y) return EAGLE_ERR_INVALID_ARG;
    if (fp8 != (l->w_scale != nullptr) || fp8 != (l->x_scale != nullptr)) return EAGLE_ERR_INVALID_ARG;
    if (off(l->w, 16) || off(l->x, 16) || off(l->w_scale, 4) || off(l->x_scale, 4) || off(l->bias, 2) || off(l->residual, 2))
        return EAGLE_ERR_INVALID_ARG;
    if (off(l->y, l->y_dtype == EAGLE_F32 ? 4 : 2) || off(d_ws, 256) || off(d_status, 4)) return EAGLE_ERR_INVALID_ARG;
    if (l->ldw < K || l->ldx < K || l->ldw % step || l->ldx % step || l->ldy < M || (l->residual && l->ldr < M))
        return EAGLE_ERR_INVALID_ARG;
    if (d_ws && ws_bytes < kLinearTicketBytes) return EAGLE_ERR_INVALID_ARG;
    const int32_t sms = linear_sms();
    if (sms < 1) return EAGLE_ERR_CUDA;
    if (d_ws && ws_bytes < linear_workspace(l->rows, sms)) return EAGLE_ERR_INVALID_ARG;
    const LinearEpilogue ep{l->x_scale, l->w_scale, static_cast<const __nv_bfloat16 *>(l->residual), l->ldr,
                            static_cast<int32_t>(l->act)};
    const cudaError_t e = launch_linear(fp8, ep, l->w, l->ldw, M, K, l->x, l->ldx, l->rows, l->bias, l->y, l->ldy,
                                        l->y_dtype == EAGLE_BF16, d_ws, d_status, sms, reinterpret_cast<cudaStream_t>(stream));
    // a row stride or a size that a tensor map does not hold
    return e == cudaSuccess ? EAGLE_OK : (e == cudaErrorInvalidValue ? EAGLE_ERR_UNSUPPORTED : EAGLE_ERR_CUDA);
}

int32_t *eagle_linear_status_word(void) {
    int32_t *word = nullptr;
    return eagle::prepare_linear_forms(&word) == cudaSuccess ? word : nullptr;
}

eagle_status eagle_linear_status(eagle_stream_t stream) {
    int32_t *d_word = eagle_linear_status_word();
    if (!d_word) return EAGLE_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int32_t word = 0;
    if (cudaMemcpyAsync(&word, d_word, sizeof(int32_t), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    if (word == 0) return EAGLE_OK;
    if (cudaMemsetAsync(d_word, 0, sizeof(int32_t), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    return (word & eagle::kDevTimeout) ? EAGLE_ERR_DEVICE_TIMEOUT : EAGLE_ERR_DEVICE_BOUNDS;
}

}  // extern "C"
