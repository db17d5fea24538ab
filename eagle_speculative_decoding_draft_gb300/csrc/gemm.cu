// gemm.cu - host side of the streamed-weight GEMM (gemm.cuh has the kernels): plans, tensor maps, launches;
// and its fp32 form.
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "gemm.cuh"

namespace eagle {
namespace {

// ---------------------------------------------------------------------------------------------
// fp32: one warp per output feature, lanes stride the reduction, 8 rows per pass.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    linear_f32_kernel(const float *__restrict__ w, int64_t ldw, const float *__restrict__ x,
                      int64_t ldx, const float *__restrict__ bias, float *__restrict__ y,
                      int64_t ldy, int32_t M, int32_t K, int32_t rows) {
    pdl_launch_dependents();  // dependents still wait for this grid to finish
    pdl_wait();
    const int32_t o = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    const int32_t lane = threadIdx.x & 31;
    if (o >= M) return;
    const float *wr = w + static_cast<int64_t>(o) * ldw;
    const float b = bias ? bias[o] : 0.0f;
    for (int32_t r0 = 0; r0 < rows; r0 += 8) {
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        for (int32_t i = lane; i < K; i += 32) {
            const float wi = wr[i];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r0 + j < rows) acc[j] = fmaf(wi, x[static_cast<int64_t>(r0 + j) * ldx + i], acc[j]);
        }
        float mine = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = acc[j];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (lane == j) mine = v;
        }
        if (lane < 8 && r0 + lane < rows) y[static_cast<int64_t>(r0 + lane) * ldy + o] = mine + b;
    }
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// A matrix in swizzled boxes, by 64 bytes where a box's rows have 64, else by 128; elements outside it read
// as 0.
bool encode_rows_2d(CUtensorMap *map, uint64_t es, const void *ptr, uint64_t inner, uint64_t outer, uint64_t row_stride_elems,
                    uint32_t box_inner, uint32_t box_outer) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0) return false;
    if ((row_stride_elems * es) % 16 != 0) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_stride_elems * es};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                           : (es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32),
              2, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_inner * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_bf16_2d(CUtensorMap *map, const void *ptr, uint64_t inner, uint64_t outer,
                    uint64_t row_stride_elems, uint32_t box_inner, uint32_t box_outer) {
    return encode_rows_2d(map, 2, ptr, inner, outer, row_stride_elems, box_inner, box_outer);
}

// Gated weights, M gate rows and behind them M up rows, as [2][M][K]: a box is `box_rows` gates and their
// ups.  Gates and ups outside their M rows read as 0.
bool encode_gated(CUtensorMap *map, bool fp8, const void *ptr, uint64_t K, uint64_t M, uint64_t ld, uint32_t box_rows) {
    EncodeTiledFn fn = encoder();
    const uint64_t es = fp8 ? 1 : 2;
    if (!fn || reinterpret_cast<uintptr_t>(ptr) % 16 != 0 || (ld * es) % 16 != 0) return false;
    cuuint64_t dims[3] = {K, M, 2};
    cuuint64_t strides[2] = {ld * es, M * ld * es};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), box_rows, 2};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Y [rows][ldo] (fp32 or bf16) for TMA stores of {box_cols columns, box_rows rows}, no swizzle.
bool encode_out_2d(CUtensorMap *map, const void *ptr, int32_t out_bf16, uint64_t inner, uint64_t outer,
                   uint64_t row_stride_elems, uint32_t box_cols, uint32_t box_rows) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    const uint64_t es = out_bf16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0) return false;
    if ((row_stride_elems * es) % 16 != 0) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {row_stride_elems * es};
    if ((box_cols * es) % 16 != 0 || box_cols > 256 || box_rows > 256 || box_rows < 1) return false;
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
              const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output map of a plan: {128, 32} boxes for the epilogue's 32-row groups.
bool encode_plan_out(LinearPlan *p, const void *out) {
    return encode_out_2d(&p->tmap_y, out, p->out_bf16, static_cast<uint64_t>(p->M), static_cast<uint64_t>(p->rows),
                         static_cast<uint64_t>(p->ldo), p->ep.act == kActSwiglu ? BM / 2 : BM,
                         static_cast<uint32_t>(kGroupRows));
}

}  // namespace

bool encode_bf16_rows_map(CUtensorMap *map, const void *ptr, uint64_t cols, uint64_t rows, uint64_t ld,
                          uint32_t box_cols, uint32_t box_rows) {
    return encode_bf16_2d(map, ptr, cols, rows, ld, box_cols, box_rows);
}

bool encode_swizzled_rows(CUtensorMap *map, int32_t es, const void *ptr, int64_t cols, int64_t rows, int64_t ld,
                          int32_t box_cols, int32_t box_rows) {
    return encode_rows_2d(map, static_cast<uint64_t>(es), ptr, static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                          static_cast<uint64_t>(ld), static_cast<uint32_t>(box_cols), static_cast<uint32_t>(box_rows));
}

bool encode_gated_rows(CUtensorMap *map, int32_t es, const void *ptr, int64_t cols, int64_t rows, int64_t ld, int32_t box_rows) {
    return encode_gated(map, es == 1, ptr, static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(ld),
                        static_cast<uint32_t>(box_rows));
}

bool encode_kv_cache_map(CUtensorMap *map, const void *cache, int32_t B, int32_t P, int32_t Hk, int32_t D) {
    EncodeTiledFn fn = encoder();
    if (!fn || B < 1 || P < 1 || Hk < 1 || (D != 64 && D != 128)) return false;
    if (reinterpret_cast<uintptr_t>(cache) % 16 != 0) return false;
    // [B][P][Hk][D] bf16 as dims (D, Hk, P, B); one box is 64 head dims of one kv head for 64 keys
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hk), static_cast<cuuint64_t>(P),
                          static_cast<cuuint64_t>(B)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hk) * D * 2,
                             static_cast<cuuint64_t>(P) * Hk * D * 2};
    cuuint32_t box[4] = {64, 1, 64, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int32_t linear_n_tile(int32_t rows) { return ((rows + 15) / 16) * 16; }

size_t linear_partials_bytes(int32_t grid, int32_t n_tile) {
    return static_cast<size_t>(grid) * 2 * n_tile * BM * sizeof(float);
}

size_t linear_counters_bytes(int32_t M, int32_t rows) {
    const int64_t chunks = (static_cast<int64_t>(rows < 1 ? 1 : rows) + kLinearMaxRows - 1) / kLinearMaxRows;
    return static_cast<size_t>((M + BM - 1) / BM) * static_cast<size_t>(chunks) * sizeof(int32_t);
}

bool plan_linear_bf16(LinearPlan *p, const void *w, int64_t ldw, int32_t M, int32_t K, const void *x,
                      int64_t ldx, int32_t rows, const void *bias, void *out, int64_t ldo,
                      int32_t out_bf16, float *partials, int32_t *counters, int32_t *status,
                      int32_t num_sms) {
    if (!plan_linear(p, false, LinearEpilogue{}, w, ldw, M, K, x, ldx, rows, bias, out, ldo, out_bf16, partials, counters,
                     status, num_sms))
        return false;
    p->form = 0;
    return true;
}

bool plan_linear(LinearPlan *p, bool fp8, const LinearEpilogue &ep, const void *w, int64_t ldw, int32_t M, int32_t K,
                 const void *x, int64_t ldx, int32_t rows, const void *bias, void *out, int64_t ldo, int32_t out_bf16,
                 float *partials, int32_t *counters, int32_t *status, int32_t num_sms) {
    const bool gated = ep.act == kActSwiglu;
    const int32_t BK = fp8 ? k_block<EpilogueOp<true, false>>() : k_block<PlainOp>(), cols = gated ? BM / 2 : BM;
    p->form = 1 + (fp8 ? 1 : 0) + (gated ? 2 : 0);
    p->ep = ep;
    if (M < 1 || K < 1 || rows < 1 || rows > kLinearMaxLaunchRows || num_sms < 1) return false;
    if (ldw < K || ldx < K || ldo < M) return false;
    p->M = M;
    p->K = K;
    p->rows = rows;
    // more rows than one MMA's N: chunks of kLinearMaxRows rows, each a unit of the split with
    // every weight tile
    p->num_chunks = (rows + kLinearMaxRows - 1) / kLinearMaxRows;
    p->n_tile = linear_n_tile(rows < kLinearMaxRows ? rows : kLinearMaxRows);
    p->num_kb = (K + BK - 1) / BK;
    p->num_tiles = (M + cols - 1) / cols;
    const int64_t total = static_cast<int64_t>(p->num_kb) * p->num_tiles * p->num_chunks;
    p->grid = static_cast<int32_t>(total < num_sms ? total : num_sms);
    // CTA pairs (.cta_group::2) for stream-K above 16 rows when the tiles pair up: the split runs
    // over pairs of adjacent tiles and the grid is twice the pairs
    p->pair = 0;
    p->num_wtiles = p->num_tiles;
    if (rows > kLinearMaxFixupRows && p->num_tiles % 2 == 0) {
        const int32_t pairs = linear_pair_workers(num_sms);
        if (pairs > 0) {
            p->pair = 1;
            p->num_wtiles = p->num_tiles / 2;
            const int64_t total_w = static_cast<int64_t>(p->num_kb) * p->num_wtiles * p->num_chunks;
            p->grid = 2 * static_cast<int32_t>(total_w < pairs ? total_w : pairs);
        }
    }
    const size_t stage_bytes = kABytes + static_cast<size_t>(p->n_tile >> p->pair) * 128;
    // above 16 rows (stream-K), outputs and partials leave in 32-row groups by bulk stores
    const bool want_y_tma = rows > kLinearMaxFixupRows;
    p->out_stage_bytes = want_y_tma ? static_cast<int32_t>(kOutStageBytes) : 0;
    size_t stages = (kMaxDynSmem - 1024 - sizeof(SmemCtl) - p->out_stage_bytes) / stage_bytes;
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages < 2) return false;
    p->stages = static_cast<int32_t>(stages);
    p->smem_bytes = 1024 + stages * stage_bytes + p->out_stage_bytes + sizeof(SmemCtl);
    int32_t tmem_cols = 32;
    while (tmem_cols < 2 * p->n_tile) tmem_cols *= 2;
    p->tmem_cols = tmem_cols;
    p->bias = bias;
    p->out = out;
    p->ldo = ldo;
    p->out_bf16 = out_bf16;
    // Many rows: one CTA per tile cannot sum the partials fast enough (it reads CTAs x rows x 128
    // floats); a separate launch spreads the sum over tiles x row blocks.
    // Above 16 rows, split tiles are summed inside the launch when every CTA covers at least a
    // whole tile's k-blocks (then a tile is shared by at most two CTAs, and the one that reaches
    // it at the end of its range finds the other's partial in and owns the sum), else by a
    // second launch.
    const int64_t per_cta =  // fewest of any worker
        static_cast<int64_t>(p->num_kb) * p->num_wtiles * p->num_chunks / (p->grid >> p->pair);
    p->owner_fix = (rows > kLinearMaxFixupRows && per_cta >= p->num_kb) ? 1 : 0;
    p->defer = (rows > kLinearMaxFixupRows && !p->owner_fix) ? 1 : 0;
    p->partials = partials;
    p->counters = counters;
    p->status = status;
    if (gated ? !encode_gated(&p->tmap_w, fp8, w, static_cast<uint64_t>(K), static_cast<uint64_t>(M),
                              static_cast<uint64_t>(ldw), 16)
              : !encode_rows_2d(&p->tmap_w, fp8 ? 1 : 2, w, static_cast<uint64_t>(K), static_cast<uint64_t>(M),
                                static_cast<uint64_t>(ldw), BK, BM))
        return false;
    p->y_tma = (want_y_tma && encode_plan_out(p, out)) ? 1 : 0;
    if (!encode_rows_2d(&p->tmap_x, fp8 ? 1 : 2, x, static_cast<uint64_t>(K), static_cast<uint64_t>(rows),
                        static_cast<uint64_t>(ldx), BK, static_cast<uint32_t>(p->n_tile >> p->pair)))
        return false;
    return true;
}

// CTA pairs that can be resident at once (clusters of 2 with the largest shared-memory request),
// at most half the SMs; 0 disables pairs (also when EAGLE_LINEAR_PAIR=0 is set in the
// environment, to compare the two ways).  Checked once per device.
int32_t linear_pair_workers(int32_t num_sms) {
    static std::mutex mu;
    static int cached[64] = {};  // 0 unknown, else max active pair clusters + 1
    static const bool disabled = [] {
        const char *e = std::getenv("EAGLE_LINEAR_PAIR");
        return e != nullptr && e[0] == '0';
    }();
    if (disabled) return 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (prepare_kernels() != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kMaxDynSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, linear_tc_kernel<1, PlainOp>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        cached[dev] = n + 1;
    }
    const int32_t n = cached[dev] - 1;
    return n < num_sms / 2 ? n : num_sms / 2;
}

cudaError_t prepare_kernels() {
    cudaError_t e = cudaFuncSetAttribute(linear_tc_kernel<0, PlainOp>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kMaxDynSmem));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(linear_tc_kernel<1, PlainOp>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kMaxDynSmem));
}

void linear_retarget_out(LinearPlan *p, void *out) {
    p->out = out;
    if (p->y_tma) p->y_tma = encode_plan_out(p, out) ? 1 : 0;
}

cudaError_t launch_linear_bf16(const LinearPlan &p, cudaStream_t st) {
    LinearArgs a;
    a.M = p.M;
    a.K = p.K;
    a.rows = p.rows;
    a.n_tile = p.n_tile;
    a.num_kb = p.num_kb;
    a.num_tiles = p.num_tiles;
    a.stages = p.stages;
    a.tmem_cols = p.tmem_cols;
    a.bias = reinterpret_cast<const __nv_bfloat16 *>(p.bias);
    a.out = p.out;
    a.ldo = p.ldo;
    a.out_bf16 = p.out_bf16;
    a.defer = p.defer;
    a.owner_fix = p.owner_fix;
    a.pair = p.pair;
    a.num_wtiles = p.num_wtiles;
    a.num_chunks = p.num_chunks;
    a.slots = 2 * p.grid;
    a.y_tma = p.y_tma;
    a.out_stage_bytes = p.out_stage_bytes;
    a.partials = p.partials;
    a.counters = p.counters;
    a.status = p.status;
    a.ep = p.ep;
    return p.form == 0 ? launch_form<PlainOp>(p, a, st) : launch_linear_form(p, a, st);
}

cudaError_t launch_linear_f32(const float *w, int64_t ldw, const float *x, int64_t ldx,
                              const float *bias, float *y, int64_t ldy, int32_t M, int32_t K,
                              int32_t rows, cudaStream_t st) {
    if (M < 1 || rows < 1) return cudaSuccess;
    const int warps = 8;
    return launch_pdl(linear_f32_kernel, dim3((M + warps - 1) / warps), dim3(warps * 32), 0, st, w, ldw, x,
                      ldx, bias, y, ldy, M, K, rows);
}

}  // namespace eagle
