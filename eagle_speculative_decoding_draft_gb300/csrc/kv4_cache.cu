// kv4_cache.cu - writing the 4-bit key/value cache and reading it back.
//
// The engine's decoder layer hands out the keys and values of a tree's nodes; after the verify the
// accepted path's rows join the cache, in 4 bits, at the request's next positions (a prompt's rows
// in order, a path's rows through the list of its nodes).  kv4.cuh has the format.
#include "kernels.cuh"
#include "kv4.cuh"

namespace eagle {

bool kv4_view(const eagle_kv4_cache *c, Kv4View *out) {
    if (!c || c->kv_heads < 1 || c->kv_heads > 1024) return false;
    if (c->head_dim < 32 || c->head_dim > 128 || c->head_dim % 32) return false;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return false;
    if (c->num_pages < 1 || c->max_pages < 1) return false;
    if (static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t{1} << 30)) return false;
    if (!c->pages || !c->table || !c->lengths) return false;
    if (reinterpret_cast<uintptr_t>(c->pages) & 15u) return false;
    if ((reinterpret_cast<uintptr_t>(c->table) | reinterpret_cast<uintptr_t>(c->lengths)) & 3u) return false;
    int32_t shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    *out = Kv4View{static_cast<uint8_t *>(c->pages), c->table, c->lengths, c->kv_heads, c->head_dim / kKv4Group,
                   shift, c->num_pages, c->max_pages, static_cast<int64_t>(c->max_pages) << shift};
    return true;
}

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    Kv4View v;
    int32_t B, src_rows, slots, blocks, slots_block;
    const __nv_bfloat16 *k, *w;  // keys and values [B][src_rows] rows of ld elements
    int64_t ld;
    const int32_t *select;       // [B][slots] or null
    const int32_t *count;        // [B] or null
    const int32_t *start;        // [B]
    int32_t *lengths;            // written by this kernel, or null (by kv4_lengths_kernel)
    int32_t *status;
};

__device__ __forceinline__ int32_t slots_of(const AppendArgs &a, int32_t b) {
    return a.count ? min(max(a.count[b], 0), a.slots) : a.slots;
}

// Eight values of a group of 32 that four neighbouring lanes hold: their codes (the first in the
// low bits) and the group's (s, m).
__device__ __forceinline__ uint32_t quantise8(const uint4 raw, uint32_t *params) {
    float x[8];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    float lo = x[0], hi = x[0];
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        ok = ok && fabsf(x[i]) <= kKv4MaxAbs;  // false for NaN
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        ok = __shfl_xor_sync(0xffffffffu, static_cast<int>(ok), off) && ok;
    }
    if (!ok) {
        *params = 0x7fff7fffu;
        return 0;
    }
    const __half m = __float2half_rd(lo);
    const float mf = __half2float(m);
    const __half s = __float2half_ru(__fdiv_rn(hi - mf, 15.0f));
    const float sf = __half2float(s);
    *params = static_cast<uint32_t>(__half_as_ushort(s)) | (static_cast<uint32_t>(__half_as_ushort(m)) << 16);
    if (sf == 0.0f) return 0;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = rintf(__fdiv_rn(x[i] - mf, sf));
        codes |= static_cast<uint32_t>(min(static_cast<int32_t>(c), 15)) << (4 * i);
    }
    return codes;
}

// Block (request, run of slots): a thread takes 8 dims of a key row and the same 8 of the value
// row (16 bytes each), so four lanes make a group and consecutive lanes read consecutive memory.
// Bound by memory: 4 bytes a value pair in, 1.25 out.
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const AppendArgs a) {
    __shared__ int32_t s_last;
    pdl_launch_dependents();
    pdl_wait();
    const int32_t b = blockIdx.x / a.blocks, part = blockIdx.x - b * a.blocks;
    const int64_t start = a.start[b];
    const int32_t cnt = slots_of(a, b);
    if (start < 0) {
        if (part == 0 && threadIdx.x == 0) latch(a.status, kDevBounds);
        return;
    }
    const int32_t G = a.v.G, D = G * kKv4Group, per_row = a.v.Hk * D / 8;  // a multiple of 4
    const int32_t j0 = part * a.slots_block, j1 = min(cnt, j0 + a.slots_block);
    const int64_t items = static_cast<int64_t>(max(j1 - j0, 0)) * per_row;
    for (int64_t it0 = threadIdx.x & ~31; it0 < items; it0 += kThreads) {
        const int64_t it = it0 + (threadIdx.x & 31);
        const int32_t dj = static_cast<int32_t>(it / per_row), piece = static_cast<int32_t>(it - static_cast<int64_t>(dj) * per_row);
        const int32_t j = j0 + dj;
        bool live = it < items;
        int32_t src = j;
        if (live && a.select) src = a.select[static_cast<int64_t>(b) * a.slots + j];
        live = live && src >= 0;
        const int64_t pos = start + j;
        if (live && (src >= a.src_rows || pos >= a.v.cap)) {
            latch(a.status, kDevBounds);
            live = false;
        }
        uint4 rk = make_uint4(0, 0, 0, 0), rv = rk;
        const int32_t hk = piece / (D / 8), in = piece - hk * (D / 8);
        uint8_t *chunk = nullptr;
        if (live) {
            const int64_t off = (static_cast<int64_t>(b) * a.src_rows + src) * a.ld + static_cast<int64_t>(piece) * 8;
            rk = *reinterpret_cast<const uint4 *>(a.k + off);
            rv = *reinterpret_cast<const uint4 *>(a.w + off);
            chunk = kv4_chunk(a.v, b, hk, pos);
            if (!chunk) latch(a.status, kDevBounds);
        }
        uint32_t pk, pv;
        const uint32_t ck = quantise8(rk, &pk), cv = quantise8(rv, &pv);
        if (!chunk) continue;
        const int32_t t = static_cast<int32_t>(pos & 15), ks = kv4_key_slot(t), g = in >> 2, qd = in & 3;
        *reinterpret_cast<uint32_t *>(chunk + ks * 16 * G + (qd * G + g) * 4) = ck;
        uint8_t *vrow = chunk + kv4_value_codes(G) + t * 16 * G;
        *reinterpret_cast<uint16_t *>(vrow + kv4_value_word(t, 2 * qd, g, G)) = static_cast<uint16_t>(cv);
        *reinterpret_cast<uint16_t *>(vrow + kv4_value_word(t, 2 * qd + 1, g, G)) = static_cast<uint16_t>(cv >> 16);
        if (qd == 0) *reinterpret_cast<uint32_t *>(chunk + kv4_key_params(G) + ks * 4 * G + 4 * g) = pk;
        if (qd == 1) *reinterpret_cast<uint32_t *>(chunk + kv4_value_params(G) + t * 4 * G + 4 * g) = pv;
    }
    if (!a.lengths || part != 0) return;
    // the length ends behind the last slot written
    if (threadIdx.x == 0) s_last = a.select ? 0 : cnt;
    __syncthreads();  // also: every thread has read start, which may be the lengths themselves
    if (a.select) {
        for (int32_t j = threadIdx.x; j < cnt; j += kThreads)
            if (a.select[static_cast<int64_t>(b) * a.slots + j] >= 0) atomicMax(&s_last, j + 1);
        __syncthreads();
    }
    if (threadIdx.x == 0) a.lengths[b] = static_cast<int32_t>(min(start + s_last, a.v.cap));
}

// The lengths alone, after a write whose blocks all read their starts from them.
__global__ void __launch_bounds__(32) kv4_lengths_kernel(const AppendArgs a, int32_t *lengths) {
    pdl_launch_dependents();
    pdl_wait();
    const int32_t b = blockIdx.x, lane = threadIdx.x;
    const int64_t start = lengths[b];
    if (start < 0) return;
    const int32_t cnt = slots_of(a, b);
    int32_t last = a.select ? 0 : cnt;
    if (a.select)
        for (int32_t j = lane; j < cnt; j += 32)
            if (a.select[static_cast<int64_t>(b) * a.slots + j] >= 0) last = j + 1;
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) lengths[b] = static_cast<int32_t>(min(start + last, a.v.cap));
}

struct ReadArgs {
    Kv4View v;
    int32_t B, rows, blocks, rows_block;
    const int32_t *start;  // [B] or null: 0
    void *k, *w;           // [B][rows][Hk * D]
    int32_t *status;
};

template <typename T>
__device__ __forceinline__ void store8(T *dst, uint32_t codes, uint32_t params) {
    const __half2 sm = *reinterpret_cast<const __half2 *>(&params);
    const float s = __low2float(sm), m = __high2float(sm);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(s, static_cast<float>((codes >> (4 * i)) & 15u), m);
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint4 o;
        uint32_t *ow = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            ow[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        *reinterpret_cast<uint4 *>(dst) = o;
    }
}

// Block (request, run of rows): a thread takes 8 dims of a key and of a value.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const ReadArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int32_t b = blockIdx.x / a.blocks, part = blockIdx.x - b * a.blocks;
    const int64_t start = a.start ? a.start[b] : 0, len = kv4_length(a.v, b);
    if (start < 0) {
        if (part == 0 && threadIdx.x == 0) latch(a.status, kDevBounds);
        return;
    }
    const int32_t G = a.v.G, D = G * kKv4Group, per_row = a.v.Hk * D / 8;
    const int32_t j0 = part * a.rows_block;
    const int32_t j1 = static_cast<int32_t>(min(static_cast<int64_t>(min(a.rows, j0 + a.rows_block)), len - start));
    const int64_t items = static_cast<int64_t>(max(j1 - j0, 0)) * per_row;
    for (int64_t it = threadIdx.x; it < items; it += kThreads) {
        const int32_t dj = static_cast<int32_t>(it / per_row), piece = static_cast<int32_t>(it - static_cast<int64_t>(dj) * per_row);
        const int64_t pos = start + j0 + dj;
        const int32_t hk = piece / (D / 8), in = piece - hk * (D / 8);
        const uint8_t *chunk = kv4_chunk(a.v, b, hk, pos);
        if (!chunk) {
            latch(a.status, kDevBounds);
            continue;
        }
        const int32_t t = static_cast<int32_t>(pos & 15), ks = kv4_key_slot(t), g = in >> 2, qd = in & 3;
        const uint32_t ck = *reinterpret_cast<const uint32_t *>(chunk + ks * 16 * G + (qd * G + g) * 4);
        const uint32_t pk = *reinterpret_cast<const uint32_t *>(chunk + kv4_key_params(G) + ks * 4 * G + 4 * g);
        const uint8_t *vrow = chunk + kv4_value_codes(G) + t * 16 * G;
        const uint32_t cv = *reinterpret_cast<const uint16_t *>(vrow + kv4_value_word(t, 2 * qd, g, G)) |
                            (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(vrow + kv4_value_word(t, 2 * qd + 1, g, G))) << 16);
        const uint32_t pv = *reinterpret_cast<const uint32_t *>(chunk + kv4_value_params(G) + t * 4 * G + 4 * g);
        const int64_t off = ((static_cast<int64_t>(b) * a.rows + j0 + dj) * a.v.Hk * D) + static_cast<int64_t>(piece) * 8;
        store8(reinterpret_cast<T *>(a.k) + off, ck, pk);
        store8(reinterpret_cast<T *>(a.w) + off, cv, pv);
    }
}

// Blocks a request's rows are cut into: about 8 passes of a block's threads each, fewer blocks
// than the grid can hold.
int32_t rows_a_block(int64_t rows, int64_t per_row, int32_t batch) {
    int64_t r = (8 * kThreads + per_row - 1) / per_row;
    const int64_t most = (int64_t{1} << 30) / batch;  // blocks a request
    r = r < 1 ? 1 : r;
    if ((rows + r - 1) / r > most) r = (rows + most - 1) / most;
    return static_cast<int32_t>(r < rows ? r : rows);
}

bool misaligned(const void *p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; }

}  // namespace
}  // namespace eagle

extern "C" {

size_t eagle_kv4_pages_bytes(const eagle_kv4_cache *cache) {
    eagle_kv4_cache c;
    eagle::Kv4View v;
    if (!cache) return 0;
    c = *cache;
    c.pages = reinterpret_cast<void *>(256);  // sizes alone
    c.table = reinterpret_cast<const int32_t *>(256);
    c.lengths = reinterpret_cast<int32_t *>(256);
    if (!eagle::kv4_view(&c, &v)) return 0;
    return static_cast<size_t>(c.num_pages) * c.kv_heads * (c.page_size / 16) * eagle::kv4_chunk_bytes(v.G);
}

eagle_status eagle_kv4_append(const eagle_kv4_cache *cache, int32_t batch, int32_t src_rows, int32_t slots,
                              const void *d_k, const void *d_v, int64_t ld, const int32_t *d_select,
                              const int32_t *d_count, const int32_t *d_start, int32_t *d_status,
                              eagle_stream_t stream) {
    using namespace eagle;
    NvtxRange nvtx_range("eagle_kv4_append");
    AppendArgs a{};
    if (!kv4_view(cache, &a.v) || batch < 0 || src_rows < 0 || slots < 0) return EAGLE_ERR_INVALID_ARG;
    if (!d_select && slots > src_rows) return EAGLE_ERR_INVALID_ARG;
    if (batch == 0) return EAGLE_OK;
    const int64_t row = static_cast<int64_t>(a.v.Hk) * a.v.G * kKv4Group;
    if (slots > 0 && (!d_k || !d_v || ld < row || ld % 8 || misaligned(d_k, 16) || misaligned(d_v, 16)))
        return EAGLE_ERR_INVALID_ARG;
    if (misaligned(d_select, 4) || misaligned(d_count, 4) || misaligned(d_start, 4) || misaligned(d_status, 4))
        return EAGLE_ERR_INVALID_ARG;
    a.B = batch;
    a.src_rows = src_rows;
    a.slots = slots;
    a.k = static_cast<const __nv_bfloat16 *>(d_k);
    a.w = static_cast<const __nv_bfloat16 *>(d_v);
    a.ld = ld;
    a.select = d_select;
    a.count = d_count;
    a.start = d_start ? d_start : cache->lengths;
    a.status = d_status;
    a.slots_block = slots > 0 ? rows_a_block(slots, row / 8, batch) : 1;
    a.blocks = slots > 0 ? (slots + a.slots_block - 1) / a.slots_block : 1;
    // one block a request, or starts of their own: the lengths are written in the same launch
    const bool own_lengths = a.blocks == 1 || a.start != cache->lengths;
    a.lengths = own_lengths ? cache->lengths : nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (launch_pdl(kv4_append_kernel, dim3(static_cast<unsigned>(batch) * a.blocks), dim3(kThreads), 0, st, a) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    if (!own_lengths &&
        launch_pdl(kv4_lengths_kernel, dim3(batch), dim3(32), 0, st, a, cache->lengths) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    return EAGLE_OK;
}

eagle_status eagle_kv4_read(const eagle_kv4_cache *cache, int32_t batch, int32_t rows, const int32_t *d_start,
                            void *d_k, void *d_v, eagle_dtype dtype, int32_t *d_status, eagle_stream_t stream) {
    using namespace eagle;
    NvtxRange nvtx_range("eagle_kv4_read");
    ReadArgs a{};
    if (!kv4_view(cache, &a.v) || batch < 0 || rows < 0) return EAGLE_ERR_INVALID_ARG;
    if (dtype != EAGLE_F32 && dtype != EAGLE_BF16) return EAGLE_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0) return EAGLE_OK;
    if (!d_k || !d_v || misaligned(d_k, 16) || misaligned(d_v, 16) || misaligned(d_start, 4) || misaligned(d_status, 4))
        return EAGLE_ERR_INVALID_ARG;
    a.B = batch;
    a.rows = rows;
    a.start = d_start;
    a.k = d_k;
    a.w = d_v;
    a.status = d_status;
    a.rows_block = rows_a_block(rows, static_cast<int64_t>(a.v.Hk) * a.v.G * 4, batch);
    a.blocks = (rows + a.rows_block - 1) / a.rows_block;
    const dim3 grid(static_cast<unsigned>(batch) * a.blocks), block(kThreads);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == EAGLE_F32 ? launch_pdl(kv4_read_kernel<float>, grid, block, 0, st, a)
                                             : launch_pdl(kv4_read_kernel<__nv_bfloat16>, grid, block, 0, st, a);
    return e == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}

}  // extern "C"
