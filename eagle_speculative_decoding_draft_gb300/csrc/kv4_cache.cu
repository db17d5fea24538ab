// kv4_cache.cu - writing the 4-bit key/value cache and reading it back.
//
// The engine's decoder layer hands out the keys and values of a tree's nodes; after the verify the
// accepted path's rows join the cache, in 4 bits, at the request's next positions (a prompt's rows
// in order, a path's rows through the list of its nodes).  kv4.cuh has the format.
#include <type_traits>

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

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kFull = 0xffffffffu;

// Both kernels: a warp takes one chunk (16 positions) of one kv head, whose 640 G bytes it assembles or
// unpacks in shared memory, so that the cache is written and read in whole lines whatever the order
// of the codes, and rows of the callers' tensors by 16-byte pieces of neighbouring lanes.
struct Units {
    int32_t Hk, per_request;  // per_request: kv heads x chunks that a request may touch
    int32_t total;            // warps of work
};
// The request of warp `id` of the launch, and which of the request's warps it is.
__device__ __forceinline__ bool unit_request(const Units &u, int32_t id, int32_t &b, int32_t &rest) {
    if (id >= u.total) return false;
    b = id / u.per_request;
    rest = id - b * u.per_request;
    return true;
}

struct AppendArgs {
    Kv4View v;
    Units u;
    int32_t B, src_rows, slots;
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
// The request's length after the write: behind its last written slot, which is one that names a row and
// whose position lies in a page that is there.  Looked for from the end, 32 slots at a time.  Whole warp.
__device__ __forceinline__ int32_t length_after(const AppendArgs &a, int32_t b, int64_t start, int32_t cnt) {
    int64_t end = min(static_cast<int64_t>(cnt), a.v.cap - start);  // slots up to the capacity
    for (; end > 0; end -= 32) {
        const int64_t j = end - 1 - (threadIdx.x & 31);
        const bool named = j >= 0 && (!a.select || static_cast<uint32_t>(a.select[static_cast<int64_t>(b) * a.slots + j]) <
                                                       static_cast<uint32_t>(a.src_rows));
        const uint32_t written = __ballot_sync(kFull, named && kv4_chunk(a.v, b, 0, start + j));
        if (written) {
            end -= __ffs(written) - 1;
            break;
        }
    }
    return static_cast<int32_t>(min(start + max(end, int64_t{0}), a.v.cap));
}

__device__ __forceinline__ __nv_bfloat162 as_b2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); }

// A group of 32 values: four words of eight codes (the first in the low bits) and (s, m).  A code is
// (x - m) / s rounded to the nearest whole number, ties to even.  The quotient is a product with a
// reciprocal that is a few units too large, rounded by a sum with 1.5 2^23 (whose low bits it then is):
// never too small, and too large by one only for ties and just below them.  The remainder a - c s, which
// is exact, tells: below -s / 2 the code is one too large, at -s / 2 it is a tie, of which the even
// neighbour is the one.
__device__ __forceinline__ uint32_t quantise(const uint32_t (&w)[16], uint32_t (&codes)[4]) {
    // both halves of a word at once; NaN passes on
    __nv_bfloat162 hi2 = as_b2(w[0]), lo2 = hi2;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        hi2 = __hmax2_nan(hi2, as_b2(w[i]));
        lo2 = __hmin2_nan(lo2, as_b2(w[i]));
    }
    const float h0 = __low2float(hi2), h1 = __high2float(hi2), l0 = __low2float(lo2), l1 = __high2float(lo2);
    const float hi = fmaxf(h0, h1), lo = fminf(l0, l1);
    const bool ok = fabsf(h0) <= kKv4MaxAbs && fabsf(h1) <= kKv4MaxAbs && fabsf(l0) <= kKv4MaxAbs && fabsf(l1) <= kKv4MaxAbs;
    const __half m = __float2half_rd(lo);
    const float mf = __half2float(m);
    const __half s = __float2half_ru(__fdiv_rn(hi - mf, 15.0f));
    const float sf = __half2float(s), below = -0.5f * sf;
    const float below_or_at = __int_as_float(__float_as_int(below) - 1);  // the next one up (NaN for -0: never)
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sf));  // within 2^-23: 3 units more are above 1 / s
    r = sf > 0.0f ? __int_as_float(__float_as_int(r) + 3) : 0.0f;
    constexpr float kMagic = 12582912.0f;  // bits 0x4b400000: the code adds to them
    const uint64_t r2 = pack_2(r, r), s2 = pack_2(sf, sf), m2 = pack_2(-mf, -mf), magic2 = pack_2(kMagic, kMagic);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t c8 = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {  // two values of a word at a time
            const uint32_t p = w[4 * k + i];
            const uint64_t a = add_2(pack_2(p << 16, p & 0xffff0000u), m2), t = fma_2(a, r2, magic2);
            const float2 code = unpack_2(t), rem = unpack_2(fma_2(fma_2(t, pack_2(-1.0f, -1.0f), magic2), s2, a));
            uint32_t c = __float_as_uint(code.y);
            if (rem.y < (c & 1u ? below_or_at : below)) --c;
            c8 = c8 * 16u + c;
            c = __float_as_uint(code.x);
            if (rem.x < (c & 1u ? below_or_at : below)) --c;
            c8 = c8 * 16u + c;
        }
        // without 0x4b400000 (1 + 16 + 256 + ...), of which three terms stay in the word
        codes[k] = ok ? c8 - (0x4b400000u + 0xb4000000u + 0x40000000u) : 0u;
    }
    return ok ? static_cast<uint32_t>(__half_as_ushort(s)) | (static_cast<uint32_t>(__half_as_ushort(m)) << 16) : 0x7fff7fffu;
}

// A lane takes whole groups (64 bytes): their least and largest value and parameters need no other
// lane.  The chunk's rows that are written come one behind the other, keys, then values, 32 groups a
// pass, the next pass on its way.  Bound by instruction issue (76 % of the cycles): 33 k tokens of 8 kv heads
// of 128 (176 MB) in 40 us, 0.65 of the measured copy rate; a lane a 16-byte piece with the least and
// largest value over four lanes took twice as long.  The accepted rows of 64 requests: 6 us, and 1 more
// where the lengths are the starts.
template <int G>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const AppendArgs a) {
    constexpr int kBytes = kv4_chunk_bytes(G);
    __shared__ __align__(16) uint8_t stage[kWarps][kBytes];
    __shared__ uint8_t order[kWarps][16];  // the rows that are written, in order
    pdl_launch_dependents();
    pdl_wait();
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t b, rest;
    if (!unit_request(a.u, static_cast<int32_t>(blockIdx.x) * kWarps + warp, b, rest)) return;
    const int32_t ci = rest / a.u.Hk, hk = rest - ci * a.u.Hk;
    const int64_t start = a.start[b];
    const int32_t cnt = slots_of(a, b);
    if (start < 0) {
        if (rest == 0 && lane == 0) latch(a.status, kDevBounds);
        return;
    }
    if (a.lengths && rest == 0) {
        const int32_t len = length_after(a, b, start, cnt);
        if (lane == 0) a.lengths[b] = len;
    }
    // lane t: the source row of position chunk0 + t, or -1
    const int64_t chunk0 = ((start >> 4) + ci) << 4, j0 = chunk0 - start;
    int32_t src = -1;
    {
        const int64_t j = j0 + lane;
        if (lane < 16 && j >= 0 && j < cnt) {
            src = a.select ? a.select[static_cast<int64_t>(b) * a.slots + j] : static_cast<int32_t>(j);
            if (src >= a.src_rows || (src >= 0 && chunk0 + lane >= a.v.cap)) {
                latch(a.status, kDevBounds);
                src = -1;
            }
        }
    }
    const uint32_t rows = __ballot_sync(kFull, src >= 0);
    if (rows == 0) return;
    const int32_t live = __popc(rows), items = 2 * live * G;
    if (src >= 0) order[warp][__popc(rows & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane);
    __syncwarp();
    // group `it` of the pass: row, tensor and place in the row
    auto load = [&](int32_t it, uint32_t (&w)[16]) {
        const int32_t n = it / G, g = it - n * G;
        const bool value = n >= live;
        const int32_t t = order[warp][min(value ? n - live : n, 15)], from = __shfl_sync(kFull, src, t & 15);
        if (it < items) {
            const uint4 *p = reinterpret_cast<const uint4 *>((value ? a.w : a.k) + (static_cast<int64_t>(b) * a.src_rows + from) * a.ld +
                                                             (static_cast<int64_t>(hk) * G + g) * kKv4Group);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = __ldg(p + i);
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = 0u;
        }
    };
    uint32_t now[16], ahead[16];
    load(lane, now);
    uint8_t *chunk = kv4_chunk(a.v, b, hk, chunk0);
    if (!chunk) {
        if (lane == 0) latch(a.status, kDevBounds);
        return;
    }
    uint8_t *st = stage[warp];
#pragma unroll 1
    for (int32_t it0 = 0; it0 < items; it0 += 32) {
        load(it0 + 32 + lane, ahead);
        uint32_t codes[4];
        const uint32_t params = quantise(now, codes);
        const int32_t it = it0 + lane;
        if (it < items) {
            const int32_t n = it / G, g = it - n * G;
            if (n < live) {
                const int32_t ks = kv4_key_slot(order[warp][n]);
#pragma unroll
                for (int qd = 0; qd < 4; ++qd) *reinterpret_cast<uint32_t *>(st + ks * 16 * G + (qd * G + g) * 4) = codes[qd];
                *reinterpret_cast<uint32_t *>(st + kv4_key_params(G) + ks * 4 * G + 4 * g) = params;
            } else {
                const int32_t t = order[warp][n - live];
                uint8_t *vrow = st + kv4_value_codes(G) + t * 16 * G;
#pragma unroll
                for (int gq = 0; gq < 8; ++gq)
                    *reinterpret_cast<uint16_t *>(vrow + kv4_value_word(t, gq, g, G)) = static_cast<uint16_t>(codes[gq >> 1] >> (16 * (gq & 1)));
                *reinterpret_cast<uint32_t *>(st + kv4_value_params(G) + t * 4 * G + 4 * g) = params;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) now[i] = ahead[i];
    }
    __syncwarp();
    // out in the widest words that hold one row's bytes each: a row has 16 G bytes of codes and 4 G of
    // parameters
    using Word = std::conditional_t<G == 4, uint4, std::conditional_t<G == 2, uint2, uint32_t>>;
    constexpr int kWord = sizeof(Word), kCodeWords = 16 * G / kWord, kParWords = 4 * G / kWord, kPart = 320 * G / kWord;
#pragma unroll
    for (int i = 0; i < (kBytes / kWord + 31) / 32; ++i) {
        const int32_t at = i * 32 + lane;
        if (at >= kBytes / kWord) break;
        const bool key = at < kPart;
        const int32_t in = key ? at : at - kPart;
        const int32_t row = in < 16 * kCodeWords ? in / kCodeWords : (in - 16 * kCodeWords) / kParWords;
        const int32_t t = key ? ((row & 7) >> 1) | ((row & 1) << 2) | (row & 8) : row;
        if ((rows >> t) & 1u) reinterpret_cast<Word *>(chunk)[at] = reinterpret_cast<const Word *>(st)[at];
    }
}

// The lengths alone, after a write whose blocks all read their starts from them.
__global__ void __launch_bounds__(32) kv4_lengths_kernel(const AppendArgs a, int32_t *lengths) {
    pdl_launch_dependents();
    pdl_wait();
    const int32_t b = blockIdx.x;
    const int64_t start = lengths[b];
    if (start < 0) return;
    const int32_t len = length_after(a, b, start, slots_of(a, b));
    if (threadIdx.x == 0) lengths[b] = len;
}

struct ReadArgs {
    Kv4View v;
    Units u;
    int32_t B, rows;
    const int32_t *start;  // [B] or null: 0
    void *k, *w;           // [B][rows][Hk * D]
    int32_t *status;
};

// N codes from the low bits of `codes` to m + s c, one fused product and sum each.
template <int N>
__device__ __forceinline__ void values_of(uint32_t codes, uint32_t params, float (&x)[N]) {
    const __half2 sm = *reinterpret_cast<const __half2 *>(&params);
    const float s = __low2float(sm), m = __high2float(sm);
#pragma unroll
    for (int i = 0; i < N; ++i)  // 2^23 + c has c in its low bits
        x[i] = fmaf(s, __uint_as_float(((codes >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.0f, m);
}

// T float: a lane takes 4 dims (16 bytes out), T bf16: 8.  Bound by memory: 65536 tokens of 8 kv heads
// of 128 to fp32 (621 MB) in 96 us, 0.96 of the measured copy rate; 33 k tokens to bf16 (176 MB) in 29.
template <int G, typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const ReadArgs a) {
    constexpr int N = 16 / sizeof(T), kPer = 32 * G / N, R = 32 / kPer;  // dims a lane, lanes a row, rows at once
    constexpr int kBytes = kv4_chunk_bytes(G);
    __shared__ __align__(16) uint8_t stage[kWarps][kBytes];
    pdl_launch_dependents();
    pdl_wait();
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t b, rest;
    if (!unit_request(a.u, static_cast<int32_t>(blockIdx.x) * kWarps + warp, b, rest)) return;
    const int32_t ci = rest / a.u.Hk, hk = rest - ci * a.u.Hk;
    const int64_t start = a.start ? a.start[b] : 0, len = kv4_length(a.v, b);
    if (start < 0) {
        if (rest == 0 && lane == 0) latch(a.status, kDevBounds);
        return;
    }
    const int64_t chunk0 = ((start >> 4) + ci) << 4;
    // rows t0 .. t1 - 1 of the chunk are asked for and there
    const int32_t t0 = static_cast<int32_t>(max(start - chunk0, int64_t{0}));
    const int32_t t1 = static_cast<int32_t>(min(min(start + a.rows, len) - chunk0, int64_t{16}));
    if (t0 >= t1) return;
    const uint8_t *chunk = kv4_chunk(a.v, b, hk, chunk0);
    if (!chunk) {
        if (lane == 0) latch(a.status, kDevBounds);
        return;
    }
    uint8_t *st = stage[warp];
    {
        constexpr int kPieces = kBytes / 16, kLoads = (kPieces + 31) / 32;
        uint4 x[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i * 32 + lane < kPieces) x[i] = __ldg(reinterpret_cast<const uint4 *>(chunk) + i * 32 + lane);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i * 32 + lane < kPieces) reinterpret_cast<uint4 *>(st)[i * 32 + lane] = x[i];
    }
    __syncwarp();
    const int32_t in = lane % kPer, dim = in * N, g = dim >> 5, qd = (dim >> 3) & 3;
    if (lane / kPer >= R) return;
    T *k_out = reinterpret_cast<T *>(a.k), *v_out = reinterpret_cast<T *>(a.w);
    const int64_t row_len = static_cast<int64_t>(a.u.Hk) * G * kKv4Group;
    const int64_t out0 = (static_cast<int64_t>(b) * a.rows + (chunk0 - start)) * row_len + static_cast<int64_t>(hk) * G * kKv4Group + dim;
#pragma unroll 4
    for (int32_t t = lane / kPer; t < 16; t += R) {
        if (t < t0 || t >= t1) continue;
        const int32_t ks = kv4_key_slot(t);
        uint32_t ck = *reinterpret_cast<const uint32_t *>(st + ks * 16 * G + (qd * G + g) * 4);
        const uint32_t pk = *reinterpret_cast<const uint32_t *>(st + kv4_key_params(G) + ks * 4 * G + 4 * g);
        const uint8_t *vrow = st + kv4_value_codes(G) + t * 16 * G;
        const uint32_t pv = *reinterpret_cast<const uint32_t *>(st + kv4_value_params(G) + t * 4 * G + 4 * g);
        float x[N], y[N];
        uint32_t cv;
        if constexpr (N == 4) {
            ck >>= (dim & 4) * 4;
            cv = *reinterpret_cast<const uint16_t *>(vrow + kv4_value_word(t, (dim >> 2) & 7, g, G));
        } else {
            cv = *reinterpret_cast<const uint16_t *>(vrow + kv4_value_word(t, 2 * qd, g, G)) |
                 (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(vrow + kv4_value_word(t, 2 * qd + 1, g, G))) << 16);
        }
        values_of(ck, pk, x);
        values_of(cv, pv, y);
        const int64_t out = out0 + t * row_len;
        if constexpr (N == 4) {
            *reinterpret_cast<float4 *>(k_out + out) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(v_out + out) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
            uint4 ko, vo;
            uint32_t *kw = reinterpret_cast<uint32_t *>(&ko), *vw = reinterpret_cast<uint32_t *>(&vo);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]), q = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                kw[i] = *reinterpret_cast<const uint32_t *>(&p);
                vw[i] = *reinterpret_cast<const uint32_t *>(&q);
            }
            *reinterpret_cast<uint4 *>(k_out + out) = ko;
            *reinterpret_cast<uint4 *>(v_out + out) = vo;
        }
    }
}

// A request's `rows` rows touch at most (rows + 30) / 16 chunks of each kv head.  False: more warps than
// 32 bits count (over a terabyte of cache).
bool units_of(int32_t batch, int32_t Hk, int64_t rows, Units *u) {
    const int64_t per = Hk * ((rows + 30) / 16);
    if (per * batch > INT32_MAX - kWarps) return false;
    *u = Units{Hk, static_cast<int32_t>(per), static_cast<int32_t>(per * batch)};
    return true;
}
dim3 grid_of(const Units &u) { return dim3(static_cast<unsigned>((u.total + kWarps - 1) / kWarps)); }

using AppendKernel = void (*)(const AppendArgs);
AppendKernel append_kernel(int32_t G) {
    switch (G) {
        case 1: return kv4_append_kernel<1>;
        case 2: return kv4_append_kernel<2>;
        case 3: return kv4_append_kernel<3>;
        default: return kv4_append_kernel<4>;
    }
}
using ReadKernel = void (*)(const ReadArgs);
template <typename T>
ReadKernel read_kernel(int32_t G) {
    switch (G) {
        case 1: return kv4_read_kernel<1, T>;
        case 2: return kv4_read_kernel<2, T>;
        case 3: return kv4_read_kernel<3, T>;
        default: return kv4_read_kernel<4, T>;
    }
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
    if (!units_of(batch, a.v.Hk, slots > 0 ? slots : 1, &a.u)) return EAGLE_ERR_UNSUPPORTED;
    // starts of their own: the lengths are written in the same launch
    const bool own_lengths = a.start != cache->lengths;
    a.lengths = own_lengths ? cache->lengths : nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (launch_pdl(append_kernel(a.v.G), grid_of(a.u), dim3(kThreads), 0, st, a) != cudaSuccess) return EAGLE_ERR_CUDA;
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
    if (!units_of(batch, a.v.Hk, rows, &a.u)) return EAGLE_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const ReadKernel kernel = dtype == EAGLE_F32 ? read_kernel<float>(a.v.G) : read_kernel<__nv_bfloat16>(a.v.G);
    return launch_pdl(kernel, grid_of(a.u), dim3(kThreads), 0, st, a) == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}

}  // extern "C"
