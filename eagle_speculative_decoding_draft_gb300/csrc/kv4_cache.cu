// kv4_cache.cu - writing the 4-bit key/value cache and reading it back.
//
// The engine's decoder layer hands out the keys and values of a tree's nodes; after the verify the
// accepted path's rows join the cache, in 4 bits, at the request's next positions (a prompt's rows
// in order, a path's rows through the list of its nodes).  kv4.cuh has the format.
#include <algorithm>
#include <cmath>
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

// Keys turned on the way (and the queries of the same rows): pair (j, j + D/2) of a head by position times
// theta^(-2j/D).  turn[j] is that frequency as a fraction of a whole turn in units of 2^-64, so that a
// position's angle is their product modulo 2^64: exact whole-number arithmetic whatever the position, and
// off by 2^-53 of the frequency (theta^(-2j/D) in 64 bits) times the position.
struct RotaryArgs {
    AppendArgs a;
    const int32_t *positions;  // [B][src_rows], or null: start + row
    const __nv_bfloat16 *q;    // [B][src_rows] rows of ldq elements, or null
    __nv_bfloat16 *q_out;      // [B][src_rows][H][D]
    int64_t ldq;
    int32_t H;
    int32_t slices;            // blocks of 8 kv heads a chunk
    int32_t cache_blocks;      // the launch's first blocks write the cache, the others turn queries
    int32_t q_rows;            // rows of one of those
    float minus_one;           // turn_word's
    uint64_t turn[64];
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

// Cosine and sine of a fraction of a turn in units of 2^-64, each the nearest fp32 value but for three in ten
// thousand that lie beside a tie (and but for sines below 2^-21, good to 2^-23 of themselves): a turned key that is
// one fp32 step off now and then rounds to another bf16 value, and takes another code of the cache.  The
// angle within an eighth of a turn and its Taylor series to the 14th power, what is left of 1, -1/6 and 1/24 in fp32
// and these in pairs of fp32 (hi + lo), products and sums by their exact remainders (T. J. Dekker, Numer. Math. 18,
// 1971).  No fp64: it runs at a 64th of the rate here.
__device__ __forceinline__ float2 cos_sin(uint64_t at) {
    const uint32_t quarter = static_cast<uint32_t>((at + (uint64_t{1} << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(at - (static_cast<uint64_t>(quarter) << 62));
    const uint64_t m = static_cast<uint64_t>(rest < 0 ? -rest : rest);
    const int32_t top = static_cast<int32_t>(m >> 32);
    const float hi = static_cast<float>(top);
    const float lo = fmaf(static_cast<float>(top - static_cast<int32_t>(hi)), 4294967296.0f, static_cast<float>(static_cast<uint32_t>(m)));
    // the angle t + tl: hi and lo times 2 pi / 2^32 and 2^64
    constexpr double kStep = 6.283185307179586 / 4294967296.0;
    constexpr float kHi = static_cast<float>(kStep), kLo = static_cast<float>(kStep - static_cast<double>(kHi));
    const float ph = __fmul_rn(hi, kHi), pl = __fadd_rn(fmaf(hi, kHi, -ph), fmaf(hi, kLo, __fmul_rn(lo, kHi / 4294967296.0f)));
    const float t = __fadd_rn(ph, pl), tl = __fsub_rn(pl, __fsub_rn(t, ph));
    const float u = __fmul_rn(t, t), ul = fmaf(__fmul_rn(2.0f, t), tl, fmaf(t, t, -u));  // its square
    // sine: t (1 + u a), a = -1/6 + u (1/120 - ...)
    float p = __fmul_rn(u, fmaf(u, fmaf(u, fmaf(u, fmaf(u, 1.0f / 6227020800.0f, -1.0f / 39916800.0f), 1.0f / 362880.0f), -1.0f / 5040.0f), 1.0f / 120.0f));
    constexpr float kSixth = -1.0f / 6.0f, kSixthLo = static_cast<float>(-1.0 / 6.0 - static_cast<double>(kSixth));
    float a = __fadd_rn(kSixth, p), al = __fadd_rn(__fsub_rn(p, __fsub_rn(a, kSixth)), kSixthLo);
    const float w = __fmul_rn(u, a), wl = __fadd_rn(fmaf(u, a, -w), fmaf(u, al, __fmul_rn(ul, a)));
    const float q = __fmul_rn(t, w), ql = __fadd_rn(fmaf(t, w, -q), fmaf(t, wl, __fmul_rn(tl, w)));
    const float s0 = __fadd_rn(t, q);
    const float s = __fadd_rn(s0, __fadd_rn(__fsub_rn(q, __fsub_rn(s0, t)), __fadd_rn(tl, ql)));
    // cosine: 1 - u / 2 + u^2 a, a = 1/24 - u (1/720 - ...)
    p = __fmul_rn(u, fmaf(u, fmaf(u, fmaf(u, 1.0f / 479001600.0f, -1.0f / 3628800.0f), 1.0f / 40320.0f), -1.0f / 720.0f));
    constexpr float k24th = 1.0f / 24.0f, k24thLo = static_cast<float>(1.0 / 24.0 - static_cast<double>(k24th));
    a = __fadd_rn(k24th, p), al = __fadd_rn(__fsub_rn(p, __fsub_rn(a, k24th)), k24thLo);
    const float v = __fmul_rn(u, u), vl = fmaf(__fmul_rn(2.0f, u), ul, fmaf(u, u, -v));
    const float f = __fmul_rn(v, a), fl = __fadd_rn(fmaf(v, a, -f), fmaf(v, al, __fmul_rn(vl, a)));
    const float c0 = fmaf(-0.5f, u, 1.0f), c0l = fmaf(-0.5f, u, __fsub_rn(1.0f, c0));
    const float c1 = __fadd_rn(c0, f), c1l = __fsub_rn(f, __fsub_rn(c1, c0));
    const float c = __fadd_rn(c1, __fadd_rn(c0l, __fadd_rn(c1l, fmaf(-0.5f, ul, fl))));
    const float sn = rest < 0 ? -s : s;
    const bool odd = quarter & 1;
    const float x = odd ? sn : c, y = odd ? c : sn;
    return make_float2(quarter == 1 || quarter == 2 ? -x : x, quarter & 2 ? -y : y);
}
// The table of cosines and sines: a block of 16 pairs is 128 bytes, two pairs' cosines and sines (c, c, s, s) a
// piece, and starts kTurnBlock bytes after the one before it, so that the 16-byte pieces that the lanes of a
// quarter warp take lie in other banks.
constexpr int kTurnBlock = 128 + 16;
__device__ __forceinline__ float4 *turn_entry(uint8_t *table, int32_t G, int32_t row, int32_t j) {
    return reinterpret_cast<float4 *>(table + (row * G + (j >> 4)) * kTurnBlock) + ((j & 15) >> 1);
}
// A warp works out one row's pairs.
template <int G>
__device__ __forceinline__ void turn_row(const RotaryArgs &ra, uint8_t *table, int32_t row, int32_t pos) {
    for (int32_t j = threadIdx.x & 31; j < 16 * G; j += 32) {
        const uint64_t at = ra.turn[j] * static_cast<uint64_t>(static_cast<int64_t>(pos));
        const float2 cs = cos_sin(at);
        float *entry = reinterpret_cast<float *>(turn_entry(table, G, row, j)) + (j & 1);
        entry[0] = cs.x;
        entry[2] = cs.y;
    }
}
// Turns two neighbouring values (a bf16 word) of one half of a head by the pairs' cosines and sines,
// own c - other s (the second half's `other` comes with its sign turned: kMinus), and rounds to bf16: the cache
// quantises bf16 keys, turned here or by the decoder layer.  Both products and their difference are rounded to fp32,
// as a plain form's are: one rounding less, in a fused sum, gives another bf16 value now and then.  The compiler
// fuses a product and a sum of packed pairs even where both say .rn, so the sum is a fused one with a factor
// that it does not know, -1 from the arguments.
constexpr uint32_t kMinus = 0x80008000u;  // both values' signs
__device__ __forceinline__ uint32_t turn_word(uint32_t own, uint32_t other, const float4 &cs, float minus_one) {
    const uint64_t x = pack_2(own << 16, own & 0xffff0000u), p = pack_2(other << 16, other & 0xffff0000u);
    const float2 y = unpack_2(fma_2(mul_2(p, pack_2(cs.z, cs.w)), pack_2(minus_one, minus_one), mul_2(x, pack_2(cs.x, cs.y))));
    const __nv_bfloat162 r = __floats2bfloat162_rn(y.x, y.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// A key's group g in place, w; `head` is the key as it came.  Blocks of 16 dims: block i and block i + G (i < G)
// are each other's halves.  Where a row's groups lie in neighbouring lanes of one pass, the other half comes
// from there (G 1, 2, 4: from the lane itself, or G / 2 lanes apart), else from memory.  Whole warp.
template <int G>
__device__ __forceinline__ void turn_group(uint8_t *table, int32_t row, int32_t g, bool key, const uint4 *head, float minus_one,
                                           uint32_t (&w)[16]) {
    uint32_t o[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        if constexpr (G == 1)
            o[k] = w[k ^ 8];
        else if constexpr (G != 3)
            o[k] = __shfl_xor_sync(kFull, w[k], G / 2);
    }
    if (!key) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t i = 2 * g + h;
        const bool first = i < G;
        const uint32_t sign = first ? 0u : kMinus;
        if constexpr (G == 3) {
            const uint4 *other = head + 2 * (first ? i + G : i - G);
            const uint4 o0 = __ldg(other), o1 = __ldg(other + 1);
            const uint32_t p[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) o[8 * h + k] = p[k];
        }
        const float4 *cs = turn_entry(table, G, row, 16 * (first ? i : i - G));
#pragma unroll
        for (int k = 0; k < 8; ++k) w[8 * h + k] = turn_word(w[8 * h + k], o[8 * h + k] ^ sign, cs[k], minus_one);
    }
}
// ra.q_rows rows of queries (16 at most): a thread turns 8 pairs of a head at a time.
template <int G>
__device__ __forceinline__ void turn_queries(const RotaryArgs &ra, uint8_t *table, int32_t block) {
    const AppendArgs &a = ra.a;
    const int64_t all = static_cast<int64_t>(a.B) * a.src_rows, row0 = static_cast<int64_t>(block) * ra.q_rows;
    const int32_t rows = static_cast<int32_t>(min(all - row0, static_cast<int64_t>(ra.q_rows)));
    for (int32_t t = threadIdx.x >> 5; t < rows; t += kWarps) {
        const int64_t r = row0 + t;
        const int32_t b = static_cast<int32_t>(r / a.src_rows);
        turn_row<G>(ra, table, t, ra.positions ? ra.positions[r] : a.start[b] + static_cast<int32_t>(r - static_cast<int64_t>(b) * a.src_rows));
    }
    __syncthreads();
    constexpr int kEights = 2 * G;  // of a half head
    const int32_t per_row = ra.H * kEights;
    // whole rows at once where they are short; a thread keeps its place in the row
    const int32_t at_once = max(1, kThreads / per_row), mine = per_row < kThreads ? static_cast<int32_t>(threadIdx.x) / per_row : 0;
    if (mine >= at_once) return;
    for (int32_t in = static_cast<int32_t>(threadIdx.x) - mine * per_row; in < per_row; in += kThreads) {
        const int32_t head = in / kEights, e = in - head * kEights;
        const int64_t at = static_cast<int64_t>(head) * 32 * G + 8 * e;
        constexpr int kAhead = 4;  // rows in flight (the outputs may take the queries' place: loads before stores)
        for (int32_t t0 = mine; t0 < rows; t0 += kAhead * at_once) {
            uint4 x[kAhead], y[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int32_t t = t0 + i * at_once;
                if (t >= rows) break;
                const uint4 *src = reinterpret_cast<const uint4 *>(ra.q + (row0 + t) * ra.ldq + at);
                x[i] = src[0];
                y[i] = src[2 * G];
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int32_t t = t0 + i * at_once;
                if (t >= rows) break;
                uint4 *dst = reinterpret_cast<uint4 *>(ra.q_out + (row0 + t) * ra.H * 32 * G + at);
                const float4 *cs = turn_entry(table, G, t, 8 * e);
                const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, yw[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
                uint32_t p[4], q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[k] = turn_word(xw[k], yw[k], cs[k], ra.minus_one);
                    q[k] = turn_word(yw[k], xw[k] ^ kMinus, cs[k], ra.minus_one);
                }
                dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
                dst[2 * G] = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
    }
}

// A lane takes whole groups (64 bytes): their least and largest value and parameters need no other
// lane.  The chunk's rows that are written come one behind the other, keys, then values, 32 groups a
// pass, the next pass on its way.  Bound by instruction issue (76 % of the cycles): 33 k tokens of 8 kv heads
// of 128 (176 MB) in 40 us, 0.65 of the measured copy rate; a lane a 16-byte piece with the least and
// largest value over four lanes took twice as long.  The accepted rows of 64 requests: 6 us, and 1 more
// where the lengths are the starts.
template <int G, bool kRotary>
__device__ __forceinline__ void append_chunk(const AppendArgs &a, uint8_t *st, uint8_t *order, uint8_t *table,
                                             const RotaryArgs *ra, int32_t b, int32_t rest, int32_t ci, int32_t hk) {
    constexpr int kBytes = kv4_chunk_bytes(G);
    const int32_t lane = threadIdx.x & 31;
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
    if (src >= 0) order[__popc(rows & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane);
    __syncwarp();
    // group `it` of the pass: row, tensor and place in the row
    auto load = [&](int32_t it, uint32_t (&w)[16]) {
        const int32_t n = it / G, g = it - n * G;
        const bool value = n >= live;
        const int32_t t = order[min(value ? n - live : n, 15)], from = __shfl_sync(kFull, src, t & 15);
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
    if (!kRotary || hk < a.u.Hk) load(lane, now);
    if constexpr (kRotary) {
        // the block's warps share the chunk: each does two of its rows
        int32_t pos = 0;
        if (src >= 0)
            pos = ra->positions ? ra->positions[static_cast<int64_t>(b) * a.src_rows + src] : static_cast<int32_t>(chunk0 + lane);
        for (int32_t t = threadIdx.x >> 5; t < 16; t += kWarps) {
            const int32_t p = __shfl_sync(kFull, pos, t);
            if ((rows >> t) & 1u) turn_row<G>(*ra, table, t, p);
        }
        __syncthreads();  // every warp of the block is here: what ended above it is the same for all
        if (hk >= a.u.Hk) return;
    }
    uint8_t *chunk = kv4_chunk(a.v, b, hk, chunk0);
    if (!chunk) {
        if (lane == 0) latch(a.status, kDevBounds);
        return;
    }
#pragma unroll 1
    for (int32_t it0 = 0; it0 < items; it0 += 32) {
        load(it0 + 32 + lane, ahead);
        uint32_t codes[4];
        const int32_t it = it0 + lane;
        if constexpr (kRotary) {
            const int32_t n = it / G, g = it - n * G;
            const int32_t t = order[min(n, 15)], from = __shfl_sync(kFull, src, t & 15);
            turn_group<G>(table, t, g, n < live, reinterpret_cast<const uint4 *>(a.k + (static_cast<int64_t>(b) * a.src_rows + from) * a.ld +
                                                                                 static_cast<int64_t>(hk) * G * kKv4Group), ra->minus_one, now);
        }
        const uint32_t params = quantise(now, codes);
        if (it < items) {
            const int32_t n = it / G, g = it - n * G;
            if (n < live) {
                const int32_t ks = kv4_key_slot(order[n]);
#pragma unroll
                for (int qd = 0; qd < 4; ++qd) *reinterpret_cast<uint32_t *>(st + ks * 16 * G + (qd * G + g) * 4) = codes[qd];
                *reinterpret_cast<uint32_t *>(st + kv4_key_params(G) + ks * 4 * G + 4 * g) = params;
            } else {
                const int32_t t = order[n - live];
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

template <int G>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const AppendArgs a) {
    __shared__ __align__(16) uint8_t stage[kWarps][kv4_chunk_bytes(G)];
    __shared__ uint8_t order[kWarps][16];  // the rows that are written, in order
    pdl_launch_dependents();
    pdl_wait();
    const int32_t warp = threadIdx.x >> 5;
    int32_t b, rest;
    if (!unit_request(a.u, static_cast<int32_t>(blockIdx.x) * kWarps + warp, b, rest)) return;
    const int32_t ci = rest / a.u.Hk, hk = rest - ci * a.u.Hk;
    append_chunk<G, false>(a, stage[warp], order[warp], nullptr, nullptr, b, rest, ci, hk);
}

// Blocks of one chunk and up to 8 of its kv heads, a warp a head: the chunk's cosines and sines are worked
// out once a block, with the first rows on their way.  Further blocks turn the queries.  Three blocks an SM (80
// registers): 33 k tokens of 8 kv heads and 32 heads of 128 (0.70 GB) in 135 us, 0.76 of the measured copy rate
// (132 with cosines and sines an fp32 step off; then two blocks 146); keys and values alone 63 us, 41 as they are.
template <int G>
__global__ void __launch_bounds__(kThreads, 3) kv4_rotary_kernel(const __grid_constant__ RotaryArgs ra) {
    __shared__ __align__(16) uint8_t stage[kWarps][kv4_chunk_bytes(G)];
    __shared__ __align__(16) uint8_t table[16 * G * kTurnBlock];
    __shared__ uint8_t order[kWarps][16];
    pdl_launch_dependents();
    pdl_wait();
    const AppendArgs &a = ra.a;
    const int32_t warp = threadIdx.x >> 5, block = blockIdx.x;
    if (block >= ra.cache_blocks) {
        turn_queries<G>(ra, table, block - ra.cache_blocks);
        return;
    }
    const int32_t chunks = a.u.per_request / a.u.Hk;  // that a request may touch
    const int32_t slice = block % ra.slices, unit = block / ra.slices;
    const int32_t b = unit / chunks, ci = unit - b * chunks, hk = slice * kWarps + warp;
    append_chunk<G, true>(a, stage[warp], order[warp], table, &ra, b, ci * a.u.Hk + hk, ci, hk);
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
using RotaryKernel = void (*)(const RotaryArgs);
RotaryKernel rotary_kernel(int32_t G) {
    switch (G) {
        case 1: return kv4_rotary_kernel<1>;
        case 2: return kv4_rotary_kernel<2>;
        case 3: return kv4_rotary_kernel<3>;
        default: return kv4_rotary_kernel<4>;
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

// The pairs' frequencies as RotaryArgs has them.  A thread keeps those of its last base and head size: 64
// powers in 64 bits take longer than the launch.
void frequencies(float theta, int32_t D, uint64_t (&turn)[64]) {
    static thread_local struct {
        float theta;
        int32_t D;
        uint64_t turn[64];
    } last = {};
    if (last.theta != theta || last.D != D) {
        constexpr double kTwoPi = 6.283185307179586;
        for (int32_t j = 0; j < D / 2; ++j) {
            const double turns = std::pow(static_cast<double>(theta), -2.0 * j / D) / kTwoPi, part = turns - std::floor(turns);
            last.turn[j] = static_cast<uint64_t>(std::ldexp(part, 64));  // exact: part <= 1 - 2^-53
        }
        last.theta = theta;
        last.D = D;
    }
    std::copy(last.turn, last.turn + 64, turn);
}

// What the two writes have in common.
eagle_status append_args(const eagle_kv4_cache *cache, int32_t batch, int32_t src_rows, int32_t slots, const void *d_k,
                         const void *d_v, int64_t ld, const int32_t *d_select, const int32_t *d_count,
                         const int32_t *d_start, int32_t *d_status, AppendArgs *out) {
    AppendArgs &a = *out;
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
    a.lengths = a.start != cache->lengths ? cache->lengths : nullptr;
    return EAGLE_OK;
}

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
    const eagle_status bad = append_args(cache, batch, src_rows, slots, d_k, d_v, ld, d_select, d_count, d_start, d_status, &a);
    if (bad != EAGLE_OK || batch == 0) return bad;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (launch_pdl(append_kernel(a.v.G), grid_of(a.u), dim3(kThreads), 0, st, a) != cudaSuccess) return EAGLE_ERR_CUDA;
    if (!a.lengths && launch_pdl(kv4_lengths_kernel, dim3(batch), dim3(32), 0, st, a, cache->lengths) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    return EAGLE_OK;
}

eagle_status eagle_kv4_append_rotary(const eagle_kv4_cache *cache, int32_t batch, int32_t src_rows, int32_t slots,
                                     const void *d_k, const void *d_v, int64_t ld, const int32_t *d_positions,
                                     float rope_theta, int32_t heads, const void *d_q, int64_t ldq, void *d_q_out,
                                     const int32_t *d_select, const int32_t *d_count, const int32_t *d_start,
                                     int32_t *d_status, eagle_stream_t stream) {
    using namespace eagle;
    NvtxRange nvtx_range("eagle_kv4_append_rotary");
    RotaryArgs r{};
    const eagle_status bad = append_args(cache, batch, src_rows, slots, d_k, d_v, ld, d_select, d_count, d_start, d_status, &r.a);
    if (bad != EAGLE_OK) return bad;
    if (!(rope_theta > 0.0f) || (d_select && !d_positions) || misaligned(d_positions, 4)) return EAGLE_ERR_INVALID_ARG;
    if ((d_q == nullptr) != (d_q_out == nullptr)) return EAGLE_ERR_INVALID_ARG;
    if (batch == 0) return EAGLE_OK;
    const int32_t D = r.a.v.G * kKv4Group;
    if (d_q && (heads < 1 || heads > 65536 || ldq < static_cast<int64_t>(heads) * D || ldq % 8 || misaligned(d_q, 16) ||
                misaligned(d_q_out, 16)))
        return EAGLE_ERR_INVALID_ARG;
    r.positions = d_positions;
    r.minus_one = -1.0f;
    const int64_t units = r.a.u.total / r.a.u.Hk;  // (request, chunk)
    r.slices = (r.a.u.Hk + kWarps - 1) / kWarps;
    int64_t blocks = units * r.slices;
    r.cache_blocks = static_cast<int32_t>(blocks);
    if (d_q && src_rows > 0) {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EAGLE_ERR_CUDA;
        const int64_t rows = static_cast<int64_t>(batch) * src_rows;
        r.q = static_cast<const __nv_bfloat16 *>(d_q);
        r.q_out = static_cast<__nv_bfloat16 *>(d_q_out);
        r.ldq = ldq;
        r.H = heads;
        // as many rows a block as leave two blocks an SM, 16 at most (the table's)
        r.q_rows = static_cast<int32_t>(std::min<int64_t>(16, std::max<int64_t>(1, rows / (2 * sms))));
        blocks += (rows + r.q_rows - 1) / r.q_rows;
    }
    if (blocks > INT32_MAX) return EAGLE_ERR_UNSUPPORTED;
    frequencies(rope_theta, D, r.turn);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (launch_pdl(rotary_kernel(r.a.v.G), dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st, r) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    if (!r.a.lengths && launch_pdl(kv4_lengths_kernel, dim3(batch), dim3(32), 0, st, r.a, cache->lengths) != cudaSuccess)
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
