// kv4_attn_tc.cu - attention over the 4-bit cache for many query rows a kv head (large trees, grouped
// heads, pieces of a prompt), on tcgen05 with the accumulators in tensor memory.
//
// With R query rows a key costs 4 R D flops and is unpacked once for all of them, so from a few dozen
// rows on the tensor cores and the softmax bound the work and not the cache's bytes.  A CTA works on
// 256 query rows of one (request, kv head), as two streams of 128 rows that share every key and
// value tile; where a unit has at most 128 rows, both streams hold the same rows and take the even
// and the odd tiles, each with its own maximum, sum and output.  Tiles are 128 keys.
//   warps 0-7, 8-15  softmax of stream 0 and 1, two threads a row (its TMEM lane), each on 64 of the
//                    tile's keys: two passes over the scores (maximum; exponentials), p as fp16 into
//                    TMEM over the scores it came from, the running maximum and sum in fp32.  p is
//                    held below 2^15 and its reference only moved (and O rescaled) when a tile's
//                    maximum passes that; the halves agree on the maximum through shared memory.
//                    Warps whose 32 rows lie behind the unit's last skip the softmax.
//   warps 16-19, 20-23  fill the key and the value tiles: codes become fp16 values m + s c (one fused
//                    multiply-add: half an fp16 step, 2^-11 relative); new keys and values are
//                    converted from bf16 (exact but for what is said below).
//   warp 24          issues the MMAs: S = Q K^T (128 x 128 x D, operands in shared memory) and
//                    O += P V (P from TMEM, V as stored: the MN-major B operand).  The order S0 S1
//                    [P0] O0 S0' [P1] O1 S1' ... keeps one stream's MMAs under the other's softmax,
//                    and from a p's arrival on nothing else is waited for.  The warp stays whole and
//                    one lane's instructions count, so that descriptors are in uniform registers
//                    (moving them there cost 100 cycles an MMA).
//   warp 25          copies the codes of cached tiles, one tile's keys and one tile's values at a time
//
// What bounds it: instruction issue and the chain of one stream's tile (scores, two passes, p, product):
// the next 2047 tokens of two requests over 4096 cached ones (64 heads, 8 kv heads of 128)
// take 737 us, 0.50 of the measured bf16 matrix rate; 32 requests of 65 nodes (260 rows,
// a full unit and one of 4 rows each) over 1024 tokens 118 us.  Registers are what it is short of:
// 26 warps leave 72 a thread, and what is spilled goes to L2, as shared memory takes all of L1.  So is the
// instruction cache: what the loops of the roles grow by shows in the time (with new keys by batches of 8
// instead of 4 the first takes 833 us).  So the walk over the units lies in shared memory, and masks
// and the elements that fp16 does not hold have functions of their own.
//
// Queries are scaled by a power of two so that a row's largest element is 2^9..2^10 (exact, as in
// kv4_attn.cu).  Within 8 neighbouring dims the tiles hold them in the order 0 4 1 5 2 6 3 7, in
// which masking a word of codes leaves them; queries are stored in the same order and the output's
// columns are put right as they leave.
// New keys and values come to the tiles by pieces of 8 dims.  What fp16 does not hold (elements above 65504,
// infinite or NaN, and those below 2^-17, whose bits go on behind fp16's last of 2^-24) is looked at in pieces
// with one of the first or with no element of 2^-12 or more: there it counts as 0 in the tiles, and the rows
// that see it add its terms one by one.  So nothing hidden reaches a row, whatever it is, and sizes may be
// anything: only next to an element of 2^-12 or more do those below 2^-17 round, by 2^-25 at most (2^-13 of
// it, next to 2^-11 that p's rounding takes).  Multiplying new tiles in bf16 instead, with the queries in both
// types one after the other and p as hi + lo, took 866 us where this took 715 (2047 tokens of two prompts).
// Tiles are made of blocks of 64 dims; with head_dim 32 and 96 half of the last one lies idle and the
// MMAs stop before it (1000 tokens of two prompts over 4096 cached ones, 32 heads of 96: a tenth of the time
// that the few-row kernel took with 32 rows a unit).
// TMEM: S0 S1 O0 O1, 128 columns each (O uses D).  Every wait on an mbarrier is bounded; the roles meet at
// named barriers as often as the units and tiles say, also after a wait has given up.
#include <type_traits>

#include "kernels.cuh"
#include "kv4_line.cuh"

namespace eagle {
namespace {

constexpr int kKeys = kKv4TcTile;
constexpr int kThreads = 26 * 32;
constexpr int kFillWarps = 4;  // for the keys, and as many for the values
constexpr int kRaw = 2;        // a tile's codes in flight: the keys', the values'
constexpr float kTop = 15.0f, kAim = 4.0f;  // p <= 2^15; a new reference puts the largest at 2^4
constexpr uint32_t kTmemCols = 512;

template <int G>
struct Tc {
    static constexpr int D = G * kKv4Group;
    // a tile: blocks of [128 rows][128 bytes], 64 dims each (half of the last one idle with an odd G)
    static constexpr uint32_t kTileBytes = (D + 63) / 64 * (kKeys * 128u);
    // lanes that take a bf16 row's 16-byte pieces: kPer, of which the first kPieces have one
    static constexpr int kPieces = D / 8, kPer = G == 3 ? 16 : kPieces, kRowsWarp = 32 / kPer;
    static constexpr uint32_t kQ = 0;                      // two streams
    static constexpr uint32_t kK = kQ + 2 * kTileBytes;    // two stages
    static constexpr uint32_t kV = kK + 2 * kTileBytes;    // two stages
    static constexpr uint32_t kPart = 320u * G;            // a chunk's keys or values: codes and parameters
    static constexpr uint32_t kCodes = kV + 2 * kTileBytes;  // kRaw stages of eight such parts
    static constexpr uint32_t kTotal = kCodes + kRaw * 8 * kPart + 1024;  // and alignment
};

struct TcBars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // stages
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2];    // streams
    uint64_t raw_full[kRaw], raw_empty[kRaw];
    uint64_t drain;
};

__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t chunk) {
    return (row >> 3) * 1024u + (row & 7u) * 128u + ((chunk ^ (row & 7u)) << 4);
}

// The MMAs and their commit, issued by the lane whose `leader` is set; the whole warp takes part.
// D[tmem] (+)= A[smem] * B[smem] and D[tmem] += A[tmem] * B[smem], fp16 in, fp32 accumulation.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_to(uint64_t *bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ uint32_t elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void tmem_st_8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ float tmem_ld_1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    tmem_wait_ld();
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st_1(uint32_t taddr, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
    tmem_wait_st();
}

// kind::f16 with fp16 A and B and fp32 D (common.cuh has the fields).
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24); }
__host__ __device__ constexpr uint32_t idesc_f16_bmn(uint32_t m, uint32_t n) { return idesc_f16(m, n) | (1u << 16); }

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// Eight codes to m + s c, pairs (0, 4), (1, 5), (2, 6), (3, 7).  A code in the low bits of fp16 1024
// is 1024 + c, one four bits higher 1024 + 16 c; both come down to c exactly.
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t sm) {
    const __half2 s = __low2half2(as_h2(sm)), m = __high2half2(as_h2(sm));
    const __half2 k1024 = __half2half2(__ushort_as_half(0x6400)), k64 = __half2half2(__ushort_as_half(0xd400));
    const __half2 k16th = __half2half2(__ushort_as_half(0x2c00));
    const uint32_t w8 = w >> 8;
    const __half2 c0 = __hsub2(as_h2((w & 0x000f000fu) | 0x64006400u), k1024);
    const __half2 c1 = __hfma2(as_h2((w & 0x00f000f0u) | 0x64006400u), k16th, k64);
    const __half2 c2 = __hsub2(as_h2((w8 & 0x000f000fu) | 0x64006400u), k1024);
    const __half2 c3 = __hfma2(as_h2((w8 & 0x00f000f0u) | 0x64006400u), k16th, k64);
    return make_uint4(as_u32(__hfma2(c0, s, m)), as_u32(__hfma2(c1, s, m)), as_u32(__hfma2(c2, s, m)), as_u32(__hfma2(c3, s, m)));
}
// A piece of 8 bf16 with 0 in place of what the tiles do not hold: nothing, where its largest magnitude is
// 2^-12 .. 65504; else elements above 65504 or no number, and those below 2^-17 (their fp16 steps are 2^-24).
static __device__ __noinline__ uint4 without_odd(uint4 v) {
    constexpr uint32_t kMost = 0x477fu, kSmall = 0x3980u, kExact = 0x3700u;  // bf16 65280, 2^-12, 2^-17
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = max(most, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    if (most >= kSmall && most <= kMost) return v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        if (lo > kMost || lo < kExact) w[i] &= 0xffff0000u;
        if (hi > kMost || hi < kExact) w[i] &= 0x0000ffffu;
    }
    return v;
}
// The elements that are not 0 there: what the piece holds and the tiles do not.
__device__ __forceinline__ uint4 odd_of(uint4 v) {
    const uint4 y = without_odd(v);
    return make_uint4(v.x ^ y.x, v.y ^ y.y, v.z ^ y.z, v.w ^ y.w);
}
__device__ __forceinline__ bool is_any(uint4 v) { return ((v.x | v.y | v.z | v.w) & 0x7fff7fffu) != 0u; }
// Eight bf16 to fp16 in the order of the tiles.
__device__ __forceinline__ uint4 convert8(uint4 v) {
    return make_uint4(pack_f16(bf_lo(v.x), bf_lo(v.z)), pack_f16(bf_hi(v.x), bf_hi(v.z)), pack_f16(bf_lo(v.y), bf_lo(v.w)),
                      pack_f16(bf_hi(v.y), bf_hi(v.w)));
}

// The terms of what the tiles do not hold, for the rows of the warp: of the keys into the row's scores
// (f: what the query was scaled by; keys first .. last of the tile), of the values into dims first ..
// last of its output, where the row sees the key.  `rows`: keys of the tile.  All lanes look at the same pieces.
template <int D>
static __device__ __noinline__ void add_odd_keys(const __nv_bfloat16 *kt, int64_t ld, int32_t first, int32_t last,
                                                 const __nv_bfloat16 *q, float f, uint32_t t_s) {
#pragma unroll 1
    for (int32_t key = first; key < last; ++key) {
        float add = 0.0f;
        bool any = false;
#pragma unroll 1
        for (int32_t d = 0; d < D; d += 8) {
            const uint4 z = odd_of(*reinterpret_cast<const uint4 *>(kt + key * ld + d));
            if (!is_any(z)) continue;
            any = true;
            const uint4 x = *reinterpret_cast<const uint4 *>(q + d);
            const uint32_t zw[4] = {z.x, z.y, z.z, z.w}, xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (zw[i] & 0x7fffu) add += bf_lo(xw[i]) * f * bf_lo(zw[i]);
                if (zw[i] & 0x7fff0000u) add += bf_hi(xw[i]) * f * bf_hi(zw[i]);
            }
        }
        __syncwarp();
        if (any) tmem_st_1(t_s + key, tmem_ld_1(t_s + key) + add);
    }
}
static __device__ __noinline__ void add_odd_values(const __nv_bfloat16 *vt, int64_t ld, int32_t rows, uint4 see, float mul,
                                                   float sub, uint32_t t_s, uint32_t t_o, int32_t first, int32_t last) {
#pragma unroll 1
    for (int32_t key = 0; key < rows; ++key) {
        const float pv = ex2_approx(__fadd_rn(__fmul_rn(tmem_ld_1(t_s + key), mul), sub));
        const uint32_t word = key < 64 ? (key < 32 ? see.x : see.y) : (key < 96 ? see.z : see.w);
        const bool mine = (word >> (key & 31)) & 1u;
#pragma unroll 1
        for (int32_t d = first; d < last; d += 8) {
            const uint4 z = odd_of(*reinterpret_cast<const uint4 *>(vt + key * ld + d));
            if (!is_any(z)) continue;
            const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
            uint32_t o[8];  // in the order 0 4 1 5 2 6 3 7
            tmem_ld_8(t_o + d, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = ((i & 3) << 1) | (i >> 2);
                const float x = i & 1 ? bf_hi(zw[i >> 1]) : bf_lo(zw[i >> 1]);
                if (mine && x != 0.0f) o[at] = __float_as_uint(__uint_as_float(o[at]) + pv * x);
            }
            __syncwarp();
            tmem_st_8(t_o + d, o);
            tmem_wait_st();
        }
    }
}

// The largest of three.
__device__ __forceinline__ float max_3(float a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

// Scores of keys that the row does not see become -inf: most tiles have none, and their loops know
// nothing of masks.  Warp-wide, as all of these.
static __device__ __noinline__ void hide_keys(uint32_t t, uint32_t see0, uint32_t see1) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t v[16];
        tmem_ld_16(t + 16 * c, v);
        tmem_wait_ld();
        const uint32_t bits = (c < 2 ? see0 : see1) >> (16 * (c & 1));
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = (bits >> i) & 1u ? v[i] : __float_as_uint(-INFINITY);
        tmem_st_16(t + 16 * c, v);
    }
    tmem_wait_st();
}

// p = 2^(score mul + sub) of 64 keys, as fp16 over the first 32 columns of their scores; returns the
// sum.  One product and difference; `steps`: in two, as the maximum was formed, for scores so large
// that the product's rounding matters next to their differences (and could pass for a score above
// the maximum).
__device__ __forceinline__ float probabilities(uint32_t t, float mul, float sub) {
    const uint64_t mul2 = pack_2(__float_as_uint(mul), __float_as_uint(mul)), sub2 = pack_2(__float_as_uint(sub), __float_as_uint(sub));
    uint64_t sum = 0;
#pragma unroll 2
    for (int c = 0; c < 4; ++c) {
        uint32_t v[16], pk[8];
        tmem_ld_16(t + 16 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 x = unpack_2(fma_2(pack_2(v[2 * i], v[2 * i + 1]), mul2, sub2));
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            sum = add_2(sum, pack_2(__float_as_uint(p0), __float_as_uint(p1)));
            pk[i] = pack_f16(p0, p1);
        }
        tmem_st_8(t + 8 * c, pk);
    }
    const float2 x = unpack_2(sum);
    return x.x + x.y;
}
static __device__ __noinline__ float probabilities_in_steps(uint32_t t, float mul, float sub) {
    float sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t v[16], pk[8];
        tmem_ld_16(t + 16 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p0 = ex2_approx(__fadd_rn(__fmul_rn(__uint_as_float(v[2 * i]), mul), sub));
            const float p1 = ex2_approx(__fadd_rn(__fmul_rn(__uint_as_float(v[2 * i + 1]), mul), sub));
            sum += p0 + p1;
            pk[i] = pack_f16(p0, p1);
        }
        tmem_st_8(t + 8 * c, pk);
    }
    return sum;
}

// A unit's sums from segment to segment, at a segment's end: what came before (`begun`), brought to this
// segment's reference, joins the accumulator, and if the unit goes on the sum moves to memory.  Each thread has
// its half of its row of the partial sums (stream 1's behind stream 0's) and a (ref, l) of its own, ml.
template <int D>
static __device__ __noinline__ void carry_over(const Kv4Args &k, const Walk &w, uint32_t t_o, float2 *ml) {
    const float ref = ml->x;
    float l = ml->y;
    const int32_t row = threadIdx.x >> 8 << 7 | (threadIdx.x & 127), first = (threadIdx.x >> 7 & 1) * (D / 2);
    const bool begun = w.s0 > w.from, goes_on = w.s1 < w.to;
    float *part = k.part_o + (slot_of(w) * kKv4TcRows + row) * D + first;
    float2 *at = k.carry_ml + static_cast<int64_t>(blockIdx.x) * kKv4Carry + threadIdx.x;
    float f = 0.0f;
    if (begun) {
        const float2 was = *at;
        f = was.x == -INFINITY ? 0.0f : ex2_approx(was.x - ref);
        l = fmaf(was.y, f, l);
    }
    *(goes_on ? at : ml) = make_float2(ref, l);
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 16) {
        uint32_t v[16];
        tmem_ld_16(t_o + first + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float4 x = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            float4 *to = reinterpret_cast<float4 *>(part + c + i);
            if (begun) {
                const float4 y = *to;
                x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
            }
            if (goes_on) *to = x;
            v[i] = __float_as_uint(x.x), v[i + 1] = __float_as_uint(x.y), v[i + 2] = __float_as_uint(x.z), v[i + 3] = __float_as_uint(x.w);
        }
        if (!goes_on) tmem_st_16(t_o + first + c, v);
    }
    tmem_wait_st();
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1) kv4_attention_tc_kernel(const __grid_constant__ Kv4Args k) {
    using S = Tc<G>;
    constexpr int D = S::D;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    __shared__ TcBars bar;
    __shared__ uint32_t tmem_base;
    __shared__ int32_t abort_mark;
    // By tile & 7: which of its 128 keys are there.  Written ahead of the tile itself, when the scores of
    // the tile three before are there: the other stream may not have looked at the tile four before yet.
    __shared__ __align__(8) uint8_t key_bits[8][16];
    __shared__ uint8_t raw_keys[kRaw][8];             // keys of each chunk that are there
    __shared__ __align__(4) uint8_t odd_tile[4][2][kFillWarps];  // by tile & 3, key or value, filling warp
    __shared__ int32_t row_at[2][128];        // stream, row: node << 16 | head, -1 behind the unit's last row
    __shared__ float2 q_scale[2][128];        // what a row's query and its scores are multiplied by
    __shared__ float half_max[2][2][2][128];  // stream, exchange & 1, half, row
    __shared__ float2 half_ml[2][2][128];     // stream, half, row: references and sums of a segment
    __shared__ int32_t red[kThreads / 32];
    __shared__ Spot spots[2];
    __shared__ Place place;
    __shared__ Lengths lens;
    __shared__ Walk walks[kThreads / 32];  // each warp's: in registers they would be spilled, and L1 is all shared memory here
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int32_t *abort_flag = &abort_mark;
    const Kv4Attention &a = k.a;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.k_full[i], kFillWarps);
            mbar_init(&bar.v_full[i], kFillWarps);
            mbar_init(&bar.k_empty[i], 1);
            mbar_init(&bar.v_empty[i], 1);
            mbar_init(&bar.q_full[i], 8);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 8);
            mbar_init(&bar.o_done[i], 1);
        }
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], kFillWarps);
        }
        mbar_init(&bar.drain, 1);
        abort_mark = 0;
        fence_barrier_init();
    }
    pdl_wait();  // and no early launch of dependents (kv4_attn.cu)
    if (!find_place(k, place, lens, red, spots)) {
        if (threadIdx.x == 0) k.share[blockIdx.x].kind = 0;
        return;
    }
    if (lane == 0) {
        Walk first;
        first.start(k, place, lens);
        walks[warp] = first;
        if (warp == 0) k.share[blockIdx.x] = share_of(first);
    }
    if (warp == 24) {
        tmem_alloc(&tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, tmem_base, 0);
    const Walk &w = walks[warp];
    auto next_unit = [&]() { return kv4_next(k, place, walks[warp], lens, kThreads, warp == 25); };
    auto wait = [&](uint64_t *b, uint32_t parity) -> bool { return kv4_wait(b, parity, abort_flag, a.limit_ns); };
    auto rows_of = [&]() { return min(kKv4TcRows, k.Mq - w.qt * kKv4TcRows); };  // rows of the unit

    if (warp >= 16 && warp < 24) {
        // ---------------- the tiles: four warps for the keys, four for the values ----------------
        const int32_t half = (warp - 16) >> 2, fw = warp & 3;
        uint64_t *const full = half ? bar.v_full : bar.k_full, *const empty = half ? bar.v_empty : bar.k_empty;
        uint8_t *const stages = base + (half ? S::kV : S::kK);
        uint32_t gt = 0, raw = 0;  // tiles and cached tiles so far
        do {
            int32_t s = w.s0;
            if (s < w.nt) {  // new keys or values, the next ones' loads under way
                constexpr int kPer = S::kPer, kRowsWarp = S::kRowsWarp;
                constexpr int kBatch = 4;  // with 8 the loops miss the instruction cache more: 65-node trees 123 us, not 114
                constexpr int kBatches = kKeys / (4 * kRowsWarp * kBatch);
                const int32_t ch = lane % kPer, first = fw * kRowsWarp + lane / kPer;
                const bool mine = S::kPieces == kPer || ch < S::kPieces;
                const __nv_bfloat16 *src = (half ? a.vn : a.kn) + static_cast<int64_t>(w.b) * a.n * a.ldkv + static_cast<int64_t>(w.hk) * D + ch * 8;
                uint4 v[kBatch];
                auto load = [&](int32_t row0) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int32_t row = row0 + i * 4 * kRowsWarp + first;
                        v[i] = mine && row < a.n ? *reinterpret_cast<const uint4 *>(src + row * a.ldkv) : make_uint4(0, 0, 0, 0);
                    }
                };
                load(s * kKeys);
                const int32_t last = min(w.s1, w.nt);
                bool odd = false;
#pragma unroll 1
                for (int32_t at = s * kBatches; at < last * kBatches; ++at) {
                    const uint32_t st = gt & 1u;
                    const int32_t sub = at % kBatches;
                    if (sub == 0) {
                        odd = false;
                        if (gt >= 2) wait(&empty[st], (gt >> 1) - 1);
                        __syncwarp();
                    }
                    uint8_t *dst = stages + st * S::kTileBytes + (ch >> 3) * (kKeys * 128);
                    auto store = [&](int32_t i, uint4 x) {
                        if (mine) *reinterpret_cast<uint4 *>(dst + sw128((sub * kBatch + i) * 4 * kRowsWarp + first, ch & 7)) = x;
                    };
                    // the largest magnitude of the results is infinite or NaN where an element is above fp16's,
                    // and that of a small piece is below 2^-12
                    __half2 big = as_h2(0u), small = as_h2(0x3c003c00u);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const uint4 x = convert8(v[i]);
                        const __half2 most = __hmax2_nan(__hmax2_nan(__habs2(as_h2(x.x)), __habs2(as_h2(x.y))),
                                                         __hmax2_nan(__habs2(as_h2(x.z)), __habs2(as_h2(x.w))));
                        big = __hmax2_nan(big, most);
                        small = __hmin2(small, __hmax2(most, __lowhigh2highlow(most)));
                        store(i, x);
                    }
                    if (!(__low2float(big) <= 65504.0f && __high2float(big) <= 65504.0f && __low2float(small) >= 0x1p-12f)) {
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const uint4 x = without_odd(v[i]);
                            if (((x.x ^ v[i].x) | (x.y ^ v[i].y) | (x.z ^ v[i].z) | (x.w ^ v[i].w)) & 0x7fff7fffu) {
                                odd = true;
                                store(i, convert8(x));
                            }
                        }
                    }
                    if (at + 1 < last * kBatches) load((at + 1) * (kKeys / kBatches));
                    if (sub == kBatches - 1) {
                        const bool any = __any_sync(kFull, odd);
                        if (lane == 0) odd_tile[gt & 3][half][fw] = any;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[st]);
                        ++gt;
                    }
                }
                s = last;
            }
#pragma unroll 1
            for (; s < w.s1; ++s, ++gt, ++raw) {
                const uint32_t st = gt & 1u;
                wait(&bar.raw_full[half], raw);
                const uint8_t *src = base + S::kCodes + half * 8 * S::kPart;
                // lanes: four pieces of 8 dims of rows t and t + 4: the stores of eight lanes touch
                // all banks
                const int32_t m = lane >> 2, q = lane & 3;
                const int32_t t8 = (m >> 1) | ((m & 1) << 2);          // token among the 8
                const int32_t slot8 = half ? t8 : m;                   // its row
                const int32_t qq = half && G == 4 ? q ^ (t8 & 2) : q;  // value rows' halves change places
                // group i of 8 rows: 1024 bytes on; dims 32 g + 8 q: chunk 4 g + q
                uint8_t *to = stages + st * S::kTileBytes + fw * 1024 + t8 * 128 + ((qq ^ t8) << 4);
                const int32_t odd_g = ((((4 + qq) ^ t8) - (qq ^ t8)) << 4);
                uint32_t c[4][G], sm[4][G];
#pragma unroll
                for (int32_t i = 0; i < 4; ++i) {
                    const int32_t group = 4 * i + fw;
                    const uint8_t *part = src + (group >> 1) * S::kPart;
                    const int32_t slot = (group & 1) * 8 + slot8;
                    const int32_t here = max(0, min(8, static_cast<int32_t>(raw_keys[half][group >> 1]) - 8 * (group & 1)));
                    load_words<G>(part + slot * 16 * G + q * 4 * G, c[i]);
                    load_words<G>(part + 256 * G + slot * 4 * G, sm[i]);
                    if (!half && lane == 0) key_bits[gt & 7][group] = static_cast<uint8_t>((1u << here) - 1u);
                    if (t8 >= here) {  // rows that are not there hold 0
#pragma unroll
                        for (int g = 0; g < G; ++g) c[i][g] = sm[i][g] = 0u;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.raw_empty[half]);
                if (gt >= 2) wait(&empty[st], (gt >> 1) - 1);
                __syncwarp();
#pragma unroll
                for (int32_t i = 0; i < 4; ++i) {
                    if (half) {  // two 16-bit words of four dims each, G apart, to the keys' words of eight
                        uint32_t x[G];
#pragma unroll
                        for (int g = 0; g < G; ++g)
                            x[g] = __byte_perm(c[i][g / 2], c[i][(G + g) / 2], (g & 1 ? 0x32 : 0x10) | ((G + g) & 1 ? 0x7600 : 0x5400));
#pragma unroll
                        for (int g = 0; g < G; ++g) c[i][g] = x[g];
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        *reinterpret_cast<uint4 *>(to + i * 4096 + (g >> 1) * (kKeys * 128) + (g & 1 ? odd_g : 0)) = dequant8(c[i][g], sm[i][g]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
            }
        } while (next_unit());
    } else if (warp == 25) {
        // ---------------- copies of codes: a stage is the keys or the values of a cached tile -------
        uint32_t raw = 0;
        bool dead = false;
        do {
            if (lane == 0 && w.len != lens.of(w.b)) latch(a.status, kDevBounds);  // clamped
            const int32_t k0 = max(w.s0 - w.nt, 0), k1 = w.s1 - w.nt;
            for (int32_t kt = k0; kt < k1 && !dead; kt += 4) {
                // the chunks of four tiles, one a lane
                const int32_t key = kt * kKeys + lane * 16;
                int32_t nv = min(max(w.len - key, 0), 16);
                const uint8_t *src = nullptr;
                if (nv > 0 && kt + (lane >> 3) < k1) {
                    src = kv4_chunk(a.cache, w.b, w.hk, key);
                    if (!src) latch(a.status, kDevBounds);  // its keys count as absent
                }
                if (!src) nv = 0;
                const int32_t halves = 2 * min(k1 - kt, 4);
                for (int32_t hh = 0; hh < halves; ++hh, ++raw) {
                    const uint32_t rs = raw % kRaw;
                    if (raw >= kRaw && lane == 0) wait(&bar.raw_empty[rs], raw / kRaw - 1);
                    dead = __shfl_sync(kFull, static_cast<int>(*abort_flag), 0) != 0;
                    dead = dead || static_cast<int32_t>(raw >> 1) >= a.stall;
                    if (dead) break;
                    const bool my = (lane >> 3) == (hh >> 1);
                    const uint32_t have = __ballot_sync(kFull, my && src);
                    if (my) raw_keys[rs][lane & 7] = static_cast<uint8_t>(nv);
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&bar.raw_full[rs], __popc(have) * S::kPart);
                    __syncwarp();
                    if (my && src)
                        bulk_load(base + S::kCodes + rs * 8 * S::kPart + (lane & 7) * S::kPart, src + (hh & 1 ? S::kPart : 0u), S::kPart,
                                  &bar.raw_full[rs]);
                }
            }
        } while (next_unit());
        // every copy has landed before the block's memory is handed on
        if (lane == 0)
            for (uint32_t i = raw > kRaw ? raw - kRaw : 0; i < raw; ++i) mbar_wait(&bar.raw_full[i % kRaw], (i / kRaw) & 1u, nullptr);
        __syncwarp();
    } else if (warp == 24) {
        // ---------------- MMA issue ----------------
        constexpr uint32_t idesc_s = idesc_f16(128, kKeys), idesc_o = idesc_f16_bmn(128, D);
        constexpr uint32_t kStep = S::kTileBytes >> 4;  // descriptors count in 16 bytes
        const uint32_t leader = elected();
        uint32_t gt = 0, seg = 0, jobs0 = 0, jobs1 = 0;  // tiles, segments, P's of each stream so far
        const uint64_t q_desc = sw128_kmajor_desc(smem_u32(base + S::kQ)), k_desc = sw128_kmajor_desc(smem_u32(base + S::kK));
        const uint64_t v_desc = sw128_desc(smem_u32(base + S::kV), kKeys * 128u, 1024u);
        // the warp stays whole when a wait gives up, too
        auto wait_all = [&](uint64_t *b, uint32_t parity) -> bool { return __all_sync(kFull, wait(b, parity)); };
        bool ok = true;
        do {
            if (!ok) continue;
            const int32_t tiles = __shfl_sync(kFull, w.s1 - w.s0, 0);
            const uint32_t both = __shfl_sync(kFull, rows_of() > 128 ? 1 : 0, 0);
            const int32_t n = tiles << both;
            auto key_tile = [&](int32_t q) -> bool {  // the first of a tile's jobs waits for both
                const uint32_t t = gt + (q >> both);
                return (both && (q & 1)) || wait_all(&bar.k_full[t & 1u], t >> 1);
            };
            auto issue_s = [&](int32_t q) {
                const uint32_t t = gt + (q >> both), st = t & 1u, j = q & 1;
                const uint64_t qd = q_desc + j * kStep, kd = k_desc + st * kStep;
                const uint32_t d = tmem + j * 128u;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * (kKeys * 128u) + (kk & 3) * 32u) >> 4;
                    mma_ss(d, qd + off, kd + off, idesc_s, kk > 0, leader);
                }
                commit_to(&bar.s_full[j], leader);
                if (!both || j) commit_to(&bar.k_empty[st], leader);  // the tile's last reader
            };
            ok = wait_all(&bar.q_full[0], seg) && key_tile(0);
            tc_fence_after();
            if (ok) issue_s(0);
            ok = ok && wait_all(&bar.q_full[1], seg) && (n < 2 || key_tile(1));
            tc_fence_after();
            if (ok && n >= 2) issue_s(1);
            for (int32_t q = 0; q < n && ok; ++q) {
                const uint32_t t = gt + (q >> both), st = t & 1u, j = q & 1;
                // everything but p is waited for ahead of it: from its arrival the products of the
                // job and the scores of the stream's next one follow each other
                ok = ((both && j) || wait_all(&bar.v_full[st], t >> 1)) && (q + 2 >= n || key_tile(q + 2)) &&
                     wait_all(&bar.p_full[j], j ? jobs1 : jobs0);
                if (!ok) break;
                if (j) ++jobs1;
                else ++jobs0;
                tc_fence_after();
                const uint64_t vd = v_desc + st * kStep;
                const uint32_t d = tmem + 256u + j * 128u, pa = tmem + j * 128u;
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)  // keys 64 .. 127 lie 64 columns on
                    mma_ts(d, pa + (kk & 3) * 8u + (kk >> 2) * 64u, vd + kk * 128u, idesc_o, leader);
                if (!both || j) commit_to(&bar.v_empty[st], leader);
                if (q + 2 < n) issue_s(q + 2);
                else commit_to(&bar.o_done[j], leader);
            }
            gt += tiles;
            ++seg;
        } while (next_unit());
        // what was issued lands before the block's memory is handed on
        commit_to(&bar.drain, leader);
        mbar_wait(&bar.drain, 0, nullptr);
        __syncwarp();
    } else if (warp < 16) {
        // ---------------- softmax and output ----------------
        // stream, half of a tile's keys (and of the output's columns), row of the stream
        const int32_t j = warp >> 3, h = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + j * 128u, t_h = t_s + 64 * h, t_o = tmem + lanes + 256u + j * 128u;
        uint32_t gt = 0, n_s = 0, n_o = 0;  // tiles, scores and outputs of this stream so far
        do {
            const bool both = rows_of() > 128;
            bool live, used;  // the thread's row, any of the warp's
            {
                const int32_t unit_rows = rows_of(), ur = both ? j * 128 + r : r, row = w.qt * kKv4TcRows + ur;
                live = ur < unit_rows;
                used = ur - lane < unit_rows;
                const int32_t node = row / k.group;
                if (h == 0) row_at[j][r] = live ? (node << 16) | (w.hk * k.group + row - node * k.group) : -1;
            }
            __syncwarp();
            named_barrier_sync(1 + j, 256);
            // the stream's queries, whole rows at a time: scaled, to fp16, and what turns a row's
            // scores to base 2
            constexpr int kPer = S::kPer, kRowsLoad = S::kRowsWarp, kBatch = 16 / kRowsLoad < 4 ? 16 / kRowsLoad : 4;
            const int32_t w8 = warp & 7, piece = lane % kPer;
            const bool mine = S::kPieces == kPer || piece < S::kPieces;
#pragma unroll 1
            for (int32_t i0 = 0; i0 < 16 / kRowsLoad; i0 += kBatch) {
                uint4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int32_t at = row_at[j][(i0 + i) * kRowsLoad + w8 * 16 + lane / kPer];
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (mine && at >= 0)
                        v[i] = *reinterpret_cast<const uint4 *>(a.q + (static_cast<int64_t>(w.b) * a.n + (at >> 16)) * a.ldq +
                                                                 static_cast<int64_t>(at & 0xffff) * D + 8 * piece);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int32_t qr = (i0 + i) * kRowsLoad + w8 * 16 + lane / kPer;
                    const uint32_t vw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t big = 0;  // magnitudes compare as whole numbers, NaN above all
#pragma unroll
                    for (int u = 0; u < 4; ++u) big = max(big, max((vw[u] << 16) & 0x7fffffffu, vw[u] & 0x7fff0000u));
#pragma unroll
                    for (int off = 1; off < kPer; off <<= 1) big = max(big, __shfl_xor_sync(kFull, big, off));
                    const int32_t e = max(static_cast<int32_t>(big >> 23), 10);
                    const float f = __uint_as_float(static_cast<uint32_t>(263 - e) << 23);
                    if (mine)
                        *reinterpret_cast<uint4 *>(base + S::kQ + j * S::kTileBytes + (piece >> 3) * (kKeys * 128) + sw128(qr, piece & 7)) =
                            make_uint4(pack_f16(bf_lo(v[i].x) * f, bf_lo(v[i].z) * f), pack_f16(bf_hi(v[i].x) * f, bf_hi(v[i].z) * f),
                                   pack_f16(bf_lo(v[i].y) * f, bf_lo(v[i].w) * f), pack_f16(bf_hi(v[i].y) * f, bf_hi(v[i].w) * f));
                    if (piece == 0) q_scale[j][qr] = make_float2(f, __uint_as_float(static_cast<uint32_t>(e - 9) << 23) * k.scale2);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_full[j]);
            __syncwarp();
            {
                uint32_t z[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tmem_st_16(t_o + h * (D / 2) + 16 * c, z);
                tmem_wait_st();
            }
            named_barrier_sync(1 + j, 256);
            const float mul = q_scale[j][r].y;
            // which of new keys k0 .. k0 + 31 the row sees
            auto new_seen = [&](int32_t k0) {
                const int32_t node = max(row_at[j][r], 0) >> 16;
                const uint32_t *mrow = a.mask ? a.mask + (static_cast<int64_t>(w.b) * a.n + node) * k.W : nullptr;
                const int32_t left = a.n - k0, own = node - k0;  // causal: nodes 0..node
                uint32_t v = own >= 31 ? kFull : (own >= 0 ? (2u << own) - 1u : 0u);
                if (mrow) v = left > 0 ? mrow[k0 >> 5] : 0u;
                return v & (left >= 32 ? kFull : (left > 0 ? (1u << left) - 1u : 0u));
            };
            // the first of new tile s's keys or values
            auto new_row = [&](int32_t s) {
                return (static_cast<int64_t>(w.b) * a.n + s * kKeys) * a.ldkv + static_cast<int64_t>(w.hk) * D;
            };
            float ref = -INFINITY, l = 0.0f;
            if (w.s0 > w.from) ref = half_ml[j][h][r].x;  // the unit goes on
            // the segment's tiles, those of new keys among them, and the stream's first and step
            const int32_t tiles = w.s1 - w.s0, fresh = max(w.nt - w.s0, 0), from = both ? 0 : j, step = both ? 1 : 2;
            for (int32_t i = from; i < tiles; i += step) {
                const uint32_t t = gt + i;
                // which of this half's keys the row sees
                uint32_t see0 = 0u, see1 = 0u;
                if (i < fresh) {
                    const int32_t key0 = (w.s0 + i) * kKeys + 64 * h;
                    see0 = new_seen(key0);
                    see1 = new_seen(key0 + 32);
                }
                wait(&bar.s_full[j], n_s);
                __syncwarp();
                tc_fence_after();
                if (i >= fresh) {
                    const uint2 b = *reinterpret_cast<const uint2 *>(key_bits[t & 7] + 8 * h);
                    see0 = b.x;
                    see1 = b.y;
                } else if (used && *reinterpret_cast<const volatile uint32_t *>(odd_tile[t & 3][0]) != 0) {
                    const int32_t at = max(row_at[j][r], 0);  // rows that are not there read a query that is
                    const int32_t s = w.s0 + i;
                    add_odd_keys<D>(a.kn + new_row(s), a.ldkv, 64 * h, min(a.n - s * kKeys, 64 * h + 64),
                                    a.q + (static_cast<int64_t>(w.b) * a.n + (at >> 16)) * a.ldq + static_cast<int64_t>(at & 0xffff) * D, q_scale[j][r].x, t_s);
                }
                if (!live) see0 = see1 = 0u;
                float mx = -INFINITY;
                if (used) {
                    if (!__all_sync(kFull, (see0 & see1) == kFull)) hide_keys(t_h, see0, see1);
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t v[32];
                        tmem_ld_32(t_h + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) m4[(i >> 1) & 3] = max_3(m4[(i >> 1) & 3], v[i], v[i + 1]);
                    }
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                }
                // the row's maximum over both halves
                half_max[j][n_s & 1u][h][r] = mx;  // the other one at every second tile
                bool odd_values = false;  // whether a new tile's values are not all held
                if (i < fresh) {
                    // one answer for the stream, whose threads all go on to the next barrier or none: where the
                    // wait has given up, the mark may be changing
                    const bool come = wait(&bar.v_full[t & 1], t >> 1);
                    const bool odd = *reinterpret_cast<const volatile uint32_t *>(odd_tile[t & 3][1]) != 0;
                    __syncwarp();
                    odd_values = named_barrier_or(1 + j, 256, come && odd);
                } else {
                    named_barrier_sync(1 + j, 256);
                }
                mx = fmaxf(mx, half_max[j][n_s & 1u][h ^ 1][r]);
                ++n_s;
                mx = mx == -INFINITY ? mx : mx * mul;  // mul may underflow to 0
                float corr = 1.0f;
                if (mx - ref > kTop) {
                    const float nr = mx - kAim;
                    corr = ref == -INFINITY ? 0.0f : ex2_approx(ref - nr);
                    l *= corr;
                    ref = nr;
                }
                const float sub = ref == -INFINITY ? 0.0f : -ref;
                if (used && i > from && __any_sync(kFull, corr != 1.0f)) {
                    // the scores' arrival says that the stream's earlier products are complete
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[16];
                        tmem_ld_16(t_o + h * (D / 2) + 16 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * corr);
                        tmem_st_16(t_o + h * (D / 2) + 16 * c, v);
                    }
                    tmem_wait_st();
                }
                if (odd_values) {
                    const int32_t s = w.s0 + i, key0 = s * kKeys;
                    uint4 see = make_uint4(0u, 0u, 0u, 0u);
                    if (live) see = make_uint4(new_seen(key0), new_seen(key0 + 32), new_seen(key0 + 64), new_seen(key0 + 96));
                    __syncwarp();
                    if (used)
                        add_odd_values(a.vn + new_row(s), a.ldkv, min(a.n - s * kKeys, kKeys), see, mul, sub, t_s, t_o, h * (D / 2), (h + 1) * (D / 2));
                    named_barrier_sync(1 + j, 256);  // both halves have read the scores that p overwrites
                }
                if (used) l += __any_sync(kFull, fabsf(sub) > 1048576.0f) ? probabilities_in_steps(t_h, mul, sub) : probabilities(t_h, mul, sub);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[j]);
                __syncwarp();
            }
            gt += tiles;
            // ---------------- the segment's output ----------------
            if (from < tiles) {
                wait(&bar.o_done[j], n_o);
                ++n_o;
            }
            __syncwarp();
            // the halves' sums, and of a unit of at most 128 rows both streams' shares
            half_ml[j][h][r] = make_float2(ref, l);
            if (w.s0 > w.from || w.s1 < w.to) {
                tc_fence_after();
                carry_over<D>(k, w, t_o, &half_ml[j][h][r]);
                if (w.s1 < w.to) continue;
            }
            tc_fence_before();
            if (both) named_barrier_sync(1 + j, 256);
            else named_barrier_sync(3, 512);
            tc_fence_after();
            const bool whole = w.from == 0 && w.s1 == w.unit;
            const int32_t ur = both ? j * 128 + r : r;
            const int64_t slot = slot_of(w);
            const uint32_t o_first = tmem + lanes + 256u;
            float M, L, w0 = 1.0f, w1 = 0.0f;
            if (both) {
                M = ref;
                L = half_ml[j][0][r].y + half_ml[j][1][r].y;
            } else {
                const float m0 = half_ml[0][0][r].x, m1 = half_ml[1][0][r].x;
                const float l0 = half_ml[0][0][r].y + half_ml[0][1][r].y, l1 = half_ml[1][0][r].y + half_ml[1][1][r].y;
                M = fmaxf(m0, m1);
                w0 = weight_of(m0, l0, M);
                w1 = weight_of(m1, l1, M);
                L = w0 * l0 + w1 * l1;
            }
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            const bool ok = __all_sync(kFull, !*abort_flag);
            // 16 columns at a time: a half of the stream's, or a quarter of both streams' sum, with
            // head_dim 32 and 96 every fourth 16 of it (for all it took the 2047-token piece 5 % longer)
            constexpr bool kQuarters = D % 64 == 0;
            const int32_t first = both ? h * (D / 2) : (2 * j + h) * (kQuarters ? D / 4 : 16);
            const int32_t end = both ? first + D / 2 : (kQuarters ? first + D / 4 : D), stride = kQuarters || both ? 16 : 64;
#pragma unroll 1
            for (int32_t c = first; c < end; c += stride) {
                float x[16];
                {
                    uint32_t v[16];
                    tmem_ld_16((both ? t_o : o_first) + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = w0 == 0.0f ? 0.0f : w0 * __uint_as_float(v[i]);
                    if (!both) {
                        tmem_ld_16(o_first + 128u + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = w1 == 0.0f ? x[i] : fmaf(w1, __uint_as_float(v[i]), x[i]);
                    }
                }
                if (L == 0.0f) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = 0.0f;
                }
                // columns 8 i + (0 .. 7) are dims 8 i + (0 4 1 5 2 6 3 7)
                if (live && ok && whole) {
                    // over the stream's queries, which no MMA reads any more; a unit of at most 128
                    // rows over those of stream 0
                    uint8_t *dst = base + S::kQ + (both ? j * S::kTileBytes : 0u);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<uint4 *>(dst + (c >> 6) * (kKeys * 128) + sw128(r, ((c >> 3) & 7) + i)) =
                            make_uint4(pack_b16(x[8 * i] * inv, x[8 * i + 2] * inv), pack_b16(x[8 * i + 4] * inv, x[8 * i + 6] * inv),
                                       pack_b16(x[8 * i + 1] * inv, x[8 * i + 3] * inv), pack_b16(x[8 * i + 5] * inv, x[8 * i + 7] * inv));
                } else if (live && ok) {
                    float *dst = k.part_o + (slot * k.rows + ur) * D + c;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        *reinterpret_cast<float4 *>(dst + 8 * i) = make_float4(x[8 * i], x[8 * i + 2], x[8 * i + 4], x[8 * i + 6]);
                        *reinterpret_cast<float4 *>(dst + 8 * i + 4) = make_float4(x[8 * i + 1], x[8 * i + 3], x[8 * i + 5], x[8 * i + 7]);
                    }
                }
                __syncwarp();  // lanes behind the unit's last row meet the others: the next columns are loaded by the warp as one
            }
            if (!whole && live && ok && h == 0 && (both || j == 0)) k.part_ml[slot * k.rows + ur] = make_float2(M, L);
            __syncwarp();
            tc_fence_before();
            // no output column or sum is overwritten before all of its readers have it, and the rows
            // to be written are all there
            if (both) named_barrier_sync(1 + j, 256);
            else named_barrier_sync(3, 512);
            if (whole) {
                const uint8_t *src = base + S::kQ + (both ? j * S::kTileBytes : 0u);
                const int32_t warps = both ? 8 : 16, wi = both ? w8 : warp;
#pragma unroll 4
                for (int32_t r0 = wi * kRowsLoad; r0 < 128; r0 += warps * kRowsLoad) {
                    const int32_t orow = r0 + lane / kPer, at = row_at[both ? j : 0][orow];
                    if (mine && at >= 0 && ok)
                        *reinterpret_cast<uint4 *>(a.o + ((static_cast<int64_t>(w.b) * a.n + (at >> 16)) * a.H + (at & 0xffff)) * D + 8 * piece) =
                            *reinterpret_cast<const uint4 *>(src + (piece >> 3) * (kKeys * 128) + sw128(orow, piece & 7));
                }
                __syncwarp();
                if (both) named_barrier_sync(1 + j, 256);
                else named_barrier_sync(3, 512);
            }
        } while (next_unit());
    }

    // ---------------- teardown ----------------
    if (*abort_flag && threadIdx.x == 0) latch(a.status, kDevTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 24) {
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t prepare_kv4_attention_tc() {
    auto set = [](auto *kernel, uint32_t bytes) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)); };
    cudaError_t e = set(kv4_attention_tc_kernel<1>, Tc<1>::kTotal);
    if (e == cudaSuccess) e = set(kv4_attention_tc_kernel<2>, Tc<2>::kTotal);
    if (e == cudaSuccess) e = set(kv4_attention_tc_kernel<3>, Tc<3>::kTotal);
    if (e == cudaSuccess) e = set(kv4_attention_tc_kernel<4>, Tc<4>::kTotal);
    return e;
}

cudaError_t launch_kv4_attention_tc(const Kv4Args &k, int32_t grid, cudaStream_t st) {
    switch (k.a.cache.G) {
        case 1: return launch_pdl(kv4_attention_tc_kernel<1>, dim3(grid), dim3(kThreads), Tc<1>::kTotal, st, k);
        case 2: return launch_pdl(kv4_attention_tc_kernel<2>, dim3(grid), dim3(kThreads), Tc<2>::kTotal, st, k);
        case 3: return launch_pdl(kv4_attention_tc_kernel<3>, dim3(grid), dim3(kThreads), Tc<3>::kTotal, st, k);
        default: return launch_pdl(kv4_attention_tc_kernel<4>, dim3(grid), dim3(kThreads), Tc<4>::kTotal, st, k);
    }
}

}  // namespace eagle
