// kv4_attn_tc.cu - attention over the 4-bit cache for many query rows a kv head (large trees, grouped
// heads, pieces of a prompt), on tcgen05 with the accumulators in tensor memory.
//
// With R query rows a key costs 4 R D flops and is unpacked once for all of them, so from a few dozen
// rows on the tensor cores and the softmax bound the work and not the cache's bytes.  A CTA works on
// 256 query rows of one (request, kv head), as two streams of 128 rows that share every key and
// value tile; where a unit has at most 128 rows, both streams hold the same rows and take the even
// and the odd tiles, each with its own maximum, sum and output.  Tiles are 128 keys.
//   warps 0-3, 4-7  softmax of stream 0 and 1, a row a thread (its TMEM lane): two passes over the
//                   row of scores (maximum; exponentials), p as fp16 into TMEM over the scores it
//                   came from, the running maximum and sum in fp32.  p is held below 2^12 and its
//                   reference only moved (and O rescaled) when a tile's maximum passes that.
//   warps 8-11      fill the tiles: codes become fp16 values m + s c (one fused multiply-add: half an
//                   fp16 step, 2^-11 relative); new keys and values are converted from bf16 (exact
//                   but for magnitudes below 2^-14).
//   warp 13         copies the codes of cached tiles into a ring of three halves of tiles
//   warp 12         one thread issues the MMAs: S = Q K^T (128 x 128 x D, operands in shared memory)
//                   and O += P V (P from TMEM, V as stored: the MN-major B operand).  The order S0 S1
//                   [P0] O0 S0' [P1] O1 S1' ... keeps one stream's MMAs under the other's softmax.
// Queries are scaled by a power of two so that a row's largest element is 2^9..2^10 (exact, as in
// kv4_attn.cu).  Within 8 neighbouring dims the tiles hold them in the order 0 4 1 5 2 6 3 7, in
// which masking a word of codes leaves them; queries are stored in the same order and the output's
// columns are put right as they leave.
// New keys or values that fp16 cannot hold (above 65504, infinite, NaN) count as 0 in the tiles, and
// the rows that see them add their terms one by one: nothing hidden reaches a row, whatever it is.
// TMEM: S0 S1 O0 O1, 128 columns each (O uses D).  Every wait is bounded.
#include <type_traits>

#include "kernels.cuh"
#include "kv4_line.cuh"

namespace eagle {
namespace {

constexpr int kKeys = kKv4TcTile;
constexpr int kThreads = 14 * 32;
constexpr int kRaw = 3;  // halves of tiles (keys or values) of codes in flight
constexpr float kTop = 12.0f, kAim = 9.0f;  // p <= 2^12; a new reference puts the largest at 2^9
constexpr uint32_t kTmemCols = 512;

template <int G>
struct Tc {
    static constexpr int D = G * kKv4Group;
    static constexpr uint32_t kTileBytes = kKeys * D * 2;  // D / 64 blocks of [128 rows][128 bytes]
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

// D[tmem] (+)= A[tmem] * B[smem]: fp16 in, fp32 accumulation.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
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
// Whether fp16 cannot hold x.
__device__ __forceinline__ bool is_odd(float x) { return !(fabsf(x) <= 65504.0f); }

// Eight bf16 to fp16 in the same order; what fp16 cannot hold becomes 0 and sets `odd`.
__device__ __forceinline__ uint4 convert8(uint4 v, bool &odd) {
    auto abs2 = [](uint32_t x) { return x & 0x7fff7fffu; };
    auto b2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); };
    const __nv_bfloat162 big = __hmax2_nan(__hmax2_nan(b2(abs2(v.x)), b2(abs2(v.y))), __hmax2_nan(b2(abs2(v.z)), b2(abs2(v.w))));
    if (!(__low2float(big) <= 65504.0f && __high2float(big) <= 65504.0f)) {
        odd = true;
        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
        for (int i = 0; i < 4; ++i) {
            if (is_odd(bf_lo(w[i]))) w[i] &= 0xffff0000u;
            if (is_odd(bf_hi(w[i]))) w[i] &= 0x0000ffffu;
        }
    }
    return make_uint4(pack_f16(bf_lo(v.x), bf_lo(v.z)), pack_f16(bf_hi(v.x), bf_hi(v.z)), pack_f16(bf_lo(v.y), bf_lo(v.w)),
                      pack_f16(bf_hi(v.y), bf_hi(v.w)));
}

// The terms of elements that fp16 cannot hold, which count as 0 in the tiles: for the keys into the
// row's scores (f: what the query was scaled by), for the values into its output, where the row sees
// the key.  Warp-wide; `rows`: keys of the tile.
template <int D>
static __device__ __noinline__ void add_odd_keys(const __nv_bfloat16 *kt, int64_t ld, int32_t rows, const __nv_bfloat16 *q,
                                                 float f, uint32_t t_s) {
    for (int32_t key = 0; key < rows; ++key) {
        float add = 0.0f;
        bool any = false;
        for (int32_t d = 0; d < D; ++d) {
            const float x = __bfloat162float(kt[key * ld + d]);
            if (!is_odd(x)) continue;
            any = true;
            add += __bfloat162float(q[d]) * f * x;
        }
        if (any) tmem_st_1(t_s + key, tmem_ld_1(t_s + key) + add);
    }
}
template <int D>
static __device__ __noinline__ void add_odd_values(const __nv_bfloat16 *vt, int64_t ld, int32_t rows, uint4 see, float mul,
                                                   float sub, uint32_t t_s, uint32_t t_o) {
    for (int32_t key = 0; key < rows; ++key) {
        const float pv = ex2_approx(__fadd_rn(__fmul_rn(tmem_ld_1(t_s + key), mul), sub));
        const uint32_t word = key < 64 ? (key < 32 ? see.x : see.y) : (key < 96 ? see.z : see.w);
        const bool mine = (word >> (key & 31)) & 1u;
        for (int32_t d = 0; d < D; ++d) {
            const float x = __bfloat162float(vt[key * ld + d]);
            if (!is_odd(x)) continue;
            const uint32_t col = (d & ~7) + ((d & 3) << 1) + ((d >> 2) & 1);  // the order 0 4 1 5 2 6 3 7
            const float o = tmem_ld_1(t_o + col);
            tmem_st_1(t_o + col, mine ? o + pv * x : o);
        }
    }
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
    __shared__ __align__(4) uint8_t key_bits[4][16];  // by tile & 3: which of its 128 keys are there
    __shared__ uint8_t raw_keys[kRaw][8];             // keys of each chunk that are there
    __shared__ __align__(4) uint8_t odd_tile[4][2][4];     // by tile & 3, key or value, filling warp
    __shared__ float2 stream_ml[2][128];      // one unit of at most 128 rows: maxima and sums
    __shared__ Place place;
    __shared__ int64_t red[kThreads / 32];
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int32_t *abort_flag = &abort_mark;
    const Kv4Attention &a = k.a;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.k_full[i], 4);
            mbar_init(&bar.v_full[i], 4);
            mbar_init(&bar.k_empty[i], 1);
            mbar_init(&bar.v_empty[i], 1);
            mbar_init(&bar.q_full[i], 128);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 128);
            mbar_init(&bar.o_done[i], 1);
        }
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], 4);
        }
        mbar_init(&bar.drain, 1);
        abort_mark = 0;
        fence_barrier_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    const bool busy = find_place(k, &place, red);
    if (!busy) {
        if (threadIdx.x == 0) k.share[blockIdx.x].b = -1;
        return;
    }
    if (warp == 12) {
        tmem_alloc(&tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const Place p = place;
    Walk w;
    w.start(k, p);
    if (threadIdx.x == 0) k.share[blockIdx.x] = share_of(k, p, w);
    auto wait = [&](uint64_t *b, uint32_t parity) -> bool { return kv4_wait(b, parity, abort_flag); };
    auto rows_of = [&]() { return min(kKv4TcRows, k.Mq - w.qt * kKv4TcRows); };  // rows of the unit

    if (warp >= 8 && warp < 12) {
        // ---------------- the tiles ----------------
        const int32_t fw = warp - 8;
        uint32_t gt = 0, raw = 0;  // tiles and halves of cached tiles so far
        do {
            for (int64_t s = w.s0; s < w.s1; ++s, ++gt) {
                const uint32_t st = gt & 1u;
#pragma unroll 1
                for (int32_t half = 0; half < 2; ++half) {
                    uint8_t *dst = base + (half ? S::kV : S::kK) + st * S::kTileBytes;
                    bool odd = false;
                    if (s >= w.nt) {
                        const uint32_t rs = raw % kRaw;
                        wait(&bar.raw_full[rs], raw / kRaw);
                        if (gt >= 2) wait(half ? &bar.v_empty[st] : &bar.k_empty[st], (gt >> 1) - 1);
                        __syncwarp();
                        const uint8_t *src = base + S::kCodes + rs * 8 * S::kPart;
                        // lanes: four pieces of 8 dims of rows t and t + 4: the stores of eight
                        // lanes touch all banks
                        const int32_t m = lane >> 2, q = lane & 3;
                        const int32_t t8 = (m >> 1) | ((m & 1) << 2);          // token among the 8
                        const int32_t slot8 = half ? t8 : m;                   // its row
                        const int32_t qq = half && G == 4 ? q ^ (t8 & 2) : q;  // value rows' halves change places
                        // group i of 8 rows: 1024 bytes on; dims 32 g + 8 q: chunk 4 g + q
                        uint8_t *to = dst + fw * 1024 + t8 * 128 + ((qq ^ t8) << 4);
                        const int32_t odd_g = ((((4 + qq) ^ t8) - (qq ^ t8)) << 4);
#pragma unroll 2
                        for (int32_t i = 0; i < 4; ++i) {
                            const int32_t group = 4 * i + fw;
                            const uint8_t *part = src + (group >> 1) * S::kPart;
                            const int32_t slot = (group & 1) * 8 + slot8;
                            const int32_t here = max(0, min(8, static_cast<int32_t>(raw_keys[rs][group >> 1]) - 8 * (group & 1)));
                            uint32_t c[G], sm[G];
                            if constexpr (G == 4) {
                                const uint4 cv = *reinterpret_cast<const uint4 *>(part + slot * 64 + q * 16);
                                const uint4 mv = *reinterpret_cast<const uint4 *>(part + 1024 + slot * 16);
                                c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
                                sm[0] = mv.x, sm[1] = mv.y, sm[2] = mv.z, sm[3] = mv.w;
                            } else {
                                const uint2 cv = *reinterpret_cast<const uint2 *>(part + slot * 32 + q * 8);
                                const uint2 mv = *reinterpret_cast<const uint2 *>(part + 512 + slot * 8);
                                c[0] = cv.x, c[1] = cv.y;
                                sm[0] = mv.x, sm[1] = mv.y;
                            }
                            if (half) {  // two 16-bit words of four dims each to the keys' words of eight
                                uint32_t x[G];
#pragma unroll
                                for (int g = 0; g < G; ++g) x[g] = __byte_perm(c[g / 2], c[G / 2 + g / 2], g & 1 ? 0x7632 : 0x5410);
#pragma unroll
                                for (int g = 0; g < G; ++g) c[g] = x[g];
                            } else if (lane == 0) {
                                key_bits[gt & 3][group] = static_cast<uint8_t>((1u << here) - 1u);
                            }
                            if (here < 8) {  // rows that are not there hold 0
#pragma unroll
                                for (int g = 0; g < G; ++g)
                                    if (t8 >= here) c[g] = sm[g] = 0u;
                            }
#pragma unroll
                            for (int g = 0; g < G; ++g)
                                *reinterpret_cast<uint4 *>(to + i * 4096 + (g >> 1) * (kKeys * 128) + (g & 1 ? odd_g : 0)) = dequant8(c[g], sm[g]);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.raw_empty[rs]);
                        ++raw;
                    } else {
                        constexpr int kPer = D / 8, kRowsWarp = 32 / kPer;  // pieces a row; rows a warp takes at once
                        const int32_t ch = lane % kPer, first = fw * kRowsWarp + lane / kPer;
                        const __nv_bfloat16 *src = (half ? a.vn : a.kn) + (static_cast<int64_t>(w.b) * a.n + s * kKeys) * a.ldkv +
                                                   static_cast<int64_t>(w.hk) * D + ch * 8;
                        const int32_t rows = static_cast<int32_t>(min(a.n - s * kKeys, int64_t{kKeys}));
#pragma unroll 1
                        for (int32_t sub = 0; sub < D / 64; ++sub) {
                            uint4 v[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int32_t row = (sub * 8 + i) * 4 * kRowsWarp + first;
                                v[i] = row < rows ? *reinterpret_cast<const uint4 *>(src + row * a.ldkv) : make_uint4(0, 0, 0, 0);
                            }
                            if (sub == 0) {
                                if (gt >= 2) wait(half ? &bar.v_empty[st] : &bar.k_empty[st], (gt >> 1) - 1);
                                __syncwarp();
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int32_t row = (sub * 8 + i) * 4 * kRowsWarp + first;
                                *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (kKeys * 128) + sw128(row, ch & 7)) = convert8(v[i], odd);
                            }
                        }
                    }
                    const bool any = __any_sync(kFull, odd);
                    if (lane == 0) odd_tile[gt & 3][half][fw] = any;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half ? &bar.v_full[st] : &bar.k_full[st]);
                }
            }
        } while (w.next(k, p));
    } else if (warp == 13) {
        // ---------------- copies of codes: a stage is the keys or the values of a cached tile -------
        uint32_t raw = 0;
        bool dead = false;
        do {
            if (lane == 0 && w.len != a.cache.lengths[w.b]) latch(a.status, kDevBounds);  // clamped
            const int64_t k0 = max(w.s0 - w.nt, int64_t{0}), k1 = w.s1 - w.nt;
            for (int64_t kt = k0; kt < k1 && !dead; kt += 4) {
                // the chunks of four tiles, one a lane
                const int64_t key = kt * kKeys + lane * 16;
                int32_t nv = static_cast<int32_t>(min(max(w.len - key, int64_t{0}), int64_t{16}));
                const uint8_t *src = nullptr;
                if (nv > 0 && kt + (lane >> 3) < k1) {
                    src = kv4_chunk(a.cache, w.b, w.hk, key);
                    if (!src) latch(a.status, kDevBounds);  // its keys count as absent
                }
                if (!src) nv = 0;
                const int32_t halves = 2 * static_cast<int32_t>(min(k1 - kt, int64_t{4}));
                for (int32_t hh = 0; hh < halves; ++hh, ++raw) {
                    const uint32_t rs = raw % kRaw;
                    if (raw >= kRaw && lane == 0) wait(&bar.raw_empty[rs], raw / kRaw - 1);
                    dead = __shfl_sync(kFull, static_cast<int>(*abort_flag), 0) != 0;
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
        } while (!dead && w.next(k, p));
        // every copy has landed before the block's memory is handed on
        if (lane == 0)
            for (uint32_t i = raw > kRaw ? raw - kRaw : 0; i < raw; ++i) mbar_wait(&bar.raw_full[i % kRaw], (i / kRaw) & 1u, nullptr);
        __syncwarp();
    } else if (warp == 12) {
        // ---------------- MMA issue (one thread) ----------------
        if (lane == 0) {
            constexpr uint32_t idesc_s = idesc_f16(128, kKeys), idesc_o = idesc_f16_bmn(128, D);
            uint32_t gt = 0, seg = 0, jobs[2] = {0, 0};  // tiles, segments, P's of each stream so far
            bool ok = true;
            do {
                const int32_t tiles = static_cast<int32_t>(w.s1 - w.s0);
                const bool both = rows_of() > 128;
                const int32_t n = both ? 2 * tiles : tiles;
                auto tile_of = [&](int32_t q) { return both ? q >> 1 : q; };
                // the last job that reads a tile's keys or values
                auto last_of_tile = [&](int32_t q) { return !both || (q & 1); };
                auto issue_s = [&](int32_t q) -> bool {
                    const uint32_t t = gt + tile_of(q), st = t & 1u, j = q & 1;
                    if (!wait(&bar.k_full[st], t >> 1)) return false;
                    tc_fence_after();
                    const uint32_t q0 = smem_u32(base + S::kQ + j * S::kTileBytes), k0 = smem_u32(base + S::kK + st * S::kTileBytes);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * (kKeys * 128u) + (kk & 3) * 32u;
                        mma_bf16_ss(tmem + j * 128u, sw128_kmajor_desc(q0 + off), sw128_kmajor_desc(k0 + off), idesc_s, kk > 0);
                    }
                    mma_commit(&bar.s_full[j]);
                    if (last_of_tile(q)) mma_commit(&bar.k_empty[st]);
                    return true;
                };
                for (int32_t j = 0; j < 2 && ok; ++j) {
                    ok = wait(&bar.q_full[j], seg);
                    if (ok && j < n) ok = issue_s(j);
                }
                for (int32_t q = 0; q < n && ok; ++q) {
                    const uint32_t t = gt + tile_of(q), st = t & 1u, j = q & 1;
                    ok = wait(&bar.v_full[st], t >> 1) && wait(&bar.p_full[j], jobs[j]);
                    if (!ok) break;
                    ++jobs[j];
                    tc_fence_after();
                    const uint32_t v0 = smem_u32(base + S::kV + st * S::kTileBytes);
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        mma_f16_ts(tmem + 256u + j * 128u, tmem + j * 128u + kk * 8u, sw128_desc(v0 + kk * 2048u, kKeys * 128u, 1024u),
                                   idesc_o, 1u);
                    if (q + 2 >= n) mma_commit(&bar.o_done[j]);
                    if (last_of_tile(q)) mma_commit(&bar.v_empty[st]);
                    if (q + 2 < n) ok = issue_s(q + 2);
                }
                gt += tiles;
                ++seg;
            } while (ok && w.next(k, p));
            // what was issued lands before the block's memory is handed on
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, nullptr);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---------------- softmax and output ----------------
        const int32_t j = warp >> 2, r = threadIdx.x & 127;  // stream, row of the stream
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + j * 128u, t_o = tmem + lanes + 256u + j * 128u;
        uint32_t gt = 0, n_s = 0, n_o = 0;  // tiles, scores and outputs of this stream so far
        do {
            const int32_t unit_rows = rows_of();
            const bool both = unit_rows > 128;
            const int32_t ur = both ? j * 128 + r : r, row = w.qt * kKv4TcRows + ur;
            const bool live = ur < unit_rows;
            const int32_t node = live ? row / k.group : 0, head = w.hk * k.group + (live ? row - node * k.group : 0);
            const __nv_bfloat16 *q_src = a.q + (static_cast<int64_t>(w.b) * a.n + node) * a.ldq + static_cast<int64_t>(head) * D;
            float f, mul;  // what the query was scaled by; what makes its scores base 2
            {
                float big = 0.0f;
                auto piece = [&](int c) { return live ? *reinterpret_cast<const uint4 *>(q_src + 8 * c) : make_uint4(0, 0, 0, 0); };
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = piece(c);
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(bf_lo(vw[i])), fabsf(bf_hi(vw[i]))));
                }
                const int32_t e = max(static_cast<int32_t>(__float_as_uint(big) >> 23), 10);
                f = __uint_as_float(static_cast<uint32_t>(263 - e) << 23);
                mul = __uint_as_float(static_cast<uint32_t>(e - 9) << 23) * k.scale2;
                uint8_t *dst = base + S::kQ + j * S::kTileBytes;
#pragma unroll 2
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = piece(c);
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * (kKeys * 128) + sw128(r, c & 7)) =
                        make_uint4(pack_f16(bf_lo(v.x) * f, bf_lo(v.z) * f), pack_f16(bf_hi(v.x) * f, bf_hi(v.z) * f),
                                   pack_f16(bf_lo(v.y) * f, bf_lo(v.w) * f), pack_f16(bf_hi(v.y) * f, bf_hi(v.w) * f));
                }
                fence_proxy_async_smem();
                mbar_arrive(&bar.q_full[j]);
            }
            const uint32_t *mrow = a.mask ? a.mask + (static_cast<int64_t>(w.b) * a.n + node) * k.W : nullptr;
            {
                uint32_t z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tmem_st_32(t_o + 32 * c, z);
                tmem_wait_st();
            }
            float ref = -INFINITY, l = 0.0f;
            const int32_t tiles = static_cast<int32_t>(w.s1 - w.s0);
            int32_t done = 0;  // tiles of this segment that this stream took
            for (int32_t ti = both ? 0 : j; ti < tiles; ti += both ? 1 : 2, ++done) {
                const int64_t s = w.s0 + ti;
                const uint32_t t = gt + ti;
                wait(&bar.s_full[j], n_s);
                ++n_s;
                __syncwarp();
                tc_fence_after();
                // which keys of the tile the row sees
                uint32_t see[4];
                bool all = true, odd_k = false, odd_v = false;
                if (s >= w.nt) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) see[i] = reinterpret_cast<const volatile uint32_t *>(key_bits[t & 3])[i];
                } else {
                    const int32_t key0 = static_cast<int32_t>(s) * kKeys;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t k0 = key0 + 32 * i, left = a.n - k0;
                        const uint32_t in = left >= 32 ? kFull : (left > 0 ? (1u << left) - 1u : 0u);
                        const int32_t own = node - k0;  // causal: nodes 0..node
                        uint32_t v = own >= 31 ? kFull : (own >= 0 ? (2u << own) - 1u : 0u);
                        if (mrow) v = left > 0 ? mrow[k0 >> 5] : 0u;
                        see[i] = v & in;
                    }
                    // the tile's values have come too: whether it holds what fp16 does not
                    wait(&bar.v_full[t & 1], t >> 1);
                    __syncwarp();
                    odd_k = *reinterpret_cast<const volatile uint32_t *>(odd_tile[t & 3][0]) != 0;
                    odd_v = *reinterpret_cast<const volatile uint32_t *>(odd_tile[t & 3][1]) != 0;
                }
                if (!live) see[0] = see[1] = see[2] = see[3] = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) all = all && see[i] == kFull;
                all = __all_sync(kFull, all);
                const int64_t new_row = (static_cast<int64_t>(w.b) * a.n + s * kKeys) * a.ldkv + static_cast<int64_t>(w.hk) * D;
                const int32_t new_rows = static_cast<int32_t>(min(a.n - s * kKeys, int64_t{kKeys}));
                if (odd_k) add_odd_keys<D>(a.kn + new_row, a.ldkv, new_rows, q_src, f, t_s);
                float mx = -INFINITY;
                if (all) {
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld_32(t_s + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(v[i]));
                    }
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                } else {
                    uint32_t bits[4] = {see[0], see[1], see[2], see[3]};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld_32(t_s + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, (bits[0] >> i) & 1u ? __uint_as_float(v[i]) : -INFINITY);
                        bits[0] = bits[1], bits[1] = bits[2], bits[2] = bits[3];
                    }
                }
                mx = mx == -INFINITY ? mx : mx * mul;  // mul may underflow to 0
                float corr = 1.0f;
                if (mx - ref > kTop) {
                    const float nr = mx - kAim;
                    corr = ref == -INFINITY ? 0.0f : ex2_approx(ref - nr);
                    l *= corr;
                    ref = nr;
                }
                const float sub = ref == -INFINITY ? 0.0f : -ref;
                if (done > 0 && __any_sync(kFull, corr != 1.0f)) {
                    // the scores' arrival says that the stream's earlier products are complete
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld_32(t_o + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * corr);
                        tmem_st_32(t_o + 32 * c, v);
                    }
                    tmem_wait_st();
                }
                if (odd_v)
                    add_odd_values<D>(a.vn + new_row, a.ldkv, new_rows, make_uint4(see[0], see[1], see[2], see[3]), mul, sub, t_s, t_o);
                // One product and difference; scores so large that the product's rounding matters next
                // to their differences (and could pass for a score above the maximum) in two steps,
                // as the maximum was formed.
                auto exponentials = [&](auto exponent, auto masked) {
                    uint32_t bits[4] = {see[0], see[1], see[2], see[3]};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32], pk[16];
                        tmem_ld_32(t_s + 32 * c, v);
                        tmem_wait_ld();
                        float sum[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float p0 = ex2_approx(exponent(__uint_as_float(v[2 * i])));
                            float p1 = ex2_approx(exponent(__uint_as_float(v[2 * i + 1])));
                            if constexpr (decltype(masked)::value) {
                                p0 = (bits[0] >> (2 * i)) & 1u ? p0 : 0.0f;
                                p1 = (bits[0] >> (2 * i + 1)) & 1u ? p1 : 0.0f;
                            }
                            sum[i & 1] += p0 + p1;
                            pk[i] = pack_f16(p0, p1);
                        }
                        l += sum[0] + sum[1];
                        tmem_st_16(t_s + 16 * c, pk);
                        if constexpr (decltype(masked)::value) bits[0] = bits[1], bits[1] = bits[2], bits[2] = bits[3];
                    }
                };
                if (__any_sync(kFull, fabsf(sub) > 1048576.0f))
                    exponentials([&](float x) { return __fadd_rn(__fmul_rn(x, mul), sub); }, std::true_type{});
                else if (all)
                    exponentials([&](float x) { return fmaf(x, mul, sub); }, std::false_type{});
                else
                    exponentials([&](float x) { return fmaf(x, mul, sub); }, std::true_type{});
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bar.p_full[j]);
            }
            gt += tiles;
            // ---------------- the segment's output ----------------
            if (done > 0) {
                wait(&bar.o_done[j], n_o);
                ++n_o;
            }
            __syncwarp();
            tc_fence_after();
            const bool whole = w.s0 == 0 && w.s1 == w.unit;
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.t == p.begin ? 0 : 1);
            float M = ref, L = l, w0 = 1.0f, w1 = 0.0f;
            const uint32_t o_first = tmem + lanes + 256u;
            if (!both) {
                // the two streams' shares: each thread sees both and writes half of the columns
                stream_ml[j][r] = make_float2(ref, l);
                tc_fence_before();
                named_barrier_sync(1, 256);
                tc_fence_after();
                const float2 m0 = stream_ml[0][r], m1 = stream_ml[1][r];
                M = fmaxf(m0.x, m1.x);
                // a stream whose scores are all NaN has no maximum and a sum of NaN
                w0 = m0.x == -INFINITY ? (m0.y == 0.0f ? 0.0f : m0.y) : ex2_approx(m0.x - M);
                w1 = m1.x == -INFINITY ? (m1.y == 0.0f ? 0.0f : m1.y) : ex2_approx(m1.x - M);
                L = w0 * m0.y + w1 * m1.y;
            }
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            const bool ok = !*abort_flag;
            const int32_t c_begin = both ? 0 : j * (D / 64), c_end = both ? D / 32 : (j + 1) * (D / 64);
#pragma unroll 1
            for (int32_t c = c_begin; c < c_end; ++c) {
                float x[32];
                {
                    uint32_t v[32];
                    if (both) {
                        tmem_ld_32(t_o + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]);
                    } else {
                        tmem_ld_32(o_first + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = w0 == 0.0f ? 0.0f : w0 * __uint_as_float(v[i]);
                        tmem_ld_32(o_first + 128u + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = w1 == 0.0f ? x[i] : fmaf(w1, __uint_as_float(v[i]), x[i]);
                    }
                }
                if (L == 0.0f) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = 0.0f;
                }
                if (!live || !ok) continue;
                // columns 8 i + (0 .. 7) are dims 8 i + (0 4 1 5 2 6 3 7)
                if (whole) {
                    __nv_bfloat16 *dst = a.o + ((static_cast<int64_t>(w.b) * a.n + node) * a.H + head) * D + 32 * c;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(dst + 8 * i) =
                            make_uint4(pack_b16(x[8 * i] * inv, x[8 * i + 2] * inv), pack_b16(x[8 * i + 4] * inv, x[8 * i + 6] * inv),
                                       pack_b16(x[8 * i + 1] * inv, x[8 * i + 3] * inv), pack_b16(x[8 * i + 5] * inv, x[8 * i + 7] * inv));
                } else {
                    float *dst = k.part_o + (slot * k.rows + ur) * D + 32 * c;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *reinterpret_cast<float4 *>(dst + 8 * i) = make_float4(x[8 * i], x[8 * i + 2], x[8 * i + 4], x[8 * i + 6]);
                        *reinterpret_cast<float4 *>(dst + 8 * i + 4) = make_float4(x[8 * i + 1], x[8 * i + 3], x[8 * i + 5], x[8 * i + 7]);
                    }
                }
            }
            if (!whole && live && ok && (both || j == 0)) k.part_ml[slot * k.rows + ur] = make_float2(M, L);
            tc_fence_before();
            // neither stream's outputs are overwritten before both have been read
            if (!both) named_barrier_sync(1, 256);
        } while (w.next(k, p));
    }

    // ---------------- teardown ----------------
    if (*abort_flag && threadIdx.x == 0) latch(a.status, kDevTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) {
        __syncwarp();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t prepare_kv4_attention_tc() {
    cudaError_t e = cudaFuncSetAttribute(kv4_attention_tc_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<4>::kTotal);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kv4_attention_tc_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<2>::kTotal);
    return e;
}

cudaError_t launch_kv4_attention_tc(const Kv4Args &k, int32_t grid, cudaStream_t st) {
    if (k.a.cache.G == 4) return launch_pdl(kv4_attention_tc_kernel<4>, dim3(grid), dim3(kThreads), Tc<4>::kTotal, st, k);
    return launch_pdl(kv4_attention_tc_kernel<2>, dim3(grid), dim3(kThreads), Tc<2>::kTotal, st, k);
}

}  // namespace eagle
