// kv4_attn.cu - attention over the 4-bit key/value cache and the new keys of each request's nodes.
//
// For node i of request b and query head h (kv head hk = h / (H / Hk)):
//     o = sum_j p_j v_j / sum_j p_j,  p_j = exp(q . k_j / sqrt(D) - max)
// over the lengths[b] cached positions, whose keys and values are m + s c (kv4.cuh), and the new
// keys that the node sees, which are bf16.  A row that sees nothing gives 0.
//
// What bounds it: reading the cache, 2 (D / 2 + D / 8) bytes a token and kv head.  At 6.8 TB/s that
// is 11 T values a second on 152 SMs x 128 lanes x 1.9 GHz, so a value may cost at most 3.4
// lane-instructions, the softmax and everything else included: unpacking codes to bf16 and scaling
// them one by one would take most of that.  Hence the cached tiles are multiplied as codes:
//   * an fp16 whose bits are a code (0..15) in its lowest bits is the subnormal c 2^-24, exactly, and
//     with the code four bits higher 16 c 2^-24.  Masking a 32-bit word of eight codes twice before
//     and twice after a shift by 8 gives four fp16 pairs: 5 instructions for 8 values.  The factor
//     16 is taken out of the query (a power of two, exact) or of the output rows.
//   * scores: q . k = sum_g s_g (q . c)_g + sum_g m_g (sum of q over the group).  The MMAs of a group
//     (32 dims, two k-steps) start from zero and the sum over groups is fp32 with the key's s_g; the
//     second sum is one more MMA with the m_g of a key against fp16 hi + lo of the query's sums.
//     Queries are scaled by a power of two to fp16 (bf16 has 8 significand bits: exact but for
//     elements 2^-19 below the row's largest).
//   * output: o_d = sum_j (p_j s_gj) c_jd + sum_j p_j m_gj.  For each group p s_g is the B operand
//     (two fp16 products a key pair), the codes again the A operand; the second sum is one MMA whose
//     rows are the groups.  p and p s are rounded to fp16 (half a step is 2^-11 relative, against
//     2^-8 of the bf16 output); sums, the running maximum and p's sum are fp32.  So that p s keeps its bits
//     whatever the values' size, s is lifted by the power of two (up to 2^15) that puts the largest one so far
//     at 8 .. 16, and the first sum carries that power: a p of 2^-26 of the row's largest still has 11 bits
//     of p s (without it four heavy keys among 65536 that weigh a fifth were off by 3 % at values of 3e-5).  One
//     lift for all groups: one a group took 123 us where this takes 115 (64 8-node trees).
// Scores are formed transposed (16 keys on the MMA's M side, 8 query rows on N), so few query rows
// waste no MMA rows, and the accumulators turn into the value product's operand by movmatrix.
//
// Measured: 64 trees of 8 nodes, 32 heads of 128 over 1024 tokens each (352 MB) in 115 us, 0.45 of the
// measured copy rate; 16 requests of 1 .. 65536 tokens under groups of 8 heads in 163 us, 0.61 of it.
// Three CTAs of 128 registers a thread stay on an SM; it issues in 41 % of the cycles, waiting for
// memory in the new keys' part (95 us without new keys) and for fixed latencies in the rest.
//
// kv4_line.cuh: how the work is split.  kv4_attn_tc.cu: the kernel for many query rows.
#include <algorithm>
#include <mutex>

#include "kernels.cuh"
#include "kv4_line.cuh"

namespace eagle {
namespace {

constexpr int kTile = 64;       // keys of a tile: a chunk of 16 for each of the 4 warps
constexpr int kWarps = 4;       // warps that multiply
constexpr int kThreads = kWarps * 32 + 32;  // and one that copies
constexpr int kStages = 5;
constexpr int kMinTiles = 2;    // tiles a CTA takes at least: a single tile's CTA is merging more than work
constexpr float kLog2e = 1.4426950408889634f;
constexpr int32_t kSegment = 1024;  // tiles summed in one go (kv4_line.cuh)
constexpr int32_t kLift = 15;   // the most by which values' scales are lifted: a power of two that fp16 holds

__device__ __forceinline__ float power_of_2(int32_t e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a sum: from zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float low_f16(uint32_t x) { return __half2float(__ushort_as_half(static_cast<uint16_t>(x))); }
// ---------------------------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------------------------
template <int G, int NQ>
struct Shape {
    static constexpr int D = G * kKv4Group;
    static constexpr int kRows = 8 * NQ;
    static constexpr uint32_t kStageBytes = 4u * kv4_chunk_bytes(G);
    static constexpr uint32_t kMergeStride = D + 4;  // floats a row: no bank conflicts
    static constexpr uint32_t kRing = 0;
    static constexpr uint32_t kMerge = kRing + kStages * kStageBytes;
    static constexpr uint32_t kMl = kMerge + kWarps * kRows * kMergeStride * 4;
    static constexpr uint32_t kTotal = kMl + kWarps * kRows * 8;
    static constexpr int kBlocks = NQ == 1 ? 3 : 2;
};

template <int G, int NQ>
__global__ void __launch_bounds__(kThreads, Shape<G, NQ>::kBlocks) kv4_attention_kernel(const __grid_constant__ Kv4Args k) {
    using S = Shape<G, NQ>;
    constexpr int D = S::D, kRows = S::kRows;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int32_t valid[kStages][4];  // keys of each chunk of the stage (0..16)
    __shared__ int32_t abort_mark;
    __shared__ int32_t red[kThreads / 32];
    __shared__ Spot spots[2];
    __shared__ Place place;
    __shared__ Lengths lens;
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        abort_mark = 0;
        fence_barrier_init();
    }
    // no early launch of dependents: their blocks would take the places of the next call's CTAs, of
    // which all must be resident at once (64 8-node trees back to back took 30 % longer with it)
    pdl_wait();
    const Kv4Attention &a = k.a;
    if (!find_place(k, place, lens, red, spots)) {  // all threads meet there: the mbarriers are ready, too
        if (threadIdx.x == 0) k.share[blockIdx.x].kind = 0;
        return;
    }
    const Place p = place;
    volatile int32_t *abort_flag = &abort_mark;
    Walk w;
    w.start(k, p, lens);
    auto next_unit = [&]() {
        meet(k, p, w, lens, kThreads, warp == kWarps);
        return w.next(k, p, lens);
    };
    if (threadIdx.x == 0) k.share[blockIdx.x] = share_of(w);

    if (warp == kWarps) {
        // ---------------- copies: a stage is up to four chunks of cached keys and values ----------
        int32_t issued = 0;
        bool dead = false;
        do {
            if (lane == 0 && w.len != lens.of(w.b)) latch(a.status, kDevBounds);  // clamped
            const int32_t k0 = max(w.s0 - w.nt, 0), k1 = w.s1 - w.nt;
            for (int32_t kt = k0; kt < k1 && !dead; kt += 8) {
                // the chunks of 8 tiles, one a lane
                const int32_t key = kt * kTile + lane * kKv4Chunk;
                int32_t nv = min(max(w.len - key, 0), kKv4Chunk);
                const uint8_t *src = nullptr;
                if (nv > 0 && kt + (lane >> 2) < k1) {
                    src = kv4_chunk(a.cache, w.b, w.hk, key);
                    if (!src) latch(a.status, kDevBounds);  // its keys count as absent
                }
                if (!src) nv = 0;
                const int32_t tiles = min(k1 - kt, 8);
                for (int32_t j = 0; j < tiles; ++j, ++issued) {
                    const int32_t st = issued % kStages;
                    if (issued >= kStages && lane == 0) kv4_wait(&empty[st], issued / kStages - 1, abort_flag, a.limit_ns);
                    dead = __shfl_sync(kFull, static_cast<int>(*abort_flag), 0) != 0;
                    dead = dead || issued >= a.stall;
                    if (dead) break;
                    const bool my = (lane >> 2) == j;
                    const uint32_t have = __ballot_sync(kFull, my && src);
                    if (my) valid[st][lane & 3] = nv;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(__popc(have)) * kv4_chunk_bytes(G));
                    __syncwarp();
                    if (my && src)
                        bulk_load(smem + S::kRing + st * S::kStageBytes + (lane & 3) * kv4_chunk_bytes(G), src,
                                  kv4_chunk_bytes(G), &full[st]);
                }
            }
        } while (next_unit());
        // every copy has landed before the block's memory is handed on
        if (lane == 0)
            for (int32_t i = max(issued - kStages, 0); i < issued; ++i)
                mbar_wait(&full[i % kStages], static_cast<uint32_t>(i / kStages) & 1u, nullptr);
        if (lane == 0 && *abort_flag) latch(a.status, kDevTimeout);
        return;
    }

    // ---------------- multiplication: warp `warp` takes chunk `warp` of each tile ----------------
    const int32_t gq = lane >> 2, qd = lane & 3;
    float *merge = reinterpret_cast<float *>(smem + S::kMerge);
    float2 *merge_ml = reinterpret_cast<float2 *>(smem + S::kMl);
    int32_t stage = 0;  // the next one, and how often the ring has come round
    uint32_t turn = 0;
    do {
        uint32_t qf[2 * G][NQ][2];  // fp16 queries, the score MMAs' B operand
        uint32_t qs[NQ];            // fp16 hi + lo of the sum of group qd's elements
        float qk[NQ][2];            // what turns a column's accumulated score into base 2
        float o[2 * G][NQ][4];      // dims (rows) x queries
        float om[NQ][4];            // groups (rows gq < G) x queries: sum of p m
        float ref[NQ][2], l[NQ][2];
        int32_t node_of[NQ][2];     // the columns' nodes, -1 behind the last row
        // p = 2^(score - ref), at most 2^top; a new ref puts the largest at 2^aim
        float aim = 9.0f, top = 12.0f;
        int32_t lift = kLift;  // values' scales are multiplied by 2^lift, and so is o
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const int32_t row = w.qt * kRows + nq * 8 + gq;
            const bool live = row < k.Mq;
            const int32_t node = live ? row / k.group : 0, head = w.hk * k.group + (live ? row - node * k.group : 0);
            const __nv_bfloat16 *src = a.q + (static_cast<int64_t>(w.b) * a.n + node) * a.ldq + static_cast<int64_t>(head) * D + 8 * qd;
            float x[G][8];
            float big = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint4 v = live ? *reinterpret_cast<const uint4 *>(src + 32 * g) : make_uint4(0, 0, 0, 0);
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[g][2 * i] = bf_lo(vw[i]);
                    x[g][2 * i + 1] = bf_hi(vw[i]);
                    big = fmaxf(big, fmaxf(fabsf(x[g][2 * i]), fabsf(x[g][2 * i + 1])));
                }
            }
            big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
            big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
            // 2^(9 - floor(log2 big)): the row's largest element becomes 2^9 .. 2^10
            const int32_t e = max(static_cast<int32_t>(__float_as_uint(big) >> 23), 10);
            const float f = __uint_as_float(static_cast<uint32_t>(263 - e) << 23);
            const float inv = __uint_as_float(static_cast<uint32_t>(e - 9) << 23);
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[g][i] *= f;
                    t += x[g][i];
                }
                t += __shfl_xor_sync(kFull, t, 1);
                t += __shfl_xor_sync(kFull, t, 2);
                if (g == qd) sum = t;
                // pairs (0, 4), (1, 5), (2, 6), (3, 7) of the word's codes; 1, 3, 5, 7 come as 16 c
                qf[2 * g][nq][0] = pack_f16(x[g][0], x[g][4]);
                qf[2 * g][nq][1] = pack_f16(x[g][1] * 0.0625f, x[g][5] * 0.0625f);
                qf[2 * g + 1][nq][0] = pack_f16(x[g][2], x[g][6]);
                qf[2 * g + 1][nq][1] = pack_f16(x[g][3] * 0.0625f, x[g][7] * 0.0625f);
            }
            const float hi = __half2float(__float2half_rn(sum));
            qs[nq] = pack_f16(hi, sum - hi);
            const float mul = inv * k.scale2 * 16777216.0f;
            node_of[nq][0] = __shfl_sync(kFull, live ? node : -1, 8 * qd);
            node_of[nq][1] = __shfl_sync(kFull, live ? node : -1, 8 * qd + 4);
            qk[nq][0] = __shfl_sync(kFull, mul, 8 * qd);
            qk[nq][1] = __shfl_sync(kFull, mul, 8 * qd + 4);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                ref[nq][c] = -INFINITY;
                l[nq][c] = 0.0f;
            }
#pragma unroll
            for (int e2 = 0; e2 < 4; ++e2) om[nq][e2] = 0.0f;
#pragma unroll
            for (int t = 0; t < 2 * G; ++t)
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) o[t][nq][e2] = 0.0f;
        }

        // scores in base 2 (t: pairs of two keys x queries 2 qd, 2 qd + 1) to p, with the running
        // maximum, the sum and what was accumulated so far brought to the same reference
        auto softmax = [&](auto &t) {
            constexpr int N = sizeof(t[0]) / sizeof(float);
            bool raise = false;
            float corr[NQ][2];
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = t[nq][c];
#pragma unroll
                    for (int e = c + 2; e < N; e += 2) mx = fmaxf(mx, t[nq][e]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
                    corr[nq][c] = 1.0f;
                    if (mx - ref[nq][c] > top) {
                        const float nr = mx - aim;
                        corr[nq][c] = ref[nq][c] == -INFINITY ? 0.0f : ex2_approx(ref[nq][c] - nr);
                        ref[nq][c] = nr;
                        raise = true;
                    }
                }
            if (__any_sync(kFull, raise)) {
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) {
                    l[nq][0] *= corr[nq][0];
                    l[nq][1] *= corr[nq][1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) om[nq][e] *= corr[nq][e & 1];
#pragma unroll
                    for (int i = 0; i < 2 * G; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][nq][e] *= corr[nq][e & 1];
                }
            }
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                const float r0 = ref[nq][0] == -INFINITY ? 0.0f : ref[nq][0], r1 = ref[nq][1] == -INFINITY ? 0.0f : ref[nq][1];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float pv = ex2_approx(t[nq][e] - (e & 1 ? r1 : r0));
                    t[nq][e] = pv;
                    l[nq][e & 1] += pv;
                }
            }
        };

        int32_t s = w.s0;
        // ---------------- new keys: bf16, straight from memory ----------------
        for (; s < w.s1 && s < w.nt; ++s) {
            const int32_t key0 = s * kTile + warp * 16;
            if (key0 >= a.n) continue;
            const int64_t krow = static_cast<int64_t>(w.b) * a.n;
            float sc[NQ][4];
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nq][e] = 0.0f;
            const int32_t ka = key0 + gq, kb = ka + 8;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint4 z = make_uint4(0, 0, 0, 0);
                const __nv_bfloat16 *src = a.kn + krow * a.ldkv + static_cast<int64_t>(w.hk) * D + 32 * g + 8 * qd;
                const uint4 va = ka < a.n ? *reinterpret_cast<const uint4 *>(src + ka * a.ldkv) : z;
                const uint4 vb = kb < a.n ? *reinterpret_cast<const uint4 *>(src + kb * a.ldkv) : z;
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) {
                    const int32_t row = w.qt * kRows + nq * 8 + gq;
                    const bool live = row < k.Mq;
                    const int32_t node = live ? row / k.group : 0, head = w.hk * k.group + (live ? row - node * k.group : 0);
                    const uint4 vq = live ? *reinterpret_cast<const uint4 *>(a.q + (krow + node) * a.ldq + static_cast<int64_t>(head) * D + 32 * g + 8 * qd) : z;
                    mma_bf16(sc[nq], va.x, vb.x, va.y, vb.y, vq.x, vq.y);
                    mma_bf16(sc[nq], va.z, vb.z, va.w, vb.w, vq.z, vq.w);
                }
            }
            // which of the two keys each of the two queries sees
            bool see[NQ][4];
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t node = node_of[nq][e & 1], key = e < 2 ? ka : kb;
                    bool vis = node >= 0 && key < a.n;
                    if (vis) {
                        vis = a.mask ? (a.mask[(krow + node) * k.W + (key >> 5)] >> (key & 31)) & 1u : key <= node;
                    }
                    see[nq][e] = vis;
                    sc[nq][e] = vis ? sc[nq][e] * k.scale2 : -INFINITY;
                }
            softmax(sc);
            // values: dims 32 g + 4 gq .. + 3 of keys 2 qd, 2 qd + 1, 2 qd + 8, 2 qd + 9
            uint2 v[G][4];
            bool odd = false;  // a NaN or an infinity among them
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t key = key0 + 2 * qd + (u & 1) + 8 * (u >> 1);
                const __nv_bfloat16 *src = a.vn + (krow + key) * a.ldkv + static_cast<int64_t>(w.hk) * D + 4 * gq;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    v[g][u] = key < a.n ? *reinterpret_cast<const uint2 *>(src + 32 * g) : make_uint2(0, 0);
                    const uint32_t x = v[g][u].x, y = v[g][u].y;
                    odd = odd || (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u ||
                          (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
                }
            }
            if (__any_sync(kFull, odd)) {
                // A hidden key's NaN or infinity must not reach the rows that do not see it (0 x NaN
                // is NaN): such elements join the rows that see them one by one, and count as 0 below.
                for (int kk = 0; kk < 16 && key0 + kk < a.n; ++kk) {
                    const __nv_bfloat16 *src = a.vn + (krow + key0 + kk) * a.ldkv + static_cast<int64_t>(w.hk) * D + 4 * gq;
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int from = (kk & 7) * 4 + qd;
                            const float p0 = __shfl_sync(kFull, sc[nq][c], from), p1 = __shfl_sync(kFull, sc[nq][2 + c], from);
                            const int s0 = __shfl_sync(kFull, static_cast<int>(see[nq][c]), from);
                            const int s1 = __shfl_sync(kFull, static_cast<int>(see[nq][2 + c]), from);
                            const float pk = kk < 8 ? p0 : p1;
                            if (!(kk < 8 ? s0 : s1)) continue;
#pragma unroll
                            for (int g = 0; g < G; ++g)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float x = __bfloat162float(src[32 * g + i]);
                                    if (!isfinite(x)) o[2 * g + (i >> 1)][nq][2 * (i & 1) + c] += pk * x;
                                }
                        }
                }
                __syncwarp();  // lanes whose queries see different keys took different ways; the MMAs take the warp as one
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t &x = v[g][u].x, &y = v[g][u].y;
                        if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                        if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
                        if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
                        if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
                    }
            }
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                // p as bf16 hi + lo: 2^-16 relative
                float hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hi[e] = __bfloat162float(__float2bfloat16_rn(sc[nq][e]));
                    lo[e] = sc[nq][e] - hi[e];
                }
                const uint32_t h0 = transpose8(pack_b16(hi[0], hi[1])), h1 = transpose8(pack_b16(hi[2], hi[3]));
                const uint32_t l0 = transpose8(pack_b16(lo[0], lo[1])), l1 = transpose8(pack_b16(lo[2], lo[3]));
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t a0 = __byte_perm(v[g][0].x, v[g][1].x, 0x5410), a1 = __byte_perm(v[g][0].x, v[g][1].x, 0x7632);
                    const uint32_t a2 = __byte_perm(v[g][2].x, v[g][3].x, 0x5410), a3 = __byte_perm(v[g][2].x, v[g][3].x, 0x7632);
                    mma_bf16(o[2 * g][nq], a0, a1, a2, a3, h0, h1);
                    mma_bf16(o[2 * g][nq], a0, a1, a2, a3, l0, l1);
                    const uint32_t c0 = __byte_perm(v[g][0].y, v[g][1].y, 0x5410), c1 = __byte_perm(v[g][0].y, v[g][1].y, 0x7632);
                    const uint32_t c2 = __byte_perm(v[g][2].y, v[g][3].y, 0x5410), c3 = __byte_perm(v[g][2].y, v[g][3].y, 0x7632);
                    mma_bf16(o[2 * g + 1][nq], c0, c1, c2, c3, h0, h1);
                    mma_bf16(o[2 * g + 1][nq], c0, c1, c2, c3, l0, l1);
                }
            }
        }
        // the cached tiles accumulate c 2^(lift - 24) (rows 0-7: even dims) and 16 c 2^(lift - 24) (rows 8-15: odd dims)
#pragma unroll
        for (int i = 0; i < 2 * G; ++i)
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nq][e] *= e < 2 ? power_of_2(kLift - 24) : power_of_2(kLift - 20);

        // ---------------- cached keys: two stages, i.e. two chunks of the warp, at a time ----------
#pragma unroll 1
        for (; s < w.s1; s += 2) {
            const int32_t count = min(w.s1 - s, 2);
            const int32_t st0 = stage, st1 = stage + 1 == kStages ? 0 : stage + 1;
            const uint32_t turn1 = turn + (st1 == 0 ? 1 : 0);
            const bool come = kv4_wait(&full[st0], turn, abort_flag, a.limit_ns) &&
                              (count < 2 || kv4_wait(&full[st1], turn1, abort_flag, a.limit_ns));
            int32_t nv[2];  // keys of the chunks that are there
            nv[0] = valid[st0][warp];
            nv[1] = count == 2 ? valid[st1][warp] : 0;
            if (!__all_sync(kFull, come)) nv[0] = nv[1] = 0;
            if (nv[0] + nv[1] > 0) {
                const uint8_t *ch[2] = {smem + S::kRing + st0 * S::kStageBytes + warp * kv4_chunk_bytes(G),
                                        smem + S::kRing + st1 * S::kStageBytes + warp * kv4_chunk_bytes(G)};
                // scores of each chunk's key rows gq, gq + 8
                float sc[NQ][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint8_t *kp = ch[u] + kv4_key_params(G);
                    uint64_t x[NQ][2];  // pairs of columns: key rows gq, gq + 8
                    {
                        const uint32_t ma = qd < G ? *reinterpret_cast<const uint32_t *>(kp + gq * 4 * G + 4 * qd) : 0u;
                        const uint32_t mb = qd < G ? *reinterpret_cast<const uint32_t *>(kp + (gq + 8) * 4 * G + 4 * qd) : 0u;
                        const uint32_t a0 = __byte_perm(ma, ma, 0x3232), a1 = __byte_perm(mb, mb, 0x3232);
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq) {
                            float m[4];
                            mma_f16_first(m, a0, a1, 0u, 0u, qs[nq], 0u);
                            x[nq][0] = mul_2(pack_2(m[0], m[1]), pack_2(0x1p-24f, 0x1p-24f));
                            x[nq][1] = mul_2(pack_2(m[2], m[3]), pack_2(0x1p-24f, 0x1p-24f));
                        }
                    }
                    uint32_t wa[G], wb[G], pa[G], pb[G];
                    load_words<G>(ch[u] + gq * 16 * G + qd * 4 * G, wa);
                    load_words<G>(ch[u] + (gq + 8) * 16 * G + qd * 4 * G, wb);
                    load_words<G>(kp + gq * 4 * G, pa);
                    load_words<G>(kp + (gq + 8) * 4 * G, pb);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint32_t xa = wa[g] >> 8, xb = wb[g] >> 8;
                        const float sa = low_f16(pa[g]), sb = low_f16(pb[g]);
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq) {
                            float acc[4];
                            mma_f16_first(acc, wa[g] & 0x000f000fu, wb[g] & 0x000f000fu, wa[g] & 0x00f000f0u,
                                    wb[g] & 0x00f000f0u, qf[2 * g][nq][0], qf[2 * g][nq][1]);
                            mma_f16(acc, xa & 0x000f000fu, xb & 0x000f000fu, xa & 0x00f000f0u, xb & 0x00f000f0u,
                                    qf[2 * g + 1][nq][0], qf[2 * g + 1][nq][1]);
                            x[nq][0] = fma_2(pack_2(sa, sa), pack_2(acc[0], acc[1]), x[nq][0]);
                            x[nq][1] = fma_2(pack_2(sb, sb), pack_2(acc[2], acc[3]), x[nq][1]);
                        }
                    }
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 y = unpack_2(mul_2(x[nq][e], pack_2(qk[nq][0], qk[nq][1])));
                            sc[nq][4 * u + 2 * e] = y.x;
                            sc[nq][4 * u + 2 * e + 1] = y.y;
                        }
                }
                const bool tail = nv[0] + nv[1] < 32;
                if (tail) {
                    // MMA row i is key t with kv4_key_slot(t) = i
                    const int32_t ta = (gq >> 1) | ((gq & 1) << 2);
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (ta + (e & 2 ? 8 : 0) >= nv[e >> 2]) sc[nq][e] = -INFINITY;
                }
                // p s must stay below fp16's largest: with p up to 2^12, lifted s below 16, so a larger
                // one lowers the lift.  Steeper values (s from 16 to 2^12.1) take p up to 2^3 from here on.
                // Each lane looks at its share of the chunks' 16 G scales.
                if (aim != 0.0f) {
                    uint32_t most = 0;  // bits of the largest; NaN above all
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < (G + 1) / 2; ++i) {
                            const int32_t at = lane + 32 * i;
                            if (at < 16 * G && at / G < nv[u])
                                most = max(most, reinterpret_cast<const uint32_t *>(ch[u] + kv4_value_params(G))[at] & 0xffffu);
                        }
                    if (__any_sync(kFull, most >= static_cast<uint32_t>(19 - lift) << 10)) {  // 2^(4 - lift)
                        most = __reduce_max_sync(kFull, most);
                        const int32_t to = max(18 - static_cast<int32_t>(most >> 10), 0);
                        const float down = power_of_2(to - lift);
                        lift = to;
#pragma unroll
                        for (int i = 0; i < 2 * G; ++i)
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[i][nq][e] *= down;
                    }
                    if (most >= 0x4c00u && lift == 0) {  // 16
                        aim = 0.0f;
                        top = 3.0f;
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq) {
                            ref[nq][0] += 9.0f;
                            ref[nq][1] += 9.0f;
                            l[nq][0] *= 0x1p-9f;
                            l[nq][1] *= 0x1p-9f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                om[nq][e] *= 0x1p-9f;
#pragma unroll
                                for (int i = 0; i < 2 * G; ++i) o[i][nq][e] *= 0x1p-9f;
                            }
                        }
                    }
                }
                softmax(sc);
                // values: keys qd, qd + 4, qd + 8, qd + 12 of each chunk
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint8_t *vp = ch[u] + kv4_value_params(G);
                    uint32_t par[4][G];
#pragma unroll
                    for (int i = 0; i < 4; ++i) load_words<G>(vp + (qd + 4 * i) * 4 * G, par[i]);
                    uint32_t mm[4] = {0u, 0u, 0u, 0u};
                    if (gq < G) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) mm[i] = *reinterpret_cast<const uint32_t *>(vp + (qd + 4 * i) * 4 * G + 4 * gq);
                    }
                    if (tail) {  // what lies behind the last key is not a number that may be used
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (qd + 4 * i >= nv[u]) {
                                mm[i] = 0u;
#pragma unroll
                                for (int g = 0; g < G; ++g) par[i][g] = 0u;
                            }
                    }
                    uint32_t b0[NQ], b1[NQ];
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq) {
                        b0[nq] = transpose8(pack_f16(sc[nq][4 * u], sc[nq][4 * u + 1]));
                        b1[nq] = transpose8(pack_f16(sc[nq][4 * u + 2], sc[nq][4 * u + 3]));
                        mma_f16(om[nq], __byte_perm(mm[0], mm[1], 0x7632), 0u, __byte_perm(mm[2], mm[3], 0x7632), 0u, b0[nq], b1[nq]);
                    }
                    const uint32_t up = 0x04000400u * static_cast<uint32_t>(15 + lift);  // 2^lift, twice
                    const uint8_t *vc = ch[u] + kv4_value_codes(G);
                    uint32_t vw[4][(G + 1) / 2];  // two groups a word
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t t = qd + 4 * i;
                        const uint8_t *src = vc + t * 16 * G + kv4_value_word(t, gq, 0, G);
                        if constexpr (G == 4 || G == 2) {
                            load_words<G / 2>(src, vw[i]);
                        } else {
#pragma unroll
                            for (int g = 0; g < G; ++g) {
                                const uint32_t x = reinterpret_cast<const uint16_t *>(src)[g];
                                vw[i][g / 2] = g & 1 ? vw[i][g / 2] | (x << 16) : x;
                            }
                        }
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
                        const uint32_t x = __byte_perm(vw[0][g / 2], vw[1][g / 2], sel), y = __byte_perm(vw[2][g / 2], vw[3][g / 2], sel);
                        const uint32_t x8 = x >> 8, y8 = y >> 8;
                        const uint32_t s01 = mul_f16x2(__byte_perm(par[0][g], par[1][g], 0x5410), up);
                        const uint32_t s23 = mul_f16x2(__byte_perm(par[2][g], par[3][g], 0x5410), up);
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq) {
                            const uint32_t p0 = mul_f16x2(b0[nq], s01), p1 = mul_f16x2(b1[nq], s23);
                            mma_f16(o[2 * g][nq], x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u, p0, p1);
                            mma_f16(o[2 * g + 1][nq], x8 & 0x000f000fu, x8 & 0x00f000f0u, y8 & 0x000f000fu, y8 & 0x00f000f0u, p0, p1);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[st0]);
                if (count == 2) mbar_arrive(&empty[st1]);
            }
            stage = count == 2 ? (st1 + 1 == kStages ? 0 : st1 + 1) : st1;
            turn = count == 2 ? turn1 + (stage == 0 ? 1 : 0) : turn1;
        }

        // ---------------- the warps' shares of the segment meet ----------------
        named_barrier_sync(1, kWarps * 32);  // the previous segment's sums have been read
        const float even = power_of_2(24 - lift), odd = power_of_2(20 - lift);
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nq][c] += __shfl_xor_sync(kFull, l[nq][c], off);
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float add = __shfl_sync(kFull, om[nq][c], g * 4 + qd);
                    float4 v;  // dims 32 g + 4 gq .. + 3
                    v.x = fmaf(o[2 * g][nq][c], even, add);
                    v.y = fmaf(o[2 * g][nq][2 + c], odd, add);
                    v.z = fmaf(o[2 * g + 1][nq][c], even, add);
                    v.w = fmaf(o[2 * g + 1][nq][2 + c], odd, add);
                    *reinterpret_cast<float4 *>(merge + (warp * kRows + nq * 8 + 2 * qd + c) * S::kMergeStride + 32 * g + 4 * gq) = v;
                }
            if (gq < 2) merge_ml[warp * kRows + nq * 8 + 2 * qd + gq] = gq ? make_float2(ref[nq][1], l[nq][1]) : make_float2(ref[nq][0], l[nq][0]);
        }
        named_barrier_sync(1, kWarps * 32);
        if (*abort_flag) {
            if (threadIdx.x == 0) latch(a.status, kDevTimeout);
        } else {
            const bool whole = w.from == 0 && w.s1 == w.unit, begun = w.s0 > w.from;
            const int64_t slot = slot_of(w);
            for (int32_t it = threadIdx.x; it < kRows * (D / 4); it += kWarps * 32) {
                const int32_t r = it / (D / 4), c4 = it - r * (D / 4), row = w.qt * kRows + r;
                if (row >= k.Mq) break;
                float M = -INFINITY, L = 0.0f, wt[kWarps];
#pragma unroll
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, merge_ml[i * kRows + r].x);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float2 ml = merge_ml[i * kRows + r];
                    wt[i] = weight_of(ml.x, ml.y, M);
                    L += wt[i] * ml.y;
                    if (wt[i] == 0.0f) continue;
                    const float4 x = *reinterpret_cast<const float4 *>(merge + (i * kRows + r) * S::kMergeStride + 4 * c4);
                    v.x = fmaf(wt[i], x.x, v.x);
                    v.y = fmaf(wt[i], x.y, v.y);
                    v.z = fmaf(wt[i], x.z, v.z);
                    v.w = fmaf(wt[i], x.w, v.w);
                }
                float2 *carry = k.carry_ml + static_cast<int64_t>(blockIdx.x) * kKv4Carry + it;
                float4 *part = reinterpret_cast<float4 *>(k.part_o + (slot * kRows + r) * D + 4 * c4);
                if (begun) {
                    float now, before;
                    join(*carry, M, L, now, before);
                    const float4 was = *part;
                    if (now == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    else v = make_float4(now * v.x, now * v.y, now * v.z, now * v.w);
                    if (before != 0.0f)
                        v = make_float4(fmaf(before, was.x, v.x), fmaf(before, was.y, v.y), fmaf(before, was.z, v.z), fmaf(before, was.w, v.w));
                }
                if (whole) {
                    const int32_t node = row / k.group, head = w.hk * k.group + row - node * k.group;
                    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                    *reinterpret_cast<uint2 *>(a.o + ((static_cast<int64_t>(w.b) * a.n + node) * a.H + head) * D + 4 * c4) =
                        make_uint2(pack_b16(v.x * inv, v.y * inv), pack_b16(v.z * inv, v.w * inv));
                } else {
                    *part = v;
                    *carry = make_float2(M, L);
                    if (c4 == 0) k.part_ml[slot * kRows + r] = make_float2(M, L);
                }
            }
        }
        __syncwarp();  // lanes without a row meet the others
    } while (next_unit());
}

// Units that several CTAs worked on: block (c, .) merges the unit that CTA c is the second to work on.
// o = sum_i w_i O_i / sum_i w_i l_i, w_i = 2^(m_i - max m), over its CTAs in order.  A warp a row: a lane
// a part for the weights, then four dims a lane over all parts.  Bound by latency (two dependent
// reads from L2): 8 us by itself for 1952 rows of 2 to 3 parts.
constexpr int kMergeRows = 4;
__global__ void __launch_bounds__(kMergeRows * 32) kv4_merge_kernel(const __grid_constant__ Kv4Args k) {
    pdl_wait();
    const int32_t lane = threadIdx.x & 31, grid = gridDim.x;
    // CTA c continues a unit that CTA c - 1 began, and that goes on while the kind is 2
    const Kv4Share sh = k.share[blockIdx.x];
    const int32_t before = blockIdx.x > 0 ? k.share[blockIdx.x - 1].kind : 2;
    if (sh.kind == 0 || before == 2) return;
    const int32_t first = blockIdx.x - 1;
    int32_t last = blockIdx.x;
    for (bool more = true; more;) {
        const int32_t c = last + lane;
        const uint32_t ends = __ballot_sync(kFull, c >= grid - 1 || k.share[min(c, grid - 1)].kind != 2);
        more = ends == 0;
        last += more ? 32 : __ffs(ends) - 1;
    }
    const int32_t parts = last - first + 1;
    const int32_t D = k.a.cache.G * kKv4Group, rows = min(k.rows, k.Mq - sh.qt * k.rows);
    // part i is slot 0 of CTA first + i, but slot 1 of the first
    auto slot = [&](int32_t i) { return 2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0); };
    for (int32_t r = blockIdx.y * kMergeRows + (threadIdx.x >> 5); r < rows; r += kMergeRows * gridDim.y) {
        float M = -INFINITY, L = 0.0f;
        for (int32_t i = lane; i < parts; i += 32) M = fmaxf(M, k.part_ml[slot(i) * k.rows + r].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int32_t i0 = 0; i0 < parts; i0 += 32) {
            float wt = 0.0f;
            if (i0 + lane < parts) {
                const float2 ml = k.part_ml[slot(i0 + lane) * k.rows + r];
                wt = weight_of(ml.x, ml.y, M);
                if (wt != 0.0f) L += wt * ml.y;
            }
            const int32_t n = min(parts - i0, 32);
#pragma unroll 8
            for (int32_t i = 0; i < n; ++i) {
                const float x = __shfl_sync(kFull, wt, i);
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (4 * lane < D) o = *reinterpret_cast<const float4 *>(k.part_o + (slot(i0 + i) * k.rows + r) * D + 4 * lane);
                if (x != 0.0f) {
                    v.x = fmaf(x, o.x, v.x);
                    v.y = fmaf(x, o.y, v.y);
                    v.z = fmaf(x, o.z, v.z);
                    v.w = fmaf(x, o.w, v.w);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(kFull, L, off);
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const int32_t row = sh.qt * k.rows + r, node = row / k.group, head = sh.hk * k.group + row - node * k.group;
        if (4 * lane < D)
            *reinterpret_cast<uint2 *>(k.a.o + ((static_cast<int64_t>(sh.b) * k.a.n + node) * k.a.H + head) * D + 4 * lane) =
                make_uint2(pack_b16(v.x * inv, v.y * inv), pack_b16(v.z * inv, v.w * inv));
    }
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
struct Variant {
    int32_t rows, threads;
    size_t smem;
    void (*kernel)(const Kv4Args);  // null: the tcgen05 kernel
};

template <int G>
Variant variant_of(int32_t mq) {
    // Query rows a unit takes: 8 or 16; from 17 rows on tcgen05 takes over.  us for 32 requests of 8 kv heads
    // over 1024 / 8192 tokens each, this kernel (32 rows: with units of 32) and the tcgen05 one:
    //     head_dim    16 rows here    there       17 here    there       32 here    there
    //     32             21 /  79    36 / 146     41 / 183   36 / 145    42 / 185   34 / 141
    //     64             24 /  95    40 / 184     48 / 215   40 / 184    50 / 220   38 / 181
    //     96             30 / 117    49 / 222     66 / 286   49 / 223    69 / 290   46 / 200
    //     128            39 / 147    50 / 214     87 / 365   50 / 214    91 / 377   47 / 208
    if (mq <= 8) return Variant{8, kThreads, Shape<G, 1>::kTotal, kv4_attention_kernel<G, 1>};
    if (mq <= 16) return Variant{16, kThreads, Shape<G, 2>::kTotal, kv4_attention_kernel<G, 2>};
    return Variant{kKv4TcRows, 0, 0, nullptr};
}
Variant variant(int32_t G, int32_t mq) {
    switch (G) {
        case 1: return variant_of<1>(mq);
        case 2: return variant_of<2>(mq);
        case 3: return variant_of<3>(mq);
        default: return variant_of<4>(mq);
    }
}

struct Device {
    int32_t sms = 0;
    int32_t blocks[5][2] = {};  // CTAs an SM holds, by groups and rows
};
std::mutex g_mu;
Device g_dev[64];

// The device's SM count and each variant's CTAs an SM (attributes set once).
const Device *device_now() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(g_mu);
    Device &d = g_dev[dev];
    if (d.sms) return &d;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return nullptr;
    for (int g = 1; g <= 4; ++g)
        for (int i = 0; i < 2; ++i) {
            const Variant v = variant(g, 8 << i);
            int n = 0;
            if (cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(v.smem)) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, v.kernel, v.threads, v.smem) != cudaSuccess || n < 1)
                return nullptr;
            d.blocks[g][i] = n;
        }
    if (prepare_kv4_attention_tc() != cudaSuccess) return nullptr;
    d.sms = sms;
    return &d;
}

int32_t grid_of(const Device &d, int32_t G, const Variant &v) {
    if (!v.kernel) return d.sms;
    return d.sms * d.blocks[G][v.rows == 8 ? 0 : 1];
}

// Key tiles of all units where every request fills its pages.
int64_t longest_line(const Kv4View &cache, int32_t B, int32_t n, int32_t H, bool new_keys) {
    const int64_t mq = static_cast<int64_t>(n) * (H / cache.Hk);
    const Variant v = variant(cache.G, static_cast<int32_t>(mq));
    const int64_t tile = v.kernel ? kTile : kKv4TcTile, units = static_cast<int64_t>(B) * cache.Hk * ((mq + v.rows - 1) / v.rows);
    const int64_t tiles = (cache.cap + tile - 1) / tile + (new_keys ? (n + tile - 1) / tile : 0);
    return units >= (int64_t{1} << 31) ? units : units * tiles;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t kv4_attention_workspace(int32_t Hk, int32_t G, int32_t H, int32_t n) {
    const Device *d = device_now();
    if (!d) return 0;
    const Variant v = variant(G, static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(n) * (H / Hk), 1 << 20)));
    const size_t grid = grid_of(*d, G, v);
    return align256(grid * sizeof(Kv4Share)) + align256(grid * 2 * v.rows * sizeof(float2)) + grid * 2 * v.rows * G * kKv4Group * 4 +
           grid * kKv4Carry * sizeof(float2);
}

bool kv4_attention_fits(const Kv4View &cache, int32_t B, int32_t n, int32_t H, bool new_keys) {
    return longest_line(cache, B, n, H, new_keys) < (int64_t{1} << 31);
}

cudaError_t launch_kv4_attention(const Kv4Attention &a, cudaStream_t st) {
    const Device *d = device_now();
    if (!d) return cudaErrorInvalidDevice;
    if (!kv4_attention_fits(a.cache, a.B, a.n, a.H, a.kn != nullptr)) return cudaErrorNotSupported;
    const int32_t G = a.cache.G;
    Kv4Args k;
    k.a = a;
    k.group = a.H / a.cache.Hk;
    k.Mq = a.n * k.group;
    const Variant v = variant(G, k.Mq);
    k.rows = v.rows;
    k.QT = (k.Mq + v.rows - 1) / v.rows;
    k.W = (a.n + 31) / 32;
    static_assert(kTile == 1 << 6 && kKv4TcTile == 1 << 7, "tile_shift");
    k.tile_shift = v.kernel ? 6 : 7;
    k.min_tiles = v.kernel ? kMinTiles : 1;
    // cuts move to a unit's end from so many tiles: a unit cut in two writes and reads partial sums of
    // all its rows.  With 0, 2, 5 and 8 on tcgen05: 32 requests of 64 nodes 96, 85, 62 and 62 us, of 65 nodes
    // 143, 135, 114 and 114, 2047 tokens of two prompts 737, 736, 725 and 732
    k.snap = v.kernel ? 1 : 5;
    k.scale2 = kLog2e / sqrtf(static_cast<float>(G * kKv4Group));
    const int32_t full = grid_of(*d, G, v);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    k.share = reinterpret_cast<Kv4Share *>(ws);
    ws += align256(full * sizeof(Kv4Share));
    k.part_ml = reinterpret_cast<float2 *>(ws);
    ws += align256(static_cast<size_t>(full) * 2 * v.rows * sizeof(float2));
    k.part_o = reinterpret_cast<float *>(ws);
    ws += static_cast<size_t>(full) * 2 * v.rows * G * kKv4Group * 4;
    k.carry_ml = reinterpret_cast<float2 *>(ws);
    k.segment = v.kernel ? kSegment : kKv4TcSegment;
    // no more CTAs than the longest possible line gives work to
    const int64_t most = (longest_line(a.cache, a.B, a.n, a.H, a.kn != nullptr) + k.min_tiles - 1) / k.min_tiles;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(full, std::max<int64_t>(most, 1)));
    const cudaError_t e = v.kernel ? launch_pdl(v.kernel, dim3(grid), dim3(v.threads), v.smem, st, k)
                                   : launch_kv4_attention_tc(k, static_cast<int32_t>(grid), st);
    if (e != cudaSuccess || grid == 1) return e;
    return launch_pdl(kv4_merge_kernel, dim3(grid, std::min(k.rows / kMergeRows, 16)), dim3(kMergeRows * 32), 0, st, k);
}

namespace {

// The call on the host: checks, and the launches.  `a` holds what differs from an ordinary call.
eagle_status attention(Kv4Attention a, const eagle_kv4_cache *cache, int32_t batch, int32_t nodes, int32_t heads, const void *d_q,
                       int64_t ldq, const void *d_k, const void *d_v, int64_t ldkv, const uint32_t *d_mask, void *d_out,
                       void *d_ws, size_t ws_bytes, int32_t *d_status, eagle_stream_t stream) {
    if (!kv4_view(cache, &a.cache) || batch < 0 || nodes < 1 || nodes > kMaxCandidates + 1) return EAGLE_ERR_INVALID_ARG;
    if (heads < 1 || heads > 65536 || heads % a.cache.Hk) return EAGLE_ERR_INVALID_ARG;
    if (batch == 0) return EAGLE_OK;
    const int64_t D = a.cache.G * kKv4Group;
    if (!d_q || !d_out || !d_ws || (d_k == nullptr) != (d_v == nullptr)) return EAGLE_ERR_INVALID_ARG;
    if (d_mask && !d_k) return EAGLE_ERR_INVALID_ARG;
    if (ldq < heads * D || ldq % 8 || (d_k && (ldkv < a.cache.Hk * D || ldkv % 8))) return EAGLE_ERR_INVALID_ARG;
    const void *p16[] = {d_q, d_k, d_v, d_out};
    for (const void *p : p16)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return EAGLE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_ws) & 255u) return EAGLE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(d_mask) | reinterpret_cast<uintptr_t>(d_status)) & 3u) return EAGLE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(nodes) * (heads / a.cache.Hk) > (1 << 24)) return EAGLE_ERR_INVALID_ARG;
    const size_t need = kv4_attention_workspace(a.cache.Hk, a.cache.G, heads, nodes);
    if (need == 0) return EAGLE_ERR_CUDA;
    if (ws_bytes < need) return EAGLE_ERR_INVALID_ARG;
    a.B = batch;
    a.n = nodes;
    a.H = heads;
    a.q = static_cast<const __nv_bfloat16 *>(d_q);
    a.kn = static_cast<const __nv_bfloat16 *>(d_k);
    a.vn = static_cast<const __nv_bfloat16 *>(d_v);
    a.ldq = ldq;
    a.ldkv = ldkv;
    a.mask = d_mask;
    a.o = static_cast<__nv_bfloat16 *>(d_out);
    a.ws = d_ws;
    a.status = d_status;
    const cudaError_t e = launch_kv4_attention(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? EAGLE_OK : (e == cudaErrorNotSupported ? EAGLE_ERR_UNSUPPORTED : EAGLE_ERR_CUDA);
}

}  // namespace
}  // namespace eagle

extern "C" {

size_t eagle_kv4_attention_workspace_bytes(const eagle_kv4_cache *cache, int32_t nodes, int32_t heads) {
    eagle::Kv4View v;
    if (!eagle::kv4_view(cache, &v) || nodes < 1 || nodes > eagle::kMaxCandidates + 1) return 0;
    if (heads < 1 || heads > 65536 || heads % v.Hk) return 0;
    return eagle::kv4_attention_workspace(v.Hk, v.G, heads, nodes);
}

eagle_status eagle_kv4_attention(const eagle_kv4_cache *cache, int32_t batch, int32_t nodes, int32_t heads,
                                 const void *d_q, int64_t ldq, const void *d_k, const void *d_v, int64_t ldkv,
                                 const uint32_t *d_mask, void *d_out, void *d_ws, size_t ws_bytes, int32_t *d_status,
                                 eagle_stream_t stream) {
    eagle::NvtxRange nvtx_range("eagle_kv4_attention");
    return eagle::attention(eagle::Kv4Attention{}, cache, batch, nodes, heads, d_q, ldq, d_k, d_v, ldkv, d_mask, d_out, d_ws,
                            ws_bytes, d_status, stream);
}

eagle_status eagle_test_kv4_stall(const eagle_kv4_cache *cache, int32_t batch, int32_t nodes, int32_t heads, const void *d_q,
                                  const void *d_k, const void *d_v, const uint32_t *d_mask, void *d_out, void *d_ws,
                                  size_t ws_bytes, int64_t limit_ns, int32_t tile, int32_t *d_status, eagle_stream_t stream) {
    if (!cache || limit_ns < 1 || limit_ns > 10000000000ll || tile < 0) return EAGLE_ERR_INVALID_ARG;
    eagle::Kv4Attention a{};
    a.limit_ns = static_cast<uint64_t>(limit_ns);
    a.stall = tile;
    return eagle::attention(a, cache, batch, nodes, heads, d_q, static_cast<int64_t>(heads) * cache->head_dim, d_k, d_v,
                            static_cast<int64_t>(cache->kv_heads) * cache->head_dim, d_mask, d_out, d_ws, ws_bytes, d_status,
                            stream);
}

}  // extern "C"
