// kv4.cuh - the 4-bit key/value cache: the layout of a page and what the kernels over it share.
//
// A group is 32 neighbouring head dimensions of one token of one kv head.  With lo and hi its least
// and largest value,
//     m = fp16(lo) rounded down,  s = fp16((hi - m) / 15) rounded up,
//     c = round_half_even((x - m) / s) in 0..15 (0 where s = 0)
// and the group stands for the values m + s c, which differ from x by at most s / 2 (s is rounded up,
// so no value is clamped).  A group with a NaN, an infinity or a value beyond 2^15 in magnitude has
// m = s = NaN: it reads back as NaN.  4 bits a value, 32 bits a group: 0.31 of bf16.
//
// A page holds page_size tokens of every kv head, [kv_heads][page_size / 16] chunks of 16 tokens.  A
// chunk (640 G bytes, G = head_dim / 32 groups a row) is what one warp takes at a time, and its
// parts lie so that the attention kernel's fragments are single conflict-free loads:
//     256 G  key codes    row kv4_key_slot(t) of 16 G bytes: 32-bit word qd * G + g holds the codes of
//                         dims 32 g + 8 qd .. + 7, the first in the low bits
//      64 G  key params   row kv4_key_slot(t): (s, m) as two fp16 for each group
//     256 G  value codes  row t of 16 G bytes: 16-bit word gq * G + g holds dims 32 g + 4 gq .. + 3
//                         (with G = 4 the halves of the row change places where t & 2 is set)
//      64 G  value params row t
// Bytes of a chunk that no token has filled are never used.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "../../include/eagle_tree.h"
#include "common.cuh"

namespace eagle {

constexpr int kKv4Group = 32;
constexpr int kKv4Chunk = 16;             // tokens of a chunk
constexpr float kKv4MaxAbs = 32768.0f;    // values beyond this have no fp16 parameters

struct Kv4View {
    uint8_t *pages;
    const int32_t *table;
    const int32_t *lengths;
    int32_t Hk, G, page_shift, num_pages, max_pages;
    int64_t cap;  // positions a request can hold: max_pages << page_shift
};

__host__ __device__ constexpr int32_t kv4_chunk_bytes(int32_t G) { return 640 * G; }
__host__ __device__ constexpr int32_t kv4_key_params(int32_t G) { return 256 * G; }
__host__ __device__ constexpr int32_t kv4_value_codes(int32_t G) { return 320 * G; }
__host__ __device__ constexpr int32_t kv4_value_params(int32_t G) { return 576 * G; }

// Row of token t (0..15) among a chunk's key rows: the order in which the score MMA's rows take
// the keys, so that after the transpose of its accumulators thread qd of the value product has
// keys qd, qd + 4, qd + 8 and qd + 12.
__host__ __device__ constexpr int32_t kv4_key_slot(int32_t t) { return ((t & 3) << 1) | ((t >> 2) & 1) | (t & 8); }

// Byte of 16-bit word (gq, g) in the value row of token t.
__host__ __device__ __forceinline__ int32_t kv4_value_word(int32_t t, int32_t gq, int32_t g, int32_t G) {
    const int32_t off = (gq * G + g) * 2;
    return G == 4 ? off ^ ((t & 2) << 4) : off;
}

// The chunk that holds position `pos` (< cap) of request b and kv head hk, or null when the table
// names no page of the pool.
__device__ __forceinline__ uint8_t *kv4_chunk(const Kv4View &v, int32_t b, int32_t hk, int64_t pos) {
    const int32_t page = v.table[static_cast<int64_t>(b) * v.max_pages + (pos >> v.page_shift)];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(v.num_pages)) return nullptr;
    const int64_t per = int64_t{1} << (v.page_shift - 4);
    const int64_t in_page = (pos >> 4) & (per - 1);
    return v.pages + ((static_cast<int64_t>(page) * v.Hk + hk) * per + in_page) * kv4_chunk_bytes(v.G);
}

// A length as lengths[] gives it, clamped to what a request's pages can hold.
__device__ __forceinline__ int64_t kv4_clamped(const Kv4View &v, int64_t len) { return len < 0 ? 0 : (len > v.cap ? v.cap : len); }
// Cached positions of request b.
__device__ __forceinline__ int64_t kv4_length(const Kv4View &v, int32_t b) { return kv4_clamped(v, v.lengths[b]); }

// Host: fills a view from the caller's description.  False when a size or pointer is unusable.
bool kv4_view(const eagle_kv4_cache *c, Kv4View *out);

// Two fp32 operations by one instruction.
__device__ __forceinline__ uint64_t pack_2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pack_2(float lo, float hi) { return pack_2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 unpack_2(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma_2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---------------------------------------------------------------------------------------------
// Attention over the cache and the new keys of each request's nodes (kv4_attn.cu)
// ---------------------------------------------------------------------------------------------
struct Kv4Attention {
    Kv4View cache;
    int32_t B, n, H;
    const __nv_bfloat16 *q;        // [B][n] rows of ldq elements, H * D used
    const __nv_bfloat16 *kn, *vn;  // [B][n] rows of ldkv elements, Hk * D used; both null: no new keys
    int64_t ldq, ldkv;
    const uint32_t *mask;          // [B][n][ceil(n / 32)], or null: node i sees nodes 0..i
    __nv_bfloat16 *o;              // [B][n][H * D]
    void *ws;
    int32_t *status;
    uint64_t limit_ns = kWaitLimitNs;  // of every wait
    int32_t stall = INT32_MAX;         // (tests) the tile from which a CTA's copying warp sends nothing
};
// False: more key tiles over all units than 32 bits count (launch_kv4_attention then refuses).
bool kv4_attention_fits(const Kv4View &cache, int32_t B, int32_t n, int32_t H, bool new_keys);
size_t kv4_attention_workspace(int32_t Hk, int32_t G, int32_t H, int32_t n);
cudaError_t launch_kv4_attention(const Kv4Attention &a, cudaStream_t st);

}  // namespace eagle
