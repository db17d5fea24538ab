// kv4_line.cuh - how the attention kernels over the 4-bit cache share their work out.
//
// A unit is (request, kv head, tile of query rows); its keys come in tiles: new keys first, then
// cached ones.  All units' tiles, in order, form one line that the CTAs cut evenly, whatever the
// requests' lengths; the line is laid out on the device from the lengths, so the host needs none of
// them.  A unit that more than one CTA works on is merged by a second kernel (kv4_attn.cu) from
// partial sums in the workspace: each CTA leaves at most two.
#pragma once

#include "kv4.cuh"

namespace eagle {

constexpr uint32_t kFull = 0xffffffffu;

// What each CTA of the attention kernel leaves for the merge: the unit that it continues (begun by
// an earlier CTA) if it is the first to do so, and the CTAs first..last that share it.
struct Kv4Share {
    int32_t b, hk, qt;       // b < 0: nothing to merge here
    int32_t first, last, first_slot;
};

struct Kv4Args {
    Kv4Attention a;
    int32_t group, Mq, rows, QT, W;
    int32_t tile_shift;      // log2 of the keys of a tile
    int32_t min_tiles;       // tiles a CTA takes at least
    float scale2;            // log2(e) / sqrt(D)
    Kv4Share *share;         // [grid]
    float2 *part_ml;         // [grid * 2][rows]: running maximum (base 2) and sum
    float *part_o;           // [grid * 2][rows][D]
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_b16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N 32-bit words at p, whose address is a multiple of 4 N bytes (N 1, 2 or 4) or of 4 (N 3).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
}

// Waits for `parity` (its lowest bit) on `bar`.  Gives up when *abort is set, and sets it after
// kWaitLimitNs.  Small, so that the kernels' loops stay in the instruction cache: the clock is looked
// at once in a thousand tries.
__device__ __forceinline__ bool kv4_wait(uint64_t *bar, uint32_t parity, volatile int32_t *abort) {
    uint64_t since = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity & 1u)) return true;
        if (*abort) return false;
        if ((i & 1023u) == 0) {
            const uint64_t now = global_timer_ns();
            if (since == 0) {
                since = now;
            } else if (now - since > kWaitLimitNs) {
                *abort = 1;
                return false;
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The line of tiles
// ---------------------------------------------------------------------------------------------
// Tiles of new keys that the rows of query tile qt need.
__device__ __forceinline__ int32_t new_tiles(const Kv4Args &k, int32_t qt) {
    if (!k.a.kn) return 0;
    if (k.a.mask) return ((k.a.n - 1) >> k.tile_shift) + 1;
    const int32_t last = min(k.a.n - 1, ((qt + 1) * k.rows - 1) / k.group);
    return (last >> k.tile_shift) + 1;
}
// Tiles of cached keys of request b; at least one where a unit would have none.
__device__ __forceinline__ int64_t cached_tiles(const Kv4Args &k, int32_t b) {
    const int64_t t = (kv4_length(k.a.cache, b) + (1 << k.tile_shift) - 1) >> k.tile_shift;
    return t < 1 && !k.a.kn ? 1 : t;
}

// Where a CTA begins and ends, and the unit that its first tile belongs to.
struct Place {
    int64_t total, begin, end;  // tiles of the line
    int64_t ctas;               // CTAs that share it
    int32_t b, hk, qt;
    int64_t off;                // the first tile's place in its unit
};

// Sum over the block; every thread gets it.  `red`: one slot a warp.
static __device__ __noinline__ int64_t block_sum64(int64_t v, int64_t *red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) t += red[w];
    return t;
}

// All threads of the block; the result is in *out after the last barrier.  Returns false when this
// CTA has nothing to do.
static __device__ __noinline__ bool find_place(const Kv4Args &k, Place *out, int64_t *red) {
    const int32_t tid = threadIdx.x, nt = blockDim.x, B = k.a.B;
    const int64_t Hk = k.a.cache.Hk;
    int64_t per = 0;  // tiles of new keys of one (request, kv head)
    if (k.a.mask || !k.a.kn) {
        per = static_cast<int64_t>(k.QT) * new_tiles(k, 0);
    } else {
        for (int32_t q = tid; q < k.QT; q += nt) per += new_tiles(k, q);
        per = block_sum64(per, red);
    }
    int64_t mine = 0;
    for (int32_t b = tid; b < B; b += nt) mine += Hk * (k.QT * cached_tiles(k, b) + per);
    const int64_t total = block_sum64(mine, red);
    const int64_t want = (total + k.min_tiles - 1) / k.min_tiles;
    const int64_t ctas = want < gridDim.x ? (want < 1 ? 1 : want) : gridDim.x;
    const int64_t c = blockIdx.x;
    if (c >= ctas) return false;
    const int64_t begin = c * total / ctas, end = (c + 1) * total / ctas;
    // the request that holds tile `begin`
    int64_t base = 0;
    for (int32_t b0 = 0; b0 < B; b0 += nt) {
        const int32_t b = b0 + tid;
        const int64_t w = b < B ? Hk * (k.QT * cached_tiles(k, b) + per) : 0;
        int64_t inc = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(kFull, inc, off);
            if ((tid & 31) >= off) inc += o;
        }
        __syncthreads();
        if ((tid & 31) == 31) red[tid >> 5] = inc;
        __syncthreads();
        int64_t before = base, all = base;
        for (int w2 = 0; w2 < nt / 32; ++w2) {
            if (w2 < (tid >> 5)) before += red[w2];
            all += red[w2];
        }
        const int64_t lo = before + inc - w;
        if (b < B && begin >= lo && begin < lo + w) {
            int64_t off = begin - lo;
            const int64_t ct = cached_tiles(k, b), block = k.QT * ct + per;
            Place p;
            p.total = total;
            p.begin = begin;
            p.end = end;
            p.ctas = ctas;
            p.b = b;
            p.hk = static_cast<int32_t>(off / block);
            off -= p.hk * block;
            if (k.a.mask || !k.a.kn) {
                const int64_t u = ct + new_tiles(k, 0);
                p.qt = static_cast<int32_t>(off / u);
                off -= p.qt * u;
            } else {
                p.qt = 0;
                for (int64_t u; off >= (u = ct + new_tiles(k, p.qt)); ++p.qt) off -= u;
            }
            p.off = off;
            *out = p;
        }
        base = all;
        if (begin < base) break;
    }
    __syncthreads();
    return true;
}

// A CTA's run through the line, unit by unit: [s0, s1) of the unit's tiles.
struct Walk {
    int32_t b, hk, qt;
    int64_t t, s0, s1, unit;
    int32_t nt;  // tiles of new keys (the unit's first)
    int64_t len;

    __device__ __forceinline__ void start(const Kv4Args &k, const Place &p) {
        b = p.b;
        hk = p.hk;
        qt = p.qt;
        t = p.begin;
        s0 = p.off;
        fill(k, p);
    }
    __device__ __forceinline__ void fill(const Kv4Args &k, const Place &p) {
        nt = new_tiles(k, qt);
        len = kv4_length(k.a.cache, b);
        unit = cached_tiles(k, b) + nt;
        s1 = min(unit, s0 + (p.end - t));
    }
    __device__ __forceinline__ bool next(const Kv4Args &k, const Place &p) {
        t += s1 - s0;
        if (t >= p.end) return false;
        s0 = 0;
        if (++qt == k.QT) {
            qt = 0;
            if (++hk == k.a.cache.Hk) {
                hk = 0;
                if (++b == k.a.B) return false;  // lengths changed under the call
            }
        }
        fill(k, p);
        return true;
    }
};

// What CTA blockIdx.x leaves for the merge.
static __device__ __noinline__ Kv4Share share_of(const Kv4Args &k, const Place &p, const Walk &w) {
    Kv4Share sh{-1, 0, 0, 0, 0, 0};
    if (w.s0 > 0) {
        const int64_t u0 = p.begin - w.s0;  // the unit's first tile
        const int64_t c0 = ((u0 + 1) * p.ctas - 1) / p.total, c1 = ((u0 + w.unit) * p.ctas - 1) / p.total;
        if (c0 == static_cast<int64_t>(blockIdx.x) - 1)
            sh = Kv4Share{w.b, w.hk, w.qt, static_cast<int32_t>(c0), static_cast<int32_t>(c1),
                          c0 * p.total / p.ctas == u0 ? 0 : 1};
    }
    return sh;
}

// The tcgen05 kernel (kv4_attn_tc.cu): head_dim 64 or 128, units of 256 query rows, tiles of 128 keys.
constexpr int32_t kKv4TcRows = 256;
constexpr int32_t kKv4TcTile = 128;
cudaError_t prepare_kv4_attention_tc();
cudaError_t launch_kv4_attention_tc(const Kv4Args &k, int32_t grid, cudaStream_t st);

}  // namespace eagle
