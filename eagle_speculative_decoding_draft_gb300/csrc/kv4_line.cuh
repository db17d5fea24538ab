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
    int32_t first, last;
};

struct Kv4Args {
    Kv4Attention a;
    int32_t group, Mq, rows, QT, W;
    int32_t tile_shift;      // log2 of the keys of a tile
    int32_t min_tiles;       // tiles a CTA takes at least
    int32_t snap;            // how far a cut may move to a unit's end
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
    int64_t snap;               // how far cuts were moved at most
    int64_t off;                // the first tile's place in its unit
    int32_t b, hk, qt;
};
struct Spot {
    int32_t b, hk, qt;
    int64_t off, unit;  // place in the unit, and its tiles
};

__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {  // x >= 0, y > 0
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

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

// The unit `off` tiles into request b, which has ct tiles of cached keys and `per` of new keys for each
// kv head.
static __device__ __noinline__ Spot spot_of(const Kv4Args &k, int32_t b, int64_t ct, int64_t off, int64_t per) {
    const int64_t block = k.QT * ct + per;
    Spot s;
    s.b = b;
    s.hk = static_cast<int32_t>(quotient(off, block));
    off -= s.hk * block;
    if (k.a.mask || !k.a.kn) {
        s.unit = ct + new_tiles(k, 0);
        s.qt = static_cast<int32_t>(quotient(off, s.unit));
        off -= s.qt * s.unit;
    } else {
        s.qt = 0;
        for (; off >= (s.unit = ct + new_tiles(k, s.qt)); ++s.qt) off -= s.unit;
    }
    s.off = off;
    return s;
}

// Moves a cut that falls within `snap` tiles of a unit's end to the nearer end: a unit cut in two costs
// partial sums of all its rows, written and read again.  True: to the unit's own end.
__device__ __forceinline__ bool move_cut(int64_t &cut, const Spot &s, int64_t snap) {
    const int64_t left = s.unit - s.off;
    if (s.off <= left) {
        if (s.off <= snap) cut -= s.off;
        return false;
    }
    if (left > snap) return false;
    cut += left;
    return true;
}
// The place of the CTA whose share runs from cut[0] to cut[1], which lie at the given spots.  False:
// nothing to do.
__device__ __forceinline__ bool place_at(const Kv4Args &k, Place *p, int64_t total, int64_t ctas, int64_t cut0, int64_t cut1,
                                         Spot s0, const Spot &s1) {
    // at most a third of a CTA's share, so that few tiles still spread over all CTAs
    const int64_t snap = min(static_cast<int64_t>(k.snap), quotient(total, 3 * ctas));
    const int64_t was = cut0;
    if (move_cut(cut0, s0, snap)) {  // the next unit's first tile
        s0.off = 0;
        if (++s0.qt == k.QT) {
            s0.qt = 0;
            if (++s0.hk == k.a.cache.Hk) {
                s0.hk = 0;
                ++s0.b;
            }
        }
    } else {
        s0.off -= was - cut0;
    }
    if (cut1 < total) move_cut(cut1, s1, snap);
    *p = Place{total, cut0, cut1, ctas, snap, s0.off, s0.b, s0.hk, s0.qt};
    return cut0 < cut1;
}
__device__ __forceinline__ int64_t ctas_of(const Kv4Args &k, int64_t total) {
    const int64_t want = quotient(total + k.min_tiles - 1, k.min_tiles);
    return want < gridDim.x ? (want < 1 ? 1 : want) : gridDim.x;
}

// At most 32 requests: every warp finds the place by itself (one request a lane), with no barrier.
static __device__ __noinline__ bool find_place_warp(const Kv4Args &k, Place *p) {
    const int32_t lane = threadIdx.x & 31;
    const int64_t ct = lane < k.a.B ? cached_tiles(k, lane) : 0;
    int64_t per = 0;
    if (k.a.mask || !k.a.kn) {
        per = static_cast<int64_t>(k.QT) * new_tiles(k, 0);
    } else {
        for (int32_t q = lane; q < k.QT; q += 32) per += new_tiles(k, q);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) per += __shfl_xor_sync(kFull, per, off);
    }
    const int64_t w = lane < k.a.B ? k.a.cache.Hk * (k.QT * ct + per) : 0;
    int64_t inc = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += o;
    }
    const int64_t total = __shfl_sync(kFull, inc, 31), ctas = ctas_of(k, total), c = blockIdx.x;
    if (c >= ctas) return false;
    const int64_t cut0 = quotient(c * total, ctas), cut1 = quotient((c + 1) * total, ctas);
    // the lanes' runs are ascending: the first whose end lies behind the cut holds it
    const int32_t b0 = __ffs(__ballot_sync(kFull, inc > cut0)) - 1;
    const int32_t b1 = cut1 < total ? __ffs(__ballot_sync(kFull, inc > cut1)) - 1 : b0;
    const int64_t lo = inc - w;
    const int64_t lo0 = __shfl_sync(kFull, lo, b0), lo1 = __shfl_sync(kFull, lo, b1);
    const int64_t ct0 = __shfl_sync(kFull, ct, b0), ct1 = __shfl_sync(kFull, ct, b1);
    const Spot s0 = spot_of(k, b0, ct0, cut0 - lo0, per);
    const Spot s1 = cut1 < total ? spot_of(k, b1, ct1, cut1 - lo1, per) : s0;
    return place_at(k, p, total, ctas, cut0, cut1, s0, s1);
}

// More: all threads of the block together.  `red`: a slot a warp.
static __device__ __noinline__ bool find_place_block(const Kv4Args &k, Place *p, int64_t *red, Spot *spots) {
    const int32_t tid = threadIdx.x, nt = blockDim.x, B = k.a.B;
    const int64_t Hk = k.a.cache.Hk;
    int64_t per = 0;
    if (k.a.mask || !k.a.kn) {
        per = static_cast<int64_t>(k.QT) * new_tiles(k, 0);
    } else {
        for (int32_t q = tid; q < k.QT; q += nt) per += new_tiles(k, q);
        per = block_sum64(per, red);
    }
    int64_t mine = 0;
    for (int32_t b = tid; b < B; b += nt) mine += Hk * (k.QT * cached_tiles(k, b) + per);
    const int64_t total = block_sum64(mine, red), ctas = ctas_of(k, total), c = blockIdx.x;
    if (c >= ctas) return false;
    const int64_t cut[2] = {quotient(c * total, ctas), quotient((c + 1) * total, ctas)};
    // the requests that hold the tiles behind the two cuts
    int64_t base = 0;
    for (int32_t b0 = 0; b0 < B; b0 += nt) {
        const int32_t b = b0 + tid;
        const int64_t ct = b < B ? cached_tiles(k, b) : 0, w = b < B ? Hk * (k.QT * ct + per) : 0;
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
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
            if (cut[i] >= lo && cut[i] < lo + w) spots[i] = spot_of(k, b, ct, cut[i] - lo, per);
        base = all;
        if (cut[1] < base) break;
    }
    __syncthreads();
    return place_at(k, p, total, ctas, cut[0], cut[1], spots[0], spots[cut[1] < total]);
}
__device__ __forceinline__ bool find_place(const Kv4Args &k, Place *p, int64_t *red, Spot *spots) {
    return k.a.B <= 32 ? find_place_warp(k, p) : find_place_block(k, p, red, spots);
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
        len = kv4_length(k.a.cache, b);
        fill(k, p);
    }
    __device__ __forceinline__ void fill(const Kv4Args &k, const Place &p) {
        nt = new_tiles(k, qt);
        unit = ((len + (1 << k.tile_shift) - 1) >> k.tile_shift) + nt;
        unit = unit < 1 ? 1 : unit;  // nothing cached and no new keys: a tile with no keys
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
                len = kv4_length(k.a.cache, b);
            }
        }
        fill(k, p);
        return true;
    }
};

// What CTA blockIdx.x leaves for the merge, given that its first unit was begun by an earlier one.  The
// cuts left inside a unit [u0, u1) are those of CTAs c with u0 + snap < c total / ctas < u1 - snap; the
// CTA before the first of them began the unit.
static __device__ __noinline__ Kv4Share share_of(const Kv4Args &k, const Place &p, const Walk &w) {
    Kv4Share sh{-1, 0, 0, 0, 0};
    if (w.s0 > 0) {
        const int64_t u0 = p.begin - w.s0, c = blockIdx.x;
        if (quotient((c - 1) * p.total, p.ctas) <= u0 + p.snap)
            sh = Kv4Share{w.b, w.hk, w.qt, static_cast<int32_t>(c) - 1,
                          static_cast<int32_t>(quotient((u0 + w.unit - p.snap) * p.ctas - 1, p.total))};
    }
    return sh;
}
// Where a segment's partial sums go: slot 0 of its CTA for a unit that an earlier CTA began, else 1.
__device__ __forceinline__ int64_t slot_of(const Walk &w) { return 2 * static_cast<int64_t>(blockIdx.x) + (w.s0 > 0 ? 0 : 1); }

// The tcgen05 kernel (kv4_attn_tc.cu): head_dim 64 or 128, units of 256 query rows, tiles of 128 keys.
constexpr int32_t kKv4TcRows = 256;
constexpr int32_t kKv4TcTile = 128;
cudaError_t prepare_kv4_attention_tc();
cudaError_t launch_kv4_attention_tc(const Kv4Args &k, int32_t grid, cudaStream_t st);

}  // namespace eagle
