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

// What each CTA leaves for the merge: of the unit that its first segment belongs to, where that one was
// begun by an earlier CTA.
struct Kv4Share {
    int32_t kind;  // 0: begun here (or nothing to do), 1: begun earlier and ended here, 2: ended later
    int32_t b, hk, qt;
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
    float2 *carry_ml;        // [grid][kKv4Carry]: part_ml of a unit's earlier segments, for each thread or item its own
    int32_t segment;         // tiles summed in one go
};
constexpr int32_t kKv4Carry = 512;

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

// True once the phase with the given parity has completed; sleeps on the barrier up to 20 us.
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
// Waits for `parity` (its lowest bit) on `bar`.  Gives up when *abort is set, and sets it after
// limit_ns.  Small, so that the kernels' loops stay in the instruction cache: the clock is looked
// at once in 64 tries.
__device__ __forceinline__ bool kv4_wait(uint64_t *bar, uint32_t parity, volatile int32_t *abort, uint64_t limit_ns) {
    uint64_t since = 0;
    for (uint32_t i = 1;; ++i) {
        if (try_wait_long(bar, parity & 1u)) return true;
        if (*abort) return false;
        if ((i & 63u) == 0) {
            const uint64_t now = global_timer_ns();
            if (since == 0) {
                since = now;
            } else if (now - since > limit_ns) {
                *abort = 1;
                return false;
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The line of tiles
// ---------------------------------------------------------------------------------------------
// Everything is counted in 32 bits: the host refuses calls whose line could be longer.
// Tiles of new keys that the rows of query tile qt need.
__device__ __forceinline__ int32_t new_tiles(const Kv4Args &k, int32_t qt) {
    if (!k.a.kn) return 0;
    if (k.a.mask) return ((k.a.n - 1) >> k.tile_shift) + 1;
    const int32_t last = min(k.a.n - 1, ((qt + 1) * k.rows - 1) / k.group);
    return (last >> k.tile_shift) + 1;
}
// Tiles of `len` cached keys; at least one where a unit would have none.
__device__ __forceinline__ int32_t cached_tiles(const Kv4Args &k, int32_t len) {
    const int32_t t = (len + (1 << k.tile_shift) - 1) >> k.tile_shift;
    return t < 1 && !k.a.kn ? 1 : t;
}
__device__ __forceinline__ int32_t length_of(const Kv4Args &k, int32_t b) { return static_cast<int32_t>(kv4_length(k.a.cache, b)); }

// The lengths that a CTA goes by, as lengths[] gave them: those of the 32 requests that it is at and of the
// next 32, in shared memory.  One reading for all of its warps: they meet at barriers, so they have to
// take the same units and tiles even if the lengths are written to under the call.
struct Lengths {
    int32_t raw[2][32];
    __device__ __forceinline__ int32_t of(int32_t b) const { return raw[(b >> 5) & 1][b & 31]; }
};
constexpr uint32_t kLengthsBarrier = 4;
// The 32 requests from b on, a multiple of 32.  One warp.
__device__ __forceinline__ void read_lengths(const Kv4Args &k, Lengths &lens, int32_t b) {
    const int32_t lane = threadIdx.x & 31;
    lens.raw[(b >> 5) & 1][lane] = b + lane < k.a.B ? k.a.cache.lengths[b + lane] : 0;
}

// A CTA's tiles [begin, end) of the line, and the unit that the first of them belongs to.
struct Place {
    int32_t begin, end;
    int32_t b, hk, qt;
    int32_t off;  // the first tile's place in its unit
};
struct Spot {
    int32_t b, hk, qt;
    int32_t off, unit;  // place in the unit, and its tiles
};

// The unit `off` tiles into request b, which has ct tiles of cached keys and `per` of new keys for each
// kv head.
__device__ __forceinline__ Spot spot_of(const Kv4Args &k, int32_t b, int32_t ct, int32_t off, int32_t per) {
    Spot s;
    s.b = b;
    const uint32_t block = k.QT * ct + per;
    s.hk = static_cast<uint32_t>(off) / block;
    off -= s.hk * block;
    if (k.QT == 1 || k.a.mask || !k.a.kn) {
        s.unit = ct + new_tiles(k, 0);
        s.qt = k.QT == 1 ? 0 : static_cast<uint32_t>(off) / static_cast<uint32_t>(s.unit);
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
__device__ __forceinline__ bool move_cut(int32_t &cut, const Spot &s, int32_t snap) {
    const int32_t left = s.unit - s.off;
    if (s.off <= left) {
        if (s.off <= snap) cut -= s.off;
        return false;
    }
    if (left > snap) return false;
    cut += left;
    return true;
}
// CTA c's raw cuts: c total / ctas and the next, rounded down.
__device__ __forceinline__ void raw_cuts(const Kv4Args &k, uint32_t total, uint32_t &ctas, int32_t &cut0, int32_t &cut1) {
    const uint32_t want = (total + k.min_tiles - 1) / k.min_tiles, c = blockIdx.x;
    ctas = min(max(want, 1u), gridDim.x);
    const uint32_t q = total / ctas, r = total - q * ctas;
    cut0 = c * q + c * r / ctas;
    cut1 = (c + 1) * q + (c + 1) * r / ctas;
}
// The place of the CTA whose raw cuts lie at the given spots.  False: nothing to do.
__device__ __forceinline__ bool place_at(const Kv4Args &k, Place *p, uint32_t total, uint32_t ctas, int32_t cut0, int32_t cut1,
                                         Spot s0, const Spot &s1) {
    // at most a third of a CTA's share, so that few tiles still spread over all CTAs
    const int32_t snap = min(static_cast<uint32_t>(k.snap), total / (3 * ctas));
    const int32_t was = cut0;
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
    if (static_cast<uint32_t>(cut1) < total) move_cut(cut1, s1, snap);
    *p = Place{cut0, cut1, s0.b, s0.hk, s0.qt, s0.off};
    return cut0 < cut1;
}

// At most 32 requests: one warp, a request a lane.
__device__ __forceinline__ bool find_place_warp(const Kv4Args &k, Place *p, const Lengths &lens) {
    const int32_t lane = threadIdx.x & 31;
    const int32_t ct = lane < k.a.B ? cached_tiles(k, static_cast<int32_t>(kv4_clamped(k.a.cache, lens.of(lane)))) : 0;
    int32_t per;
    if (k.QT == 1 || k.a.mask || !k.a.kn) {
        per = k.QT * new_tiles(k, 0);
    } else {
        per = 0;
        for (int32_t q = lane; q < k.QT; q += 32) per += new_tiles(k, q);
        per = __reduce_add_sync(kFull, per);
    }
    const int32_t w = lane < k.a.B ? k.a.cache.Hk * (k.QT * ct + per) : 0;
    int32_t inc = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t o = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += o;
    }
    const uint32_t total = __shfl_sync(kFull, inc, 31);
    uint32_t ctas;
    int32_t cut0, cut1;
    raw_cuts(k, total, ctas, cut0, cut1);
    if (blockIdx.x >= ctas) return false;
    // the lanes' runs are ascending: the first whose end lies behind a cut holds it
    Spot s[2];
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int32_t cut = min(i ? cut1 : cut0, static_cast<int32_t>(total) - 1);
        const int32_t b = __ffs(__ballot_sync(kFull, inc > cut)) - 1;
        const Spot x = spot_of(k, b, __shfl_sync(kFull, ct, b), cut - __shfl_sync(kFull, inc - w, b), per);
        if (i) s[1] = x;
        else s[0] = x;
    }
    return place_at(k, p, total, ctas, cut0, cut1, s[0], s[1]);
}

// Sum over the block; every thread gets it.  `red`: one slot a warp.
static __device__ __noinline__ int32_t block_sum(int32_t v, int32_t *red) {
    v = __reduce_add_sync(kFull, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int32_t t = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) t += red[w];
    return t;
}
// More: all threads of the block together.
static __device__ __noinline__ bool find_place_block(const Kv4Args &k, Place *p, int32_t *red, Spot *spots) {
    const int32_t tid = threadIdx.x, nt = blockDim.x, B = k.a.B, Hk = k.a.cache.Hk;
    // kept where lengths that were written to between the two looks at them put no request behind a cut
    if (tid < 2) spots[tid] = Spot{B - 1, Hk - 1, k.QT - 1, 0, 1};
    int32_t per = 0;
    if (k.a.mask || !k.a.kn) {
        per = k.QT * new_tiles(k, 0);
    } else {
        for (int32_t q = tid; q < k.QT; q += nt) per += new_tiles(k, q);
        per = block_sum(per, red);
    }
    int32_t mine = 0;
    for (int32_t b = tid; b < B; b += nt) mine += Hk * (k.QT * cached_tiles(k, length_of(k, b)) + per);
    const uint32_t total = block_sum(mine, red);
    uint32_t ctas;
    int32_t cut[2];
    raw_cuts(k, total, ctas, cut[0], cut[1]);
    if (blockIdx.x >= ctas) return false;
    // the requests that hold the tiles behind the two cuts
    int32_t base = 0;
    for (int32_t b0 = 0; b0 < B; b0 += nt) {
        const int32_t b = b0 + tid;
        const int32_t ct = b < B ? cached_tiles(k, length_of(k, b)) : 0, w = b < B ? Hk * (k.QT * ct + per) : 0;
        int32_t inc = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t o = __shfl_up_sync(kFull, inc, off);
            if ((tid & 31) >= off) inc += o;
        }
        __syncthreads();
        if ((tid & 31) == 31) red[tid >> 5] = inc;
        __syncthreads();
        int32_t before = base, all = base;
        for (int w2 = 0; w2 < nt / 32; ++w2) {
            if (w2 < (tid >> 5)) before += red[w2];
            all += red[w2];
        }
        const int32_t lo = before + inc - w;
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
            if (cut[i] >= lo && cut[i] < lo + w) spots[i] = spot_of(k, b, ct, cut[i] - lo, per);
        base = all;
        if (cut[1] < base) break;
    }
    __syncthreads();
    return place_at(k, p, total, ctas, cut[0], cut[1], spots[0], spots[static_cast<uint32_t>(cut[1]) < total]) && p->b < B;
}
// The CTA's place and the lengths there, in shared memory; all threads together.  False: nothing to do.
__device__ __forceinline__ bool find_place(const Kv4Args &k, Place &place, Lengths &lens, int32_t *red, Spot *spots) {
    const Place none{0, 0, 0, 0, 0, 0};
    if (k.a.B <= 32) {
        if (threadIdx.x < 32) {
            Place p;
            read_lengths(k, lens, 0);
            __syncwarp();
            const bool busy = find_place_warp(k, &p, lens);
            if (threadIdx.x == 0) place = busy ? p : none;
        }
    } else {
        Place p;
        const bool busy = find_place_block(k, &p, red, spots);
        if (busy && threadIdx.x < 64) read_lengths(k, lens, (p.b & ~31) + static_cast<int32_t>(threadIdx.x & 32));
        if (threadIdx.x == 0) place = busy ? p : none;
    }
    __syncthreads();
    return place.begin < place.end;
}

// A CTA's run through the line, unit by unit: tiles [from, to) of the unit, of which [s0, s1) is a segment.
// Accumulators of matrix products cut off what lies below their last bit: 2^-24 of themselves or so each time
// (4 M cached keys in one sum: 2.6 % over 16 query rows, 0.6 % up to 16).  So a segment has k.segment tiles at
// most, 256 or 1024: under 2^-12.  The segments of a unit join in the CTA's partial sums, in fp32 rounded to
// the nearest.
struct Walk {
    int32_t b, hk, qt;
    int32_t t, from, to, s0, s1, unit;
    int32_t nt;  // tiles of new keys (the unit's first)
    int32_t len;

    __device__ __forceinline__ void start(const Kv4Args &k, const Place &p, const Lengths &lens) {
        b = p.b;
        hk = p.hk;
        qt = p.qt;
        t = p.begin;
        s0 = p.off;
        len = static_cast<int32_t>(kv4_clamped(k.a.cache, lens.of(b)));
        fill(k, p);
    }
    __device__ __forceinline__ void fill(const Kv4Args &k, const Place &p) {
        nt = new_tiles(k, qt);
        unit = cached_tiles(k, len) + nt;
        from = s0 = min(s0, unit - 1);  // the place may come from an earlier length
        to = min(unit, s0 + (p.end - t));
        s1 = min(to, s0 + k.segment);
    }
    // Whether the next unit is of a request of another 32.
    __device__ __forceinline__ bool leaves(const Kv4Args &k, const Place &p) const {
        return s1 == to && ((b + 1) & 31) == 0 && b + 1 < k.a.B && hk + 1 == k.a.cache.Hk && qt + 1 == k.QT && t + s1 - s0 < p.end;
    }
    // (meet comes first)
    __device__ __forceinline__ bool next(const Kv4Args &k, const Place &p, const Lengths &lens) {
        t += s1 - s0;
        if (s1 < to) {
            s0 = s1;
            s1 = min(to, s0 + k.segment);
            return true;
        }
        if (t >= p.end) return false;
        s0 = 0;
        if (++qt == k.QT) {
            qt = 0;
            if (++hk == k.a.cache.Hk) {
                hk = 0;
                if (++b == k.a.B) return false;  // lengths were written to under the call
                len = static_cast<int32_t>(kv4_clamped(k.a.cache, lens.of(b)));
            }
        }
        fill(k, p);
        return true;
    }
};

// Ahead of the next unit: where its request is of another 32, all of the CTA's `threads` meet, after which
// none needs the 32 before, and the warp with `reads` set brings the lengths of those after.  Every warp
// comes here for every unit, also once a wait has given up.
__device__ __forceinline__ void meet(const Kv4Args &k, const Place &p, const Walk &w, Lengths &lens, uint32_t threads, bool reads) {
    if (!w.leaves(k, p)) return;
    __syncwarp();
    named_barrier_sync(kLengthsBarrier, threads);
    if (reads) read_lengths(k, lens, w.b + 33);
}

// On to the next unit of a walk in shared memory that the warp's lanes read; false behind the last.
__device__ __forceinline__ bool kv4_next(const Kv4Args &k, const Place &p, Walk &walk, Lengths &lens, uint32_t threads, bool reads) {
    meet(k, p, walk, lens, threads, reads);
    __syncwarp();  // every lane is through with the last
    int more = 0;
    if ((threadIdx.x & 31) == 0) {
        Walk w = walk;
        more = w.next(k, p, lens);
        walk = w;
    }
    more = __shfl_sync(kFull, more, 0);
    __syncwarp();
    return more != 0;
}

// What CTA blockIdx.x leaves for the merge.
__device__ __forceinline__ Kv4Share share_of(const Walk &w) {
    return Kv4Share{w.from == 0 ? 0 : (w.to == w.unit ? 1 : 2), w.b, w.hk, w.qt};
}
// Where a segment's partial sums go: slot 0 of its CTA for a unit that an earlier CTA began, else 1 (which
// only the CTA's last unit leaves to the merge).
__device__ __forceinline__ int64_t slot_of(const Walk &w) { return 2 * static_cast<int64_t>(blockIdx.x) + (w.from > 0 ? 0 : 1); }

// What a part with maximum m and sum l counts beside the maximum M of all: one that is all hidden has neither,
// one whose scores are all NaN has no maximum and a sum of NaN.
__device__ __forceinline__ float weight_of(float m, float l, float M) { return m == -INFINITY ? (l == 0.0f ? 0.0f : l) : ex2_approx(m - M); }
// Joins the part `was` of earlier segments to this one's (M, L).  now, before: the two parts' weights.
__device__ __forceinline__ void join(float2 was, float &M, float &L, float &now, float &before) {
    const float most = fmaxf(M, was.x);
    now = weight_of(M, L, most);
    before = weight_of(was.x, was.y, most);
    L = (now == 0.0f ? 0.0f : now * L) + (before == 0.0f ? 0.0f : before * was.y);
    M = most;
}

// The tcgen05 kernel (kv4_attn_tc.cu): units of 256 query rows, tiles of 128 keys.
constexpr int32_t kKv4TcRows = 256;
constexpr int32_t kKv4TcTile = 128;
constexpr int32_t kKv4TcSegment = 256;
cudaError_t prepare_kv4_attention_tc();
cudaError_t launch_kv4_attention_tc(const Kv4Args &k, int32_t grid, cudaStream_t st);

}  // namespace eagle
