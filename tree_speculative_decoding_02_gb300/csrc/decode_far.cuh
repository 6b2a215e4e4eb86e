// decode_far.cuh -- single-token attention over an 8-bit cache: the rows of blocks of V whose scales are far from
// their segment's (far blocks), which k_decode_quant leaves out of its products: their weights would need more
// parts than the products have.  Shared by its clusters and by k_decode_finish.
//
// Bound by latency, a few rows at a time.  Of a batch of 32 requests of 1K to 32K rows, 24 heads over 4 of 256, blocks of 64
// rows: 0.1 % of them far 191 us (146 without), 1 % 351, 10 % 2790.
#pragma once

#include <math.h>

#include "decode.cuh"
#include "quant.cuh"

namespace ddt {

constexpr int kNear = 4;    // powers of two from the segment's unit up to which a block of V goes through the products
constexpr int kApart = 80;  // between two far blocks, or one and the unit, above which there is no result

// The byte that V's scales of a segment count from, its unit, by a warp whose lanes have the bytes of its first 32 blocks (0:
// none, or of zeros; of zeros alone: those of a later tile): the first block's, or if that one is far from the median of first,
// middle and last, the median; 0 if there is none.
__device__ __forceinline__ int v_unit_of(int byte) {
    const unsigned some = __ballot_sync(kFull, byte > 0);
    const int x = __ffs(some) - 1, z = 31 - __clz(some);  // (none: any lane)
    const int a = __shfl_sync(kFull, byte, x), m = __shfl_sync(kFull, byte, (x + z) / 2), c = __shfl_sync(kFull, byte, z), b = m ? m : a;
    const int median = max(min(a, b), min(max(a, b), c));
    return !some ? 0 : (abs(a - median) > kNear ? median : a);
}
__device__ __forceinline__ bool is_far(int byte, int unit) { return byte && abs(byte - unit) > kNear; }

// E channels of a query as they lie in memory (2, 4 or 8; aligned to their bytes)
template <typename T, int E>
struct QueryRun {
    static constexpr int W = E * (int)sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (W == 1) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x; w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
                w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    // bits of the largest |x| (integers order as the values do)
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) m = sizeof(T) == 4 ? max(m, w[i] & 0x7fffffffu) : __vmaxu2(m, w[i] & 0x7fff7fffu);
        return sizeof(T) == 4 ? m : max(m & 0xffffu, m >> 16) << 16;
    }
    __device__ __forceinline__ float get(int i) const {
        if (sizeof(T) == 4) return __uint_as_float(w[i % W]);
        return __uint_as_float(i % 2 ? w[i / 2 % W] & 0xffff0000u : w[i / 2 % W] << 16);
    }
    __device__ __forceinline__ uint32_t top_finite() const {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) m = fabsf(get(i)) < INFINITY ? fmaxf(m, fabsf(get(i))) : m;
        return __float_as_uint(m);
    }
    __device__ __forceinline__ void without_infinities() {  // what has all bits of the exponent set becomes NaN
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (sizeof(T) == 4) {
                if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] = 0x7fffffffu;
            } else {
                if ((w[i] & 0x7f80u) == 0x7f80u) w[i] |= 0x7fffu;
                if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] |= 0x7fff0000u;
            }
        }
    }
};

// E codes as they lie in memory
template <int E>
struct CodeRun {
    uint32_t w[(E + 3) / 4];
    __device__ __forceinline__ void load(const unsigned char* p) {
        if constexpr (E == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else if constexpr (E == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x; w[1] = x.y;
        }
    }
    __device__ __forceinline__ float get(int i) const {
        const float2 x = e4m3_values(w[i / 4] >> (i % 4 / 2 * 16) & 0xffffu);
        return i % 2 ? x.y : x.x;
    }
};

// One warp: the far rows of tiles [t0, t1) of (layer, request) lb and kv head g join the partial of query head hq of g's, in
// `slot` at place h: a segment's tiles.  Scores, weights and products in fp32 from the codes in HBM, a few rows at once.
template <typename Tin, int D>
__device__ __forceinline__ void far_rows(const DecodeParams& p, int lb, int g, int hq, int t0, int t1, long long slot, int h, int lane) {
    constexpr int E = D / 32, R = E == 8 ? 4 : 8;  // consecutive channels a lane; rows at once, the next ones on their way
    float2* const ml = p.part_ml + slot * p.HT + h;
    float2 part = *ml;
    if (part.y < 0.f) return;  // a bad page, or a wait that gave up
    const int l = lb / p.B, b = lb - l * p.B, end = min(p.prefix_len[b], t1 * kDecTile), per_page = p.page_rows / p.block;
    const int32_t* table = p.block_table + (long long)b * p.max_pages;
    QueryRun<Tin, E> q;
    q.load(static_cast<const Tin*>(p.q) + ((long long)lb * p.Hq + g * p.G + hq) * D + lane * E);
    float* const out = p.part_o + (slot * p.HT + h) * D + lane * E;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = out[e];
    int unit = 0, low = 255, high = 0;  // of the far blocks' scales
    // 32 blocks at a time, one a lane; tile after tile while all are of zeros, as k_decode_quant looks for the unit
    for (int r0 = t0 * kDecTile, step; r0 < end; r0 += step) {
        step = unit || r0 == t0 * kDecTile ? 32 * p.block : kDecTile;
        const int pos = r0 + lane * p.block;
        const bool there = pos < min(end, r0 + step);
        const long long plane = there ? ((long long)l * p.num_pages + table[pos / p.page_rows]) * p.Hkv + g : 0;
        const long long at = plane * per_page + pos % p.page_rows / p.block;
        const int vb = there ? p.vs[at] : 0, kb = there ? p.ks[at] : 0;
        if (!unit) unit = v_unit_of(vb);
        const bool mine = is_far(vb, unit);
        if (mine) low = min(low, vb), high = max(high, vb);
        for (unsigned far = __ballot_sync(kFull, mine); far; far &= far - 1) {
            const int of = __ffs(far) - 1, first = r0 + of * p.block, n = min(p.block, end - first);
            const float k_unit = scale_of(__shfl_sync(kFull, kb, of)) * p.scale_log2, v_unit = scale_of(__shfl_sync(kFull, vb, of));
            const long long row = __shfl_sync(kFull, plane, of) * p.page_rows + first % p.page_rows;
            const unsigned char* kc = static_cast<const unsigned char*>(p.k_pages) + row * D + lane * E;
            const unsigned char* vc = static_cast<const unsigned char*>(p.v_pages) + row * D + lane * E;
            struct Rows {
                CodeRun<E> k[R], v[R];
            } x, y;
            auto load = [&](int i0, Rows& z) {  // (a block is of a multiple of 8 rows: all are there to be read)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    z.k[i].load(kc + (i0 + i) * D);
                    z.v[i].load(vc + (i0 + i) * D);
                }
            };
            auto add = [&](int i0, const Rows& z) {
                float s[R], most = part.x;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    s[i] = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) s[i] = fmaf(q.get(e), z.k[i].get(e), s[i]);
                    s[i] = warp_sum(s[i]) * k_unit;
                    if (i0 + i >= n) s[i] = -INFINITY;
                    most = fmaxf(most, s[i]);
                }
                const float f = tc::ex2(part.x - most);
                part = make_float2(most, part.y * f);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (i0 + i >= n) break;  // (rows behind the prefix may hold NaN)
                    const float w = tc::ex2(s[i] - most);
                    part.y += w;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, z.v[i].get(e) * v_unit, acc[e]);
                }
            };
            load(0, x);
            for (int i0 = 0; i0 < n; i0 += 2 * R) {
                if (i0 + R < n) load(i0 + R, y);
                add(i0, x);
                if (i0 + 2 * R < n) load(i0 + 2 * R, x);
                if (i0 + R < n) add(i0 + R, y);
            }
        }
    }
    if (max(__reduce_max_sync(kFull, high), unit) - min(__reduce_min_sync(kFull, low), unit) > kApart) part.y = __int_as_float(0x7fffffff);  // NaN
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = acc[e];
    if (lane == 0) *ml = part;
    __syncwarp();
}

}  // namespace ddt
