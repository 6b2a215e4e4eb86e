// decode.cuh -- what the kernels of ddt_decode_attn_paged share: the parameters, the split
// of the cached rows over the CTAs, and the layout of the partial results.
//
// A unit is one (layer, request, kv head, block of up to HBS of the kv head's query heads);
// its cached rows are cut into tiles of 128.  The tiles of all units, unit after unit, form
// one line, and CTA c of C takes the tiles [c T / C, (c + 1) T / C) of it: every CTA streams
// the same number of bytes (to a tile) whatever the requests' lengths are, with no plan from
// the host, so a captured call follows the lengths it is replayed with.  A CTA's run of one
// unit's tiles is a segment; it leaves a partial result (per head: the reference of its
// exponents, their sum, and the sum of the weighted value rows) in slot u + c, which no
// other segment has: from one segment to the next either u or c grows.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace ddt {

constexpr int kDecTile = 128;  // cached rows a tile

struct DecodeParams {
    int L, B, Hq, Hkv, G, d;
    int hbs, HB, HT;  // heads a block (of the kernel), blocks a kv head, heads a partial slot holds: min(G, hbs)
    int page_rows, num_pages, max_pages, cap;
    int C;            // CTAs of the split kernel
    const int32_t* block_table;
    const int32_t* prefix_len;
    const void* q;
    const void* k_new;
    const void* v_new;
    const void* k_pages;
    const void* v_pages;
    void* o;
    float* weight;   // [L][B][Hkv][cap], or null
    int32_t* status;
    float scale_log2;
    // workspace
    long long* pre;   // [B + 1] tiles of the requests before b
    float2* part_ml;  // [U + C][HT] (reference in log2 units, sum); sum < 0: see kSeg*
    float* part_o;    // [U + C][HT][d]
    float* score;     // [L][B][Hq][cap] scores in log2 units (weight only)
};

// values of a partial's sum that say why there is none
constexpr float kSegBadPage = -1.f;  // a block-table entry outside [0, num_pages)
constexpr float kSegTimeout = -2.f;  // a bounded wait gave up

__host__ __device__ __forceinline__ int dec_tiles(int P, int cap) {
    return (P < 0 || P > cap) ? 0 : (P + kDecTile - 1) / kDecTile;
}

// A CTA's place on the line of tiles.
struct DecodeWalk {
    long long left;  // tiles this CTA still has
    int l, b, g;     // g: kv head and head block together
    int P, t, nt;    // rows of the request, first tile of the segment, tiles of the unit
};

// First tile of CTA c, and the CTA that owns tile x, of T tiles over C CTAs, every one of
// which has a tile (where T < C the CTAs from T on have none: C is then T).
// (A 64-bit division takes about 100 instructions; ordinary calls fit in 32 bits.)
__device__ __forceinline__ long long dec_first(long long T, int C, int c) {
    return T <= 0xffffffffu / (unsigned)C ? (unsigned)T * (unsigned)c / (unsigned)C : T * c / C;
}
__device__ __forceinline__ int dec_owner(long long T, int C, long long x) {
    return T <= 0xffffffffu / (unsigned)C ? (int)(((unsigned)(x + 1) * (unsigned)C - 1u) / (unsigned)T)
                                          : (int)(((x + 1) * C - 1) / T);
}

// All threads of the block: finds this CTA's run.  CTA 0 also writes pre[] and the statuses.
template <int NT>
__device__ __forceinline__ DecodeWalk dec_plan(const DecodeParams& p) {
    __shared__ long long s_sum[NT / 32];
    __shared__ long long s_pre;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT;  // consecutive requests a thread counts
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += dec_tiles(p.prefix_len[b], p.cap);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    if (tid == 0) s_b = -1;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += s_sum[w];
        all += s_sum[w];
    }
    const long long excl = before + incl - mine;
    if (blockIdx.x == 0) {
        long long at = excl;
        for (int b = b0; b < b1; ++b) {
            const int P = p.prefix_len[b];
            p.pre[b] = at;
            at += dec_tiles(P, p.cap);
            p.status[b] = (P < 0 || P > p.cap) ? DDT_ERR_CAPACITY : DDT_OK;
        }
        if (tid == 0) p.pre[p.B] = all;
    }
    const int HH = p.Hkv * p.HB;
    const long long T = all * HH * p.L;
    const int C = (int)min((long long)p.C, T), c = blockIdx.x;
    DecodeWalk w;
    const long long s = c < C ? dec_first(T, C, c) : 0;
    w.left = c < C ? dec_first(T, C, c + 1) - s : 0;
    w.l = w.b = w.g = w.P = w.t = w.nt = 0;
    if (w.left <= 0) return w;  // the same for the whole block
    w.l = (int)(s / (all * HH));
    const long long r = s % (all * HH), y = r / HH;
    if (y >= excl && y < excl + mine) {
        long long at = excl;
        for (int b = b0; b < b1; ++b) {
            const int t = dec_tiles(p.prefix_len[b], p.cap);
            if (y < at + t) {
                s_b = b;
                s_pre = at;
                break;
            }
            at += t;
        }
    }
    __syncthreads();
    w.b = s_b;
    w.P = p.prefix_len[w.b];
    w.nt = dec_tiles(w.P, p.cap);
    const long long r2 = r - s_pre * HH;
    w.g = (int)(r2 / w.nt);
    w.t = (int)(r2 % w.nt);
    return w;
}

// Tiles of the current segment, and the step to the next one.
__device__ __forceinline__ int dec_seg_tiles(const DecodeWalk& w) { return (int)min((long long)(w.nt - w.t), w.left); }
__device__ __forceinline__ void dec_next(const DecodeParams& p, DecodeWalk& w) {
    w.left -= dec_seg_tiles(w);
    if (w.left <= 0) return;
    w.t = 0;
    if (++w.g < p.Hkv * p.HB) return;
    w.g = 0;
    do {
        if (++w.b == p.B) {
            w.b = 0;
            ++w.l;
        }
        w.P = p.prefix_len[w.b];
        w.nt = dec_tiles(w.P, p.cap);
    } while (w.nt == 0);
}
__device__ __forceinline__ long long dec_unit(const DecodeParams& p, const DecodeWalk& w) {
    return ((long long)w.l * p.B + w.b) * (p.Hkv * p.HB) + w.g;
}

bool decode_tc_supported(int d, ddt_dtype in);
int decode_tc_heads(int G, int d);
cudaError_t launch_decode_tc(DecodeParams& p, cudaStream_t st);

}  // namespace ddt
