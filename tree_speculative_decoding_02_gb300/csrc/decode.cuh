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
//
// Small calls (p.cl) are bound by latency instead: a cluster of CTAs takes a unit, and joins its
// partials behind a cluster barrier, in the same launch.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace ddt {

constexpr int kDecTile = 128;  // cached rows a tile

struct DecodeParams {
    int L, B, Hq, Hkv, G, d;
    int hbs, HB, HT;  // heads a block (of the kernel), blocks a kv head, heads a partial slot holds: min(G, hbs)
    int page_rows, num_pages, max_pages, cap;
    int C;            // CTAs of the split kernel
    int cl;           // 0, or small calls: a cluster of cl CTAs a unit, which also joins (HB is 1)
    ddt_dtype out;
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
    // caches in 8 bits
    const uint8_t* ks;  // [L][num_pages][Hkv][page_rows / block]
    const uint8_t* vs;
    int block;          // rows a scale
    int* far;           // [C] (workspace) whether a CTA's segments have far blocks
};

// values of a partial's sum that say why there is none
constexpr float kSegBadPage = -1.f;  // a block-table entry outside [0, num_pages)
constexpr float kSegTimeout = -2.f;  // a bounded wait gave up

// A segment's first reference, the lowest finite value: a head's scores may all be -inf so far, and
// 2^(-inf - kNoRef) is 0 where 2^(-inf + inf) is NaN.
constexpr float kNoRef = -3.402823466e38f;

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
    if (p.cl) {  // a unit a cluster, its tiles over the CTAs of the cluster
        const int u = blockIdx.x / p.cl, rank = blockIdx.x % p.cl;
        DecodeWalk w;
        w.g = u % p.Hkv;
        w.b = u / p.Hkv % p.B;
        w.l = u / p.Hkv / p.B;
        w.P = p.prefix_len[w.b];
        w.nt = dec_tiles(w.P, p.cap);
        const int c = min(p.cl, w.nt);
        w.t = rank < c ? w.nt * rank / c : 0;
        w.left = rank < c ? w.nt * (rank + 1) / c - w.t : 0;
        // The request's status.  What its lengths and pages raise, this unit raises too, behind
        // its cluster's barrier.  A wait that gives up in another unit does so a second after its
        // CTA began, and all CTAs of the grid are resident.
        if (w.l == 0 && w.g == 0 && rank == 0 && tid == 0) p.status[w.b] = DDT_OK;
        return w;
    }
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
// the segment's slot
__device__ __forceinline__ long long dec_slot(const DecodeParams& p, const DecodeWalk& w) {
    return p.cl ? blockIdx.x : ((long long)w.l * p.B + w.b) * (p.Hkv * p.HB) + w.g + blockIdx.x;
}

// The new row's part of head h of kv head g, by one warp: its score (log2 units), and its value.
template <typename Tin, int D>
struct DecNew {
    float tn, v[D / 32];
    __device__ __forceinline__ void load(const DecodeParams& p, long long lb, int g, int h, int lane) {
        tn = -INFINITY;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
        if (!p.k_new || h >= p.G) return;
        const Tin* q = static_cast<const Tin*>(p.q) + (lb * p.Hq + g * p.G + h) * D + lane;
        const Tin* k = static_cast<const Tin*>(p.k_new) + (lb * p.Hkv + g) * D + lane;
        const Tin* vn = static_cast<const Tin*>(p.v_new) + (lb * p.Hkv + g) * D + lane;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            s = fmaf(to_f32(q[e * 32]), to_f32(k[e * 32]), s);
            v[e] = to_f32(vn[e * 32]);
        }
        tn = warp_sum(s) * p.scale_log2;
    }
};
// One head's joined softmax, by one warp.
struct HeadJoin {
    float ref, z;      // reference, sum
    int err;           // a status for the request, or DDT_OK
    int ns;            // segments, from slot `first` on
    long long first;
    int c0;            // the first one's CTA
    bool far;          // FAR: one of their CTAs has far blocks
};

template <bool FAR = false>
__device__ __forceinline__ HeadJoin head_join(const DecodeParams& p, int lb, int hq, float tn, int lane) {
    const int l = lb / p.B, b = lb - l * p.B, g = hq / p.G, hb = (hq % p.G) / p.hbs, h = (hq % p.G) % p.hbs;
    // loads that do not wait for one another first
    const int P = p.prefix_len[b];
    const long long pre = p.cl ? 0 : p.pre[b], all = p.cl ? 0 : p.pre[p.B];
    HeadJoin j;
    j.ref = j.z = 0.f;
    j.ns = j.c0 = 0;
    j.first = 0;
    j.far = false;
    j.err = (P < 0 || P > p.cap) ? DDT_ERR_CAPACITY : DDT_OK;
    if (j.err) return j;
    const int nt = dec_tiles(P, p.cap);
    if (p.cl) {
        j.ns = min(p.cl, nt);
        j.first = ((long long)lb * p.Hkv + g) * p.cl;
    } else if (nt > 0) {
        const int HH = p.Hkv * p.HB;
        const long long T = all * HH * p.L;
        const long long first = l * all * HH + pre * HH + (long long)(g * p.HB + hb) * nt;
        const int C = (int)min((long long)p.C, T);
        j.c0 = dec_owner(T, C, first);
        j.ns = dec_owner(T, C, first + nt - 1) - j.c0 + 1;
        j.first = (long long)lb * HH + g * p.HB + hb + j.c0;
    }
    const float2* ml = p.part_ml + j.first * p.HT + h;
    float m = tn, low = 0.f;
    for (int s = lane; s < j.ns; s += 32) {
        const float2 v = ml[(long long)s * p.HT];
        if (FAR) j.far |= p.far[j.c0 + s] != 0;
        m = fmaxf(m, v.x);
        low = fminf(low, v.y);
    }
    if (FAR) j.far = __any_sync(kFull, j.far);
    m = warp_max(m);
    low = -warp_max(-low);
    if (low < 0.f) j.err = low == kSegTimeout ? DDT_ERR_TIMEOUT : DDT_ERR_INVALID_ARG;
    j.ref = m == -INFINITY ? 0.f : m;
    float z = 0.f;
    for (int s = lane; s < j.ns; s += 32) {
        const float2 v = ml[(long long)s * p.HT];
        z = fmaf(tc::ex2(v.x - j.ref), v.y, z);
    }
    j.z = warp_sum(z) + tc::ex2(tn - j.ref);
    return j;
}

// A cluster's finish (p.cl): the heads of its unit over its warps, the weight sums of each CTA's
// own rows.  All threads of all its CTAs, behind a cluster barrier; `w` as dec_plan gave it.  What
// needs no partials (the new row's part of a warp's first head) comes before the barrier.
__device__ __forceinline__ int dec_first_head(const DecodeParams& p) {
    return (int)(blockIdx.x % p.cl) + p.cl * (int)(threadIdx.x >> 5);
}

template <typename Tin, int D, int NT>
__device__ __forceinline__ void dec_finish(const DecodeParams& p, const DecodeWalk& w, DecNew<Tin, D> x, float* s_x) {
    constexpr int E = D / 32, kCh = E == 8 ? 4 : 8;  // segments whose O is in flight
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x % p.cl;
    const int lb = w.l * p.B + w.b, g = w.g, ns = min(p.cl, w.nt);
    const long long first = ((long long)lb * p.Hkv + g) * p.cl;  // slot
    for (int h = dec_first_head(p); h < p.G; h += p.cl * (NT / 32)) {
        if (h >= p.cl * (NT / 32)) x.load(p, lb, g, h, lane);
        const float* po = p.part_o + (first * p.HT + h) * D + lane;
        const float2 ml = lane < ns ? p.part_ml[(first + lane) * p.HT + h] : make_float2(-INFINITY, 0.f);
        float o[kCh][E], acc[E];
#pragma unroll
        for (int s = 0; s < kCh; ++s)
#pragma unroll
            for (int e = 0; e < E; ++e) o[s][e] = s < ns ? po[(long long)s * p.HT * D + e * 32] : 0.f;
        const float m = fmaxf(warp_max(ml.x), x.tn), ref = m == -INFINITY ? 0.f : m, low = -warp_max(-fminf(ml.y, 0.f));
        const float f = lane < ns ? tc::ex2(ml.x - ref) : 0.f, fn = tc::ex2(x.tn - ref);
        const float z = warp_sum(f * ml.y) + fn;
        const int err = (w.P < 0 || w.P > p.cap) ? DDT_ERR_CAPACITY
                                                 : (low < 0.f ? (low == kSegTimeout ? DDT_ERR_TIMEOUT : DDT_ERR_INVALID_ARG) : DDT_OK);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fn * x.v[e];
#pragma unroll
        for (int s0 = 0; s0 < 8; s0 += kCh) {
            if (s0 >= ns) break;
            if (s0) {
#pragma unroll
                for (int s = 0; s < kCh; ++s)
#pragma unroll
                    for (int e = 0; e < E; ++e) o[s][e] = s0 + s < ns ? po[(long long)(s0 + s) * p.HT * D + e * 32] : 0.f;
            }
#pragma unroll
            for (int s = 0; s < kCh; ++s) {
                const float fs = __shfl_sync(kFull, f, s0 + s);
                if (s0 + s < ns)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(fs, o[s][e], acc[e]);
            }
        }
        const float inv = z > 0.f ? 1.f / z : z;  // no rows at all: 0; NaN stays
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = err ? 0.f : acc[e] * inv;
        if (err && lane == 0) atomicMax(p.status + w.b, err);
        const long long at = ((long long)lb * p.Hq + g * p.G + h) * D;
        if (p.out == DDT_BF16) {
#pragma unroll
            for (int e = 0; e < E; ++e) static_cast<__nv_bfloat16*>(p.o)[at + e * 32 + lane] = from_f32<__nv_bfloat16>(acc[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) static_cast<float*>(p.o)[at + e * 32 + lane] = acc[e];
        }
    }
    if (!p.weight) return;
    float* s_ref = s_x;
    float* s_inv = s_ref + p.G;
    float* s_tn = s_inv + p.G;
    int bad = 0;
    for (int h = warp; h < p.G; h += NT / 32) {
        x.load(p, lb, g, h, lane);
        const HeadJoin j = head_join(p, lb, g * p.G + h, x.tn, lane);
        bad |= j.err;
        if (lane == 0) {
            s_ref[h] = j.ref;
            s_inv[h] = j.z > 0.f ? 1.f / j.z : j.z;  // (NaN stays)
            s_tn[h] = x.tn;
        }
    }
    if (__syncthreads_or(bad)) return;
    const float* sc = p.score + ((long long)lb * p.Hq + g * p.G) * p.cap;
    float* wt = p.weight + ((long long)lb * p.Hkv + g) * p.cap;
    const int end = min(w.P, (w.t + (int)w.left) * kDecTile);
    if (w.left > 0)
        for (int r = w.t * kDecTile + tid; r < end; r += NT) {
            float sum = 0.f;
#pragma unroll 4
            for (int h = 0; h < p.G; ++h) sum = fmaf(tc::ex2(sc[(long long)h * p.cap + r] - s_ref[h]), s_inv[h], sum);
            wt[r] += sum;
        }
    if (p.k_new && w.P < p.cap && rank == 0 && tid == 0) {  // the new token's own row
        float sum = 0.f;
        for (int h = 0; h < p.G; ++h) sum = fmaf(tc::ex2(s_tn[h] - s_ref[h]), s_inv[h], sum);
        wt[w.P] += sum;
    }
}

// ---- what the tensor-core kernels share
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!tc::mbar_try(bar, parity))
        if (clock64() - t0 > tc::kWaitCycles) return;
}

// the warp's maximum in one instruction
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// barrier of the 128 softmax threads that also tells whether any of them passed true
__device__ __forceinline__ bool bar_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return r != 0;
}

// 8 consecutive 32-bit columns of this thread's lane
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn decode_encode_fn();  // cuTensorMapEncodeTiled, or null
bool decode_tc_supported(int d, ddt_dtype in);
int decode_tc_heads(int G, int d);
cudaError_t launch_decode_tc(DecodeParams& p, cudaStream_t st);
int decode_quant_heads(int G, ddt_dtype in);
cudaError_t launch_decode_quant_tiles(DecodeParams& p, ddt_dtype in, cudaStream_t st);
struct DecodeSmall {
    double most, excess;  // channels of a CTA's rows, in tiles, and of those above an even split's, up to which a call is small
};
void decode_clusters(DecodeParams& p, DecodeSmall small, int ctas);
cudaLaunchConfig_t decode_grid(const DecodeParams& p, int threads, int smem, cudaLaunchAttribute& at, cudaStream_t st);

}  // namespace ddt
