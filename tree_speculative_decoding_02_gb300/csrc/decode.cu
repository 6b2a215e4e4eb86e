// decode.cu -- ddt_decode_attn_paged: attention of one new token a request over the paged
// prefix cache, split over the cached rows and joined.
//
// "DDTree on vLLM: candid research notes", section "Where the next step is": attention over
// paged KV blocks.  This is the round's step for a request that has no drafts: one query row
// a head instead of a tree of them, so nothing is left to share a K/V row but the G query
// heads of its kv head, and the call is bound by reading the cache once.
//
//   k_decode_tc     grid C (decode_tc.cu): the tiles of a CTA's run on the tensor cores, bf16.
//   k_decode_simt   grid C: the same on the CUDA cores, fp32 caches.
//                   (small calls: a cluster a unit, which joins by itself, decode.cuh)
//   k_decode_finish join: a head's partials with the new token's own row,
//                     O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s;
//                   and, from the scores the split kernel left, sum_h 2^(t_h(p) - M_h) / Z_h
//                   added to the running sum of row p's attention weights.
#include <math.h>

#include "decode_far.cuh"
#include "tc.cuh"

namespace ddt {

namespace {
constexpr int kSimtThreads = 256;
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtMaxCtas = 512;
}  // namespace

// Up to 4 heads a kv head bound by HBM and the latency of a tile's steps: 16 requests of 4000 to 8000
// rows (105787 in all), 32 heads over 8 kv heads of 128 (867 MB of K and V), 166 us, 5.2 TB/s.  Above,
// bound by reads of shared memory: a lane has one row, so a piece of K is multiplied with 8 or 16
// pieces of q from there.  24 heads over 4 of 256 (867 MB) 233 us, 3.7 TB/s; 32 over 2 of 256 (433 MB)
// 216 us and 48 over 3 of 128 (325 MB) 170 us, 2.0 and 1.9 TB/s: half of the warps' waiting is for
// shared memory, its data pipe is 61 % busy, the FMA pipe 23 to 26 % (the arithmetic alone, 2.6 Gflop
// of the first and the last, would take 35 us).  Before the ring, with each row's copies behind its own
// page lookup, the first two took 265 and 305 us.  A block is 4, 8 or 16 heads, the smallest that holds
// the group: sums for more do not fit in the registers of two CTAs an SM (128 a thread; blocks of 8
// heads spill 120 to 144 bytes, of 16 196 to 288: 0.2 % of the instructions at most).
//
// Tiles of 32 KB of K and V (R rows), three on their way by cp.async; two barriers a tile.
//   scores   D / 16 lanes a row, 16 channels a lane, all heads; the sums over the lanes scatter
//            the heads over them, so a lane ends up with the scores (and the exponentials) of
//            its row for a few heads
//   values   a thread owns four channels and four consecutive rows of the tile
// As in the tensor-core kernel the exponents' reference moves only when a score is 2^8 above it.
template <int D, int HBS>
struct SimtCfg {
    static constexpr int R = 4096 / D;                       // rows a tile
    static constexpr int LPR = D / 16;                       // lanes a row
    static constexpr int kStages = D == 256 && HBS == 16 ? 2 : 3;
    static constexpr int NV = HBS > LPR ? HBS / LPR : 1;     // heads a lane ends up with
    static constexpr int kSets = kSimtThreads / (D / 4);     // row sets of the values
    static constexpr int kLeft = D == 64 ? kSets / 2 : kSets;  // of them through shared memory at a segment's end
    static constexpr int kQ = HBS * D > 1024 ? HBS * D : 1024;  // floats: the queries, then those sums
    static constexpr int kSumHeads = kQ / (kLeft * D) < HBS ? kQ / (kLeft * D) : HBS;  // heads at a time
    static constexpr int kSmem = kStages * 32768 + kQ * 4 + 2 * HBS * R * 4;
    static_assert(2 * (kSmem + 2048) <= 228 * 1024 && kSumHeads >= 1 && HBS % kSumHeads == 0, "shared memory");
};

template <int D, int HBS>
__global__ void __launch_bounds__(kSimtThreads, 2) k_decode_simt(const DecodeParams p) {
    using Cfg = SimtCfg<D, HBS>;
    constexpr int R = Cfg::R, LPR = Cfg::LPR, NV = Cfg::NV, kStages = Cfg::kStages;
    extern __shared__ __align__(16) float s_ring[];   // [kStages][K, V][R][D]
    float* s_q = s_ring + kStages * 8192;             // [HBS][D]
    float* s_p = s_q + Cfg::kQ;                       // [HBS][R] exponentials
    float* s_t = s_p + HBS * R;                       // [HBS][R] scores
    __shared__ float s_m[HBS], s_f[HBS], s_l[kSimtWarps][HBS];
    __shared__ long long s_row[4][R];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float* kp = static_cast<const float*>(p.k_pages);
    const float* vp = static_cast<const float*>(p.v_pages);
    const DecodeWalk mine = dec_plan<kSimtThreads>(p);
    DecodeWalk w = mine;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_decode_finish may be set up

    // ---- the copies, kStages - 1 tiles ahead of the sums, and one tile ahead of them the rows'
    //      places: the tile at row fy of segment f
    DecodeWalk f = w;
    auto seg_end = [&](const DecodeWalk& x) { return min(x.P, (x.t + dec_seg_tiles(x)) * kDecTile); };
    int fy = f.t * kDecTile, seg_f = 0, seg_w = 0;
    int bad_bits = 0;  // bit (segment & 31): this thread met a page that does not exist
    uint32_t there = 0;  // bit slot: it holds a tile's places
    auto places = [&](int slot) {
        there &= ~(1u << slot);
        if (f.left <= 0) return;
        there |= 1u << slot;
        const int end = seg_end(f), y = fy + tid;
        if (tid < R) {
            long long row = -1;  // not there: zeros
            if (y < end) {
                const int lp = y / p.page_rows, phys = p.block_table[(long long)f.b * p.max_pages + lp];
                if (phys >= 0 && phys < p.num_pages)
                    row = ((((long long)f.l * p.num_pages + phys) * p.Hkv + f.g / p.HB) * p.page_rows + (y - lp * p.page_rows)) * D;
                else
                    bad_bits |= 1 << (seg_f & 31);
            }
            s_row[slot][tid] = row;
        }
        fy += R;
        if (fy >= end) {
            dec_next(p, f);
            fy = f.t * kDecTile;
            ++seg_f;
        }
    };
    auto fetch = [&](int stage, int slot) {
        if (there >> slot & 1u) {
            const uint32_t dst = tc::smem_u32(s_ring + stage * 8192 + tid * 4);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = tid + q * kSimtThreads;
                const long long row = s_row[slot][e / (D / 4)];
                const uint32_t n = row >= 0 ? 16 : 0, to = dst + q * kSimtThreads * 16;
                const long long at = (row >= 0 ? row : 0) + (e % (D / 4)) * 4;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(kp + at), "r"(n) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + R * D * 4), "l"(vp + at), "r"(n) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) places(s);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(s, s);
    int stage = 0, slot = kStages - 1;  // the next tile's places

    const int r = tid / LPR, lr = tid % LPR;           // scores: this lane's row and place in it
    const int c4 = (tid % (D / 4)) * 4, set = tid / (D / 4);  // values: channels, rows 4 set ..
    int hb = 0;  // scores: first of the heads this lane ends up with
#pragma unroll
    for (int o = LPR / 2, nv = HBS; o > 0; o >>= 1)
        if (nv > 1) {
            nv >>= 1;
            if (lane & o) hb += nv;
        }
    // of lanes with the same heads (fewer heads than lanes) the first one counts
    const bool owner = HBS >= LPR || (lr % (LPR / (HBS < LPR ? HBS : LPR))) == 0;
    for (; w.left > 0; dec_next(p, w), ++seg_w) {
        const int g = w.g / p.HB, h0 = (w.g % p.HB) * HBS, nh = min(HBS, p.G - h0), end = seg_end(w);
        const float* q = static_cast<const float*>(p.q) + (((long long)w.l * p.B + w.b) * p.Hq + g * p.G + h0) * D;
        __syncthreads();  // the previous segment is done with shared memory
        for (int e = tid; e < HBS * D; e += kSimtThreads) s_q[e] = e < nh * D ? q[e] : 0.f;
        if (tid < HBS) s_m[tid] = kNoRef;
        float acc[HBS][4], l[NV];
#pragma unroll
        for (int h = 0; h < HBS; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][i] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) l[v] = 0.f;
        for (int y = w.t * kDecTile; y < end; y += R) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncthreads();  // everyone's copies have landed, and the tile before is done with
            fetch((stage + kStages - 1) % kStages, slot);
            slot = (slot + 1) & 3;
            places(slot);
            const float* K = s_ring + stage * 8192;
            const float* V = K + R * D;
            stage = (stage + 1) % kStages;
            // ---- scores
            float s[HBS];
#pragma unroll
            for (int h = 0; h < HBS; ++h) s[h] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // (head size 64: rows of the other parity take the pieces in another order, so
                // that the two rows of a quarter warp are in different banks)
                const int c = (lr + LPR * (D == 64 ? i ^ (r & 1) : i)) * 4;
                const float4 k = *reinterpret_cast<const float4*>(K + r * D + c);
#pragma unroll
                for (int h = 0; h < HBS; ++h) {
                    const float4 x = *reinterpret_cast<const float4*>(s_q + h * D + c);
                    s[h] = fmaf(k.x, x.x, fmaf(k.y, x.y, fmaf(k.z, x.z, fmaf(k.w, x.w, s[h]))));
                }
            }
#pragma unroll
            for (int o = LPR / 2, nv = HBS; o > 0; o >>= 1) {
                if (nv > 1) {
                    nv >>= 1;
#pragma unroll
                    for (int v = 0; v < HBS / 2; ++v)
                        if (v < nv) {
                            const float send = (lane & o) ? s[v] : s[v + nv], keep = (lane & o) ? s[v + nv] : s[v];
                            s[v] = keep + __shfl_xor_sync(kFull, send, o);
                        }
                } else {
                    s[0] += __shfl_xor_sync(kFull, s[0], o);
                }
            }
            bool above = false;
            float e[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float m = s_m[hb + v];
                s[v] = y + r < end ? s[v] * p.scale_log2 : -INFINITY;
                above |= s[v] > m + 8.f;
                e[v] = tc::ex2(s[v] - m);
                if (owner) {
                    s_p[(hb + v) * R + r] = e[v];
                    if (p.score) s_t[(hb + v) * R + r] = s[v];
                }
            }
            if (__syncthreads_or(above)) {
                // the segment's first tile, or a growing maximum: new references
                if (owner)
#pragma unroll
                    for (int v = 0; v < NV; ++v) s_t[(hb + v) * R + r] = s[v];
                __syncthreads();
                for (int h = warp; h < HBS; h += kSimtWarps) {
                    float m = -INFINITY;
                    for (int x = lane; x < R; x += 32) m = fmaxf(m, s_t[h * R + x]);
                    m = warp_max(m);
                    const float old = s_m[h];
                    __syncwarp();
                    if (lane == 0) {
                        s_f[h] = m > old + 8.f ? tc::ex2(old - m) : 1.f;
                        if (m > old + 8.f) s_m[h] = m;
                    }
                }
                __syncthreads();
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    e[v] = tc::ex2(s[v] - s_m[hb + v]);
                    l[v] *= s_f[hb + v];
                    if (owner) s_p[(hb + v) * R + r] = e[v];
                }
#pragma unroll
                for (int h = 0; h < HBS; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[h][i] *= s_f[h];
                __syncthreads();
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) l[v] += e[v];
            if (p.score) {
                float* sc = p.score + (((long long)w.l * p.B + w.b) * p.Hq + g * p.G + h0) * p.cap + y;
                const int n = min(R, end - y);
                for (int x = tid; x < nh * R; x += kSimtThreads)
                    if (x % R < n) sc[(long long)(x / R) * p.cap + x % R] = s_t[x];
            }
            // ---- values
            float4 v4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v4[i] = *reinterpret_cast<const float4*>(V + (set * 4 + i) * D + c4);
#pragma unroll
            for (int h = 0; h < HBS; ++h) {
                const float4 x = *reinterpret_cast<const float4*>(s_p + h * R + set * 4);
                acc[h][0] = fmaf(x.x, v4[0].x, fmaf(x.y, v4[1].x, fmaf(x.z, v4[2].x, fmaf(x.w, v4[3].x, acc[h][0]))));
                acc[h][1] = fmaf(x.x, v4[0].y, fmaf(x.y, v4[1].y, fmaf(x.z, v4[2].y, fmaf(x.w, v4[3].y, acc[h][1]))));
                acc[h][2] = fmaf(x.x, v4[0].z, fmaf(x.y, v4[1].z, fmaf(x.z, v4[2].z, fmaf(x.w, v4[3].z, acc[h][2]))));
                acc[h][3] = fmaf(x.x, v4[0].w, fmaf(x.y, v4[1].w, fmaf(x.z, v4[2].w, fmaf(x.w, v4[3].w, acc[h][3]))));
            }
        }
        // ---- the segment's partial: sums of the exponentials over the rows of a warp, then of
        //      the warps; the row sets' O a few heads at a time, a warp's own two sets (head
        //      size 64) by a shuffle
        const long long slot = dec_slot(p, w);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) l[v] += __shfl_xor_sync(kFull, l[v], o);
            if (lane < LPR && owner) s_l[warp][hb + v] = l[v];
        }
        const int bad = __syncthreads_or(bad_bits >> (seg_w & 31) & 1);
        bad_bits &= ~(1 << (seg_w & 31));
#pragma unroll
        for (int h4 = 0; h4 < HBS; h4 += Cfg::kSumHeads) {
            if (h4) __syncthreads();
            const int to = D == 64 ? warp : set;
#pragma unroll
            for (int h = 0; h < Cfg::kSumHeads; ++h) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = acc[h4 + h][i];
                    if (D == 64) x[i] += __shfl_xor_sync(kFull, x[i], 16);
                }
                if (D != 64 || lane < 16)
                    *reinterpret_cast<float4*>(s_q + (to * Cfg::kSumHeads + h) * D + c4) = make_float4(x[0], x[1], x[2], x[3]);
            }
            __syncthreads();
            for (int x = tid; x < Cfg::kSumHeads * D; x += kSimtThreads) {
                float o = 0.f;
#pragma unroll
                for (int s = 0; s < Cfg::kLeft; ++s) o += s_q[s * Cfg::kSumHeads * D + x];
                if (h4 + x / D < nh) p.part_o[(slot * p.HT + h4) * D + x] = o;
            }
        }
        if (tid < nh) {
            float z = 0.f;
#pragma unroll
            for (int x = 0; x < kSimtWarps; ++x) z += s_l[x][tid];
            p.part_ml[slot * p.HT + tid] = make_float2(s_m[tid], bad ? kSegBadPage : z);
        }
    }
    if (p.cl) {
        DecNew<float, D> mine_new;
        mine_new.load(p, (long long)mine.l * p.B + mine.b, mine.g, dec_first_head(p), lane);
        if (p.cl > 1) tc::cluster_sync();
        else __syncthreads();
        dec_finish<float, D, kSimtThreads>(p, mine, mine_new, s_q);
    }
}

// A head's output from its joined softmax, by WPH warps (8: all of a block; s_x [8][D]).
template <typename Tin, typename Tout, int D, int WPH>
__device__ __forceinline__ void write_head(const DecodeParams& p, int lb, int hq, const DecNew<Tin, D>& x, const HeadJoin& j, float* s_x) {
    constexpr int E = D / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Tout* out = static_cast<Tout*>(p.o) + ((long long)lb * p.Hq + hq) * D;
    if (j.err) {
        if (WPH == 1 || warp == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) out[e * 32 + lane] = from_f32<Tout>(0.f);
            if (lane == 0) p.status[lb % p.B] = j.err;
        }
        return;  // (WPH 8: all warps)
    }
    const int h = (hq % p.G) % p.hbs;
    const float w = WPH == 1 || warp == 0 ? tc::ex2(x.tn - j.ref) : 0.f;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = w * x.v[e];
    const float2* ml = p.part_ml + j.first * p.HT + h;
    const float* po = p.part_o + (j.first * p.HT + h) * D;
#pragma unroll 4
    for (int s = WPH == 1 ? 0 : warp; s < j.ns; s += WPH) {
        const float f = tc::ex2(ml[(long long)s * p.HT].x - j.ref);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(f, po[(long long)s * p.HT * D + e * 32 + lane], acc[e]);
    }
    const float inv = j.z > 0.f ? 1.f / j.z : j.z;  // no rows at all: 0; NaN stays
    if (WPH == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) out[e * 32 + lane] = from_f32<Tout>(acc[e] * inv);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) s_x[warp * D + e * 32 + lane] = acc[e];
        __syncthreads();
        if (tid < D) {
            float o = s_x[tid];
#pragma unroll
            for (int w = 1; w < 8; ++w) o += s_x[w * D + tid];
            out[tid] = from_f32<Tout>(o * inv);
        }
    }
}

// The same of a head whose segments have far blocks, which join their partials first.  (A function of its own, called last: the
// kernel's ordinary way has no registers to spare.)
template <typename Tin, typename Tout, int D, int WPH>
__device__ __noinline__ void far_join(const DecodeParams& p, int lb, int hq, float* s_x) {
    const int l = lb / p.B, b = lb - l * p.B, g = hq / p.G, hb = hq % p.G / p.hbs, nt = dec_tiles(p.prefix_len[b], p.cap), HH = p.Hkv * p.HB;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const HeadJoin j = head_join(p, lb, hq, 0.f, lane);  // (for its segments)
    // the head's tiles on the line
    const long long all = p.pre[p.B], T = all * HH * p.L, from = l * all * HH + p.pre[b] * HH + (long long)(g * p.HB + hb) * nt;
    const int C = (int)min((long long)p.C, T);
    for (int s = WPH == 1 ? 0 : warp; s < j.ns; s += WPH) {
        const int c = j.c0 + s;
        if (p.far[c])
            far_rows<Tin, D>(p, lb, g, hq % p.G, (int)(max(dec_first(T, C, c), from) - from), (int)(min(dec_first(T, C, c + 1), from + nt) - from),
                             j.first + s, hq % p.G % p.hbs, lane);
    }
    DecNew<Tin, D> mine;
    mine.load(p, lb, g, hq % p.G, lane);
    if (WPH == 1) __syncwarp();
    else __syncthreads();  // (all warps are of this head)
    write_head<Tin, Tout, D, WPH>(p, lb, hq, mine, head_join(p, lb, hq, mine.tn, lane), s_x);
}

// Blocks below n_join: WPH warps a head, O of the head.  The others: the weight sums of some rows
// of one (layer, request, kv head); with them the kernel is bound by HBM (4 bytes a head and row,
// written by the split and read here: about 20 us of 415 for 500000 rows of 24 heads), else by
// the latency of the join.
// QUANT: of a cache in 8 bits, without weight sums; the far blocks' rows join their segments' partials first, where there are any.
template <typename Tin, typename Tout, int D, int WPH, bool QUANT>
__global__ void __launch_bounds__(256, QUANT ? 3 : 4) k_decode_finish(const __grid_constant__ DecodeParams p, unsigned n_join, int chunks) {
    extern __shared__ float s_x[];  // [8][D] sums of the warps of a head, or 3 floats a head of a group
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    DecNew<Tin, D> mine;
    // launched ahead: the partials are there from here on (the call's inputs were before)
    auto partials = [&]() { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (blockIdx.x < n_join) {
        const unsigned x = WPH == 1 ? blockIdx.x * 8 + warp : blockIdx.x;
        const int lb = (int)(x / p.Hq), hq = (int)(x - (unsigned)lb * p.Hq);
        if (lb < p.L * p.B) mine.load(p, lb, hq / p.G, hq % p.G, lane);
        partials();
        if (lb >= p.L * p.B) return;  // (WPH 1: whole warps, no barrier follows)
        const HeadJoin j = head_join<QUANT>(p, lb, hq, mine.tn, lane);
        if (QUANT && j.far) return far_join<Tin, Tout, D, WPH>(p, lb, hq, s_x);
        write_head<Tin, Tout, D, WPH>(p, lb, hq, mine, j, s_x);
        return;
    }
    if (QUANT) return;
    const unsigned y = blockIdx.x - n_join;
    const int lbg = (int)(y / chunks), part = (int)(y - (unsigned)lbg * chunks), lb = lbg / p.Hkv, g = lbg - lb * p.Hkv;
    float* s_ref = s_x;
    float* s_inv = s_ref + p.G;
    float* s_tn = s_inv + p.G;
    mine.load(p, lb, g, warp, lane);
    const int P = p.prefix_len[lb % p.B];
    partials();
    // blocks behind the unit's rows (the first also has the new token's)
    if (part && part * 1024LL >= P) return;
    int bad = 0;
    for (int h = warp; h < p.G; h += 8) {
        if (h >= 8) mine.load(p, lb, g, h, lane);
        const HeadJoin j = head_join(p, lb, g * p.G + h, mine.tn, lane);
        bad |= j.err;
        if (lane == 0) {
            s_ref[h] = j.ref;
            s_inv[h] = j.z > 0.f ? 1.f / j.z : j.z;  // (NaN stays)
            s_tn[h] = mine.tn;
        }
    }
    if (__syncthreads_or(bad)) return;
    const float* sc = p.score + ((long long)lb * p.Hq + g * p.G) * p.cap;
    float* wt = p.weight + (long long)lbg * p.cap;
    for (int r = (part * 256 + tid) * 4; r < P; r += chunks * 1024) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int h0 = 0; h0 < p.G; h0 += 4) {  // four heads' scores are in flight
            float4 t[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)  // the rows are padded to whole pages: r + 3 < cap
                if (h0 + h < p.G) t[h] = *reinterpret_cast<const float4*>(sc + (long long)(h0 + h) * p.cap + r);
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (h0 + h < p.G) {
                    const float ref = s_ref[h0 + h], inv = s_inv[h0 + h];
                    sum.x = fmaf(tc::ex2(t[h].x - ref), inv, sum.x);
                    sum.y = fmaf(tc::ex2(t[h].y - ref), inv, sum.y);
                    sum.z = fmaf(tc::ex2(t[h].z - ref), inv, sum.z);
                    sum.w = fmaf(tc::ex2(t[h].w - ref), inv, sum.w);
                }
        }
        if (r + 3 < P) {
            float4 w = *reinterpret_cast<float4*>(wt + r);
            *reinterpret_cast<float4*>(wt + r) = make_float4(w.x + sum.x, w.y + sum.y, w.z + sum.z, w.w + sum.w);
        } else {  // entries past the prefix stay as they are
            wt[r] += sum.x;
            if (r + 1 < P) wt[r + 1] += sum.y;
            if (r + 2 < P) wt[r + 2] += sum.z;
        }
    }
    if (p.k_new && P < p.cap && part == 0 && tid == 0) {  // the new token's own row
        float sum = 0.f;
        for (int h = 0; h < p.G; ++h) sum = fmaf(tc::ex2(s_tn[h] - s_ref[h]), s_inv[h], sum);
        wt[P] += sum;
    }
}

// ------------------------------------------------------------------------------ host
constexpr int kTcMaxCtas = 512;  // two an SM, for up to 256 SMs
constexpr int kQuantMaxCtas = 640;  // four an SM, for up to 160 SMs
static int simt_heads(int G) { return G <= 4 ? 4 : (G <= 8 ? 8 : 16); }

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// fills the workspace pointers; returns the bytes
static size_t decode_layout(DecodeParams& p, int hbs, int ctas, bool weight, unsigned char* ws, bool far = false) {
    p.hbs = hbs;
    p.HB = (p.G + hbs - 1) / hbs;
    p.HT = p.G < hbs ? p.G : hbs;
    const size_t units = (size_t)p.L * p.B * p.Hkv, slots = units * p.HB + ctas;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* r = ws + at;
        at += al256(bytes);
        return r;
    };
    p.pre = reinterpret_cast<long long*>(take(((size_t)p.B + 1) * sizeof(long long)));
    p.part_ml = reinterpret_cast<float2*>(take(slots * p.HT * sizeof(float2)));
    p.part_o = reinterpret_cast<float*>(take(slots * p.HT * p.d * sizeof(float)));
    p.score = weight ? reinterpret_cast<float*>(take(units * p.cap * p.G * sizeof(float))) : nullptr;
    p.far = far ? reinterpret_cast<int*>(take(ctas * sizeof(int))) : nullptr;
    return at;
}

size_t decode_ws_bytes(int L, int B, int Hq, int Hkv, int d, int cap, ddt_dtype in, bool weight) {
    DecodeParams p{};
    p.L = L;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.d = d;
    p.cap = cap;
    return decode_tc_supported(d, in) ? decode_layout(p, decode_tc_heads(p.G, d), kTcMaxCtas, weight, nullptr)
                                      : decode_layout(p, simt_heads(p.G), kSimtMaxCtas, weight, nullptr);
}

// p.C (SMs on entry) and p.cl of a split kernel with `ctas` CTAs an SM.  A cluster a unit saves the second kernel (2.7
// us), but a CTA of it takes nt / cl tiles of a full table where an even split over all CTAs takes
// units nt / C (one at least), and a tile takes about 1.2 us at head size 128 and 1.6 at 256 (fp32
// 4.7 and 12): a call is small if the excess, times the head size, is within 384 (fp32 96).
// Replayed from a graph, as clusters and as two kernels: one request, 32 heads over 8 of 128, 1000
// rows 7.5 and 10.0 us, 4000 rows 10.7 and 11.1, 6000 rows (4.8 tiles of excess) 13.1 and 12.8; four
// requests of 4000 rows (0.6) 12.2 and 16.2; 24 heads over 4 of 256, one request of 4000 rows (3)
// 13.4 and 12.0; fp32, 32 over 8 of 128, one request of 2000 rows (1) 15.1 and 13.7, four (0.3) 20.3
// and 25.8.  Clusters of 8 stay below the number of CTAs that the GPU's clusters of SMs have room for:
// 16 of them with a CTA an SM do not run at once (16 units of 256, 1000 rows: 15.1 and 12.1 us).
// Requests may be shorter than the table, and of different lengths: the even split follows them, so
// the tiles of a CTA are bounded too (512 channels' worth, fp32 256).  With lengths spread from an
// eighth of the table's rows to all of them, 16 requests of up to 1000 rows, 32 heads over 8 of 128,
// take 12.5 and 15.1 us; one of 160 shapes is slower as clusters (fp32, 16 units of 256, 1000 rows:
// 26.7 and 22.2 us).
// A tile of an 8-bit cache is half of bf16's bytes, and the second kernel as long: 1024 and 896.  24 heads over 4 of 256, 4
// requests of 4000 rows 13.0 and 15.9 us, 16 of 2000 14.8 and 19.5; 32 over 8 of 128, one request of 8000 rows (6.3 tiles of
// excess) 11.5 and 13.0, four 13.2 and 17.9, 16 of 2000 14.1 and 17.2; with lengths from an eighth of those on the gains are
// larger; 24 over 4 of 256, one request of 8000 rows (7 tiles of excess) 17.0 and 14.4.
void decode_clusters(DecodeParams& p, DecodeSmall small, int ctas) {
    p.C *= ctas;
    const long units = (long)p.L * p.B * p.Hkv;
    const int nt = (p.cap + kDecTile - 1) / kDecTile;
    int cl = 1;
    while (cl < 8 && units * 2 * cl <= (cl < 4 ? p.C : p.C - p.C / (ctas == 1 ? 4 : 8)) && cl < nt) cl *= 2;
    const double tiles = (nt + cl - 1) / cl, even = (double)units * nt / p.C;
    p.cl = p.HB == 1 && units * cl <= p.C && tiles * p.d <= small.most && (tiles - (even > 1. ? even : 1.)) * p.d <= small.excess ? cl : 0;
}

cudaLaunchConfig_t decode_grid(const DecodeParams& p, int threads, int smem, cudaLaunchAttribute& at, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(counted(p.cl ? (unsigned)(p.L * p.B * p.Hkv * p.cl) : (unsigned)p.C));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    at = cudaLaunchAttribute{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.cl ? p.cl : 1;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cfg;
}

template <int D, int HBS>
static cudaError_t simt_go(DecodeParams& p, cudaStream_t st) {
    constexpr int smem = SimtCfg<D, HBS>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(k_decode_simt<D, HBS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    decode_clusters(p, DecodeSmall{256., 96.}, 2);
    cudaLaunchConfig_t cfg = decode_grid(p, kSimtThreads, smem, at, st);
    return cudaLaunchKernelEx(&cfg, k_decode_simt<D, HBS>, p);
}
template <int D>
static cudaError_t simt_heads_go(DecodeParams& p, cudaStream_t st) {
    return p.hbs == 4 ? simt_go<D, 4>(p, st) : (p.hbs == 8 ? simt_go<D, 8>(p, st) : simt_go<D, 16>(p, st));
}
static cudaError_t simt_d_go(DecodeParams& p, cudaStream_t st) {
    return p.d == 64 ? simt_heads_go<64>(p, st) : (p.d == 128 ? simt_heads_go<128>(p, st) : simt_heads_go<256>(p, st));
}

template <typename Tin, typename Tout, int D, int WPH, bool QUANT>
static cudaError_t finish_launch(const DecodeParams& p, int sms, cudaStream_t st) {
    const size_t heads = (size_t)p.L * p.B * p.Hq;
    const unsigned n_join = (unsigned)(WPH == 1 ? (heads + 7) / 8 : heads), units = (unsigned)p.L * p.B * p.Hkv;
    // 2048 rows a block, so that long requests get more of them (131071 rows: the call takes 103 us,
    // 109 with 8192); not too many for units that may be short
    const unsigned most = (p.cap + 2047) / 2048, room = 24u * sms / units + 1;
    const int chunks = (int)(most < room ? most : room);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(counted(n_join + (p.weight ? units * chunks : 0)));
    cfg.blockDim = dim3(256);
    const size_t join_smem = WPH == 1 ? 0 : 8 * D * sizeof(float), weight_smem = p.weight ? 3 * p.G * sizeof(float) : 0;
    cfg.dynamicSmemBytes = join_smem > weight_smem ? join_smem : weight_smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};  // may be set up while the split kernel ends
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_decode_finish<Tin, Tout, D, WPH, QUANT>, p, n_join, chunks);
}
template <typename Tin, typename Tout, bool QUANT>
static cudaError_t finish_go(const DecodeParams& p, int sms, cudaStream_t st) {
    // Eight warps a head where it has a dozen segments (C / units) or more: whole calls with 8 and
    // with 1, one request of 131071 rows, 8 heads over one of 128 (304 segments) 21.2 and 44.1 us, 32
    // over 8 (39) 85.0 and 88.6; but 2 x 96 short requests of 16 heads (1 or 2) 182 and 166.
    const bool many = p.C >= 12L * p.L * p.B * p.Hkv * p.HB;
    switch (p.d) {
        case 64: return many ? finish_launch<Tin, Tout, 64, 8, QUANT>(p, sms, st) : finish_launch<Tin, Tout, 64, 1, QUANT>(p, sms, st);
        case 128: return many ? finish_launch<Tin, Tout, 128, 8, QUANT>(p, sms, st) : finish_launch<Tin, Tout, 128, 1, QUANT>(p, sms, st);
    }
    return many ? finish_launch<Tin, Tout, 256, 8, QUANT>(p, sms, st) : finish_launch<Tin, Tout, 256, 1, QUANT>(p, sms, st);
}

template <bool QUANT>
static cudaError_t finish_any(const DecodeParams& p, ddt_dtype in, int sms, cudaStream_t st) {
    if (in == DDT_BF16)
        return p.out == DDT_BF16 ? finish_go<__nv_bfloat16, __nv_bfloat16, QUANT>(p, sms, st)
                                 : finish_go<__nv_bfloat16, float, QUANT>(p, sms, st);
    return p.out == DDT_BF16 ? finish_go<float, __nv_bfloat16, QUANT>(p, sms, st) : finish_go<float, float, QUANT>(p, sms, st);
}

static DecodeParams decode_params(int L, int B, int Hq, int Hkv, int d, const AttnPaging& pg, ddt_dtype out, const void* q,
                                  const void* k_new, const void* v_new, const void* k_pages, const void* v_pages,
                                  const int32_t* prefix_len, float scale, void* o, float* weight, int32_t* status) {
    DecodeParams p{};
    p.L = L;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.d = d;
    p.page_rows = pg.page_rows;
    p.num_pages = pg.num_pages;
    p.max_pages = pg.max_pages;
    p.cap = pg.page_rows * pg.max_pages;
    p.block_table = pg.block_table;
    p.prefix_len = prefix_len;
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.o = o;
    p.weight = weight;
    p.status = status;
    p.out = out;
    p.scale_log2 = scale * 1.4426950408889634f;
    return p;
}

static int sm_count() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

cudaError_t launch_decode(int L, int B, int Hq, int Hkv, int d, const AttnPaging& pg, ddt_dtype in, ddt_dtype out,
                          const void* q, const void* k_new, const void* v_new, const void* k_pages,
                          const void* v_pages, const int32_t* prefix_len, float scale, void* o, float* weight,
                          int32_t* status, void* ws, cudaStream_t st) {
    DecodeParams p = decode_params(L, B, Hq, Hkv, d, pg, out, q, k_new, v_new, k_pages, v_pages, prefix_len, scale, o, weight, status);
    const int sms = sm_count();
    unsigned char* w = static_cast<unsigned char*>(ws);
    cudaError_t e;
    if (decode_tc_supported(d, in)) {  // bf16: persistent CTAs
        p.C = sms < kTcMaxCtas / 2 ? sms : kTcMaxCtas / 2;
        decode_layout(p, decode_tc_heads(p.G, d), kTcMaxCtas, weight != nullptr, w);
        e = launch_decode_tc(p, st);
    } else {
        p.C = sms < kSimtMaxCtas / 2 ? sms : kSimtMaxCtas / 2;
        decode_layout(p, simt_heads(p.G), kSimtMaxCtas, weight != nullptr, w);
        e = simt_d_go(p, st);
    }
    return e != cudaSuccess || p.cl ? e : finish_any<false>(p, in, sms, st);
}

// ---- the same over a cache held in 8 bits: the split kernel is another, the join the same
size_t decode_quant_ws_bytes(int L, int B, int Hq, int Hkv, int d, ddt_dtype in) {
    DecodeParams p{};
    p.L = L;
    p.B = B;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.d = d;
    return decode_layout(p, decode_quant_heads(p.G, in), kQuantMaxCtas, false, nullptr, true);
}

cudaError_t launch_decode_quant(int L, int B, int Hq, int Hkv, int d, int block, const AttnPaging& pg, ddt_dtype in,
                                ddt_dtype out, const void* q, const void* k_new, const void* v_new, const void* k_pages,
                                const void* v_pages, const uint8_t* k_scale, const uint8_t* v_scale,
                                const int32_t* prefix_len, float scale, void* o, int32_t* status, void* ws, cudaStream_t st) {
    DecodeParams p = decode_params(L, B, Hq, Hkv, d, pg, out, q, k_new, v_new, k_pages, v_pages, prefix_len, scale, o, nullptr, status);
    const int sms = sm_count();
    p.C = sms < kQuantMaxCtas / 4 ? sms : kQuantMaxCtas / 4;
    decode_layout(p, decode_quant_heads(p.G, in), kQuantMaxCtas, false, static_cast<unsigned char*>(ws), true);
    p.ks = k_scale;
    p.vs = v_scale;
    p.block = block;
    const cudaError_t e = launch_decode_quant_tiles(p, in, st);
    return e != cudaSuccess || p.cl ? e : finish_any<true>(p, in, sms, st);
}

}  // namespace ddt
