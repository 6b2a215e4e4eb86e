// decode_quant.cuh -- k_decode_quant: ddt_decode_attn_paged_quant's pass over the cached rows, a
// cache of e4m3 codes with a power of two for each block of rows and head.
//
// As for bf16 caches (decode_tc.cu) the cache is the M = 128 operand of the products and the few
// heads are N, so no thread touches a cached element; here the codes go to the tensor cores as
// they lie in HBM, one byte an element (kind::f8f6f4, 32 channels or rows an MMA):
//   S^T [128 rows x heads]  = K codes [rows x d] . Q^T        (K-major)
//   O^T [d x heads]        += V codes^T [d x rows] . P^T      (V and P as they lie, M- and N-major)
// The other operand of such an MMA is e4m3 as well, 4 significant bits, so Q and P are sums of
// parts in N columns of their own, each part the rounding error of those before it times 16:
//   x = x_0 + x_1 / 16 + x_2 / 256 + ..,  x_i = e4m3(16 (x_{i-1} residue)).
// A part takes 4 bits at least, and what lies below e4m3's normal range is made up for by the next:
// bf16 queries (scaled by a power of two to at most 256) are whole in 2 parts, the weights get 4
// (2^-16, as with bf16 caches); fp32 calls take 6 of each (2^-24).  With up to 8 heads the parts of
// Q fill the MMA's smallest N, 16.
//
// The scales.  A block's power of two 2^a of K multiplies its rows' scores.  That of V, 2^v, goes
// into the weights: t' = t + v (base 2), P = 2^(t' - m) with one reference m a head for all t', so
// that P is at most 2^8; the softmax sum gets 2^-v P = 2^(t - m).  v counts from the segment's unit
// (v_unit_of).  The parts hold P to 2^-26 of the largest, and so a weight to 2^-26 2^(difference of
// the v) of the largest weight: only blocks with |v| <= kNear go this way.  The rows of the others, far
// blocks, have no weight here; they join the partials afterwards (far_rows), where a call has any.
//
//   warp 0      producer: block-table entries, TMA of K and V tiles into one ring
//   warp 1      MMA issuer: Q K^T of tile j + 1 ahead of P V of tile j
//   warp 2      queries: the parts of a segment's heads (for 16 heads or more and one CTA an SM three more warps, the last)
//   warp 3      scales: the bytes of a tile's blocks, two tiles ahead of the softmax
//   warps 4-7, 8-11 ..  softmax, eight heads a warpgroup, a thread a cached row
// The split of the rows over the CTAs, the partials and the join are those of decode.cuh.
// Every wait is bounded, as there.
//
// Bound by HBM for groups of up to 8 heads (heads of 128 and 256: 16): 32 requests of 1K to 32K rows, 24 heads over 4 of 256
// (901 MB), 138 us, 6.5 TB/s; one of 131071 rows, 32 over 8 of 128 (269 MB), 46 us; 2 x 96 of up to 2500 rows, 16 over 16 of
// 64 (453 MB), 83 us.  A tile is half as many bytes as in bf16 and its softmax as long, so two to four CTAs share an SM (heads
// of 64, one head a kv head: 98 us with three, 93 with four), and instances for groups of up to 2 and 4 heads leave out what
// the others would compute for nobody (139 -> 98).  Larger groups are bound by the softmax's instructions, 323 a warp for a
// tile and eight heads: 16 heads of 64 read 4.3 TB/s.  Pairs of heads go through packed fp32 instructions, weights four a word.
#pragma once

#include <cuda.h>
#include <math.h>

#include "decode_far.cuh"
#include "quant.cuh"
#include "tc.cuh"

namespace ddt {

constexpr float kLift = 4.f;  // a reference is this far below the score that set it: P = 2^kLift there
constexpr float kTau = 4.f;   // and moves when a score is this much above it

constexpr int pow2_at_least(int x, int y) { return x <= y ? y : pow2_at_least(x, 2 * y); }

// HP: heads a block; GH: of the eight of a warpgroup, those that there are; QP, PP: parts of Q and of P
template <int D, int HP, int GH, int QP, int PP>
struct QuantCfg {
    static constexpr int kGroups = HP / 8;                // softmax warpgroups
    static constexpr int kRow = D < 128 ? D : 128;        // bytes of a swizzled row
    static constexpr int kBlocks = D / kRow;              // of a cached row
    static constexpr int kStageBytes = kDecTile * D;      // a K or V tile
    static constexpr int NQ = QP * HP;                    // N of Q K^T
    static constexpr int NP = pow2_at_least(PP * HP, 32); // N of P V, and the bytes of a row of P
    static constexpr int kCtas = QP == 6 ? (HP == 8 && D < 256 ? 2 : 1) : HP == 8 ? (D == 64 ? (GH < 8 ? 4 : 3) : 2) : (HP == 16 && D < 256 ? 2 : 1);  // an SM
    // warps of queries, those but the first behind the softmax.  One takes 4 us for 16 heads of 256, and longer than the tiles
    // of a short segment (96 requests of up to 493 rows, 64 heads over 4: 40 us with one, 29 with four; 64 over 2: 38 and 26).
    // Where a second CTA shares the SM, more of them would take registers from the softmax (16 heads of 64: 141 us, 151).
    static constexpr int kQWarps = kCtas == 1 && HP > 8 ? 4 : 1;
    static constexpr int kThreads = 128 + 128 * kGroups + 32 * (kQWarps - 1);
    static constexpr int kQBufs = kCtas == 2 && D == 256 ? 1 : 2;
    static constexpr int kQBytes = NQ * D;
    static constexpr int kPBytes = NP * kDecTile;
    static constexpr int kMB = D > 128 ? D / 128 : 1;     // M blocks of P V
    static constexpr int kOCol = 2 * NQ;                  // tensor memory: S x 2, O
    static constexpr int kTmemCols = pow2_at_least(2 * NQ + kMB * NP, 32);
    static constexpr int kFixed = 1024 + kQBufs * kQBytes + 2 * kPBytes + 1408 + (8 + 4 * 2 + 4) * HP * 4;
    static constexpr int kRing = (228 * 1024 / kCtas - 1024 - 256 - kFixed) / kStageBytes;
    static constexpr int kStages = kRing > 12 ? 12 : kRing;
    static constexpr int kSmem = kFixed + kStages * kStageBytes;
    static_assert(kStages >= 3 && kSmem <= 227 * 1024, "shared memory");
    static_assert(kCtas * kTmemCols <= 512, "tensor memory");
    static_assert((2 * kStages + 15) * 8 + 40 + 15 + 4 * 256 <= 1408, "barriers and scales");
    // bad_tile and q_unit are kept for 8 tiles (segments): the producer is up to 6 tiles ahead of the products, they two of
    // the softmax
    static_assert(kStages <= 12, "rings of 8");
    static_assert(NQ % 16 == 0 && NQ <= 256 && NP <= 128, "N of the products");
    // head size 64: lanes 64-127 of O read on behind a tile, into Q and P at the end of the ring
    static_assert(D != 64 || kQBufs * kQBytes + 2 * kPBytes >= kStageBytes, "shared memory behind the ring");
};

struct DecQuantArgs {
    int sub;  // rows of a box: the largest of 128, 64, ... that pages are made of
};

// x[0..3] as PARTS codes each, a word a part.  Up to four parts: what the first one leaves is rounded to fp16, 11 bits
// of at most 2^-4 x (2^-16 of x), which three more parts hold; more: fp32 throughout.
template <int PARTS>
__device__ __forceinline__ void split4(const float (&x)[4], uint32_t (&c)[PARTS]) {
    F2 u = f2(x[0], x[1]), v = f2(x[2], x[3]);
    c[0] = e4m3x4(x[0], x[1], x[2], x[3]);
    __half2 p, q;
    e4m3x4_values(c[0], p, q);
    if constexpr (PARTS <= 4) {
        const float2 fp = __half22float2(p), fq = __half22float2(q);
        const float2 ru = f2_get(u - f2(fp.x, fp.y)), rv = f2_get(v - f2(fq.x, fq.y));
        const __half2 k16 = __float2half2_rn(16.f);
        __half2 hu = __hmul2(__floats2half2_rn(ru.x, ru.y), k16), hv = __hmul2(__floats2half2_rn(rv.x, rv.y), k16);
#pragma unroll
        for (int i = 1; i < PARTS; ++i) {
            c[i] = e4m3x4(hu, hv);
            if (i + 1 < PARTS) {
                e4m3x4_values(c[i], p, q);
                hu = __hmul2(__hsub2(hu, p), k16);
                hv = __hmul2(__hsub2(hv, q), k16);
            }
        }
    } else {
        const F2 k16 = f2(16.f, 16.f);
#pragma unroll
        for (int i = 1; i < PARTS; ++i) {
            const float2 fp = __half22float2(p), fq = __half22float2(q);
            u = (u - f2(fp.x, fp.y)) * k16;
            v = (v - f2(fq.x, fq.y)) * k16;
            const float2 a = f2_get(u), b = f2_get(v);
            c[i] = e4m3x4(a.x, a.y, b.x, b.y);
            if (i + 1 < PARTS) e4m3x4_values(c[i], p, q);
        }
    }
}

// The end of a CTA of a cluster that has far blocks: its only segment's partials with them, then the join.
template <typename Tin, int D, int THREADS>
__device__ __forceinline__ void far_tail(const DecodeParams& p, const DecodeWalk& w, float* s_x) {
    const int lb = w.l * p.B + w.b, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int h = warp; h < p.G; h += THREADS / 32) far_rows<Tin, D>(p, lb, w.g, h, w.t, w.t + (int)w.left, blockIdx.x, h, lane);
    DecNew<Tin, D> mine_new;
    mine_new.load(p, lb, w.g, dec_first_head(p), lane);
    __syncthreads();
    if (p.cl > 1) tc::cluster_sync();
    dec_finish<Tin, D, THREADS>(p, w, mine_new, s_x);
}

// CLUSTER: a unit a cluster, which joins its partials itself; else k_decode_finish does.  (Two instances: registers are short,
// and what the one does behind its roles costs the other's roles up to 15 % of a call.)
template <typename Tin, int D, int HP, int GH, int QP, int PP, bool CLUSTER>
__global__ void __launch_bounds__(QuantCfg<D, HP, GH, QP, PP>::kThreads, QuantCfg<D, HP, GH, QP, PP>::kCtas)
    k_decode_quant(const DecodeParams p, const DecQuantArgs a, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
    using Cfg = QuantCfg<D, HP, GH, QP, PP>;
    constexpr int kStages = Cfg::kStages, NQ = Cfg::NQ, NP = Cfg::NP, kMB = Cfg::kMB, kRow = Cfg::kRow, kQBufs = Cfg::kQBufs;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sQ = ring + kStages * Cfg::kStageBytes;  // [kQBufs]
    unsigned char* sP = sQ + kQBufs * Cfg::kQBytes;         // [2]
    uint64_t* full = reinterpret_cast<uint64_t*>(sP + 2 * Cfg::kPBytes);  // [kStages] a tile landed
    uint64_t* empty = full + kStages;                                      // [kStages] its MMAs are done
    uint64_t* q_full = empty + kStages;  // [2] a segment's queries are there
    uint64_t* q_free = q_full + 2;       // [2] its last Q K^T is done
    uint64_t* s_full = q_free + 2;       // [2] S of a tile in tensor memory
    uint64_t* p_full = s_full + 2;       // [2] P of a tile in shared memory (the softmax warps)
    uint64_t* p_free = p_full + 2;       // [2] its P V is done
    uint64_t* x_full = p_free + 2;       // [4] a tile's scales are there
    uint64_t* drain = x_full + 4;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    int* bad_tile = abort_flag + 1;                            // [8] a page of the tile does not exist
    // [4][16] a tile's scales by block: 2^a, v (of a far block -inf: its rows have no weight here), 2^-v, and the byte of V's unit
    float4* scales = reinterpret_cast<float4*>(smem_raw + (reinterpret_cast<unsigned char*>(bad_tile + 8) - smem_raw + 15) / 16 * 16);
    float* q_unit = reinterpret_cast<float*>(scales + 4 * 16);  // [8][HP] log2 scores of a unit of Q K^T, by segment
    float* xm = q_unit + 8 * HP;                               // [2][4][HP] warps' tile maxima
    float* sm_l = xm + 2 * 4 * HP;                             // [4][HP] warps' sums of a segment

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2 * kStages; ++i) tc::mbar_init(full + i, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + i, Cfg::kQWarps);
            tc::mbar_init(q_free + i, 1);
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_full + i, 4 * Cfg::kGroups);
            tc::mbar_init(p_free + i, 1);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(x_full + i, 1);
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&tm_k);
        tc::prefetch_tmap(&tm_v);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, Cfg::kTmemCols);
        tc::tmem_relinquish();
    }
    DecodeWalk w = dec_plan<Cfg::kThreads>(p);
    __shared__ DecodeWalk s_mine;  // the same, kept for the end
    __shared__ int s_any_far;      // some block is far from its segment's unit
    if (CLUSTER && tid == 0) s_mine = w;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int* abort = abort_flag;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_decode_finish may be set up

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        const int n_box = kDecTile / a.sub;
        int u = 0, j = 0;  // stages and tiles issued
        bool ok = true;
        for (; w.left > 0 && ok; dec_next(p, w)) {
            const int g = w.g / p.HB, n_seg = dec_seg_tiles(w);
            const int32_t* table = p.block_table + (long long)w.b * p.max_pages;
            auto entry = [&](int t) {  // this lane's page of tile t, -1 past the prefix
                const int pos = t * kDecTile + lane * a.sub;
                return lane < n_box && pos < w.P ? table[pos / p.page_rows] : -1;
            };
            int phys = entry(w.t);
            for (int t = w.t; t < w.t + n_seg; ++t, ++j) {
                const int pos = t * kDecTile + lane * a.sub;
                const bool mine = lane < n_box && pos < w.P;
                const bool good = mine && phys >= 0 && phys < p.num_pages;
                const int plane = (int)(((long long)w.l * p.num_pages + phys) * p.Hkv + g);
                const int row = good ? pos % p.page_rows : 0;
                const unsigned goods = __ballot_sync(kFull, good), bads = __ballot_sync(kFull, mine && !good);
                if (t + 1 < w.t + n_seg) phys = entry(t + 1);
                if (lane == 0) bad_tile[j & 7] = bads != 0;
#pragma unroll
                for (int kv = 0; kv < 2 && ok; ++kv, ++u) {
                    const int st = u % kStages;
                    ok = tc::mbar_wait(empty + st, ((u / kStages) & 1) ^ 1, abort);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    if (lane == 0) tc::mbar_expect_tx(full + st, __popc(goods) * a.sub * D);
                    __syncwarp();
                    if (good) {
                        unsigned char* dst = ring + st * Cfg::kStageBytes + lane * a.sub * kRow;
#pragma unroll
                        for (int blk = 0; blk < Cfg::kBlocks; ++blk)
                            tc::tma_load_3d(dst + blk * (kDecTile * kRow), kv ? &tm_v : &tm_k, full + st, blk * kRow, row, plane);
                    }
                }
                if (!ok) break;
            }
        }
        // no copy may be under way when the CTA leaves
        for (int i = max(0, u - kStages); i < u; ++i) drain_wait(full + i % kStages, (i / kStages) & 1);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_qk = tc::idesc_e4m3(128, NQ, false, false);
            constexpr uint32_t idesc_pv = tc::idesc_e4m3(128, NP, true, true);
            const uint64_t kdesc = tc::desc_sw(kRow, tc::smem_u32(ring), 16, 8 * kRow);
            const uint64_t vdesc = tc::desc_sw(kRow, tc::smem_u32(ring), kDecTile * kRow, 8 * kRow);
            const uint64_t qdesc = tc::desc_sw(kRow, tc::smem_u32(sQ), 16, 8 * kRow);
            const uint64_t pdesc = tc::desc_sw(NP, tc::smem_u32(sP), 16, 8 * NP);
            int j = 0, seg = 0;
            bool ok = true;
            // P V of tile i; `first`: of a segment, so O starts anew (its warps have read the
            // last segment's O before they hand over this P)
            auto pv = [&](int i, bool first) {
                const int st = (2 * i + 1) % kStages;
                if (!tc::mbar_wait(full + st, ((2 * i + 1) / kStages) & 1, abort)) return false;
                if (!tc::mbar_wait(p_full + (i & 1), (i >> 1) & 1, abort)) return false;
                tc::tc_fence_after();
                const uint64_t vd = vdesc + (uint64_t)((st * Cfg::kStageBytes) >> 4);
                const uint64_t pd = pdesc + (uint64_t)(((i & 1) * Cfg::kPBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kDecTile / 32; ++kk)
#pragma unroll
                    for (int mb = 0; mb < kMB; ++mb)
                        tc::mma_f8_ss(tmem + Cfg::kOCol + mb * NP, vd + (uint64_t)((mb * kDecTile * kRow + kk * 32 * kRow) >> 4),
                                      pd + (uint64_t)((kk * 32 * NP) >> 4), idesc_pv, !first || kk > 0);
                tc::mma_commit(empty + st);
                tc::mma_commit(p_free + (i & 1));
                return true;
            };
            bool prev_first = false;
            for (; w.left > 0 && ok; dec_next(p, w), ++seg) {
                const int n_seg = dec_seg_tiles(w), qb = seg % kQBufs;
                ok = tc::mbar_wait(q_full + qb, (seg / kQBufs) & 1, abort);
                for (int i = 0; i < n_seg && ok; ++i, ++j) {
                    const int st = (2 * j) % kStages;
                    // (the scales for the softmax's sake, which waits for S alone)
                    ok = tc::mbar_wait(full + st, ((2 * j) / kStages) & 1, abort) && tc::mbar_wait(x_full + (j & 3), (j >> 2) & 1, abort);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint64_t kd = kdesc + (uint64_t)((st * Cfg::kStageBytes) >> 4);
                    const uint64_t qd = qdesc + (uint64_t)((qb * Cfg::kQBytes) >> 4);
                    constexpr int kSteps = kRow / 32;  // of a swizzled row
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        tc::mma_f8_ss(tmem + (j & 1) * NQ,
                                      kd + (uint64_t)(((kk / kSteps) * (kDecTile * kRow) + (kk % kSteps) * 32) >> 4),
                                      qd + (uint64_t)(((kk / kSteps) * (NQ * kRow) + (kk % kSteps) * 32) >> 4), idesc_qk, kk > 0);
                    tc::mma_commit(empty + st);
                    tc::mma_commit(s_full + (j & 1));
                    if (i == n_seg - 1) tc::mma_commit(q_free + qb);
                    // S of tile j + 1 may overwrite that of tile j - 1 once P of j - 1 is there
                    if (j > 0) ok = pv(j - 1, prev_first);
                    prev_first = i == 0;
                }
            }
            if (ok && j > 0) pv(j - 1, prev_first);
            tc::mma_commit(drain);
            drain_wait(drain, 0);
        }
    } else if (warp == 2 || warp >= 4 + 4 * Cfg::kGroups) {
        // -------------------------------------------------------------------- queries
        constexpr int E = D / 32;                                     // consecutive channels a lane
        constexpr int HW = HP / Cfg::kQWarps, N = GH < HW ? GH : HW;  // heads a warp, and of them at a time
        const int hw = warp == 2 ? 0 : HW * (warp - 3 - 4 * Cfg::kGroups);
        int seg = 0;
        for (; w.left > 0; dec_next(p, w), ++seg) {
            const int g = w.g / p.HB, h0 = (w.g % p.HB) * HP, nh = min(HP, p.G - h0), qb = seg % kQBufs;
            const Tin* q = static_cast<const Tin*>(p.q) + (((long long)w.l * p.B + w.b) * p.Hq + g * p.G + h0) * D + lane * E;
            bool ok = true;
            QueryRun<Tin, E> x[2][N];  // up to eight heads, and the next eight on their way
            auto load = [&](int hb) {
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    x[hb / 8 & 1][h].zero();
                    if (hw + hb + h < nh) x[hb / 8 & 1][h].load(q + (hw + hb + h) * D);
                }
            };
            load(0);
            unsigned char* const to = sQ + qb * Cfg::kQBytes + lane * E / kRow * (NQ * kRow);
#pragma unroll
            for (int hb = 0; hb < HW; hb += 8) {
                if (hb + 8 < HW) load(hb + 8);
                QueryRun<Tin, E>* v = x[hb / 8 & 1];
                // (of heads that are not there: zeros.  Steps over all heads, no branch between them: a head's own chain is long)
                uint32_t most[N], all = 0;
#pragma unroll
                for (int h = 0; h < N; ++h) most[h] = v[h].top();
#pragma unroll
                for (int h = 0; h < N; ++h) most[h] = __reduce_max_sync(kFull, most[h]);
#pragma unroll
                for (int h = 0; h < N; ++h) all = max(all, most[h]);
                if (all >= 0x7f800000u) {  // infinities or NaN: the largest of the others; they become NaN
#pragma unroll
                    for (int h = 0; h < N; ++h) {
                        v[h].without_infinities();
                        most[h] = __reduce_max_sync(kFull, v[h].top_finite());
                    }
                }
                if (hb == 0) ok = __all_sync(kFull, tc::mbar_wait(q_free + qb, ((seg / kQBufs) & 1) ^ 1, abort));
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    // the power of two that takes the largest channel to [128, 256)
                    const int up = most[h] ? min(134 - (int)(most[h] >> 23), 100) : 0;
                    const float f = __int_as_float((127 + up) << 23);
                    if (lane == 0) q_unit[(seg & 7) * HP + hw + hb + h] = p.scale_log2 * __int_as_float((127 - up) << 23);
                    uint32_t c[(E + 3) / 4][QP];
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        float y[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) y[z] = e + z < E ? v[h].get((e + z) % E) * f : 0.f;
                        split4<QP>(y, c[e / 4]);
                    }
#pragma unroll
                    for (int i = 0; i < QP; ++i) {
                        unsigned char* at = to + tc::swizzled<kRow>((i * HP + hw + hb + h) * kRow + lane * E % kRow);
                        if constexpr (E == 8)
                            *reinterpret_cast<uint2*>(at) = make_uint2(c[0][i], c[E / 4 - 1][i]);
                        else if constexpr (E == 4)
                            *reinterpret_cast<uint32_t*>(at) = c[0][i];
                        else
                            *reinterpret_cast<uint16_t*>(at) = (uint16_t)c[0][i];
                    }
                }
            }
            if (!ok) break;
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(q_full + qb);
        }
    } else if (warp == 3) {
        // --------------------------------------------------------------------- scales
        const int n_blk = kDecTile / p.block, per_page = p.page_rows / p.block;
        int j = 0;
        bool ok = true, any_far = false;
        for (; w.left > 0 && ok; dec_next(p, w)) {
            const int g = w.g / p.HB, n_seg = dec_seg_tiles(w);
            const int32_t* table = p.block_table + (long long)w.b * p.max_pages;
            // the page of this lane's block of tile t (of the first tile: and the tiles behind it), -1 past the segment
            const int end = min(w.P, (w.t + n_seg) * kDecTile);
            auto entry = [&](int t, int lanes) {
                const int pos = t * kDecTile + lane * p.block;
                return lane < lanes && pos < end ? table[pos / p.page_rows] : -1;
            };
            int phys = entry(w.t, 32), base = 0;  // base: V's unit, 0 while the segment's blocks are of zeros
            for (int t = w.t; t < w.t + n_seg; ++t, ++j) {
                const bool good = phys >= 0 && phys < p.num_pages;
                const int in = (t * kDecTile + lane * p.block) % p.page_rows / p.block;
                const long long at = good ? (((long long)w.l * p.num_pages + phys) * p.Hkv + g) * per_page + in : 0;
                const int kb = p.ks[at], vb = good ? p.vs[at] : 0;
                if (t + 1 < w.t + n_seg) phys = entry(t + 1, n_blk);
                // at most two tiles ahead of the softmax, so no slot of four is written that it still reads
                if (j >= 2) ok = __all_sync(kFull, tc::mbar_wait(p_full + (j & 1), ((j - 2) >> 1) & 1, abort));
                if (!ok) break;
                if (!base) base = v_unit_of(vb);
                // A block of zeros takes any scale: a small one, so that the weights which do count keep their bits.
                const int dv = vb ? vb - base : -60;
                const bool far = is_far(vb, base) && lane < n_blk;
                any_far |= far;
                if (lane < n_blk)
                    scales[(j & 3) * 16 + lane] = make_float4(scale_of(kb), far ? -INFINITY : (float)dv, far ? 0.f : scale_of(127 - dv), __int_as_float(base));
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(x_full + (j & 3));
            }
        }
        any_far = __any_sync(kFull, any_far);
        if (CLUSTER) s_any_far = any_far;
        else if (lane == 0) p.far[blockIdx.x] = any_far;
    } else {
        // -------------------------------------------------- softmax, and the segments' partials
        const int ws = warp & 3, r = 32 * ws + lane;  // a warp reads its quarter of the lanes
        const uint32_t lane_base = (uint32_t)(32 * ws) << 16;
        const int grp = Cfg::kGroups == 1 ? 0 : (warp - 4) >> 2, hg = grp * 8, bar = 1 + grp;  // heads hg .. hg + 7 of the block
        const int my_block = r / p.block;
        int j = 0, seg = 0;
        bool ok = true;
        for (; w.left > 0; dec_next(p, w), ++seg) {
            const int h0 = (w.g % p.HB) * HP + hg, nh = min(8, p.G - h0), n_seg = dec_seg_tiles(w);
            int base = 0;  // the byte of V's unit (0: so far there are zeros alone)
            F2 m[GH / 2], l[GH / 2];  // two heads each; m holds minus the reference
#pragma unroll
            for (int h = 0; h < GH / 2; ++h) {
                m[h] = f2(-kNoRef, -kNoRef);
                l[h] = f2(0.f, 0.f);
            }
            int bad = 0;
            for (int i = 0; i < n_seg; ++i, ++j) {
                const int n = min(kDecTile, w.P - (w.t + i) * kDecTile);
                // a warp that gave up still takes part in the barriers
                if (ok) ok = tc::mbar_wait(s_full + (j & 1), (j >> 1) & 1, abort);
                ok = __all_sync(kFull, ok);
                F2 t[GH / 2];
                float v_back = 1.f;
                bool above = false;  // a score is far above its head's reference
                if (ok) {
                    tc::tc_fence_after();
                    const float4 x = scales[(j & 3) * 16 + my_block];
                    const F2 k_unit = f2(x.x, x.x);
                    const float add = r < n ? x.y : -INFINITY;  // a row past the prefix: weight 0
                    const F2 v_add = f2(add, add);
                    v_back = x.z;
                    base = __float_as_int(x.w);
                    uint32_t sr[QP][8];
#pragma unroll
                    for (int y = 0; y < QP; ++y) tmem_ld8(tmem + lane_base + (j & 1) * NQ + y * HP + hg, sr[y]);
                    tc::tmem_wait_ld();
                    bad |= bad_tile[j & 7];
                    const float2* unit = reinterpret_cast<const float2*>(q_unit + (seg & 7) * HP + hg);
#pragma unroll
                    for (int h = 0; h < GH / 2; ++h) {
                        F2 s = f2(__uint_as_float(sr[QP - 1][2 * h]), __uint_as_float(sr[QP - 1][2 * h + 1]));
#pragma unroll
                        for (int y = QP - 2; y >= 0; --y)
                            s = fma2(s, f2(0.0625f, 0.0625f), f2(__uint_as_float(sr[y][2 * h]), __uint_as_float(sr[y][2 * h + 1])));
                        const float2 q = unit[h];
                        t[h] = fma2(s, k_unit * f2(q.x, q.y), v_add);
                        const float2 d = f2_get(t[h] + m[h]);
                        above |= d.x > kLift + kTau;
                        above |= d.y > kLift + kTau;
                    }
                    if (n < kDecTile && r >= n) {  // (what lies in the rows behind the prefix may be NaN)
                        above = false;
#pragma unroll
                        for (int h = 0; h < GH / 2; ++h) t[h] = v_add;
                    }
                }
                if (bar_any(bar, above)) {
                    // the segment's first tile, or a growing maximum: new references, the tile's
                    // maxima, for the heads that need them
                    float* x = xm + (j & 1) * 4 * HP + hg;
                    float mine = -INFINITY;
                    if (ok)
#pragma unroll
                        for (int h = 0; h < GH / 2; ++h) {
                            const float2 y = f2_get(t[h]);
                            const float v0 = redux_max(y.x), v1 = redux_max(y.y);
                            if (lane == 2 * h) mine = v0;
                            if (lane == 2 * h + 1) mine = v1;
                        }
                    if (lane < 8) x[ws * HP + lane] = mine;
                    tc::named_bar(bar, 128);
                    if (ok) {
                        float f[GH];
#pragma unroll
                        for (int h = 0; h < GH / 2; ++h) {
                            const float2 old = f2_get(m[h]);
                            float now[2] = {old.x, old.y};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int k = 2 * h + e;
                                const float mt = fmaxf(fmaxf(x[k], x[HP + k]), fmaxf(x[2 * HP + k], x[3 * HP + k])) - kLift;
                                f[k] = 1.f;
                                if (mt > kTau - now[e]) {
                                    f[k] = tc::ex2(-now[e] - mt);
                                    now[e] = -mt;
                                }
                            }
                            l[h] = l[h] * f2(f[2 * h], f[2 * h + 1]);
                            m[h] = f2(now[0], now[1]);
                        }
                        if (i > 0) {  // O holds earlier tiles of the segment: once their P V are done
                            ok = __all_sync(kFull, tc::mbar_wait(p_free + ((j - 1) & 1), ((j - 1) >> 1) & 1, abort));
                            if (ok) {
                                tc::tc_fence_after();
#pragma unroll
                                for (int c = 0; c < kMB * PP; ++c) {
                                    uint32_t o[8];
                                    const uint32_t at = tmem + lane_base + Cfg::kOCol + (c / PP) * NP + (c % PP) * HP + hg;
                                    tmem_ld8(at, o);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < GH; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
                                    tmem_st8(at, o);
                                }
                                tc::tmem_wait_st();
                            }
                        }
                    }
                }
                if (!ok) continue;
                // (the P buffer is free: S of tile j comes after P V of tile j - 2)
                uint32_t c[2][PP] = {};
#pragma unroll
                for (int h = 0; h < GH; h += 4) {
                    float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int y = 0; y < 4 && h + y < GH; y += 2) {
                        const float2 d = f2_get(t[(h + y) / 2] + m[(h + y) / 2]);
                        e[y] = tc::ex2(d.x);
                        e[y + 1] = tc::ex2(d.y);
                        l[(h + y) / 2] = fma2(f2(e[y], e[y + 1]), f2(v_back, v_back), l[(h + y) / 2]);
                    }
                    split4<PP>(e, c[h / 4]);
                }
                unsigned char* pb = sP + (j & 1) * Cfg::kPBytes;
#pragma unroll
                for (int x = 0; x < PP; ++x) {
                    const uint2 v = make_uint2(c[0][x], c[1][x]);
                    if (HP > 8 || x + 1 == PP) {
                        if (HP > 8 || x % 2 == 0) *reinterpret_cast<uint2*>(pb + tc::swizzled<NP>(r * NP + x * HP + hg)) = v;
                    } else if (x % 2 == 0) {
                        *reinterpret_cast<uint4*>(pb + tc::swizzled<NP>(r * NP + x * HP)) =
                            make_uint4(v.x, v.y, c[0][(x + 1) % PP], c[1][(x + 1) % PP]);
                    }
                }
                if (n < kDecTile) {
                    // V rows past the prefix may hold anything, even NaN, and a zero weight
                    // does not cancel NaN: zero them before the MMA reads them
                    const int st = (2 * j + 1) % kStages;
                    ok = __all_sync(kFull, tc::mbar_wait(full + st, ((2 * j + 1) / kStages) & 1, abort));
                    if (!ok) continue;
                    unsigned char* v = ring + st * Cfg::kStageBytes;
                    const int per = (kDecTile - n) * (kRow / 16);
                    for (int e = grp * 128 + r; e < per * Cfg::kBlocks; e += 128 * Cfg::kGroups)
                        *reinterpret_cast<uint4*>(v + (e / per) * (kDecTile * kRow) + n * kRow + (e % per) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_full + (j & 1));
            }
            // ---- the partial: sums through shared memory, O once the last P V is done
            float sum = 0.f, ref = 0.f;
#pragma unroll
            for (int h = 0; h < GH / 2; ++h) {
                const float2 z = f2_get(l[h]), y = f2_get(m[h]);
                const float x0 = warp_sum(z.x), x1 = warp_sum(z.y);
                if (lane == 2 * h) sum = x0, ref = -y.x;
                if (lane == 2 * h + 1) sum = x1, ref = -y.y;
            }
            if (lane < 8) sm_l[ws * HP + hg + lane] = sum;
            if (ok) ok = tc::mbar_wait(p_free + ((j - 1) & 1), ((j - 1) >> 1) & 1, abort);
            ok = __all_sync(kFull, ok);
            tc::named_bar(bar, 128);
            const long long slot = dec_slot(p, w);
            if (r < nh) {
                const float* x = sm_l + hg + r;
                const float z = (x[0] + x[HP]) + (x[2 * HP] + x[3 * HP]);
                p.part_ml[slot * p.HT + hg + r] = make_float2(ref, !ok ? kSegTimeout : (bad ? kSegBadPage : z));
            }
            if (!ok) continue;
            tc::tc_fence_after();
            const float v_unit = scale_of(base);
#pragma unroll
            for (int mb = 0; mb < kMB; ++mb) {
                uint32_t o[PP][8];
#pragma unroll
                for (int x = 0; x < PP; ++x) tmem_ld8(tmem + lane_base + Cfg::kOCol + mb * NP + x * HP + hg, o[x]);
                tc::tmem_wait_ld();
                if (D >= 128 || r < D) {
                    float* out = p.part_o + (slot * p.HT + hg) * D + mb * 128 + r;
#pragma unroll
                    for (int h = 0; h < GH; ++h)
                        if (h < nh) {
                            float s = __uint_as_float(o[PP - 1][h]);
#pragma unroll
                            for (int x = PP - 2; x >= 0; --x) s = fmaf(s, 0.0625f, __uint_as_float(o[x][h]));
                            out[h * D] = s * v_unit;
                        }
                }
            }
        }
    }

    tc::tc_fence_before();
    DecNew<Tin, D> mine_new;
    if (CLUSTER) mine_new.load(p, (long long)s_mine.l * p.B + s_mine.b, s_mine.g, dec_first_head(p), lane);
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, Cfg::kTmemCols);
    }
    if (CLUSTER) {
        if (s_any_far) return far_tail<Tin, D, Cfg::kThreads>(p, s_mine, reinterpret_cast<float*>(ring));
        if (p.cl > 1) tc::cluster_sync();
        dec_finish<Tin, D, Cfg::kThreads>(p, s_mine, mine_new, reinterpret_cast<float*>(ring));
    }
}

// ------------------------------------------------------------------------------ host
// p as decode_clusters left it
template <typename Tin, int D, int HP, int GH, int QP, int PP, bool CLUSTER>
cudaError_t quant_launch(const DecodeParams& p, const DecQuantArgs& a, const CUtensorMap* maps, cudaStream_t st) {
    using Cfg = QuantCfg<D, HP, GH, QP, PP>;
    const auto kernel = k_decode_quant<Tin, D, HP, GH, QP, PP, CLUSTER>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    cudaLaunchConfig_t cfg = decode_grid(p, Cfg::kThreads, Cfg::kSmem, at, st);
    return cudaLaunchKernelEx(&cfg, kernel, p, a, maps[0], maps[1]);
}

// the instances, F(type, head size, heads a block, of a warpgroup, parts of Q, of P)
#define DDT_QUANT_D(F, D)           \
    F(float, D, 8, 8, 6, 6)         \
    F(float, D, 16, 8, 6, 6)        \
    F(__nv_bfloat16, D, 8, 2, 2, 4) \
    F(__nv_bfloat16, D, 8, 4, 2, 4) \
    F(__nv_bfloat16, D, 8, 8, 2, 4) \
    F(__nv_bfloat16, D, 16, 8, 2, 4) \
    F(__nv_bfloat16, D, 32, 8, 2, 4)
#define DDT_QUANT_INSTANCES(F) DDT_QUANT_D(F, 64) DDT_QUANT_D(F, 128) DDT_QUANT_D(F, 256)

}  // namespace ddt
