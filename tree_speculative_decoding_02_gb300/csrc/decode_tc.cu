// decode_tc.cu -- k_decode_tc: ddt_decode_attn_paged's pass over the cached rows on the
// tensor cores (bf16 caches).
//
// One query row a head leaves G = Hq / Hkv rows to share a K/V row, so the pass is bound by
// reading the cache: 4 G d flop for 4 d bytes.  The products run with the cache as the
// M = 128 operand, straight from the tiles that TMA writes, and the few heads as N:
//   S^T [128 rows x heads]  = K tile [rows x d] . Q^T          (K as it lies, K-major)
//   O^T [d x heads]        += V tile^T [d x rows] . P^T        (V as it lies, M-major)
// so no thread ever touches a K or V element; the CUDA cores see G scores a row.  P is
// handed over as two bf16 parts, P = P_hi + P_lo, in N columns of their own (the MMA's
// smallest N is 16: for up to 8 heads the second part costs nothing), which keeps the
// weights to 2^-16 where bf16 alone would give 2^-9.
//
//   warp 0      producer: block-table entries, TMA of K and V tiles (128 rows, 128-byte
//               swizzle, a box a page slice, a lane a box) into one ring, Q by TMA
//   warp 1      MMA issuer: Q K^T of tile j + 1 ahead of P V of tile j
//   warps 2-5, 6-9 ..  softmax, eight heads a warpgroup: a thread a cached row.  The exponents' reference of a head is the
//               maximum of the segment's first tile, and moves (with O rescaled) only when a
//               score is 2^8 above it: one vote a tile instead of its maxima.  At a segment's
//               end the same warps write its partial.
// A block of heads is 8, 16 or 32 of them: the smallest that holds the group, so the cache is
// read once for up to 32 heads (16 for head size 256).  Eight heads a warpgroup, because the
// chain from S to P of a tile (about 2000 cycles, as long as an SM's share of HBM takes for
// 32 KB) grows with a thread's heads: 32 heads of 64, 16 requests of 6000 rows, 41.8 us with
// four warpgroups and 62.5 with one.  For up to eight heads and head sizes 64 and 128 the
// second warpgroup is that of a second CTA on the SM, with half the ring: 2 x 96 requests of
// up to 2500 rows, 16 heads of 64, 156 us, and 215 with one CTA.
//
// Bound by HBM: 32 requests of 1K to 32K rows, 24 heads over 4 kv heads of 256, with weights
// (2.49 GB): 394 us, 6.3 TB/s; one of 131071 rows, 32 heads over 8 of 128 (545 MB): 89 us, 6.1
// TB/s; the 2 x 96 above (937 MB) 6.0 TB/s.  On the CUDA cores the first took 2.2 ms.
// Every wait is bounded; after one gives up the CTA drains its copies and MMAs, and its
// unfinished segments say so to the join.
#include <cuda.h>
#include <math.h>

#include <mutex>

#include "decode.cuh"
#include "tc.cuh"

namespace ddt {

namespace {

constexpr float kTau = 8.f;  // rescale O only when a head's maximum grows by more than 2^kTau

template <int D, int HP>
struct DecCfg {
    static constexpr int kGroups = HP / 8;                 // softmax warpgroups
    static constexpr int kThreads = 64 + 128 * kGroups;
    static constexpr int kBlocks = D / 64;                 // 128-byte swizzle blocks of a row
    static constexpr int kStageBytes = kDecTile * D * 2;   // a K or V tile
    static constexpr int kCtas = HP == 8 && D <= 128 ? 2 : 1;  // an SM
    static constexpr int kRing = kCtas == 2 ? 98304 : (HP == 32 ? 163840 : 196608);
    static constexpr int kStages = kRing / kStageBytes;
    static constexpr int NQ = HP < 16 ? 16 : HP;           // N of Q K^T
    static constexpr int NP = 2 * HP;                      // N of P V: both parts
    static constexpr int kQPitch = HP * 128;               // a 64-channel block of Q: HP rows (for 8 of
                                                           // them N = 16 reads on: columns not used)
    static constexpr int kQBytes = HP * D * 2;
    static constexpr int kPBytes = NP * kDecTile * 2;
    static constexpr int kMB = D > 128 ? D / 128 : 1;      // M blocks of P V
    static constexpr int kOCol = 2 * NQ;                   // tensor memory: S x 2, O
    static constexpr int kCols = 2 * NQ + kMB * NP;
    static constexpr int kTmemCols = kCols <= 64 ? 64 : 128;
    static constexpr int kCtl = (2 * kStages + 16) * 8 + 12 * HP * 4;  // barriers and small arrays
    static constexpr int kSmem = 1024 + kStages * kStageBytes + 2 * kQBytes + 2 * kPBytes + kCtl;
    static_assert(kCtas * (kSmem + 1024 + 256) <= 228 * 1024, "shared memory of an SM (the plan has a little of its own)");
    static_assert(kCols <= 128, "tensor memory");
};

struct DecTcArgs {
    int sub;  // rows of a box: the largest of 128, 64, ... that pages are made of
};

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

}  // namespace

template <int D, int HP>
__global__ void __launch_bounds__(DecCfg<D, HP>::kThreads, DecCfg<D, HP>::kCtas)
    k_decode_tc(const DecodeParams p, const DecTcArgs a, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q) {
    using Cfg = DecCfg<D, HP>;
    constexpr int kStages = Cfg::kStages, NQ = Cfg::NQ, NP = Cfg::NP, kMB = Cfg::kMB;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sQ = ring + kStages * Cfg::kStageBytes;  // [2]
    unsigned char* sP = sQ + 2 * Cfg::kQBytes;              // [2]
    uint64_t* full = reinterpret_cast<uint64_t*>(sP + 2 * Cfg::kPBytes);  // [kStages] a tile landed
    uint64_t* empty = full + kStages;                                      // [kStages] its MMAs are done
    uint64_t* q_full = empty + kStages;  // [2] a segment's queries landed
    uint64_t* q_free = q_full + 2;       // [2] its last Q K^T is done
    uint64_t* s_full = q_free + 2;       // [2] S of a tile in tensor memory
    uint64_t* p_full = s_full + 2;       // [2] P of a tile in shared memory (the softmax warps)
    uint64_t* p_free = p_full + 2;       // [2] its P V is done
    uint64_t* drain = p_free + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
    int* bad_tile = abort_flag + 1;                            // [8] a page of the tile does not exist
    float* xm = reinterpret_cast<float*>(bad_tile + 8);        // [2][4][HP] warps' tile maxima
    float* sm_l = xm + 2 * 4 * HP;                             // [4][HP] warps' sums of a segment

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2 * kStages; ++i) tc::mbar_init(full + i, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + i, 1);
            tc::mbar_init(q_free + i, 1);
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_full + i, 4 * Cfg::kGroups);
            tc::mbar_init(p_free + i, 1);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&tm_k);
        tc::prefetch_tmap(&tm_v);
        tc::prefetch_tmap(&tm_q);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, Cfg::kTmemCols);
        tc::tmem_relinquish();
    }
    const DecodeWalk mine = dec_plan<Cfg::kThreads>(p);
    DecodeWalk w = mine;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int* abort = abort_flag;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_decode_finish may be set up

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        const int n_box = kDecTile / a.sub;
        int u = 0, seg = 0, j = 0;  // stages, segments and tiles issued
        bool ok = true;
        for (; w.left > 0 && ok; dec_next(p, w), ++seg) {
            const int g = w.g / p.HB, n_seg = dec_seg_tiles(w);
            const int32_t* table = p.block_table + (long long)w.b * p.max_pages;
            auto entry = [&](int t) {  // this lane's page of tile t, -1 past the prefix
                const int pos = t * kDecTile + lane * a.sub;
                return lane < n_box && pos < w.P ? table[pos / p.page_rows] : -1;
            };
            int phys = entry(w.t);
            ok = tc::mbar_wait(q_free + (seg & 1), ((seg >> 1) & 1) ^ 1, abort);
            if (!__all_sync(kFull, ok)) break;
            if (lane == 0) {
                tc::mbar_expect_tx(q_full + (seg & 1), Cfg::kBlocks * p.HT * 128);
                const long long row = ((long long)w.l * p.B + w.b) * p.Hq + g * p.G + (w.g % p.HB) * HP;
#pragma unroll
                for (int blk = 0; blk < Cfg::kBlocks; ++blk)
                    tc::tma_load_2d(sQ + (seg & 1) * Cfg::kQBytes + blk * Cfg::kQPitch, &tm_q, q_full + (seg & 1),
                                    blk * 64, (int)row);
            }
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
                    if (lane == 0) tc::mbar_expect_tx(full + st, __popc(goods) * a.sub * D * 2);
                    __syncwarp();
                    if (good) {
                        unsigned char* dst = ring + st * Cfg::kStageBytes + lane * a.sub * 128;
#pragma unroll
                        for (int blk = 0; blk < Cfg::kBlocks; ++blk)
                            tc::tma_load_3d(dst + blk * (kDecTile * 128), kv ? &tm_v : &tm_k, full + st, blk * 64, row,
                                            plane);
                    }
                }
                if (!ok) break;
            }
        }
        // no copy may be under way when the CTA leaves
        for (int i = max(0, u - kStages); i < u; ++i) drain_wait(full + i % kStages, (i / kStages) & 1);
        for (int i = max(0, seg - 1); i <= seg; ++i)
            if (*abort) drain_wait(q_full + (i & 1), (i >> 1) & 1);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_qk = tc::idesc_bf16(128, NQ, false, false);
            constexpr uint32_t idesc_pv = tc::idesc_bf16(128, NP, true, false);
            const uint64_t kdesc = tc::desc_sw128(tc::smem_u32(ring), 16, 1024);
            // head size 64: lanes 64-127 of O read on in shared memory and are not used
            const uint64_t vdesc = tc::desc_sw128(tc::smem_u32(ring), D == 64 ? 8192 : kDecTile * 128, 1024);
            const uint64_t qdesc = tc::desc_sw128(tc::smem_u32(sQ), 16, 1024);
            const uint64_t pdesc = tc::desc_sw128(tc::smem_u32(sP), 16, 1024);
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
                for (int kk = 0; kk < kDecTile / 16; ++kk)
#pragma unroll
                    for (int mb = 0; mb < kMB; ++mb)
                        tc::mma_f16_ss(tmem + Cfg::kOCol + mb * NP,
                                       vd + (uint64_t)((mb * 2 * kDecTile * 128 + kk * 2048) >> 4),
                                       pd + (uint64_t)(((kk >> 2) * (NP * 128) + (kk & 3) * 32) >> 4), idesc_pv,
                                       !first || kk > 0);
                tc::mma_commit(empty + st);
                tc::mma_commit(p_free + (i & 1));
                return true;
            };
            bool prev_first = false;
            for (; w.left > 0 && ok; dec_next(p, w), ++seg) {
                const int n_seg = dec_seg_tiles(w);
                ok = tc::mbar_wait(q_full + (seg & 1), (seg >> 1) & 1, abort);
                for (int i = 0; i < n_seg && ok; ++i, ++j) {
                    const int st = (2 * j) % kStages;
                    ok = tc::mbar_wait(full + st, ((2 * j) / kStages) & 1, abort);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint64_t kd = kdesc + (uint64_t)((st * Cfg::kStageBytes) >> 4);
                    const uint64_t qd = qdesc + (uint64_t)(((seg & 1) * Cfg::kQBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc::mma_f16_ss(tmem + (j & 1) * NQ,
                                       kd + (uint64_t)(((kk >> 2) * (kDecTile * 128) + (kk & 3) * 32) >> 4),
                                       qd + (uint64_t)(((kk >> 2) * Cfg::kQPitch + (kk & 3) * 32) >> 4), idesc_qk, kk > 0);
                    tc::mma_commit(empty + st);
                    tc::mma_commit(s_full + (j & 1));
                    if (i == n_seg - 1) tc::mma_commit(q_free + (seg & 1));
                    // S of tile j + 1 may overwrite that of tile j - 1 once P of j - 1 is there
                    if (j > 0) ok = pv(j - 1, prev_first);
                    prev_first = i == 0;
                }
            }
            if (ok && j > 0) pv(j - 1, prev_first);
            tc::mma_commit(drain);
            drain_wait(drain, 0);
        }
    } else {
        // -------------------------------------------------- softmax, and the segments' partials
        const int ws = warp & 3, r = 32 * ws + lane;  // a warp reads its quarter of the lanes
        const uint32_t lane_base = (uint32_t)(32 * ws) << 16;
        const int grp = Cfg::kGroups == 1 ? 0 : (warp - 2) >> 2, hg = grp * 8, bar = 1 + grp;  // heads hg .. hg + 7 of the block
        int j = 0;
        bool ok = true;
        for (; w.left > 0; dec_next(p, w)) {
            const int g = w.g / p.HB, h0 = (w.g % p.HB) * HP + hg, nh = min(8, p.G - h0), n_seg = dec_seg_tiles(w);
            float m[8], l[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                m[h] = kNoRef;
                l[h] = 0.f;
            }
            int bad = 0;
            for (int i = 0; i < n_seg; ++i, ++j) {
                const int y = (w.t + i) * kDecTile, n = min(kDecTile, w.P - y);
                // a warp that gave up still takes part in the barriers
                if (ok) ok = tc::mbar_wait(s_full + (j & 1), (j >> 1) & 1, abort);
                ok = __all_sync(kFull, ok);
                float t[8];
                bool above = false;  // a score is far above its head's reference
                if (ok) {
                    tc::tc_fence_after();
                    uint32_t sr[8];
                    tmem_ld8(tmem + lane_base + (j & 1) * NQ + hg, sr);
                    tc::tmem_wait_ld();
                    bad |= bad_tile[j & 7];
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        t[h] = r < n ? __uint_as_float(sr[h]) * p.scale_log2 : -INFINITY;
                        if (h < nh) above |= t[h] > m[h] + kTau;
                    }
                    if (p.score && r < n) {
                        float* sc = p.score + (((long long)w.l * p.B + w.b) * p.Hq + g * p.G + h0) * p.cap + y + r;
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            if (h < nh) sc[(long long)h * p.cap] = t[h];
                    }
                }
                if (bar_any(bar, above)) {
                    // the segment's first tile, or a growing maximum: new references, the tile's
                    // maxima, for the heads that need them
                    float* x = xm + (j & 1) * 4 * HP + hg;
                    float mine = -INFINITY;
                    if (ok)
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            if (h < nh) {
                                const float v = redux_max(t[h]);
                                if (lane == h) mine = v;
                            }
                    if (lane < 8) x[ws * HP + lane] = mine;
                    tc::named_bar(bar, 128);
                    if (ok) {
                        float f[8];
#pragma unroll
                        for (int h = 0; h < 8; ++h) {
                            const float mt = fmaxf(fmaxf(x[h], x[HP + h]), fmaxf(x[2 * HP + h], x[3 * HP + h]));
                            f[h] = 1.f;
                            if (mt > m[h] + kTau) {
                                f[h] = tc::ex2(m[h] - mt);
                                l[h] *= f[h];
                                m[h] = mt;
                            }
                        }
                        if (i > 0) {  // O holds earlier tiles of the segment: once their P V are done
                            ok = __all_sync(kFull, tc::mbar_wait(p_free + ((j - 1) & 1), ((j - 1) >> 1) & 1, abort));
                            if (ok) {
                                tc::tc_fence_after();
#pragma unroll
                                for (int c = hg; c < kMB * NP; c += HP) {
                                    uint32_t o[8];
                                    const uint32_t at = tmem + lane_base + Cfg::kOCol + c;
                                    tmem_ld8(at, o);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
                                    tmem_st8(at, o);
                                }
                                tc::tmem_wait_st();
                            }
                        }
                    }
                }
                if (!ok) continue;
                // the P buffer is free once P V of tile j - 2 is done
                ok = __all_sync(kFull, tc::mbar_wait(p_free + (j & 1), ((j >> 1) & 1) ^ 1, abort));
                if (!ok) continue;
                unsigned char* pb = sP + (j & 1) * Cfg::kPBytes + (r >> 6) * (NP * 128);
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (h < nh) {
                        const float e = tc::ex2(t[h] - m[h]);
                        l[h] += e;
                        const uint32_t hi = __float_as_uint(e) & 0xffff0000u;
                        const __nv_bfloat16 lo = __float2bfloat16_rn(e - __uint_as_float(hi));
                        const uint32_t col = ((uint32_t)(r & 63) * 2) ^ ((uint32_t)(h & 7) << 4);
                        *reinterpret_cast<uint16_t*>(pb + (hg + h) * 128 + col) = (uint16_t)(hi >> 16);
                        *reinterpret_cast<__nv_bfloat16*>(pb + (HP + hg + h) * 128 + col) = lo;
                    }
                if (n < kDecTile) {
                    // V rows past the prefix may hold anything, even NaN, and a zero weight
                    // does not cancel NaN: zero them before the MMA reads them
                    const int st = (2 * j + 1) % kStages;
                    ok = __all_sync(kFull, tc::mbar_wait(full + st, ((2 * j + 1) / kStages) & 1, abort));
                    if (!ok) continue;
                    unsigned char* v = ring + st * Cfg::kStageBytes;
                    const int per = (kDecTile - n) * 8;
                    for (int e = grp * 128 + r; e < per * Cfg::kBlocks; e += 128 * Cfg::kGroups)
                        *reinterpret_cast<uint4*>(v + (e / per) * (kDecTile * 128) + n * 128 + (e % per) * 16) =
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
            for (int h = 0; h < 8; ++h)
                if (h < nh) {
                    const float x = warp_sum(l[h]);
                    if (lane == h) sum = x;
                    if (r == h) ref = m[h];
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
#pragma unroll
            for (int mb = 0; mb < kMB; ++mb) {
                uint32_t o[16];
                tmem_ld8(tmem + lane_base + Cfg::kOCol + mb * NP + hg, o);
                tmem_ld8(tmem + lane_base + Cfg::kOCol + mb * NP + HP + hg, o + 8);
                tc::tmem_wait_ld();
                if (D >= 128 || r < D) {
                    float* out = p.part_o + (slot * p.HT + hg) * D + mb * 128 + r;
#pragma unroll
                    for (int h = 0; h < 8; ++h)
                        if (h < nh) out[h * D] = __uint_as_float(o[h]) + __uint_as_float(o[8 + h]);
                }
            }
        }
    }

    tc::tc_fence_before();
    DecNew<__nv_bfloat16, D> mine_new;
    if (p.cl) mine_new.load(p, (long long)mine.l * p.B + mine.b, mine.g, dec_first_head(p), lane);
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, Cfg::kTmemCols);
    }
    if (p.cl) {
        if (p.cl > 1) tc::cluster_sync();
        dec_finish<__nv_bfloat16, D, Cfg::kThreads>(p, mine, mine_new, reinterpret_cast<float*>(ring));
    }
}

// ------------------------------------------------------------------------------ host
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

template <int D, int HP>
cudaError_t tc_go(DecodeParams& p, const DecTcArgs& a, const CUtensorMap* maps, cudaStream_t st) {
    constexpr int smem = DecCfg<D, HP>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(k_decode_tc<D, HP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    cudaLaunchConfig_t cfg = decode_config(p, false, DecCfg<D, HP>::kCtas, DecCfg<D, HP>::kThreads, smem, at, st);
    return cudaLaunchKernelEx(&cfg, k_decode_tc<D, HP>, p, a, maps[0], maps[1], maps[2]);
}

}  // namespace

bool decode_tc_supported(int d, ddt_dtype in) { return in == DDT_BF16 && (d == 64 || d == 128 || d == 256); }

// heads a block: the smallest of 8, 16 and 32 that holds the group (16 for head size 256,
// where shared memory has no room for more)
int decode_tc_heads(int G, int d) { return G <= 8 ? 8 : (G <= 16 || d == 256 ? 16 : 32); }

// p.C: SMs on entry, CTAs on return
cudaError_t launch_decode_tc(DecodeParams& p, cudaStream_t st) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    DecTcArgs a;
    a.sub = p.page_rows % 128 == 0 ? 128 : (p.page_rows < 64 ? p.page_rows : 64);
    CUtensorMap maps[3];
    const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.page_rows, (cuuint64_t)p.L * p.num_pages * p.Hkv};
    const cuuint64_t str[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.page_rows * p.d * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.sub, 1}, es[3] = {1, 1, 1};
    const cuuint64_t qdims[2] = {(cuuint64_t)p.d, (cuuint64_t)p.L * p.B * p.Hq}, qstr[1] = {(cuuint64_t)p.d * 2};
    const cuuint32_t qbox[2] = {64, (cuuint32_t)p.HT};
    const void* base[3] = {p.k_pages, p.v_pages, p.q};
    for (int i = 0; i < 3; ++i)
        if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, i < 2 ? 3 : 2, const_cast<void*>(base[i]), i < 2 ? dims : qdims,
                i < 2 ? str : qstr, i < 2 ? box : qbox, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    switch (p.d * 100 + p.hbs) {
        case 6408: return tc_go<64, 8>(p, a, maps, st);
        case 6416: return tc_go<64, 16>(p, a, maps, st);
        case 6432: return tc_go<64, 32>(p, a, maps, st);
        case 12808: return tc_go<128, 8>(p, a, maps, st);
        case 12816: return tc_go<128, 16>(p, a, maps, st);
        case 12832: return tc_go<128, 32>(p, a, maps, st);
        case 25608: return tc_go<256, 8>(p, a, maps, st);
        case 25616: return tc_go<256, 16>(p, a, maps, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ddt
