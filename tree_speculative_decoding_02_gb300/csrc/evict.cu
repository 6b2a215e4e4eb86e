// evict.cu -- ddt_evict_paged: eviction from the paged cache by accumulated attention weight.
//
// Every (layer, request, kv head) keeps the `keep` of its cached rows whose running sums of
// attention weight are largest (the first n_sink and the last n_recent positions before all
// others).  Softmax attention does not depend on the order of the cached rows (rotary
// embedding is in the keys), so nothing is compacted: the kept rows behind the budget's last
// index fill, in order, the holes the evicted rows leave below it.  Sources (>= keep) and
// destinations (< keep) never meet, so the moves run in place and in any order, and a
// request that is r rows over its budget moves at most r rows however long its cache is.
//
//   k_evict_claim   grid B: lengths and block table checked, pages that are used twice found.
//   k_evict_select  grid L B Hkv: the keep-th largest key by three histogram passes (11, 11
//                   and 10 bits), then one pass in index order for the holes and the rows
//                   that fill them; their sums and positions follow at once.  Long caches of few
//                   units: a cluster of CTAs a unit, each with a slice of its rows, their
//                   histograms and counts summed over the cluster's shared memory.
//   k_evict_move    grid (L B Hkv, y): the K and V rows, 16 bytes a thread, and the entries behind
//                   the budget; the first layer's first head writes the request's lengths and status.
//
// The moves are bound by HBM: 695 MB (336203 moves of 512-byte K and V rows from random places, and
// the entries behind the budget) of 16 requests of up to 32768 rows cut to 8192 take 104 us, 6.7
// TB/s, beside their selection's 24 (two rows' loads in flight a thread and five blocks an SM take
// as long).  The selection is bound by latency: three
// passes and a few barriers each, 8.5 us for a unit of 2000 rows, 23 us for 1024 units of 4200
// on all SMs (its floor, 8 bytes a row, is 5 us), so it begins beside the checks and the moves
// are set up behind it.  Whole calls: 19.5 us (4 units of 2001 rows), 40 us (the 1024 units, 100
// rows over the budget each) and 133 us (the 16 requests).
#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace ddt {

namespace {
constexpr int kBins = 2048;             // bins of a histogram pass (the last one uses 1024)
constexpr int kSelCache = 45 * 1024;    // rows whose keys fit in shared memory
constexpr int kUncut = 16384;           // rows that one CTA takes in any case
constexpr int kSlice = 4096;            // rows a CTA of a cluster has at least
constexpr int kClaimThreads = 512;
constexpr int kWindow = 1 << 20;        // pages a bitmap in shared memory covers

struct EvictParams {
    int L, B, Hkv, page_rows, num_pages, max_pages, cap, keep, n_sink, n_recent;
    int pieces;  // 16-byte pieces of a cached row
    int cl;      // k_evict_select's CTAs a unit
    int most;    // moves the workspace holds a unit
    const int32_t* block_table;
    const int32_t* seq_len;
    uint4* k_pages;
    uint4* v_pages;
    float* weight;
    int32_t* row_pos;
    int32_t* prefix_len;
    int32_t* n_placed;
    int32_t* status;
    // workspace
    int32_t* state;   // [B] -P (over its budget), DDT_OK (within it), or an error
    int32_t* n_move;  // [U]
    int32_t* src;     // [U][most]
    int32_t* dst;     // [U][most]
};
}  // namespace

// Checks one request.  A page that it would rewrite may be used once only: its own pages are
// marked in a bitmap in shared memory (a window of the pages at a time, one window but for
// pools of over a million pages), and every page of the other requests is looked up there.
__global__ void __launch_bounds__(kClaimThreads) k_evict_claim(const EvictParams p) {
    extern __shared__ uint32_t s_used[];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the selection may begin
    const int P = p.prefix_len[b], np = p.n_placed[b], sq = p.seq_len[b];
    int st = (P < 0 || P > p.cap) ? DDT_ERR_CAPACITY : ((np < 0 || np > P || sq < P) ? DDT_ERR_INVALID_ARG : DDT_OK);
    auto pages = [&](int rows) { return rows < 0 || rows > p.cap ? 0 : (rows + p.page_rows - 1) / p.page_rows; };
    const int32_t* mine = p.block_table + (long long)b * p.max_pages;
    const int n = st == DDT_ERR_CAPACITY ? 0 : pages(P);
    const bool cut = st == DDT_OK && P > p.keep;
    int bad = 0, twice = 0;
    for (int w0 = 0; w0 < p.num_pages && (cut || w0 == 0); w0 += kWindow) {
        const int len = min(kWindow, p.num_pages - w0);
        auto marked = [&](int page, bool set) {
            const unsigned at = (unsigned)(page - w0);
            if (at >= (unsigned)len) return 0u;
            const uint32_t bit = 1u << (at & 31);
            return (set ? atomicOr(&s_used[at >> 5], bit) : s_used[at >> 5]) & bit;
        };
        if (cut)
            for (int i = tid; i < (len + 31) / 32; i += kClaimThreads) s_used[i] = 0;
        __syncthreads();
#pragma unroll 2
        for (int i = tid; i < n; i += kClaimThreads) {
            const int page = mine[i];
            bad |= page < 0 || page >= p.num_pages;
            if (cut) twice |= marked(page, true) != 0;
        }
        __syncthreads();
        if (!cut) break;
        for (int o = warp; o < p.B; o += kClaimThreads / 32) {
            const int32_t* other = p.block_table + (long long)o * p.max_pages;
            const int no = o == b ? 0 : pages(p.prefix_len[o]);
#pragma unroll 4
            for (int i = lane; i < no; i += 32) twice |= marked(other[i], false) != 0;
        }
        __syncthreads();
    }
    bad = __syncthreads_or(bad);
    twice = __syncthreads_or(twice);
    if (tid == 0) p.state[b] = st != DDT_OK ? st : (bad || twice ? (int)DDT_ERR_INVALID_ARG : (cut ? -P : (int)DDT_OK));
}

// The order of the rows as an unsigned key: 0 for NaN, then the sums from the smallest to
// the largest (-0 and +0 alike), and above them all the protected positions.
__device__ __forceinline__ uint32_t evict_key(const EvictParams& p, float w, int pos, int sq) {
    // n_sink <= seq_len - n_recent: both fit in the budget, which the sequence is longer than
    if ((uint32_t)(pos - p.n_sink) >= (uint32_t)(sq - p.n_recent - p.n_sink)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return w != w ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Exclusive prefix sum of v over the block and the total, with one barrier: the caller
// alternates between two arrays of warp sums.
template <int NT>
__device__ __forceinline__ int block_scan(int v, int* s_w, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_w[warp] = incl;
    __syncthreads();
    int x = lane < NT / 32 ? s_w[lane] : 0;  // every warp sums up the warps for itself
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) {
        const int up = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += up;
    }
    total = __shfl_sync(kFull, x, NT / 32 - 1);
    const int before = __shfl_sync(kFull, x, warp ? warp - 1 : 0);
    return incl - v + (warp ? before : 0);
}

// `x` of the same variable in CTA `rank` of the cluster
__device__ __forceinline__ int cluster_read(const int* x, int rank) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(tc::mapa_shared(tc::smem_u32(x), (uint32_t)rank)) : "memory");
    return v;
}

// CACHED: the slice's keys are kept in shared memory after the first pass.  The histogram
// passes take four consecutive rows a thread.
template <int NT, bool CACHED>
__global__ void __launch_bounds__(NT, NT == 256 ? 6 : 1) k_evict_select(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t s_key[];
    constexpr bool kClusters = NT == 1024;  // p.cl may be above 1
    __shared__ int s_hist[kClusters ? 2 : 1][kBins];  // while other CTAs read one, the next pass fills the other
    __shared__ uint4 s_bits[NT];
    __shared__ int s_w[2][32];
    __shared__ int s_bin, s_rest, s_count, s_all[2];
    __shared__ int s_same[2], s_cnt[4];  // of this CTA's rows: keys of 0 and protected ones; see the lists
    const int cl = kClusters ? p.cl : 1, rank = kClusters ? blockIdx.x % cl : 0;
    const unsigned unit = kClusters ? blockIdx.x / (unsigned)cl : blockIdx.x;
    const long long u = unit;
    auto sync = [&]() {
        if (kClusters && cl > 1) tc::cluster_sync();
        else __syncthreads();
    };
    const int b = (int)(unit / (unsigned)p.Hkv % (unsigned)p.B);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the moves may be set up
    const int P = p.prefix_len[b], np = p.n_placed[b], sq = p.seq_len[b], K = p.keep;
    // lengths that make no sense are refused by k_evict_claim, which may still be running: it
    // has the last word before anything is written
    const bool cut = P > K && P <= p.cap && np >= 0 && np <= P && sq >= P;
    if (!cut) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid == 0) p.n_move[u] = 0;  // (by every CTA of a cluster)
        return;
    }
    // this CTA's rows
    const int per = cl == 1 ? P : ((P + cl - 1) / cl + 31) & ~31, lo = min(rank * per, P), hi = min(lo + per, P);
    float* wt = p.weight + u * p.cap;
    int32_t* rp = p.row_pos + u * p.cap;
    const int32_t* table = p.block_table + (long long)b * p.max_pages;
    for (int i = tid; i < kBins; i += NT) s_hist[0][i] = 0;
    if (tid < 2) s_same[tid] = 0;
    if (tid < 4) s_cnt[tid] = 0;
    __syncthreads();
    auto pos_of = [&](int i) { return i < np ? rp[i] : sq - P + i; };
    // the keys of rows i .. i + 3 (rows >= P: any)
    auto keys4 = [&](int i, uint32_t (&key)[4]) {
        const float4 w = *reinterpret_cast<const float4*>(wt + i);
        int4 r = make_int4(0, 0, 0, 0);
        if (i < np) r = *reinterpret_cast<const int4*>(rp + i);
        const float ww[4] = {w.x, w.y, w.z, w.w};
        const int rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) key[q] = evict_key(p, ww[q], i + q < np ? rr[q] : sq - P + i + q, sq);
    };
    auto key_of = [&](int i) { return CACHED ? s_key[i - lo] : evict_key(p, wt[i], pos_of(i), sq); };
    // ---- the K-th largest key: its bits from the highest down.  Kept are the rows above
    //      `limit` and the first `rest` that equal it.
    uint32_t limit = 0;
    int rest = K;
    bool tie = false;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int sh = pass == 0 ? 21 : (pass == 1 ? 10 : 0), up = pass == 1 ? 21 : 10;
        const uint32_t mask = pass == 2 ? 1023 : 2047;
        int* hist = s_hist[kClusters ? pass & 1 : 0];
        int zeros = 0, safe = 0;  // the two keys that many rows share: counted in registers
#pragma unroll 2
        for (int i = lo + tid * 4; i < hi; i += NT * 4) {
            uint32_t key[4];
            if (CACHED && pass > 0) {
                const uint4 k = *reinterpret_cast<const uint4*>(s_key + i - lo);
                key[0] = k.x;
                key[1] = k.y;
                key[2] = k.z;
                key[3] = k.w;
            } else {
                keys4(i, key);
                if (CACHED) *reinterpret_cast<uint4*>(s_key + i - lo) = make_uint4(key[0], key[1], key[2], key[3]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (i + q >= P || (pass > 0 && (key[q] >> up) != limit)) continue;
                if (key[q] == 0x80000000u) ++zeros;
                else if (key[q] == 0xffffffffu) ++safe;
                else atomicAdd(&hist[(key[q] >> sh) & mask], 1);
            }
        }
        zeros = __reduce_add_sync(kFull, zeros);
        safe = __reduce_add_sync(kFull, safe);
        if (lane == 0) {
            if (zeros) {
                atomicAdd(&hist[(0x80000000u >> sh) & mask], zeros);
                if (pass == 0) atomicAdd(&s_same[0], zeros);
            }
            if (safe) {
                atomicAdd(&hist[(0xffffffffu >> sh) & mask], safe);
                if (pass == 0) atomicAdd(&s_same[1], safe);
            }
        }
        sync();
        if (pass == 0 && tid < 2) {
            int n = s_same[tid];
            if (cl > 1) {
                n = 0;
                for (int r = 0; r < cl; ++r) n += cluster_read(&s_same[tid], r);
            }
            s_all[tid] = n;
        }
        // warp i has the i-th run of bins from the top, and only the warp whose run holds the
        // K-th largest looks closer
        constexpr int kPer = kBins / NT;
        const int top = kBins - 1 - warp * (kBins / (NT / 32)) - lane;
        int c[kPer], sum = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            c[q] = cl == 1 ? hist[top - 32 * q] : 0;
            if (cl > 1)
#pragma unroll 4
                for (int r = 0; r < cl; ++r) c[q] += cluster_read(hist + top - 32 * q, r);
            s_hist[kClusters ? (pass & 1) ^ 1 : 0][top - 32 * q] = 0;  // for the next pass
            sum += c[q];
        }
        sum = __reduce_add_sync(kFull, sum);
        if (lane == 0) s_w[pass & 1][warp] = sum;
        __syncthreads();
        int above = __reduce_add_sync(kFull, lane < warp ? s_w[pass & 1][lane] : 0);
        if (above < rest && above + sum >= rest) {
#pragma unroll 1
            for (int q = 0; q < kPer; ++q) {
                int here = c[0];
#pragma unroll
                for (int r = 1; r < kPer; ++r) here = q == r ? c[r] : here;
                int incl = here;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up1 = __shfl_up_sync(kFull, incl, o);
                    if (lane >= o) incl += up1;
                }
                const int excl = above + incl - here;
                if (excl < rest && excl + here >= rest) {
                    s_bin = top - 32 * q;
                    s_rest = rest - excl;
                    s_count = here;
                }
                above = __shfl_sync(kFull, above + incl, 31);
                if (above >= rest) break;
            }
        }
        __syncthreads();
        limit = pass == 0 ? (uint32_t)s_bin : (limit << (pass == 2 ? 10 : 11)) | (uint32_t)s_bin;
        rest = s_rest;
        tie = s_count > rest;
        if (!tie) {  // all of this prefix stay
            limit = (limit << sh) - 1u;
            rest = 0;
            break;
        }
        if (pass == 0 && limit == 0x80000000u >> 21 && s_count == s_all[0]) {
            limit = 0x80000000u;
            break;
        }
        if (pass == 0 && limit == 0xffffffffu >> 21 && s_count == s_all[1]) {
            limit = 0xffffffffu;
            break;
        }
    }
    if (kClusters && cl > 1) {
        // what the lists of the CTAs before this one will hold: above the limit below K and from K on,
        // and equal to it
        int n[4] = {0, 0, 0, 0};
        for (int i = lo + tid; i < hi; i += NT) {
            const uint32_t key = key_of(i);
            n[0] += key > limit && i < K;
            n[1] += key > limit && i >= K;
            n[2] += key == limit && i < K;
            n[3] += key == limit && i >= K;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            n[q] = __reduce_add_sync(kFull, n[q]);
            if (lane == 0 && n[q]) atomicAdd(&s_cnt[q], n[q]);
        }
        sync();
    }
    int eqs = 0, holes = 0, movers = 0, all_holes = 0;
    if (kClusters && cl > 1) {
        int eq = 0;
        for (int r = 0; r < cl; ++r) {
            if (r == rank) {
                eqs = eq;
                holes = all_holes;
            }
            const int first = min(r * per, P), below = max(min(min(first + per, P), K) - first, 0);
            int n[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) n[q] = cluster_read(&s_cnt[q], r);
            const int left = tie ? max(rest - eq, 0) : 0, low = min(left, n[2]), high = min(left - low, n[3]);
            all_holes += below - n[0] - low;
            if (r < rank) movers += n[1] + high;
            eq += n[2] + n[3];
        }
        sync();  // no CTA's shared memory is read by others from here on
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.state[b] >= 0) {
        if (tid == 0) p.n_move[u] = 0;
        return;
    }
    // ---- in index order: holes below K, and the kept rows behind it that fill them.  A bit a
    //      row (above the limit, equal to it) by ballots, a thread a word of 32 rows for the
    //      counts, and a warp a word for the lists.
    int32_t* src = p.src + u * p.most;
    int32_t* dst = p.dst + u * p.most;
    for (int c0 = lo; c0 < hi; c0 += 32 * NT) {
        const int words = min(NT, (hi - c0 + 31) / 32);
#pragma unroll 4
        for (int w = warp; w < words; w += NT / 32) {
            const int i = c0 + w * 32 + lane;
            const uint32_t key = i < hi ? key_of(i) : 0u;  // no limit is below 0
            const uint32_t gt = __ballot_sync(kFull, key > limit), eq = __ballot_sync(kFull, i < hi && key == limit);
            if (lane == 0) s_bits[w] = make_uint4(gt, eq, 0u, 0u);
        }
        __syncthreads();
        const uint4 x = tid < words ? s_bits[tid] : make_uint4(0u, 0u, 0u, 0u);
        const int i = c0 + tid * 32;
        uint32_t kept = x.x;
        int total;
        if (tie) {  // the first `rest` equal rows stay
            const int before = eqs + block_scan<NT>(__popc(x.y), s_w[0], total);
            eqs += total;
            uint32_t eq = before < rest ? x.y : 0u;
            while (__popc(eq) > rest - before && eq) eq &= ~(0x80000000u >> __clz(eq));
            kept |= eq;
        }
        // the word's rows that exist, and those below K
        const uint32_t live = hi - i >= 32 ? ~0u : (hi <= i ? 0u : (1u << (hi - i)) - 1u);
        const uint32_t low = K - i >= 32 ? ~0u : (K <= i ? 0u : (1u << (K - i)) - 1u);
        const uint32_t hole = ~kept & live & low, mover = kept & ~low;
        const int at = block_scan<NT>(__popc(hole) + (__popc(mover) << 16), s_w[1], total);
        if (tid < words)
            s_bits[tid] = make_uint4(hole, mover, (uint32_t)(holes + (at & 0xffff)), movers + ((uint32_t)at >> 16));
        __syncthreads();
#pragma unroll 4
        for (int w = warp; w < words; w += NT / 32) {
            const uint4 y = s_bits[w];
            const int row = c0 + w * 32 + lane;
            if (y.x >> lane & 1u) dst[y.z + __popc(y.x & ((1u << lane) - 1u))] = row;
            if (y.y >> lane & 1u) src[y.w + __popc(y.y & ((1u << lane) - 1u))] = row;
        }
        holes += total & 0xffff;
        movers += (int)((uint32_t)total >> 16);
        __syncthreads();
    }
    for (int i = np + rank * NT + tid; i < K; i += NT * cl) rp[i] = sq - P + i;
    if (cl > 1) holes = all_holes;
    if (rank == 0 && tid == 0) p.n_move[u] = holes;
    sync();
    for (int j0 = rank * 4 * NT + tid; j0 < holes; j0 += 4 * NT * cl) {  // four moves' loads are in flight
        int s[4], d[4], pos[4], ps[4], pd[4];
        float w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = j0 + q * NT < holes ? j0 + q * NT : j0;
            s[q] = src[j];
            d[q] = dst[j];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = wt[s[q]];
            pos[q] = pos_of(s[q]);
            const int is = s[q] / p.page_rows, id = d[q] / p.page_rows;
            ps[q] = table[is] * p.page_rows + s[q] - is * p.page_rows;
            pd[q] = table[id] * p.page_rows + d[q] - id * p.page_rows;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = j0 + q * NT;
            if (j >= holes) break;
            wt[d[q]] = w[q];
            rp[d[q]] = pos[q];
            // from here on the lists hold places in the pages
            src[j] = ps[q];
            dst[j] = pd[q];
        }
    }
}

// A block moves 256 / pieces rows at a time, a thread 16 bytes of K and of V; the next
// round's places are loaded while this one's rows are on their way.
__global__ void __launch_bounds__(256, 8) k_evict_move(const EvictParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long u = blockIdx.x;
    const unsigned lb = blockIdx.x / (unsigned)p.Hkv;  // (64-bit divisions would be most of the instructions)
    const int g = (int)(blockIdx.x - lb * p.Hkv), l = (int)(lb / (unsigned)p.B), b = (int)(lb - (unsigned)l * p.B);
    const int st = p.state[b], tid = threadIdx.x, K = p.keep;
    if (l == 0 && g == 0 && blockIdx.y == 0 && tid == 0) {
        if (st < 0) {
            p.prefix_len[b] = K;
            p.n_placed[b] = K;
        }
        p.status[b] = max(st, (int)DDT_OK);
    }
    if (st < 0) {  // sums and positions of rows K .. P - 1, four at a time but for the ends
        const int P = -st, k4 = min((K + 3) & ~3, P), p4 = max(P & ~3, k4);
        float* wt = p.weight + u * p.cap;
        int32_t* rp = p.row_pos + u * p.cap;
        for (int i = k4 + (blockIdx.y * 256 + tid) * 4; i < p4; i += gridDim.y * 1024) {
            *reinterpret_cast<float4*>(wt + i) = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<int4*>(rp + i) = make_int4(-1, -1, -1, -1);
        }
        if (blockIdx.y == 0 && tid < 8) {
            const int i = tid < 4 ? K + tid : p4 + tid - 4;
            if (i < (tid < 4 ? k4 : P)) {
                wt[i] = 0.f;
                rp[i] = -1;
            }
        }
    }
    const int n = p.n_move[u];
    const int32_t* src = p.src + u * p.most;
    const int32_t* dst = p.dst + u * p.most;
    const int wide = min(p.pieces, 256), rows = 256 / wide, step = gridDim.y * rows;
    int j = blockIdx.y * rows + threadIdx.x / wide;
    if ((int)threadIdx.x >= rows * wide || j >= n) return;
    const long long layer = (long long)l * p.num_pages;
    // place -> 16-byte words: page * (Hkv * page_rows) + g * page_rows + row in the page
    auto word = [&](int place) {
        const int page = place / p.page_rows;
        return (((layer + page) * p.Hkv + g) * p.page_rows + (place - page * p.page_rows)) * p.pieces;
    };
    int s = src[j], d = dst[j];
    for (; j < n; j += step) {
        const bool more = j + step < n;
        const int s1 = more ? src[j + step] : 0, d1 = more ? dst[j + step] : 0;
        const long long from = word(s), to = word(d);
        for (int c = threadIdx.x % wide; c < p.pieces; c += wide) {
            const uint4 k = p.k_pages[from + c], v = p.v_pages[from + c];
            p.k_pages[to + c] = k;
            p.v_pages[to + c] = v;
        }
        s = s1;
        d = d1;
    }
}

// ------------------------------------------------------------------------------ host
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

static size_t evict_layout(EvictParams& p, unsigned char* ws) {
    const size_t units = (size_t)p.L * p.B * p.Hkv;
    size_t at = 0;
    auto take = [&](size_t n) {
        unsigned char* r = ws + at;
        at += al256(n * sizeof(int32_t));
        return reinterpret_cast<int32_t*>(r);
    };
    p.most = p.cap / 2;  // min(keep, cap - keep) whatever `keep` is
    p.state = take(p.B);
    p.n_move = take(units);
    p.src = take(units * p.most);
    p.dst = take(units * p.most);
    return at;
}

size_t evict_ws_bytes(int L, int B, int Hkv, const AttnPaging& pg) {
    EvictParams p{};
    p.L = L;
    p.B = B;
    p.Hkv = Hkv;
    p.num_pages = pg.num_pages;
    p.cap = pg.page_rows * pg.max_pages;
    return evict_layout(p, nullptr);
}

// a launch that may be set up while the kernel before it ends
static cudaError_t launch_behind(void (*kernel)(EvictParams), dim3 grid, int threads, int smem, const EvictParams& p,
                                 cudaStream_t st, int cluster = 1) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = counted(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int NT>
static cudaError_t select_go(const EvictParams& p, unsigned units, int keys, cudaStream_t st) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_evict_select<NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCache * 4);
    return e != cudaSuccess ? e : launch_behind(k_evict_select<NT, true>, dim3(units * p.cl), NT, keys, p, st, p.cl);
}

cudaError_t launch_evict(int L, int B, int Hkv, int row_bytes, const AttnPaging& pg, int keep, int n_sink,
                         int n_recent, void* k_pages, void* v_pages, const int32_t* seq_len, float* weight,
                         int32_t* row_pos, int32_t* prefix_len, int32_t* n_placed, int32_t* status, void* ws,
                         cudaStream_t st) {
    EvictParams p{};
    p.L = L;
    p.B = B;
    p.Hkv = Hkv;
    p.page_rows = pg.page_rows;
    p.num_pages = pg.num_pages;
    p.max_pages = pg.max_pages;
    p.cap = pg.page_rows * pg.max_pages;
    p.keep = keep;
    p.n_sink = n_sink;
    p.n_recent = n_recent;
    p.pieces = row_bytes / 16;
    p.block_table = pg.block_table;
    p.seq_len = seq_len;
    p.k_pages = static_cast<uint4*>(k_pages);
    p.v_pages = static_cast<uint4*>(v_pages);
    p.weight = weight;
    p.row_pos = row_pos;
    p.prefix_len = prefix_len;
    p.n_placed = n_placed;
    p.status = status;
    evict_layout(p, static_cast<unsigned char*>(ws));
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const unsigned units = (unsigned)L * B * Hkv;
    cudaError_t e = cudaFuncSetAttribute(k_evict_claim, cudaFuncAttributeMaxDynamicSharedMemorySize, kWindow / 8);
    if (e != cudaSuccess) return e;
    k_evict_claim<<<counted(B), kClaimThreads, ((pg.num_pages < kWindow ? pg.num_pages : kWindow) + 31) / 32 * 4, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // Many threads a unit, for its latency, if there is an SM for every unit or a unit is long;
    // else small blocks, so that several units share an SM and hide each other's barriers.  With
    // 1024 and 256 threads: 64 units of 4000 rows 10.6 and 13.4 us, of 8000 13.3 and 19.3; but 256
    // units of 4000 rows 19.0 and 15.2, of 8000 24.1 and 24.2, of 16000 33 and 42.
    const bool wide = units <= (unsigned)sms || p.cap > 8192;
    // Clusters where SMs would idle.  Of 1, 2, 4, 8 CTAs a unit: 4 units of 16000 rows 16.1, 18.3, -, -;
    // of 32000 28.4, 24.0, 21.7, 23.9; of 131000 135, -, -, 32 us.  16 clusters of 8 are not all
    // resident at once (32000 rows: 43.8 us, in clusters of 4 22.2).
    p.cl = 1;
    while (p.cl < 8 && p.cap > kUncut && units * 2 * p.cl <= (unsigned)(p.cl == 4 ? sms * 3 / 4 : sms) &&
           p.cap >= kSlice * 2 * p.cl)
        p.cl *= 2;
    const int slice = p.cl == 1 ? p.cap : ((p.cap + p.cl - 1) / p.cl + 31) & ~31, keys = (slice + 3) / 4 * 16;
    if (slice > kSelCache) e = launch_behind(k_evict_select<1024, false>, dim3(units * p.cl), 1024, 0, p, st, p.cl);
    else if (wide) e = select_go<1024>(p, units, keys, st);
    else e = select_go<256>(p, units, keys, st);
    if (e != cudaSuccess) return e;
    const int rows = 256 / (p.pieces < 256 ? p.pieces : 256);  // a block's
    // Blocks a unit: one for every eight rounds that a full table could need, so that units of all
    // lengths end together, but one place of every SM at least and eight times as many at most.
    // With one place: 16 requests of 3000 to 32768 rows cut to 8192 152 us, with eight 133; but 256
    // units cut from 1000 to 500 rows 20.5 and 25.4.
    const long moves = keep < p.cap - keep ? keep : (p.cap > keep ? p.cap - keep : 1);
    const long rounds = (moves + rows - 1) / rows, one = 8L * sms / units + 1, all = 64L * sms / units + 1;
    long y = (rounds + 7) / 8;
    y = y < one ? one : (y > all ? all : y);
    return launch_behind(k_evict_move, dim3(units, (unsigned)(y < rounds ? y : rounds)), 256, 0, p, st);
}

}  // namespace ddt
