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
//   k_evict_claim   grid B: lengths and block table checked, uses of each page counted.
//   k_evict_select  grid L B Hkv: the keep-th largest key by three histogram passes (11, 11
//                   and 10 bits), then one pass in index order for the holes and the rows
//                   that fill them; sums and positions follow at once.
//   k_evict_move    grid (L B Hkv, y): the K and V rows, 16 bytes a thread; the first layer's
//                   first head writes the request's lengths and status.
#include "common.cuh"
#include "kernels.h"

namespace ddt {

namespace {
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kEvict = -1;  // state of a request that is over its budget

struct EvictParams {
    int L, B, Hkv, page_rows, num_pages, max_pages, cap, keep, n_sink, n_recent;
    int pieces;  // 16-byte pieces of a cached row
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
    int32_t* uses;    // [num_pages]
    int32_t* state;   // [B] kEvict, DDT_OK (within the budget), or an error
    int32_t* shared;  // [B] 1: a page of the request is used more than once
    int32_t* n_move;  // [U]
    int32_t* src;     // [U][most]
    int32_t* dst;     // [U][most]
};
}  // namespace

__global__ void __launch_bounds__(256) k_evict_claim(const EvictParams p) {
    const int b = blockIdx.x;
    const int P = p.prefix_len[b], np = p.n_placed[b], sq = p.seq_len[b];
    int st = (P < 0 || P > p.cap) ? DDT_ERR_CAPACITY : ((np < 0 || np > P || sq < P) ? DDT_ERR_INVALID_ARG : DDT_OK);
    int bad = 0;
    if (st != DDT_ERR_CAPACITY) {
        const int n = (P + p.page_rows - 1) / p.page_rows;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int pg = p.block_table[(long long)b * p.max_pages + i];
            if (pg < 0 || pg >= p.num_pages) bad = 1;
            else atomicAdd(p.uses + pg, 1);
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        if (bad) st = DDT_ERR_INVALID_ARG;
        p.state[b] = st != DDT_OK ? st : (P > p.keep ? kEvict : DDT_OK);
        p.shared[b] = 0;
    }
}

// The order of the rows as an unsigned key: 0 for NaN, then the sums from the smallest to
// the largest (-0 and +0 alike), and above them all the protected positions.
__device__ __forceinline__ uint32_t evict_key(const EvictParams& p, float w, int pos, int sq) {
    if (pos < p.n_sink || pos >= sq - p.n_recent) return 0xffffffffu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the block and the total; the caller's shared array.
__device__ __forceinline__ int block_scan(int v, int* s_w, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();  // the array's last use is over
    if (lane == 31) s_w[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int x = lane < kSelWarps ? s_w[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += up;
        }
        s_w[lane] = x;
    }
    __syncthreads();
    total = s_w[kSelWarps - 1];
    return incl - v + (warp ? s_w[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const EvictParams p) {
    __shared__ int s_hist[kBins];
    __shared__ int s_w[32];
    __shared__ int s_bin, s_rest;
    const long long u = blockIdx.x;
    const int b = (int)(u / p.Hkv % p.B);
    const int tid = threadIdx.x;
    if (p.state[b] != kEvict) {
        if (tid == 0) p.n_move[u] = 0;
        return;
    }
    const int P = p.prefix_len[b], np = p.n_placed[b], sq = p.seq_len[b], K = p.keep;
    int twice = 0;
    for (int i = tid; i < (P + p.page_rows - 1) / p.page_rows; i += kSelThreads)
        twice |= p.uses[p.block_table[(long long)b * p.max_pages + i]] > 1;
    if (__syncthreads_or(twice)) {
        if (tid == 0) {
            p.n_move[u] = 0;
            p.shared[b] = 1;
        }
        return;
    }
    float* wt = p.weight + u * p.cap;
    int32_t* rp = p.row_pos + u * p.cap;
    auto pos_of = [&](int i) { return i < np ? rp[i] : sq - P + i; };
    // ---- the K-th largest key: its bits from the highest down
    uint32_t prefix = 0;
    int rest = K;  // how many of the keys with this prefix are kept
    const int shift[3] = {21, 10, 0};
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int sh = shift[pass], nb = pass == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < P; i += kSelThreads) {
            const uint32_t key = evict_key(p, wt[i], pos_of(i), sq);
            const bool in = pass == 0 || (key >> shift[pass - 1]) == prefix;
            if (in) atomicAdd(&s_hist[(key >> sh) & (nb - 1)], 1);
        }
        __syncthreads();
        // thread i looks at bins nb - 1 - 2 i and the one below: an exclusive sum from the top
        const int hi = kBins - 1 - 2 * tid;
        const int c0 = s_hist[hi], c1 = s_hist[hi - 1];
        int total;
        const int above = block_scan(c0 + c1, s_w, total);
        if (above < rest && above + c0 >= rest) {
            s_bin = hi;
            s_rest = rest - above;
        } else if (above + c0 < rest && above + c0 + c1 >= rest) {
            s_bin = hi - 1;
            s_rest = rest - above - c0;
        }
        __syncthreads();
        prefix = pass == 0 ? (uint32_t)s_bin : (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)s_bin;
        rest = s_rest;
        __syncthreads();
    }
    // ---- kept: every key above the threshold and the first `rest` equal to it
    int32_t* src = p.src + u * p.most;
    int32_t* dst = p.dst + u * p.most;
    int eq0 = 0, holes = 0, movers = 0;
    for (int i0 = 0; i0 < P; i0 += kSelThreads) {
        const int i = i0 + tid;
        uint32_t key = 0;
        int pos = 0;
        if (i < P) {
            pos = pos_of(i);
            key = evict_key(p, wt[i], pos, sq);
        }
        const int eq = i < P && key == prefix;
        int n_eq;
        const int before = block_scan(eq, s_w, n_eq);
        const bool kept = i < P && (key > prefix || (eq && eq0 + before < rest));
        eq0 += n_eq;
        const int f = i >= P ? 0 : (i < K ? (kept ? 0 : 1) : (kept ? 1 << 16 : 0));
        int both;
        const int at = block_scan(f, s_w, both);
        if (f == 1) dst[holes + (at & 0xffff)] = i;
        if (f == 1 << 16) src[movers + (at >> 16)] = i;
        if (i < K && i >= np && i < P) rp[i] = pos;
        holes += both & 0xffff;
        movers += both >> 16;
    }
    __syncthreads();
    for (int j = tid; j < holes; j += kSelThreads) {
        wt[dst[j]] = wt[src[j]];
        rp[dst[j]] = pos_of(src[j]);
    }
    __syncthreads();
    for (int i = K + tid; i < P; i += kSelThreads) {
        wt[i] = 0.f;
        rp[i] = -1;
    }
    if (tid == 0) p.n_move[u] = holes;
}

__global__ void __launch_bounds__(256) k_evict_move(const EvictParams p) {
    const long long u = blockIdx.x;
    const int g = (int)(u % p.Hkv), b = (int)(u / p.Hkv % p.B), l = (int)(u / p.Hkv / p.B);
    if (l == 0 && g == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        const int st = p.state[b];
        if (st == kEvict && !p.shared[b]) {
            p.prefix_len[b] = p.keep;
            p.n_placed[b] = p.keep;
        }
        p.status[b] = st != kEvict ? st : (p.shared[b] ? (int)DDT_ERR_INVALID_ARG : (int)DDT_OK);
    }
    const int n = p.n_move[u];
    const int32_t* table = p.block_table + (long long)b * p.max_pages;
    auto row = [&](int i) {
        return ((((long long)l * p.num_pages + table[i / p.page_rows]) * p.Hkv + g) * p.page_rows + i % p.page_rows) *
               p.pieces;
    };
    const long long all = (long long)n * p.pieces;
    for (long long e = (long long)blockIdx.y * blockDim.x + threadIdx.x; e < all; e += (long long)gridDim.y * blockDim.x) {
        const long long j = e / p.pieces;
        const int c = (int)(e % p.pieces);
        const long long from = row(p.src[u * p.most + j]) + c, to = row(p.dst[u * p.most + j]) + c;
        const uint4 k = p.k_pages[from], v = p.v_pages[from];
        p.k_pages[to] = k;
        p.v_pages[to] = v;
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
    p.uses = take(p.num_pages);
    p.state = take(p.B);
    p.shared = take(p.B);
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
    cudaError_t e = cudaMemsetAsync(p.uses, 0, (size_t)p.num_pages * sizeof(int32_t), st);
    if (e != cudaSuccess) return e;
    const unsigned units = (unsigned)L * B * Hkv;
    k_evict_claim<<<counted(B), 256, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k_evict_select<<<counted(units), kSelThreads, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long pieces = (long long)p.most * p.pieces;
    const unsigned most = (unsigned)((pieces + 255) / 256), want = 8u * sms / units + 1;
    k_evict_move<<<counted(dim3(units, most < 1 ? 1 : (most < want ? most : want))), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace ddt
