// quant.cu -- a paged key-value cache held in 8 bits: ddt_append_paged_quant, which quantises rows
// as they are written, and ddt_read_paged_quant, which reads them back.
//
// A row's channels are e4m3 codes; a block of S tokens of one head shares a power of two as its
// scale, one byte: value = code * 2^(byte - 127), and byte 0 marks a block without finite channels but zeros.
// A power of two because e4m3 is a floating-point format: a finer scale would move the rounding
// steps, not narrow them (a value keeps 4 significant bits wherever it lies between 2^-6 and 448 of
// its block's unit), and rescaling a block that a later, larger row joins is exact but for codes
// that fall below 2^-6.
// The byte is that of the smallest e in [-100, 120] with max |x| <= 448 * 2^e over the block's rows
// so far, so nothing saturates; it never falls while the block holds rows.
//
// Both are bound by HBM once their instructions are few.  Append: 6 prompts of 2001 to 16384 rows, 8 heads of 128 (299
// MB in and out), 48 us, 6.2 TB/s; its maxima on packed bf16 pairs, its codes four a word, the values in between as they
// came (as floats, with divisions for the places, it took 190 us).  Read back: 32 requests of 1K to 32K rows, 4 heads of
// 256 (2.89 GB), 432 us, 6.7 TB/s, 98 % of the copy rate; 482 with a division for each vector's page, 490 with stores
// that fill half sectors.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 8;  // vectors of 8 channels a lane has in flight

struct AppendArgs {
    int B, N, A, Hkv, S;
    int page_rows, num_pages, max_pages, cap;
    int wpi;          // warps an item (a block's K or V rows of one head)
    int run, groups;  // blocks a CTA; CTAs that share a block's items
    int advance, solo;  // solo: one CTA has all of a request
    int checked;      // a kernel of its own looks at the pages (and advances prefix_len)
    const void* k;
    const void* v;
    const int32_t* node;   // or null
    const int32_t* count;
    const int32_t* table;
    int32_t* prefix_len;
    unsigned char* kp;
    unsigned char* vp;
    unsigned char* ks;
    unsigned char* vs;
    int32_t* status;
};

// 8 channels as they lie in memory, read once
template <typename T>
struct Vec8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ld_stream_u4(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    // the largest |x| as bits, of bf16 vectors in halves of 16 bits (integers order as the values do)
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            if (sizeof(T) == 4)
                m = max(max(max(m, w[i].x & 0x7fffffffu), max(w[i].y & 0x7fffffffu, w[i].z & 0x7fffffffu)), w[i].w & 0x7fffffffu);
            else
                m = __vimax3_u16x2(__vimax3_u16x2(m, w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu), w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu);
        }
        return m;
    }
    __device__ __forceinline__ float get(int i) const {
        if (sizeof(T) == 4) {
            const uint4& x = w[i / 4 % (sizeof(T) / 2)];
            return __uint_as_float(i % 4 == 0 ? x.x : (i % 4 == 1 ? x.y : (i % 4 == 2 ? x.z : x.w)));
        }
        const uint32_t x = i / 2 == 0 ? w[0].x : (i / 2 == 1 ? w[0].y : (i / 2 == 2 ? w[0].z : w[0].w));
        return __uint_as_float(i % 2 ? x & 0xffff0000u : x << 16);
    }
    __device__ __forceinline__ uint2 codes(float inv) const {
        const F2 k = f2(inv, inv);
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = f2_get(f2(get(4 * i), get(4 * i + 1)) * k), y = f2_get(f2(get(4 * i + 2), get(4 * i + 3)) * k);
            c[i] = e4m3x4(x.x, x.y, y.x, y.y);
        }
        return make_uint2(c[0], c[1]);
    }
    // the same where an infinity may be among them: it becomes NaN
    __device__ __forceinline__ uint2 codes_any(float inv) const {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = get(2 * i), y = get(2 * i + 1);
            c[i] = e4m3x2(fmaf(x, 0.f, x) * inv, fmaf(y, 0.f, y) * inv);
        }
        return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
    }
};

}  // namespace

// All threads of a CTA: the request as a whole.  Nothing of it is written unless all of it can be.
__device__ __forceinline__ int append_check(const AppendArgs& a, int b, int P, int n) {
    int err = P < 0 || P > a.cap ? DDT_ERR_CAPACITY : DDT_OK;
    if (!err && (n < 0 || n > a.A)) err = DDT_ERR_INVALID_ARG;
    if (!err && n > a.cap - P) err = DDT_ERR_CAPACITY;
    const int32_t* table = a.table + (long long)b * a.max_pages;
    int bad = 0;
    if (!err && n > 0) {
        const int p1 = (P + n - 1) / a.page_rows;
        for (int p = P / a.page_rows + threadIdx.x; p <= p1; p += kThreads) bad |= table[p] < 0 || table[p] >= a.num_pages;
        if (a.node)
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const int r = a.node[(long long)b * a.A + i];
                bad |= r < 0 || r >= a.N;
            }
    }
    return __syncthreads_or(bad) ? DDT_ERR_INVALID_ARG : err;
}

// grid B: the check by itself, where every CTA of the next kernel would look at many pages; and prefix_len
__global__ void __launch_bounds__(kThreads) k_append_check(const AppendArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x, P = a.prefix_len[b], n = a.count[b], err = append_check(a, b, P, n);
    if (threadIdx.x == 0) {
        a.status[b] = err;
        if (a.advance && !err) a.prefix_len[b] = P + n;
    }
}

// grid (runs of blocks x item groups, 1, L * B).  A CTA takes a few blocks of one request and layer, one after
// another; wpi of its warps an item (a block's K or V rows of one head).  Up to kChunk vectors a lane stay in registers
// between the maximum and the codes; items of more (blocks of 128 rows of 256 channels, a few rows of many requests) are
// read twice.
template <typename T, int D, bool NODE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) k_append_quant(const AppendArgs a) {
    __shared__ float s_max[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.z % a.B, l = blockIdx.z / a.B, group = blockIdx.x % a.groups;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_append_advance may be set up
    if (a.checked) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (a.status[b] != DDT_OK) return;
    }
    const int n = a.count[b], P = a.prefix_len[b] - (a.checked && a.advance ? n : 0);
    int first = P / a.S + blockIdx.x / a.groups * a.run;  // block
    // a CTA without rows: none, or none so far behind the prefix (which is for others to judge)
    if ((blockIdx.x > 0 || l > 0) && (n <= 0 || (long long)first * a.S >= (long long)P + n)) return;
    const int err = a.checked ? DDT_OK : append_check(a, b, P, n);
    if (!a.checked && l == 0 && blockIdx.x == 0 && tid == 0) {
        a.status[b] = err;
        if (a.solo && a.advance && !err) a.prefix_len[b] = P + n;
    }
    if (err || n == 0) return;  // (without rows no page has been looked at)
    const int32_t* table = a.table + (long long)b * a.max_pages;
    const int item = group * (kWarps / a.wpi) + warp / a.wpi, part = warp % a.wpi;
    const bool real = item < 2 * a.Hkv;
    const int isv = item & 1, g = min(item >> 1, a.Hkv - 1);
    // vector e of the item: 8 channels of its row e / (d / 8); a lane's are the same ones of every row
    constexpr int shift = D == 64 ? 3 : (D == 128 ? 4 : 5);
    const int step = a.wpi * 32, e0 = part * 32 + lane, ch = (e0 & ((1 << shift) - 1)) * 8;
    const T* src = static_cast<const T*>(isv ? a.v : a.k) + ((long long)l * a.B + b) * a.N * a.Hkv * D + (long long)g * D + ch;
    const int pitch = a.Hkv * D;  // (below 2^23)
    const long long hop = (long long)(step >> shift) * pitch;
    // the blocks' page and the row in it
    int lp = first * a.S / a.page_rows, in = first * a.S - lp * a.page_rows;

    for (int turn = 0; turn < a.run && first * a.S < P + n; ++turn, ++first, in += a.S) {
        if (in >= a.page_rows) {
            in = 0;
            ++lp;
        }
        const int r0 = first * a.S, lo = max(P - r0, 0), hi = min(P + n - r0, a.S);  // new rows [lo, hi) of the block
        const int count = real ? (hi - lo) << shift : 0;  // the item's vectors
        Vec8<T> x[kChunk];
        auto load = [&](int e) {  // vectors e, e + step, ..
            const int j = r0 + lo - P + (e >> shift);
            const T* at = src + (long long)j * pitch;
            const int32_t* node = a.node + (long long)b * a.A + j;
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                x[i].zero();
                if (e + i * step < count) x[i].load(NODE ? src + (long long)node[i * (step >> shift)] * pitch : at);
                at += hop;
            }
        };
        uint32_t most = 0;
        for (int e = e0; e < count; e += kChunk * step) {
            load(e);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) most = x[i].top(most);
        }
        const long long plane = ((long long)l * a.num_pages + table[lp]) * a.Hkv + g;
        unsigned char* page = (isv ? a.vp : a.kp) + (plane * a.page_rows + in) * D;
        unsigned char* byte = (isv ? a.vs : a.ks) + plane * (a.page_rows / a.S) + in / a.S;
        const int old = real && lo > 0 ? *byte : 0;
        if (sizeof(T) == 2) most = max(most & 0xffffu, most >> 16) << 16;
        most = __reduce_max_sync(kFull, most);
        float m = __uint_as_float(most);
        const bool finite = most < 0x7f800000u;
        if (!finite) {  // infinities or NaN: the largest of the others
            m = 0.f;
            for (int e = e0; e < count; e += kChunk * step) {
                load(e);
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k) m = fabsf(x[i].get(k)) < INFINITY ? fmaxf(m, fabsf(x[i].get(k))) : m;
            }
            __syncwarp();
            m = warp_max(m);
        }
        if (a.wpi > 1) {
            if (lane == 0) s_max[turn & 1][warp] = m;
            __syncthreads();
            for (int i = warp / a.wpi * a.wpi, k = 0; k < a.wpi; ++k) m = fmaxf(m, s_max[turn & 1][i + k]);
        }
        if (!real) continue;
        const int now = max(old, scale_byte(m));
        if (part == 0 && lane == 0) *byte = (unsigned char)now;
        const float inv = now ? scale_of(254 - now) : 0.f;
        for (int e = e0; e < count; e += kChunk * step) {
            if (count > kChunk * step) load(e);
            unsigned char* to = page + (lo * D + (e >> shift) * D + ch);
            const int rows = (step >> shift) * D;
            if (finite) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    if (e + i * step < count) *reinterpret_cast<uint2*>(to + i * rows) = x[i].codes(inv);
            } else {
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    if (e + i * step < count) *reinterpret_cast<uint2*>(to + i * rows) = x[i].codes_any(inv);
            }
        }
        if (old && now > old) {  // the rows that the block had, under its new scale
            const float f = scale_of(max(127 + old - now, 0));
            for (int e = part * 32 + lane; e < lo << shift; e += a.wpi * 32) {
                uint2* at = reinterpret_cast<uint2*>(page + e * 8);
                const uint2 c = *at;
                float v[8];
                values8(c, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= f;
                *at = make_uint2(e4m3x2(v[0], v[1]) | e4m3x2(v[2], v[3]) << 16, e4m3x2(v[4], v[5]) | e4m3x2(v[6], v[7]) << 16);
            }
        }
    }
}

// prefix_len += count, where the rows were written (launched ahead; waits for them)
__global__ void k_append_advance(int B, const int32_t* __restrict__ count, const int32_t* status, int32_t* prefix_len) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B && status[b] == DDT_OK) prefix_len[b] += count[b];
}

template <typename T, int D>
static cudaError_t append_d_go(const cudaLaunchConfig_t& cfg, const AppendArgs& a) {
    return a.node ? cudaLaunchKernelEx(&cfg, k_append_quant<T, D, true>, a) : cudaLaunchKernelEx(&cfg, k_append_quant<T, D, false>, a);
}
template <typename T>
static cudaError_t append_go(int d, const cudaLaunchConfig_t& cfg, const AppendArgs& a) {
    return d == 64 ? append_d_go<T, 64>(cfg, a) : (d == 128 ? append_d_go<T, 128>(cfg, a) : append_d_go<T, 256>(cfg, a));
}

cudaError_t launch_append_quant(int L, int B, int N, int A, int Hkv, int d, int S, const AttnPaging& pg, ddt_dtype in,
                                const void* k, const void* v, const int32_t* node, const int32_t* count,
                                int32_t* prefix_len, int advance, void* kp, void* vp, uint8_t* ks, uint8_t* vs,
                                int32_t* status, cudaStream_t st) {
    AppendArgs a{};
    a.B = B;
    a.N = N;
    a.A = A;
    a.Hkv = Hkv;
    a.S = S;
    a.page_rows = pg.page_rows;
    a.num_pages = pg.num_pages;
    a.max_pages = pg.max_pages;
    a.cap = pg.page_rows * pg.max_pages;
    a.k = k;
    a.v = v;
    a.node = node;
    a.count = count;
    a.table = pg.block_table;
    a.prefix_len = prefix_len;
    a.advance = advance;
    a.kp = static_cast<unsigned char*>(kp);
    a.vp = static_cast<unsigned char*>(vp);
    a.ks = ks;
    a.vs = vs;
    a.status = status;
    const int vectors = (S < A ? S : A) * d / 256;  // a lane of one warp has this many of an item at most
    a.wpi = 1;
    // A few rows of many requests: one warp an item, which reads up to 16 vectors twice, from L1 the second time (blocks of 16 rows of
    // 256, bf16, by two warps and by one: 1 to 16 rows, 128 units 4.2 and 6.0 us, 512 6.9 and 7.8, 1024 10.0 and 9.4, 8192 51 and
    // 35; 1 to 32 rows, 1024 units 12.8 and 11.7, 8192 75 and 56; with 1 to 5 rows one is never slower)
    const bool few = A <= 32 && (long)L * B * Hkv >= 1024;
    while (a.wpi < kWarps && vectors > (few ? 2 : 1) * kChunk * a.wpi) a.wpi *= 2;
    const int blocks = (int)(((long long)A + S - 2) / S + 1);  // that a request's rows may fall into
    const int per = kWarps / a.wpi;
    a.groups = (2 * Hkv + per - 1) / per;
    a.solo = L == 1 && blocks == 1 && a.groups == 1;
    a.run = blocks > 64 ? 4 : 1;
    a.checked = (A + pg.page_rows - 1) / pg.page_rows > kThreads;
    if (a.checked) {
        k_append_check<<<counted(dim3(B)), kThreads, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at{};  // set up while the kernel before ends
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = counted(dim3((unsigned)((long long)(blocks + a.run - 1) / a.run * a.groups), 1, L * B));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = a.checked ? 1 : 0;
    cudaError_t e = in == DDT_BF16 ? append_go<__nv_bfloat16>(d, cfg, a) : append_go<float>(d, cfg, a);
    if (e != cudaSuccess || !advance || a.solo || a.checked) return e;
    cfg.gridDim = dim3(counted((unsigned)(B + 127) / 128));
    cfg.blockDim = dim3(128);
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_append_advance, B, count, (const int32_t*)status, prefix_len);
}

// a thread a request
__global__ void k_chain_status(int n, int B, const int32_t* __restrict__ status, const int32_t* __restrict__ length, int32_t* length_out,
                               int32_t* status_out) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= B) return;
    int s = DDT_OK;
    for (int i = n - 1; i >= 0; --i) {
        const int x = status[(long long)i * B + b];
        s = x != DDT_OK ? x : s;
    }
    if (length) length_out[b] = s == DDT_OK ? length[b] : -1;
    if (status_out) status_out[b] = s;
}

cudaError_t launch_chain_status(int n, int B, const int32_t* status, const int32_t* length, int32_t* length_out,
                                int32_t* status_out, cudaStream_t st) {
    k_chain_status<<<counted(dim3((unsigned)(((long long)B + 127) / 128))), 128, 0, st>>>(n, B, status, length, length_out, status_out);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------ read back
namespace {
struct ReadArgs {
    int B, Hkv, Pcap;
    int page_rows, num_pages, max_pages, cap;
    const int32_t* table;
    const int32_t* prefix_len;
    const unsigned char* kp;
    const unsigned char* vp;
    const unsigned char* ks;
    const unsigned char* vs;
    void* ko;
    void* vo;
    int32_t* status;
    int turns, block_shift;
    int hop_pages, hop_rows;  // a thread's next vector, in pages and rows
};
constexpr int kReadVecs = 4;   // 16 codes each, in flight a thread
}  // namespace

// grid (row chunks, 2 * Hkv, L * B): `turns` steps of kReadVecs * kThreads * 16 codes of one head's K or V a CTA.
// (The grid goes by the table's rows; CTAs behind a request's own take a few hundred cycles each, which larger ones
// make rarer.)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_read_quant(const ReadArgs a) {
    const int tid = threadIdx.x, b = blockIdx.z % a.B, l = blockIdx.z / a.B, g = blockIdx.y >> 1, isv = blockIdx.y & 1;
    const int P = a.prefix_len[b];
    const bool fits = P >= 0 && P <= a.cap && P <= a.Pcap;
    const int32_t* table = a.table + (long long)b * a.max_pages;
    if (l == 0 && blockIdx.x == 0 && blockIdx.y == 0) {  // this CTA tells of the whole request
        int bad = 0;
        if (fits)
            for (int p = tid; (long long)p * a.page_rows < P; p += kThreads) bad |= table[p] < 0 || table[p] >= a.num_pages;
        bad = __syncthreads_or(bad);
        if (tid == 0) a.status[b] = !fits ? DDT_ERR_CAPACITY : (bad ? DDT_ERR_INVALID_ARG : DDT_OK);
    }
    constexpr int vpr = D / 16, hop = kThreads / vpr, rows = kReadVecs * hop;  // vectors a row; rows apart are a thread's vectors
    int y = blockIdx.x * a.turns * rows + tid / vpr;
    if (!fits || y - tid / vpr >= P) return;
    const int ch = tid % vpr * 16;
    const unsigned char* pages = (isv ? a.vp : a.kp) + ((long long)l * a.num_pages * a.Hkv + g) * a.page_rows * D + ch;
    const unsigned char* scales = (isv ? a.vs : a.ks) + ((long long)l * a.num_pages * a.Hkv + g) * (a.page_rows >> a.block_shift);
    const int page_pitch = a.Hkv * a.page_rows, scale_pitch = a.Hkv * (a.page_rows >> a.block_shift);
    T* out = static_cast<T*>(isv ? a.vo : a.ko) + ((((long long)l * a.B + b) * a.Hkv + g) * a.Pcap + y) * D + ch;
    int lp = y / a.page_rows, r = y - lp * a.page_rows;
    for (int turn = 0; turn < a.turns && y - tid / vpr < P; ++turn) {
        uint4 c[kReadVecs];
        float f[kReadVecs];
        bool there[kReadVecs];
#pragma unroll
        for (int i = 0; i < kReadVecs; ++i, y += hop) {
            const int phys = y < P ? table[lp] : -1;
            there[i] = phys >= 0 && phys < a.num_pages;
            c[i] = make_uint4(0, 0, 0, 0);
            f[i] = 0.f;
            if (there[i]) {
                c[i] = ld_stream_u4(pages + ((long long)phys * page_pitch + r) * D);
                f[i] = scale_of(scales[(long long)phys * scale_pitch + (r >> a.block_shift)]);
            }
            lp += a.hop_pages;
            r += a.hop_rows;
            if (r >= a.page_rows) {
                r -= a.page_rows;
                ++lp;
            }
        }
#pragma unroll
        for (int i = 0; i < kReadVecs; ++i) {
            // Lanes in twos (fp32: fours), which share a row, exchange words so that each store of theirs fills 32 (64)
            // consecutive bytes: word w of lane x goes to lane w, as its word x.
            constexpr int X = sizeof(T) / 2;  // 16 bytes of output a word of X, in 8 / X codes
            uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            const int me = tid & (2 * X - 1);
            if constexpr (X == 1) {  // words of 8 codes: (w0 w1), (w2 w3)
                const uint32_t s0 = me ? w[0] : w[2], s1 = me ? w[1] : w[3];
                const uint32_t r0 = __shfl_xor_sync(kFull, s0, 1), r1 = __shfl_xor_sync(kFull, s1, 1);
                if (me) w[0] = r0, w[1] = r1;
                else w[2] = r0, w[3] = r1;
            } else {
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const uint32_t r = __shfl_xor_sync(kFull, me & 1 ? w[k] : w[k + 1], 1);
                    if (me & 1) w[k] = r;
                    else w[k + 1] = r;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t r = __shfl_xor_sync(kFull, me & 2 ? w[k] : w[k + 2], 2);
                    if (me & 2) w[k] = r;
                    else w[k + 2] = r;
                }
            }
            T* to = out + i * hop * D - me * 16 + me * (16 / (int)sizeof(T));
            if (!there[i]) continue;
#pragma unroll
            for (int x = 0; x < 2 * X; ++x) {
                uint32_t z[4];
                if constexpr (X == 1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = e4m3_values(w[2 * x + k / 2] >> (k % 2 * 16) & 0xffffu);
                        const float2 p = f2_get(f2(v.x, v.y) * f2(f[i], f[i]));
                        const __nv_bfloat162 q = __floats2bfloat162_rn(p.x, p.y);
                        z[k] = *reinterpret_cast<const uint32_t*>(&q);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 v = e4m3_values(w[x] >> (k * 16) & 0xffffu);
                        z[2 * k] = __float_as_uint(v.x * f[i]);
                        z[2 * k + 1] = __float_as_uint(v.y * f[i]);
                    }
                }
                *reinterpret_cast<uint4*>(to + x * 16) = make_uint4(z[0], z[1], z[2], z[3]);
            }
        }
        out += (long long)kReadVecs * hop * D;
    }
}

template <typename T>
static void read_go(int d, dim3 grid, const ReadArgs& a, cudaStream_t st) {
    if (d == 64) k_read_quant<T, 64><<<grid, kThreads, 0, st>>>(a);
    else if (d == 128) k_read_quant<T, 128><<<grid, kThreads, 0, st>>>(a);
    else k_read_quant<T, 256><<<grid, kThreads, 0, st>>>(a);
}

cudaError_t launch_read_quant(int L, int B, int Hkv, int d, int S, int Pcap, const AttnPaging& pg, ddt_dtype out,
                              const void* kp, const void* vp, const uint8_t* ks, const uint8_t* vs,
                              const int32_t* prefix_len, void* ko, void* vo, int32_t* status, cudaStream_t st) {
    ReadArgs a{B, Hkv, Pcap, pg.page_rows, pg.num_pages, pg.max_pages, pg.page_rows * pg.max_pages, pg.block_table, prefix_len,
               static_cast<const unsigned char*>(kp), static_cast<const unsigned char*>(vp), ks, vs, ko, vo, status};
    const int rows = kReadVecs * kThreads / (d / 16), most = Pcap < a.cap ? Pcap : a.cap;
    const long long steps = (most + rows - 1) / rows;
    a.turns = steps * 2 * Hkv * L * B > 16384 ? 4 : 1;  // 20 or more an SM's resident CTA
    const dim3 grid((unsigned)((steps + a.turns - 1) / a.turns), 2 * Hkv, L * B);
    while ((1 << a.block_shift) < S) ++a.block_shift;
    a.hop_pages = kThreads / (d / 16) / pg.page_rows;
    a.hop_rows = kThreads / (d / 16) % pg.page_rows;
    if (out == DDT_BF16) read_go<__nv_bfloat16>(d, counted(grid), a, st);
    else read_go<float>(d, counted(grid), a, st);
    return cudaGetLastError();
}

}  // namespace ddt
