// decode.cu -- ddt_decode_attn_paged: attention of one new token a request over the paged
// prefix cache, split over the cached rows and joined.
//
// "DDTree on vLLM: candid research notes", section "Where the next step is": attention over
// paged KV blocks.  This is the round's step for a request that has no drafts: one query row
// a head instead of a tree of them, so nothing is left to share a K/V row but the G query
// heads of its kv head, and the call is bound by reading the cache once.
//
//   k_decode_tc     grid C (decode_tc.cu): the tiles of a CTA's run on the tensor cores, bf16.
//   k_decode_simt   grid C: the same on the CUDA cores, fp32.
//   k_decode_join   grid L B Hq: joins a head's partials with the new token's own row:
//                   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
//   k_decode_weight grid (L B Hkv, y): adds sum_h 2^(t_h(p) - M_h) / Z_h to the running sum
//                   of row p's attention weights, from the scores the split kernel left.
#include <math.h>

#include "decode.cuh"
#include "tc.cuh"

namespace ddt {

namespace {
constexpr int kSimtThreads = 256;
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtMaxCtas = 1024;
}  // namespace

// 16 bytes of a row as floats.
__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[4], const float*) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[8], const __nv_bfloat16*) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// Four consecutive elements as floats.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(a.x << 16);
    v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16);
    v[3] = __uint_as_float(a.y & 0xffff0000u);
}

// One tile of 128 rows at a time, three phases between barriers:
//   scores   eight lanes a row: each takes every eighth 16-byte piece of the K row and of
//            the queries (shared memory, fp32), three shuffles add up the eight
//   softmax  a warp a head: tile maximum, running reference, exponentials, sum
//   values   a thread owns four channels and every (1024 / D)-th row of the tile
template <typename T, int D, int HBS>
__global__ void __launch_bounds__(kSimtThreads) k_decode_simt(const DecodeParams p) {
    constexpr int VE = 16 / (int)sizeof(T);
    constexpr int kVec = D / (8 * VE);           // 16-byte pieces a lane takes of a row
    constexpr int kSets = kSimtThreads / (D / 4);  // row sets of the value phase
    __shared__ __align__(16) float s_q[HBS][D];
    __shared__ __align__(16) float s_p[HBS][kDecTile];
    __shared__ long long s_row[kDecTile];
    __shared__ float s_m[HBS], s_l[HBS], s_f[HBS];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T* kp = static_cast<const T*>(p.k_pages);
    const T* vp = static_cast<const T*>(p.v_pages);
    DecodeWalk w = dec_plan<kSimtThreads>(p);
    for (; w.left > 0; dec_next(p, w)) {
        const int g = w.g / p.HB, h0 = (w.g % p.HB) * HBS, nh = min(HBS, p.G - h0);
        const T* q = static_cast<const T*>(p.q) + (((long long)w.l * p.B + w.b) * p.Hq + g * p.G + h0) * D;
        __syncthreads();  // the previous segment is done with shared memory
        for (int e = tid; e < HBS * D; e += kSimtThreads) s_q[e / D][e % D] = e < nh * D ? to_f32(q[e]) : 0.f;
        if (tid < HBS) {
            s_m[tid] = -INFINITY;
            s_l[tid] = 0.f;
        }
        if (tid == 0) s_bad = 0;
        float acc[HBS][4];
#pragma unroll
        for (int h = 0; h < HBS; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][i] = 0.f;
        const int n_seg = dec_seg_tiles(w);
        for (int j = 0; j < n_seg; ++j) {
            const int y = (w.t + j) * kDecTile, n = min(kDecTile, w.P - y);
            __syncthreads();
            if (tid < kDecTile) {
                long long row = -1;
                if (tid < n) {
                    const int lp = (y + tid) / p.page_rows, in = (y + tid) % p.page_rows;
                    const int phys = p.block_table[(long long)w.b * p.max_pages + lp];
                    if (phys < 0 || phys >= p.num_pages) s_bad = 1;
                    else row = ((((long long)w.l * p.num_pages + phys) * p.Hkv + g) * p.page_rows + in) * D;
                }
                s_row[tid] = row;
            }
            __syncthreads();
            // ---- scores
#pragma unroll 2
            for (int r0 = warp * 4; r0 < kDecTile; r0 += kSimtWarps * 4) {
                const int r = r0 + (lane >> 3);
                const long long row = s_row[r];
                float kv[kVec][VE];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (row >= 0) u = ld_stream_u4(kp + row + ((lane & 7) + 8 * i) * VE);
                    unpack16(u, kv[i], static_cast<const T*>(nullptr));
                }
#pragma unroll
                for (int h = 0; h < HBS; ++h) {
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
#pragma unroll
                        for (int e = 0; e < VE; ++e) s = fmaf(kv[i][e], s_q[h][((lane & 7) + 8 * i) * VE + e], s);
                    s += __shfl_xor_sync(kFull, s, 1);
                    s += __shfl_xor_sync(kFull, s, 2);
                    s += __shfl_xor_sync(kFull, s, 4);
                    if ((lane & 7) == 0) s_p[h][r] = row >= 0 ? s * p.scale_log2 : -INFINITY;
                }
            }
            __syncthreads();
            // ---- softmax
            if (p.score) {
                float* sc = p.score + (((long long)w.l * p.B + w.b) * p.Hq + g * p.G + h0) * p.cap + y;
                for (int e = tid; e < kDecTile * nh; e += kSimtThreads)
                    if (e % kDecTile < n) sc[(long long)(e / kDecTile) * p.cap + e % kDecTile] = s_p[e / kDecTile][e % kDecTile];
                __syncthreads();
            }
            for (int h = warp; h < HBS; h += kSimtWarps) {
                float v[kDecTile / 32], mt = -INFINITY;
#pragma unroll
                for (int i = 0; i < kDecTile / 32; ++i) {
                    v[i] = s_p[h][lane + 32 * i];
                    mt = fmaxf(mt, v[i]);
                }
                mt = warp_max(mt);
                const float m0 = s_m[h], m1 = fmaxf(m0, mt);
                const float ref = m1 == -INFINITY ? 0.f : m1;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kDecTile / 32; ++i) {
                    v[i] = tc::ex2(v[i] - ref);
                    sum += v[i];
                    s_p[h][lane + 32 * i] = v[i];
                }
                sum = warp_sum(sum);
                __syncwarp();
                if (lane == 0) {
                    const float f = m0 == -INFINITY ? 0.f : tc::ex2(m0 - m1);
                    s_f[h] = f;
                    s_l[h] = s_l[h] * f + sum;
                    s_m[h] = m1;
                }
            }
            __syncthreads();
            // ---- values
#pragma unroll
            for (int h = 0; h < HBS; ++h) {
                const float f = s_f[h];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[h][i] *= f;
            }
            const int c4 = (tid % (D / 4)) * 4;
#pragma unroll 4
            for (int r = tid / (D / 4); r < n; r += kSets) {
                const long long row = s_row[r];
                float vv[4] = {0.f, 0.f, 0.f, 0.f};
                if (row >= 0) load4(vp + row + c4, vv);
#pragma unroll
                for (int h = 0; h < HBS; ++h) {
                    const float pr = s_p[h][r];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[h][i] = fmaf(pr, vv[i], acc[h][i]);
                }
            }
        }
        // ---- the segment's partial: the row sets' sums, through the query array (done with)
        const long long slot = dec_unit(p, w) + blockIdx.x;
        const int c4 = (tid % (D / 4)) * 4, set = tid / (D / 4);
        for (int s = 0; s < kSets; ++s) {
            __syncthreads();
            if (set == s) {
#pragma unroll
                for (int h = 0; h < HBS; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s_q[h][c4 + i] = acc[h][i] + (s ? s_q[h][c4 + i] : 0.f);
            }
        }
        __syncthreads();
        for (int e = tid; e < nh * D; e += kSimtThreads) p.part_o[slot * p.HT * D + e] = s_q[e / D][e % D];
        if (tid < nh) p.part_ml[slot * p.HT + tid] = make_float2(s_m[tid], s_bad ? kSegBadPage : s_l[tid]);
    }
}

template <typename Tin, typename Tout, int D>
__global__ void __launch_bounds__(D) k_decode_join(const DecodeParams p) {
    __shared__ float s_w[256 / 32 * 2];
    __shared__ float s_seg[1024];  // factors of up to 1024 segments at a time
    const int hq = blockIdx.x % p.Hq;
    const long long lb = blockIdx.x / p.Hq;
    const int b = (int)(lb % p.B);
    const int g = hq / p.G, hb = (hq % p.G) / p.hbs, h = (hq % p.G) % p.hbs;
    const int c = threadIdx.x, lane = c & 31, warp = c >> 5;
    const int P = p.prefix_len[b];
    Tout* out = static_cast<Tout*>(p.o) + (lb * p.Hq + hq) * D + c;
    float4* stat = p.stat + lb * p.Hq + hq;
    if (P < 0 || P > p.cap) {
        *out = from_f32<Tout>(0.f);
        if (c == 0) *stat = make_float4(0.f, -1.f, 0.f, 0.f);
        return;
    }
    // the new token's own row
    float tn = -INFINITY;
    if (p.k_new) {
        float s = to_f32(static_cast<const Tin*>(p.q)[(lb * p.Hq + hq) * D + c]) *
                  to_f32(static_cast<const Tin*>(p.k_new)[(lb * p.Hkv + g) * D + c]);
        s = warp_sum(s);
        if (lane == 0) s_w[warp] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) s += s_w[w];
        tn = s * p.scale_log2;
    }
    // this unit's segments: CTAs c0 .. c1
    const int HH = p.Hkv * p.HB;
    const long long unit = lb * HH + g * p.HB + hb;
    const long long all = p.pre[p.B], T = all * HH * p.L;
    const int nt = dec_tiles(P, p.cap);
    int c0 = 0, ns = 0;
    if (nt > 0) {
        const long long first = (lb / p.B) * all * HH + p.pre[b] * HH + (long long)(g * p.HB + hb) * nt;
        const int C = (int)min((long long)p.C, T);
        c0 = dec_owner(T, C, first);
        ns = dec_owner(T, C, first + nt - 1) - c0 + 1;
    }
    const float2* ml = p.part_ml + (unit + c0) * p.HT + h;
    float M = tn, lmin = 0.f;
    for (int s = c; s < ns; s += D) {
        const float2 v = ml[(long long)s * p.HT];
        M = fmaxf(M, v.x);
        lmin = fminf(lmin, v.y);
    }
    M = warp_max(M);
    lmin = -warp_max(-lmin);
    __syncthreads();
    if (lane == 0) {
        s_w[warp] = M;
        s_w[8 + warp] = lmin;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        M = fmaxf(M, s_w[w]);
        lmin = fminf(lmin, s_w[8 + w]);
    }
    if (lmin < 0.f) {
        *out = from_f32<Tout>(0.f);
        if (c == 0) {
            *stat = make_float4(0.f, -1.f, 0.f, 0.f);
            p.status[b] = lmin == kSegTimeout ? DDT_ERR_TIMEOUT : DDT_ERR_INVALID_ARG;
        }
        return;
    }
    const float ref = M == -INFINITY ? 0.f : M;
    const float wn = tc::ex2(tn - ref);
    float z = wn, acc = p.k_new ? wn * to_f32(static_cast<const Tin*>(p.v_new)[(lb * p.Hkv + g) * D + c]) : 0.f;
    const float* po = p.part_o + ((unit + c0) * p.HT + h) * D + c;
    for (int s0 = 0; s0 < ns; s0 += 1024) {
        const int n = min(1024, ns - s0);
        __syncthreads();
        for (int s = c; s < n; s += D) s_seg[s] = tc::ex2(ml[(long long)(s0 + s) * p.HT].x - ref);
        __syncthreads();
#pragma unroll 8
        for (int s = 0; s < n; ++s) {
            z = fmaf(s_seg[s], ml[(long long)(s0 + s) * p.HT].y, z);
            acc = fmaf(s_seg[s], po[(long long)(s0 + s) * p.HT * D], acc);
        }
    }
    const float inv = z > 0.f ? 1.f / z : 0.f;
    *out = from_f32<Tout>(z != z ? z : acc * inv);
    if (c == 0) *stat = make_float4(ref, inv, tn, 0.f);
}

__global__ void __launch_bounds__(256) k_decode_weight(const DecodeParams p) {
    extern __shared__ float4 s_stat[];
    const long long lbg = blockIdx.x;
    const int g = (int)(lbg % p.Hkv);
    const long long lb = lbg / p.Hkv;
    const int P = p.prefix_len[lb % p.B];
    const float4* stat = p.stat + lb * p.Hq + g * p.G;
    int bad = P < 0 || P > p.cap;
    for (int h = threadIdx.x; h < p.G; h += blockDim.x) {
        s_stat[h] = stat[h];
        bad |= s_stat[h].y < 0.f;
    }
    if (__syncthreads_or(bad)) return;
    const int n = P + (p.k_new && P < p.cap ? 1 : 0);
    const float* sc = p.score + (lb * p.Hq + (long long)g * p.G) * p.cap;
    float* wt = p.weight + lbg * p.cap;
    for (int r = blockIdx.y * blockDim.x + threadIdx.x; r < n; r += gridDim.y * blockDim.x) {
        float sum = 0.f;
        for (int h = 0; h < p.G; ++h) {
            const float4 st = s_stat[h];
            const float t = r < P ? sc[(long long)h * p.cap + r] : st.z;
            sum = fmaf(tc::ex2(t - st.x), st.y, sum);
        }
        wt[r] += sum;
    }
}

// ------------------------------------------------------------------------------ host
constexpr int kTcMaxCtas = 256;  // bounds the SM count from above
static int simt_heads(int G) { return G <= 4 ? 4 : (G <= 8 ? 8 : 16); }

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// fills the workspace pointers; returns the bytes
static size_t decode_layout(DecodeParams& p, int hbs, int ctas, bool weight, unsigned char* ws) {
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
    p.stat = reinterpret_cast<float4*>(take((size_t)p.L * p.B * p.Hq * sizeof(float4)));
    p.part_o = reinterpret_cast<float*>(take(slots * p.HT * p.d * sizeof(float)));
    p.score = weight ? reinterpret_cast<float*>(take(units * p.cap * p.G * sizeof(float))) : nullptr;
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

template <typename T, int D, int HBS>
static cudaError_t simt_go(DecodeParams& p, cudaStream_t st) {
    k_decode_simt<T, D, HBS><<<counted(p.C), kSimtThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, int D>
static cudaError_t simt_heads_go(DecodeParams& p, cudaStream_t st) {
    return p.hbs == 4 ? simt_go<T, D, 4>(p, st) : (p.hbs == 8 ? simt_go<T, D, 8>(p, st) : simt_go<T, D, 16>(p, st));
}
template <typename T>
static cudaError_t simt_d_go(DecodeParams& p, cudaStream_t st) {
    return p.d == 64 ? simt_heads_go<T, 64>(p, st)
                     : (p.d == 128 ? simt_heads_go<T, 128>(p, st) : simt_heads_go<T, 256>(p, st));
}

template <typename Tin, typename Tout>
static cudaError_t join_go(const DecodeParams& p, cudaStream_t st) {
    const unsigned n = counted((unsigned)p.L * p.B * p.Hq);
    if (p.d == 64) k_decode_join<Tin, Tout, 64><<<n, 64, 0, st>>>(p);
    else if (p.d == 128) k_decode_join<Tin, Tout, 128><<<n, 128, 0, st>>>(p);
    else k_decode_join<Tin, Tout, 256><<<n, 256, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_decode(int L, int B, int Hq, int Hkv, int d, const AttnPaging& pg, ddt_dtype in, ddt_dtype out,
                          const void* q, const void* k_new, const void* v_new, const void* k_pages,
                          const void* v_pages, const int32_t* prefix_len, float scale, void* o, float* weight,
                          int32_t* status, void* ws, cudaStream_t st) {
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
    p.scale_log2 = scale * 1.4426950408889634f;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    unsigned char* w = static_cast<unsigned char*>(ws);
    cudaError_t e;
    if (decode_tc_supported(d, in)) {  // bf16: one persistent CTA an SM
        p.C = sms < kTcMaxCtas ? sms : kTcMaxCtas;
        decode_layout(p, decode_tc_heads(p.G, d), kTcMaxCtas, weight != nullptr, w);
        e = launch_decode_tc(p, st);
    } else {
        p.C = 3 * sms < kSimtMaxCtas ? 3 * sms : kSimtMaxCtas;
        decode_layout(p, simt_heads(p.G), kSimtMaxCtas, weight != nullptr, w);
        e = simt_d_go<float>(p, st);
    }
    if (e != cudaSuccess) return e;
    if (in == DDT_BF16) e = out == DDT_BF16 ? join_go<__nv_bfloat16, __nv_bfloat16>(p, st) : join_go<__nv_bfloat16, float>(p, st);
    else e = out == DDT_BF16 ? join_go<float, __nv_bfloat16>(p, st) : join_go<float, float>(p, st);
    if (e != cudaSuccess || !weight) return e;
    const unsigned units = (unsigned)L * B * Hkv;
    const unsigned most = (p.cap + 255) / 256, want = (unsigned)sms * 8 / units + 1;
    k_decode_weight<<<counted(dim3(units, most < want ? most : want)), 256, p.G * sizeof(float4), st>>>(p);
    return cudaGetLastError();
}

}  // namespace ddt
