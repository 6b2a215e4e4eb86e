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
//   k_decode_finish join: a head's partials with the new token's own row,
//                     O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s;
//                   and, from the scores the split kernel left, sum_h 2^(t_h(p) - M_h) / Z_h
//                   added to the running sum of row p's attention weights.
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
    __shared__ __align__(16) float s_sum[(D == 64 ? kSets / 2 : kSets) * 4 * D];
    __shared__ long long s_row[kDecTile];
    __shared__ float s_m[HBS], s_l[HBS], s_f[HBS];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T* kp = static_cast<const T*>(p.k_pages);
    const T* vp = static_cast<const T*>(p.v_pages);
    DecodeWalk w = dec_plan<kSimtThreads>(p);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_decode_finish may be set up
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
        // ---- the segment's partial: the row sets' sums, four heads at a time, a warp's own two
        //      sets (head size 64) by a shuffle
        const long long slot = dec_unit(p, w) + blockIdx.x;
        constexpr int kLeft = D == 64 ? kSets / 2 : kSets;  // sets that go through shared memory
        const int c4 = (tid % (D / 4)) * 4, set = D == 64 ? warp : tid / (D / 4);
#pragma unroll
        for (int h4 = 0; h4 < HBS; h4 += 4) {
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = acc[h4 + h][i];
                    if (D == 64) v[i] += __shfl_xor_sync(kFull, v[i], 16);
                }
                if (D != 64 || lane < 16)
                    *reinterpret_cast<float4*>(s_sum + (set * 4 + h) * D + c4) = make_float4(v[0], v[1], v[2], v[3]);
            }
            __syncthreads();
            for (int e = tid; e < 4 * D; e += kSimtThreads) {
                float o = 0.f;
#pragma unroll
                for (int s = 0; s < kLeft; ++s) o += s_sum[s * 4 * D + e];
                if (h4 + e / D < nh) p.part_o[(slot * p.HT + h4) * D + e] = o;
            }
        }
        if (tid < nh) p.part_ml[slot * p.HT + tid] = make_float2(s_m[tid], s_bad ? kSegBadPage : s_l[tid]);
    }
}

// One head's joined softmax, by one warp.
struct HeadJoin {
    float ref, z, tn;  // reference, sum, the new row's score (log2 units)
    int err;           // a status for the request, or DDT_OK
    int ns;            // segments, from slot `first` on
    long long first;
};

template <typename Tin, int D>
__device__ __forceinline__ HeadJoin head_join(const DecodeParams& p, int lb, int hq, int lane) {
    const int l = lb / p.B, b = lb - l * p.B, g = hq / p.G, hb = (hq % p.G) / p.hbs, h = (hq % p.G) % p.hbs;
    // loads that do not wait for one another first
    const int P = p.prefix_len[b];
    const long long pre = p.pre[b], all = p.pre[p.B];
    float s = 0.f;
    if (p.k_new) {
        const Tin* q = static_cast<const Tin*>(p.q) + ((long long)lb * p.Hq + hq) * D;
        const Tin* k = static_cast<const Tin*>(p.k_new) + ((long long)lb * p.Hkv + g) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) s = fmaf(to_f32(q[e * 32 + lane]), to_f32(k[e * 32 + lane]), s);
    }
    HeadJoin j;
    j.ref = j.z = 0.f;
    j.tn = p.k_new ? warp_sum(s) * p.scale_log2 : -INFINITY;
    j.ns = 0;
    j.first = 0;
    j.err = (P < 0 || P > p.cap) ? DDT_ERR_CAPACITY : DDT_OK;
    if (j.err) return j;
    const int nt = dec_tiles(P, p.cap);
    if (nt > 0) {
        const int HH = p.Hkv * p.HB;
        const long long T = all * HH * p.L;
        const long long first = l * all * HH + pre * HH + (long long)(g * p.HB + hb) * nt;
        const int C = (int)min((long long)p.C, T), c0 = dec_owner(T, C, first);
        j.ns = dec_owner(T, C, first + nt - 1) - c0 + 1;
        j.first = (long long)lb * HH + g * p.HB + hb + c0;
    }
    const float2* ml = p.part_ml + j.first * p.HT + h;
    float m = j.tn, low = 0.f;
    for (int s = lane; s < j.ns; s += 32) {
        const float2 v = ml[(long long)s * p.HT];
        m = fmaxf(m, v.x);
        low = fminf(low, v.y);
    }
    m = warp_max(m);
    low = -warp_max(-low);
    if (low < 0.f) j.err = low == kSegTimeout ? DDT_ERR_TIMEOUT : DDT_ERR_INVALID_ARG;
    j.ref = m == -INFINITY ? 0.f : m;
    float z = 0.f;
    for (int s = lane; s < j.ns; s += 32) {
        const float2 v = ml[(long long)s * p.HT];
        z = fmaf(tc::ex2(v.x - j.ref), v.y, z);
    }
    j.z = warp_sum(z) + tc::ex2(j.tn - j.ref);
    return j;
}

// Blocks below n_join: WPH warps a head (1, or 8 where a head has many segments), O of the
// head.  The others: the weight sums of some rows of one (layer, request, kv head).
template <typename Tin, typename Tout, int D, int WPH>
__global__ void __launch_bounds__(256, 4) k_decode_finish(const DecodeParams p, unsigned n_join, int chunks) {
    constexpr int E = D / 32;
    extern __shared__ float s_x[];  // [8][D] sums of the warps of a head, or 3 floats a head of a group
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: the partials are there from here on
    if (blockIdx.x < n_join) {
        const unsigned x = WPH == 1 ? blockIdx.x * 8 + warp : blockIdx.x;
        const int lb = (int)(x / p.Hq), hq = (int)(x - (unsigned)lb * p.Hq);
        if (lb >= p.L * p.B) return;  // (WPH 1: whole warps, no barrier follows)
        const HeadJoin j = head_join<Tin, D>(p, lb, hq, lane);
        Tout* out = static_cast<Tout*>(p.o) + (long long)x * D;
        if (j.err) {
            if (WPH == 1 || warp == 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) out[e * 32 + lane] = from_f32<Tout>(0.f);
                if (lane == 0) p.status[lb % p.B] = j.err;
            }
            return;  // (WPH 8: all warps)
        }
        const int g = hq / p.G, h = (hq % p.G) % p.hbs;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        if (p.k_new && (WPH == 1 || warp == 0)) {
            const float w = tc::ex2(j.tn - j.ref);
            const Tin* v = static_cast<const Tin*>(p.v_new) + ((long long)lb * p.Hkv + g) * D;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = w * to_f32(v[e * 32 + lane]);
        }
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
        return;
    }
    const unsigned y = blockIdx.x - n_join;
    const int lbg = (int)(y / chunks), part = (int)(y - (unsigned)lbg * chunks), lb = lbg / p.Hkv, g = lbg - lb * p.Hkv;
    float* s_ref = s_x;
    float* s_inv = s_ref + p.G;
    float* s_tn = s_inv + p.G;
    const int P = p.prefix_len[lb % p.B];
    // blocks behind the unit's rows (the first also has the new token's)
    if (part && part * 1024LL >= P) return;
    int bad = 0;
    for (int h = warp; h < p.G; h += 8) {
        const HeadJoin j = head_join<Tin, D>(p, lb, g * p.G + h, lane);
        bad |= j.err;
        if (lane == 0) {
            s_ref[h] = j.ref;
            s_inv[h] = j.z > 0.f ? 1.f / j.z : 0.f;
            s_tn[h] = j.tn;
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

template <typename Tin, typename Tout, int D, int WPH>
static cudaError_t finish_launch(const DecodeParams& p, int sms, cudaStream_t st) {
    const size_t heads = (size_t)p.L * p.B * p.Hq;
    const unsigned n_join = (unsigned)(WPH == 1 ? (heads + 7) / 8 : heads), units = (unsigned)p.L * p.B * p.Hkv;
    // 2048 rows a block, so that long requests get more of them; not too many for units that may
    // be short
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
    return cudaLaunchKernelEx(&cfg, k_decode_finish<Tin, Tout, D, WPH>, p, n_join, chunks);
}
template <typename Tin, typename Tout>
static cudaError_t finish_go(const DecodeParams& p, int sms, cudaStream_t st) {
    // segments a head: C / (units) + 1 or so
    const bool many = p.C >= 12L * p.L * p.B * p.Hkv * p.HB;
    switch (p.d) {
        case 64: return many ? finish_launch<Tin, Tout, 64, 8>(p, sms, st) : finish_launch<Tin, Tout, 64, 1>(p, sms, st);
        case 128: return many ? finish_launch<Tin, Tout, 128, 8>(p, sms, st) : finish_launch<Tin, Tout, 128, 1>(p, sms, st);
    }
    return many ? finish_launch<Tin, Tout, 256, 8>(p, sms, st) : finish_launch<Tin, Tout, 256, 1>(p, sms, st);
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
    if (decode_tc_supported(d, in)) {  // bf16: persistent CTAs
        p.C = sms < kTcMaxCtas / 2 ? sms : kTcMaxCtas / 2;
        decode_layout(p, decode_tc_heads(p.G, d), kTcMaxCtas, weight != nullptr, w);
        e = launch_decode_tc(p, st);
    } else {
        p.C = 3 * sms < kSimtMaxCtas ? 3 * sms : kSimtMaxCtas;
        decode_layout(p, simt_heads(p.G), kSimtMaxCtas, weight != nullptr, w);
        e = simt_d_go<float>(p, st);
    }
    if (e != cudaSuccess) return e;
    if (in == DDT_BF16)
        return out == DDT_BF16 ? finish_go<__nv_bfloat16, __nv_bfloat16>(p, sms, st)
                               : finish_go<__nv_bfloat16, float>(p, sms, st);
    return out == DDT_BF16 ? finish_go<float, __nv_bfloat16>(p, sms, st) : finish_go<float, float>(p, sms, st);
}

}  // namespace ddt
