// logprobs.cu -- ddt_token_logprobs: log probabilities of given tokens under the target's
// logits, the entropy of their rows, and each row's most likely tokens.
//
// With x the row's logits, m the largest, w_v = (x_v - m) log2(e) / T and Z = sum_v 2^(w_v):
//   log p(t) = (w_t - log2 Z) ln 2,   H = -sum_v p_v log p_v = (log2 Z - sum_v 2^(w_v) w_v / Z) ln 2,
// so one pass that carries (m, Z, sum 2^w w) is enough; the top tokens need a second look at
// a few entries only.
//
//   k_lp_unit   persistent warps over the (row, 4096-byte unit) pairs of the rows that are
//               asked for: one pass, the next unit's 16-byte words in registers while this
//               one's are worked on.  Packed maxima and minima on the raw words, packed fp32
//               pairs for the rest: about 4.5 instructions an entry.  Each lane's largest
//               entry goes to the second kernel.
//   k_lp_join   grid B A: joins a row's units; the n-th largest of the units' largest entries
//               bounds the n-th best entry of the row from below, so only the lanes that
//               reach it are read again (somewhat over n of 2400).
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace ddt {

namespace {
constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpCtas = 2;      // CTAs an SM of the first kernel, all resident
constexpr int kLpRows = 4096;   // rows it lists
constexpr int kLpLists = 512;   // lanes read again
constexpr int kLpCand = 1024;   // entries ranked
constexpr float kLpLow = -200.f;  // 2^w is 0 from here down
}  // namespace

struct LpPartial {
    float m;  // the unit's largest logit
    float s;  // sum of 2^w; 0: nothing above -inf; NaN: a NaN or +inf logit
    float t;  // sum of 2^w w
    float pad;
};

// A unit is 4096 bytes of a row: 8 words of 16 bytes a lane, word j of lane i being word
// 32 j + i.  Units are cut from the 16-byte boundary at or before the row's first entry, so
// rows of any length and alignment are read in whole words but for their ends.
template <typename T>
struct LpUnit {
    static constexpr int VE = 16 / (int)sizeof(T);  // entries a word
    static constexpr int kEntries = 256 * VE;
    __device__ static int lead(const T* row) { return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)); }
    __device__ static int entry(int unit, int j, int lane, int lead) {
        return unit * kEntries + (j * 32 + lane) * VE - lead;
    }
};
static inline int lp_units(int V, size_t esz) {
    const int per = 4096 / (int)esz, gap = 16 / (int)esz - 1;
    return (int)(((long long)V + gap + per - 1) / per);
}
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t logprobs_ws_bytes(int B, int A, int V, int top_n) {
    // fp32 rows have twice the units of bf16 rows: the workspace covers both
    const size_t n = (size_t)B * A * lp_units(V, 4);
    return al256(n * sizeof(LpPartial)) + (top_n > 0 ? al256(n * 32 * sizeof(float)) : 0);
}

// The word at entry e of the row; entries outside [0, V) are -inf.
__device__ __forceinline__ uint4 lp_word(const __nv_bfloat16* __restrict__ row, int e, int V) {
    if (e >= 0 && e + 8 <= V) return ld_stream_u4(row + e);
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = (e + q >= 0 && e + q < V) ? (uint32_t)__bfloat16_as_ushort(row[e + q]) : 0xff80u;
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}
__device__ __forceinline__ uint4 lp_word(const float* __restrict__ row, int e, int V) {
    if (e >= 0 && e + 4 <= V) return ld_stream_u4(row + e);
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = (e + q >= 0 && e + q < V) ? __float_as_uint(row[e + q]) : 0xff800000u;
    return make_uint4(h[0], h[1], h[2], h[3]);
}
// entry q of a word
__device__ __forceinline__ float lp_at(const uint4& w, int q, const __nv_bfloat16*) {
    const uint32_t v = q < 2 ? w.x : (q < 4 ? w.y : (q < 6 ? w.z : w.w));
    return __uint_as_float((q & 1) ? (v & 0xffff0000u) : (v << 16));
}
__device__ __forceinline__ float lp_at(const uint4& w, int q, const float*) {
    return __uint_as_float(q < 1 ? w.x : (q < 2 ? w.y : (q < 3 ? w.z : w.w)));
}
// running maximum and minimum of a lane's words (NaN entries are passed over here: they turn
// the sums NaN)
struct LpRangeBf16 {
    __nv_bfloat162 hi, lo;
    __device__ __forceinline__ void init() {
        hi = __float2bfloat162_rn(-INFINITY);
        lo = __float2bfloat162_rn(INFINITY);
    }
    __device__ __forceinline__ void see(const uint4& w) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&v[i]);
            hi = __hmax2(hi, x);
            lo = __hmin2(lo, x);
        }
    }
    __device__ __forceinline__ float max() const { return fmaxf(__low2float(hi), __high2float(hi)); }
    __device__ __forceinline__ float min() const { return fminf(__low2float(lo), __high2float(lo)); }
};
struct LpRangeF32 {
    float hi, lo;
    __device__ __forceinline__ void init() {
        hi = -INFINITY;
        lo = INFINITY;
    }
    __device__ __forceinline__ void see(const uint4& w) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi = fmaxf(hi, __uint_as_float(v[i]));
            lo = fminf(lo, __uint_as_float(v[i]));
        }
    }
    __device__ __forceinline__ float max() const { return hi; }
    __device__ __forceinline__ float min() const { return lo; }
};
template <typename T>
struct LpRange;
template <>
struct LpRange<__nv_bfloat16> : LpRangeBf16 {};
template <>
struct LpRange<float> : LpRangeF32 {};

// two fp32 values in one 64-bit register, for the packed fp32 instructions
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// One unit's words -> its partial (lane 0 writes) and the lane's largest entry.
template <typename T>
__device__ __forceinline__ void lp_reduce(const uint4 (&w)[8], float s2, int lane, LpPartial* part, T* lane_max) {
    constexpr int VE = LpUnit<T>::VE;
    LpRange<T> range;
    range.init();
#pragma unroll
    for (int j = 0; j < 8; ++j) range.see(w[j]);
    const float mt = range.max();
    const float m = redux_max(mt);
    const float ref = m * s2, base = m == -INFINITY ? 0.f : m;
    // rows with masked entries (-inf or the type's lowest) or out of fp32's range once scaled
    const bool low = !(fmaf(range.min(), s2, -ref) > kLpLow && fabsf(ref) < 1e30f);
    uint64_t s[2] = {0, 0}, t[2] = {0, 0};
    float off = 0.f;
    const uint64_t k2 = pack2(s2, s2), r2 = pack2(-ref, -ref);
    if (!__any_sync(kFull, low)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < VE; q += 2) {
                const uint64_t x = pack2(lp_at(w[j], q, static_cast<const T*>(nullptr)),
                                         lp_at(w[j], q + 1, static_cast<const T*>(nullptr)));
                const uint64_t v = fma2(x, k2, r2);
                float a, b;
                unpack2(v, a, b);
                const uint64_t e = pack2(tc::ex2(a), tc::ex2(b));
                s[(q >> 1) & 1] = add2(s[(q >> 1) & 1], e);
                t[(q >> 1) & 1] = fma2(e, v, t[(q >> 1) & 1]);
            }
        // the terms took m s2 as rounded for their reference: to the exact one, 2^-24 m s2
        // away at most (its square is nothing)
        off = fmaf(m, s2, -ref);
    } else {
        // the bound keeps 0 * -inf out of t
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int q = 0; q < VE; q += 2) {
                const float a = max_nan((lp_at(w[j], q, static_cast<const T*>(nullptr)) - base) * s2, kLpLow);
                const float b = max_nan((lp_at(w[j], q + 1, static_cast<const T*>(nullptr)) - base) * s2, kLpLow);
                const uint64_t e = pack2(tc::ex2(a), tc::ex2(b));
                s[(q >> 1) & 1] = add2(s[(q >> 1) & 1], e);
                t[(q >> 1) & 1] = fma2(e, pack2(a, b), t[(q >> 1) & 1]);
            }
    }
    float s0, s1, t0, t1;
    unpack2(add2(s[0], s[1]), s0, s1);
    unpack2(add2(t[0], t[1]), t0, t1);
    const float ss = warp_sum(s0 + s1), tt = warp_sum(t0 + t1);
    const float c = 1.f - 0.6931471805599453f * off;
    if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(m, ss * c, fmaf(-off, ss, tt) * c, 0.f);
    if (lane_max) lane_max[lane] = from_f32<T>(mt);
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) k_lp_unit(const T* __restrict__ logits, int rows, int N, int V,
                                                                 int A, int nunits, float s2,
                                                                 const int32_t* __restrict__ node,
                                                                 LpPartial* __restrict__ part,
                                                                 T* __restrict__ lane_max) {
    __shared__ int s_row[kLpRows];
    __shared__ int s_n;
    const int lane = threadIdx.x & 31;
    // a walk's rows are mostly padding: the ones that are asked for are listed first (in no
    // order: the partials go to the rows' own places), so that all warps share them evenly
    const bool listed = node && rows <= kLpRows;
    if (listed) {
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < rows; i += kLpThreads) {
            const int r = node[i];
            if (r >= 0 && r < N) s_row[atomicAdd(&s_n, 1)] = i;
        }
        __syncthreads();
    }
    // rows * nunits < 2^31
    const unsigned total = (unsigned)(listed ? s_n : rows) * nunits, step = gridDim.x * kLpWarps;
    // the words of pair x, if its row is asked for; `at`: the place of its results
    auto load = [&](unsigned x, uint4 (&w)[8], unsigned& at) {
        unsigned i = x / nunits;
        const int u = (int)(x - i * nunits);
        if (listed) i = s_row[i];
        const int r = node ? node[i] : (int)(i % A);
        at = i * nunits + u;
        if (r < 0 || r >= N) return false;
        const T* row = logits + ((long long)(i / A) * N + r) * V;
        const int e0 = LpUnit<T>::entry(u, 0, lane, LpUnit<T>::lead(row));
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = lp_word(row, e0 + j * 32 * LpUnit<T>::VE, V);
        return true;
    };
    unsigned x = blockIdx.x * kLpWarps + (threadIdx.x >> 5), at = 0, at1 = 0;
    uint4 w[8];
    bool have = x < total && load(x, w, at);
    for (; x < total; x += step) {
        uint4 next[8];
        const bool more = x + step < total && load(x + step, next, at1);
        if (have) lp_reduce<T>(w, s2, lane, part + at, lane_max ? lane_max + (long long)at * 32 : nullptr);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = next[j];
        have = more;
        at = at1;
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_lp_join(const T* __restrict__ logits, int N, int V, int A, int nunits,
                                                        int top_n, float s2, float inv_t,
                                                        const int32_t* __restrict__ node,
                                                        const int32_t* __restrict__ token,
                                                        const LpPartial* __restrict__ part,
                                                        const T* __restrict__ lane_max, float* __restrict__ logprob,
                                                        float* __restrict__ entropy, int32_t* __restrict__ top_token,
                                                        float* __restrict__ top_logprob, int32_t* __restrict__ status) {
    constexpr int VE = LpUnit<T>::VE;
    __shared__ float s_m[kLpWarps], s_z[kLpWarps], s_t[kLpWarps];
    __shared__ float s_sorted[kLpWarps * 32];
    __shared__ int s_list[kLpLists];
    __shared__ float s_cv[kLpCand];
    __shared__ int s_ci[kLpCand];
    __shared__ int s_nl, s_nc;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long i = blockIdx.x;
    const int b = (int)(i / A);
    const int r = node ? node[i] : (int)(i % A), tok = token[i];
    int32_t* tt = top_token + i * top_n;
    float* tl = top_logprob + i * top_n;
    const bool outside = r >= N || (r >= 0 && tok >= V);
    if (r < 0 || outside) {  // a padding entry, or one that names no row or no token
        for (int j = tid; j < top_n; j += kLpThreads) {
            tt[j] = -1;
            tl[j] = 0.f;
        }
        if (tid == 0) {
            logprob[i] = 0.f;
            if (entropy) entropy[i] = 0.f;
            status[i] = outside ? DDT_ERR_INVALID_ARG : DDT_OK;
        }
        return;
    }
    const T* row = logits + ((long long)b * N + r) * V;
    const float xt = tok >= 0 ? to_f32(row[tok]) : 0.f;
    const float4* P = reinterpret_cast<const float4*>(part + i * nunits);
    // ---- the row's maximum, Z and sum 2^w w (a NaN sum stays NaN)
    float m = -INFINITY;
    for (int u = tid; u < nunits; u += kLpThreads) m = fmaxf(m, P[u].x);
    m = redux_max(m);
    if (lane == 0) s_m[warp] = m;
    if (tid == 0) s_nl = s_nc = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) m = fmaxf(m, s_m[w]);
    float z = 0.f, t = 0.f;
    for (int u = tid; u < nunits; u += kLpThreads) {
        const float4 p = P[u];
        if (p.y == 0.f) continue;
        const float d = fmaxf((p.x - m) * s2, kLpLow), f = tc::ex2(d);
        z = fmaf(f, p.y, z);
        t = fmaf(f, fmaf(d, p.y, p.z), t);
    }
    z = warp_sum(z);
    t = warp_sum(t);
    if (lane == 0) {
        s_z[warp] = z;
        s_t[warp] = t;
    }
    __syncthreads();
    z = t = 0.f;
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) {
        z += s_z[w];
        t += s_t[w];
    }
    if (!(z > 0.f)) {  // NaN, +inf, or nothing above -inf
        for (int j = tid; j < top_n; j += kLpThreads) {
            tt[j] = -1;
            tl[j] = NAN;
        }
        if (tid == 0) {
            logprob[i] = NAN;
            if (entropy) entropy[i] = NAN;
            status[i] = DDT_ERR_NONFINITE;
        }
        return;
    }
    const float LN2 = 0.6931471805599453f, lz = log2f(z);
    if (tid == 0) {
        logprob[i] = tok >= 0 ? (xt - m) * inv_t - lz * LN2 : 0.f;
        if (entropy) entropy[i] = (lz - t / z) * LN2;
        status[i] = DDT_OK;
    }
    if (top_n == 0) return;
    // ---- a bound from below on the row's n-th best value: the n-th largest of the units'
    //      largest entries, or of the threads' where there are few units (each of those n has
    //      an entry that reaches it)
    const T* LM = lane_max + i * nunits * 32;
    const bool by_unit = nunits >= top_n;
    float tm = -INFINITY;
    if (by_unit) {
        for (int u = tid; u < nunits; u += kLpThreads) tm = fmaxf(tm, P[u].x);
    } else {
        for (int x = tid * VE; x < nunits * 32; x += kLpThreads * VE) {
            const uint4 v = *reinterpret_cast<const uint4*>(LM + x);
#pragma unroll
            for (int q = 0; q < VE; ++q) tm = fmaxf(tm, lp_at(v, q, static_cast<const T*>(nullptr)));
        }
    }
    float sv = tm;
    int si = lane;
    warp_sort_best_first(sv, si);
    s_sorted[warp * 32 + lane] = sv;
    __syncthreads();
    float tau = -INFINITY;
    {
        int at = 0;
        float head = lane < kLpWarps ? s_sorted[lane * 32] : -INFINITY;
        for (int n = 0; n < top_n; ++n) {
            tau = redux_max(head);
            const unsigned who = __ballot_sync(kFull, head == tau);
            if (lane == __ffs(who) - 1) head = ++at < 32 ? s_sorted[lane * 32 + at] : -INFINITY;
        }
    }
    // ---- the lanes that reach it, and their entries that do
    const int lead = LpUnit<T>::lead(row);
    if (by_unit) {  // a warp looks at the lanes of one unit at a time
        for (int u = warp; u < nunits; u += kLpWarps) {
            if (!(P[u].x >= tau)) continue;
            if (to_f32(LM[u * 32 + lane]) >= tau) {
                const int at = atomicAdd(&s_nl, 1);
                if (at < kLpLists) s_list[at] = u * 32 + lane;
            }
        }
    } else if (tm >= tau) {
        for (int x = tid * VE; x < nunits * 32; x += kLpThreads * VE) {
            const uint4 v = *reinterpret_cast<const uint4*>(LM + x);
#pragma unroll
            for (int q = 0; q < VE; ++q)
                if (lp_at(v, q, static_cast<const T*>(nullptr)) >= tau) {
                    const int at = atomicAdd(&s_nl, 1);
                    if (at < kLpLists) s_list[at] = x + q;
                }
        }
    }
    __syncthreads();
    const int nl = s_nl;
    if (nl <= kLpLists)
        for (int x = tid; x < nl * 8; x += kLpThreads) {
            const int l = s_list[x >> 3];
            const int e = LpUnit<T>::entry(l >> 5, x & 7, l & 31, lead);
            const uint4 v = lp_word(row, e, V);
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const float y = lp_at(v, q, static_cast<const T*>(nullptr));
                if (y >= tau && e + q >= 0 && e + q < V) {
                    const int at = atomicAdd(&s_nc, 1);
                    if (at < kLpCand) {
                        s_cv[at] = y;
                        s_ci[at] = e + q;
                    }
                }
            }
        }
    __syncthreads();
    const VId none = vid_empty();
    float bv = none.v;
    int bi = none.id;
    if (nl > kLpLists || s_nc > kLpCand) {
        // many entries tie with the bound (a masked row, say): every warp ranks its part of
        // the whole row, and the first warp merges the warps' lists
        WarpTopK k;
        k.init(32);
        for (int e0 = warp * 32 * VE - lead; e0 < V; e0 += kLpThreads * VE) {
            const int e = e0 + lane * VE;
            const uint4 v = lp_word(row, e, V);
            float most = -INFINITY;
#pragma unroll
            for (int q = 0; q < VE; ++q) most = fmaxf(most, lp_at(v, q, static_cast<const T*>(nullptr)));
            const float last = __shfl_sync(kFull, k.v, 31);
            const int last_id = __shfl_sync(kFull, k.id, 31);
            if (__any_sync(kFull, most > last || (most == last && e < last_id)))
#pragma unroll
                for (int q = 0; q < VE; ++q) {
                    const bool in = e + q >= 0 && e + q < V;
                    k.insert(in ? lp_at(v, q, static_cast<const T*>(nullptr)) : none.v, in ? e + q : none.id);
                }
        }
        __syncthreads();
        s_cv[warp * 32 + lane] = k.v;
        s_ci[warp * 32 + lane] = k.id;
        __syncthreads();
        if (warp) return;
        bv = k.v;
        bi = k.id;
        for (int w = 1; w < kLpWarps; ++w) warp_merge_best_first(bv, bi, s_cv[w * 32 + lane], s_ci[w * 32 + lane]);
    } else {
        if (warp) return;
        const int nc = s_nc;
        for (int c0 = 0; c0 < nc; c0 += 32) {
            float cv = c0 + lane < nc ? s_cv[c0 + lane] : none.v;
            int ci = c0 + lane < nc ? s_ci[c0 + lane] : none.id;
            warp_sort_best_first(cv, ci);
            warp_merge_best_first(bv, bi, cv, ci);
        }
    }
    if (lane < top_n) {
        tt[lane] = bi;
        tl[lane] = (bv - m) * inv_t - lz * LN2;
    }
}

template <typename T>
static cudaError_t lp_go(int B, int N, int V, int A, int top_n, float temperature, const void* logits,
                         const int32_t* node, const int32_t* token, float* logprob, float* entropy,
                         int32_t* top_token, float* top_logprob, int32_t* status, void* ws, cudaStream_t st) {
    const int nunits = lp_units(V, sizeof(T)), rows = B * A;
    LpPartial* part = static_cast<LpPartial*>(ws);
    T* lane_max = top_n > 0 ? reinterpret_cast<T*>(static_cast<unsigned char*>(ws) +
                                                   al256((size_t)rows * nunits * sizeof(LpPartial)))
                            : nullptr;
    const float s2 = (float)(1.4426950408889634 / (double)temperature);
    const T* x = static_cast<const T*>(logits);
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long want = ((long long)rows * nunits + kLpWarps - 1) / kLpWarps;
    const int grid = (int)(want < (long long)kLpCtas * sms ? want : (long long)kLpCtas * sms);
    k_lp_unit<T><<<counted(grid), kLpThreads, 0, st>>>(x, rows, N, V, A, nunits, s2, node, part, lane_max);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_lp_join<T><<<counted((unsigned)rows), kLpThreads, 0, st>>>(x, N, V, A, nunits, top_n, s2,
                                                               (float)(1.0 / (double)temperature), node, token, part, lane_max,
                                                               logprob, entropy, top_token, top_logprob, status);
    return cudaGetLastError();
}

cudaError_t launch_token_logprobs(int B, int N, int V, int A, int top_n, float temperature, ddt_dtype dtype,
                                  const void* logits, const int32_t* node, const int32_t* token, float* logprob,
                                  float* entropy, int32_t* top_token, float* top_logprob, int32_t* status, void* ws,
                                  cudaStream_t st) {
    return dtype == DDT_BF16
               ? lp_go<__nv_bfloat16>(B, N, V, A, top_n, temperature, logits, node, token, logprob, entropy, top_token,
                                      top_logprob, status, ws, st)
               : lp_go<float>(B, N, V, A, top_n, temperature, logits, node, token, logprob, entropy, top_token,
                              top_logprob, status, ws, st);
}

}  // namespace ddt
