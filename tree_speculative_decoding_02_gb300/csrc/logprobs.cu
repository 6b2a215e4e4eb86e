// logprobs.cu -- ddt_token_logprobs: log probabilities of given tokens under the target's
// logits, the entropy of their rows, and each row's most likely tokens.
//
// With x the row's logits, m their maximum, u_v = (x_v - m) / T and Z = sum_v e^(u_v):
//   log p(t) = u_t - log Z,    H = -sum_v p_v log p_v = log Z - sum_v e^(u_v) u_v / Z,
// so one pass that carries (m, Z, sum e^u u) is enough; the top tokens need a second look at
// a few entries only.
//
//   k_lp_unit   grid (B A, units / 8): one pass over the rows that are asked for.  A warp
//               reduces 2048 entries to (m, sum 2^w, sum 2^w w), w = (x - m) log2(e) / T, in
//               fp32, and leaves each lane's largest entry for the second kernel.
//   k_lp_join   grid B A: joins a row's units in fp64; the n-th largest of the threads'
//               largest lane entries bounds the n-th best entry of the row from below, so
//               only the lanes that reach it are read again (about n of 2400).
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace ddt {

namespace {
constexpr int kLpUnit = 2048;
constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpLists = 512;   // lanes read again
constexpr int kLpCand = 1024;   // entries ranked
constexpr int kLpGap = 7;       // entries an aligned start may lie before the row's
}  // namespace

struct LpPartial {
    float m;  // largest logit of the unit (-inf: none)
    float s;  // sum of 2^w; -1: a NaN or +inf logit
    float t;  // sum of 2^w w
    float pad;
};

static inline int lp_units(int V) { return (V + kLpGap + kLpUnit - 1) / kLpUnit; }
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t logprobs_ws_bytes(int B, int A, int V, int top_n) {
    const size_t n = (size_t)B * A * lp_units(V);
    return al256(n * sizeof(LpPartial)) + (top_n > 0 ? al256(n * 32 * sizeof(float)) : 0);
}

// Row r's first entry sits `lead` entries behind a 16-byte boundary: units are cut from
// that boundary, so rows of any length are read in whole 16-byte words but for their ends.
template <typename T>
__device__ __forceinline__ int row_lead(const T* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// Eight consecutive entries e .. e + 7 of the row (entries outside [0, V): -inf).
__device__ __forceinline__ void entries8(const __nv_bfloat16* __restrict__ row, int e, int V, float (&v)[8]) {
    if (e >= 0 && e + 8 <= V) {
        load8_stream(row + e, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = (e + q >= 0 && e + q < V) ? to_f32(row[e + q]) : -INFINITY;
    }
}
__device__ __forceinline__ void entries8(const float* __restrict__ row, int e, int V, float (&v)[8]) {
    if (e >= 0 && e + 8 <= V) {
        load8_stream(row + e, v);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = (e + q >= 0 && e + q < V) ? row[e + q] : -INFINITY;
    }
}

__device__ __forceinline__ int lp_node(const int32_t* node, long long i, int a) { return node ? node[i] : a; }

template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_lp_unit(const T* __restrict__ logits, int N, int V, int A, int nunits,
                                                        float s2, const int32_t* __restrict__ node,
                                                        LpPartial* __restrict__ part, float* __restrict__ lane_max) {
    const long long i = blockIdx.x;
    const int b = (int)(i / A), lane = threadIdx.x & 31;
    const int u = blockIdx.y * kLpWarps + (threadIdx.x >> 5);
    const int r = lp_node(node, i, (int)(i % A));
    if (r < 0 || r >= N || u >= nunits) return;
    const T* row = logits + ((long long)b * N + r) * V;
    const int e0 = u * kLpUnit - row_lead(row) + lane * 8;
    float v[8][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) entries8(row, e0 + j * 256, V, v[j]);
    float mt = -INFINITY;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            bad |= !(v[j][q] < INFINITY);
            mt = fmaxf(mt, v[j][q]);
        }
    const float m = warp_max(mt);
    const float ref = m == -INFINITY ? 0.f : m;
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float sj = 0.f, tj = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            // a term below 2^-200 is 0 either way; the bound keeps 0 * -inf out of t
            const float w = fmaxf((v[j][q] - ref) * s2, -200.f);
            const float e = tc::ex2(w);
            sj += e;
            tj = fmaf(e, w, tj);
        }
        s += sj;
        t += tj;
    }
    s = warp_sum(s);
    t = warp_sum(t);
    bad = __any_sync(kFull, bad);
    if (lane == 0) part[i * nunits + u] = LpPartial{m, bad ? -1.f : s, t, 0.f};
    if (lane_max) lane_max[(i * nunits + u) * 32 + lane] = mt;
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_lp_join(const T* __restrict__ logits, int N, int V, int A, int nunits,
                                                        int top_n, float s2, double inv_t,
                                                        const int32_t* __restrict__ node,
                                                        const int32_t* __restrict__ token,
                                                        const LpPartial* __restrict__ part,
                                                        const float* __restrict__ lane_max,
                                                        float* __restrict__ logprob, float* __restrict__ entropy,
                                                        int32_t* __restrict__ top_token,
                                                        float* __restrict__ top_logprob, int32_t* __restrict__ status) {
    __shared__ double s_z[kLpWarps], s_t[kLpWarps];
    __shared__ float s_m[kLpWarps];
    __shared__ float s_sorted[kLpWarps * 32];
    __shared__ int s_list[kLpLists];
    __shared__ float s_cv[kLpCand];
    __shared__ int s_ci[kLpCand];
    __shared__ int s_nl, s_nc;
    __shared__ double s_lse;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long i = blockIdx.x;
    const int b = (int)(i / A);
    const int r = lp_node(node, i, (int)(i % A)), tok = token[i];
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
    const LpPartial* P = part + i * nunits;
    // ---- the row's maximum, Z and sum 2^w w
    float m = -INFINITY;
    int bad = 0;
    for (int u = tid; u < nunits; u += kLpThreads) {
        m = fmaxf(m, P[u].m);
        bad |= P[u].s < 0.f;
    }
    m = warp_max(m);
    if (lane == 0) s_m[warp] = m;
    if (tid == 0) s_nl = s_nc = 0;
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) m = fmaxf(m, s_m[w]);
    bad |= m == -INFINITY;
    if (bad) {
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
    double z = 0.0, t = 0.0;
    for (int u = tid; u < nunits; u += kLpThreads) {
        const LpPartial x = P[u];
        if (!(x.s > 0.f)) continue;
        const float d = fmaxf((x.m - m) * s2, -200.f);
        const double f = (double)tc::ex2(d);
        z += f * (double)x.s;
        t += f * ((double)x.t + (double)d * (double)x.s);
    }
    z = warp_sum(z);
    t = warp_sum(t);
    if (lane == 0) {
        s_z[warp] = z;
        s_t[warp] = t;
    }
    __syncthreads();
    if (tid == 0) {
        z = t = 0.0;
        for (int w = 0; w < kLpWarps; ++w) {
            z += s_z[w];
            t += s_t[w];
        }
        const double lse = log(z);
        s_lse = lse;
        logprob[i] = tok >= 0 ? (float)(((double)to_f32(row[tok]) - (double)m) * inv_t - lse) : 0.f;
        if (entropy) entropy[i] = (float)(lse - t / z * 0.6931471805599453);
        status[i] = DDT_OK;
    }
    if (top_n == 0) return;
    // ---- a bound from below on the row's n-th best value: the n-th largest of the threads'
    //      largest entries (each of those n threads has an entry that reaches it)
    const float* LM = lane_max + i * nunits * 32;
    float tm = -INFINITY;
    for (int x = tid; x < nunits * 32; x += kLpThreads) tm = fmaxf(tm, LM[x]);
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
            tau = warp_max(head);
            const unsigned who = __ballot_sync(kFull, head == tau);
            if (lane == __ffs(who) - 1) head = ++at < 32 ? s_sorted[lane * 32 + at] : -INFINITY;
        }
    }
    // ---- the lanes that reach it, and their entries that do
    const int lead = row_lead(row);
    for (int x = tid; x < nunits * 32; x += kLpThreads)
        if (LM[x] >= tau) {
            const int at = atomicAdd(&s_nl, 1);
            if (at < kLpLists) s_list[at] = x;
        }
    __syncthreads();
    const int nl = s_nl;
    if (nl <= kLpLists)
        for (int x = tid; x < nl * 8; x += kLpThreads) {
            const int w = s_list[x >> 3];
            const int e = (w >> 5) * kLpUnit - lead + (w & 31) * 8 + (x & 7) * 256;
            float v[8];
            entries8(row, e, V, v);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (v[q] >= tau && e + q >= 0 && e + q < V) {
                    const int at = atomicAdd(&s_nc, 1);
                    if (at < kLpCand) {
                        s_cv[at] = v[q];
                        s_ci[at] = e + q;
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
        for (int e0 = warp * 256 - lead; e0 < V; e0 += kLpThreads * 8) {
            float v[8];
            entries8(row, e0 + lane * 8, V, v);
            float most = -INFINITY;
#pragma unroll
            for (int q = 0; q < 8; ++q) most = fmaxf(most, v[q]);
            const float last = __shfl_sync(kFull, k.v, 31);
            const int last_id = __shfl_sync(kFull, k.id, 31);
            if (__any_sync(kFull, most > last || (most == last && e0 + lane * 8 < last_id)))
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                    const int e = e0 + lane * 8 + q;
                    float x = v[0];
#pragma unroll
                    for (int y = 1; y < 8; ++y) x = q == y ? v[y] : x;
                    const bool in = e >= 0 && e < V;
                    k.insert(in ? x : none.v, in ? e : none.id);
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
        for (int c0 = 0; c0 < s_nc; c0 += 32) {
            float cv = c0 + lane < s_nc ? s_cv[c0 + lane] : none.v;
            int ci = c0 + lane < s_nc ? s_ci[c0 + lane] : none.id;
            warp_sort_best_first(cv, ci);
            warp_merge_best_first(bv, bi, cv, ci);
        }
    }
    if (lane < top_n) {
        tt[lane] = bi;
        tl[lane] = (float)(((double)bv - (double)m) * inv_t - s_lse);
    }
}

template <typename T>
static cudaError_t lp_go(int B, int N, int V, int A, int top_n, float temperature, const void* logits,
                         const int32_t* node, const int32_t* token, float* logprob, float* entropy,
                         int32_t* top_token, float* top_logprob, int32_t* status, void* ws, cudaStream_t st) {
    const int nunits = lp_units(V);
    LpPartial* part = static_cast<LpPartial*>(ws);
    float* lane_max = top_n > 0 ? reinterpret_cast<float*>(static_cast<unsigned char*>(ws) +
                                                           al256((size_t)B * A * nunits * sizeof(LpPartial)))
                                : nullptr;
    const double inv_t = 1.0 / (double)temperature;
    const float s2 = (float)(1.4426950408889634 * inv_t);
    const T* x = static_cast<const T*>(logits);
    k_lp_unit<T><<<counted(dim3((unsigned)(B * A), (nunits + kLpWarps - 1) / kLpWarps)), kLpThreads, 0, st>>>(x, N, V, A, nunits, s2,
                                                                                               node, part, lane_max);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_lp_join<T><<<counted((unsigned)(B * A)), kLpThreads, 0, st>>>(x, N, V, A, nunits, top_n, s2, inv_t, node, token, part,
                                                           lane_max, logprob, entropy, top_token, top_logprob, status);
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
