// logprobs.cu -- ddt_token_logprobs: log probabilities of given tokens under the target's
// logits, the entropy of their rows, and each row's most likely tokens.
//
// With x the row's logits, m the largest, w_v = (x_v - m) log2(e) / T and Z = sum_v 2^(w_v):
//   log p(t) = (w_t - log2 Z) ln 2,   H = -sum_v p_v log p_v = (log2 Z - sum_v 2^(w_v) w_v / Z) ln 2,
// so one pass that carries (m, Z, sum 2^w w) is enough; the top tokens need a second look at
// a few entries only.
//
// k_token_logprobs: a CTA a row, or a cluster of up to eight CTAs a row in calls of few rows,
// which are bound by latency.
//   stream  the row is cut into 4096-byte units, a warp a unit.  A warp keeps two units on
//           their way into shared memory (cp.async, each thread its own words, so no barrier).
//           Each thread carries a reference near its largest entry, moved only when an entry is
//           2^8 above it, and its two sums: packed maxima on the raw words, packed fp32 pairs
//           for the rest, nothing across the warp.  It leaves its share of the row's sums, and
//           its largest entry of every unit.
//   finish  joins the shares; the n-th largest of the threads' largest entries bounds the n-th
//           best entry of the row from below, so only the few (unit, thread) words that hold
//           an entry that reaches it are read again.  Six CTAs an SM: most stream while one or
//           two finish their rows (a chain of reads that depend on one another).
//
// Bound by HBM without alternatives: 1800 rows of 151936 bf16 logits (547 MB, two rounds of the
// resident CTAs) 87 us, 6.3 TB/s; with 20 alternatives 101 us, the rest being the finishing of a
// row by warps that do not stream, half of it the words read again.  2000 rows: 96 and 110 us, the
// third round being short of CTAs.  Small calls are bound by latency: one request's walk 9.5 us, 300
// rows 20 us.  Measured and dropped: finishing in a kernel of its own 135 us, by warps of the CTA that
// do nothing else 150 to 174; resident CTAs that fetch the next row's first units before they finish
// one 3 % slower (all rows end at once); a lane's words in one 128-byte line the same; the bound by
// counting instead of sorting 10 % slower at 32000 entries a row; eight warps and three CTAs an SM
// as much as this.
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace ddt {

namespace {
constexpr int kLpWarps = 4;
constexpr int kLpThreads = kLpWarps * 32;
constexpr int kLpCtas = 6;      // CTAs an SM
constexpr int kLpStages = 2;    // units on their way a warp
constexpr int kLpClusters = 256 * kLpCtas;  // CTAs of a call with several a row, at most
constexpr int kLpLists = 256;   // (unit, thread) pairs read again
constexpr int kLpCand = 512;    // entries ranked
constexpr float kLpLow = -200.f;  // 2^w is 0 from here down
}  // namespace

// A thread's share of a row.
struct LpPartial {
    float m;   // reference, a logit (-inf: no entry above -inf so far)
    float s;   // sum of 2^w with this reference; 0: nothing above -inf; NaN: a NaN or +inf logit
    float t;   // sum of 2^w w
    float mx;  // largest entry
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
    // all of the unit's words lie within the row
    __device__ static bool whole(int unit, int lead, int V) {
        return unit * kEntries >= lead && (unit + 1) * kEntries - lead <= V;
    }
};
static inline int lp_units(int V, size_t esz) {
    const int per = 4096 / (int)esz, gap = 16 / (int)esz - 1;
    return (int)(((long long)V + gap + per - 1) / per);
}
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// the shares of rows with several CTAs
static constexpr size_t kLpPartBytes = (size_t)kLpClusters * kLpThreads * sizeof(LpPartial);

// workspace: shares, the threads' largest entries of every unit.  fp32 rows have twice the
// units of bf16 rows: the size covers both.
size_t logprobs_ws_bytes(int B, int A, int V, int top_n) {
    const size_t rows = (size_t)B * A;
    return kLpPartBytes + (top_n > 0 ? al256(rows * lp_units(V, 4) * 32 * sizeof(float)) : 0);
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
// running maximum of a lane's words (NaN entries are passed over here: they turn the sums NaN)
template <typename T>
struct LpMax;
template <>
struct LpMax<__nv_bfloat16> {
    __nv_bfloat162 hi = __float2bfloat162_rn(-INFINITY);
    __device__ __forceinline__ void see(const uint4& w) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) hi = __hmax2(hi, *reinterpret_cast<const __nv_bfloat162*>(&v[i]));
    }
    __device__ __forceinline__ float max() const { return fmaxf(__low2float(hi), __high2float(hi)); }
};
template <>
struct LpMax<float> {
    float hi = -INFINITY;
    __device__ __forceinline__ void see(const uint4& w) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) hi = fmaxf(hi, __uint_as_float(v[i]));
    }
    __device__ __forceinline__ float max() const { return hi; }
};

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

// A thread's running share of a row.
struct LpRun {
    float m, ref, s, t, mx;  // ref = m log2(e) / T as rounded, which the terms take as it is
    __device__ __forceinline__ void start() {
        m = ref = mx = -INFINITY;
        s = t = 0.f;
    }
};
// The terms take the reference as m log2(e) / T rounds, and lp_share puts that right.  From here on
// (off by up to 1/8) differences to it are taken before scaling instead, term by term: 2047 rows of
// 151936 take 163 us there instead of 114.  Logits of 29 at a temperature of 1e-5 are still below.
constexpr float kLpFar = 4194304.f;
__device__ __forceinline__ bool lp_far(float ref) { return !(fabsf(ref) < kLpFar); }
// what the terms of a near reference took too much
__device__ __forceinline__ float lp_off(float m, float ref, float s2) { return lp_far(ref) ? 0.f : fmaf(m, s2, -ref); }

// One unit's words of this thread, from shared memory (read twice: keeping them in registers
// costs a third of the warps); returns the largest entry.
template <typename T>
__device__ __forceinline__ float lp_add(LpRun& r, const uint4* from, float s2) {
    constexpr int VE = LpUnit<T>::VE;
    const T* kT = nullptr;
    LpMax<T> top;
#pragma unroll
    for (int j = 0; j < 8; ++j) top.see(from[j * 32]);
    const float mt = top.max();
    r.mx = fmaxf(r.mx, mt);
    if ((mt - r.m) * s2 > 8.f) {  // the first unit, or an entry far above the reference
        const float ref = mt * s2;
        if (r.s != 0.f) {
            const float d = !lp_far(ref) && !lp_far(r.ref)
                                ? r.ref - ref
                                : fmaxf((r.m - mt) * s2 - lp_off(r.m, r.ref, s2) + lp_off(mt, ref, s2), kLpLow);
            const float f = tc::ex2(d);
            r.t = f * fmaf(d, r.s, r.t);
            r.s *= f;
        }
        r.m = mt;
        r.ref = ref;
    }
    const uint64_t k2 = pack2(s2, s2), r2 = pack2(-r.ref, -r.ref);
    uint64_t s[2] = {0, 0}, t[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 w = from[j * 32];
#pragma unroll
        for (int q = 0; q < VE; q += 2) {
            const uint64_t v = fma2(pack2(lp_at(w, q, kT), lp_at(w, q + 1, kT)), k2, r2);
            float a, b;
            unpack2(v, a, b);
            const uint64_t e = pack2(tc::ex2(a), tc::ex2(b));
            s[(q >> 1) & 1] = add2(s[(q >> 1) & 1], e);
            t[(q >> 1) & 1] = fma2(e, v, t[(q >> 1) & 1]);
        }
    }
    float s0, s1, t0, t1;
    unpack2(add2(s[0], s[1]), s0, s1);
    unpack2(add2(t[0], t[1]), t0, t1);
    s0 += s1;
    t0 += t1;
    if (__any_sync(kFull, t0 != t0 || lp_far(r.ref))) {
        // masked entries (0 * -inf in t), or a far reference (a low temperature, logits far from
        // zero, the type's lowest value as a mask): again, term by term and with a bound
        const bool far = lp_far(r.ref);
        const float base = r.m == -INFINITY ? 0.f : r.m;
        s0 = t0 = 0.f;
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            const uint4 w = from[j * 32];
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const float x = lp_at(w, q, kT);
                const float a = max_nan(far ? (x - base) * s2 : fmaf(x, s2, -r.ref), kLpLow), e = tc::ex2(a);
                s0 += e;
                t0 = fmaf(e, a, t0);
            }
        }
    }
    r.s += s0;
    r.t += t0;
    return mt;
}

// The share with the exact reference m: a term 2^a a was to be 2^(a - off) (a - off).
__device__ __forceinline__ float4 lp_share(const LpRun& r, float s2) {
    const float off = lp_off(r.m, r.ref, s2), c = 1.f + expm1f(-0.6931471805599453f * off);
    return make_float4(r.m, r.s * c, fmaf(-off, r.s, r.t) * c, r.mx);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

struct LpArgs {
    int N, V, A, nunits, top_n;
    bool near;  // the units' largest entries behind the ring, not in the workspace
    float s2, inv_t;
    const int32_t* node;
    const int32_t* token;
    float4* part;    // LpPartial
    float* logprob;
    float* entropy;
    int32_t* top_token;
    float* top_logprob;
    int32_t* status;
};

__device__ __forceinline__ int lp_node(const LpArgs& p, int i) { return p.node ? p.node[i] : i % p.A; }
// entry i names a row and no impossible token
__device__ __forceinline__ bool lp_asked(const LpArgs& p, int i) {
    const int r = lp_node(p, i);
    return r >= 0 && r < p.N && p.token[i] < p.V;
}
template <typename T>
__device__ __forceinline__ const T* lp_row(const LpArgs& p, const T* logits, int i) {
    return logits + ((long long)(i / p.A) * p.N + lp_node(p, i)) * p.V;
}
// the results of an entry that does not
__device__ __forceinline__ void lp_padding(const LpArgs& p, int i, int tid) {
    if (tid == 0) {
        p.logprob[i] = 0.f;
        if (p.entropy) p.entropy[i] = 0.f;
        p.status[i] = lp_node(p, i) < 0 ? DDT_OK : DDT_ERR_INVALID_ARG;
    }
    if (tid < p.top_n) {
        p.top_token[(long long)i * p.top_n + tid] = -1;
        p.top_logprob[(long long)i * p.top_n + tid] = 0.f;
    }
}

struct LpScratch {
    float m[kLpWarps], z[kLpWarps], t[kLpWarps], sorted[kLpThreads];
    int list[kLpLists];
    float cv[kLpCand];
    int ci[kLpCand];
    int nl, nc;
};

// A unit's words: on their way into a warp's place of the ring, and from there.
template <typename T>
__device__ __forceinline__ void lp_fetch(uint4* dst, const T* row, int u, int lane, int V) {
    constexpr int VE = LpUnit<T>::VE;
    const int lead = LpUnit<T>::lead(row), e0 = LpUnit<T>::entry(u, 0, lane, lead);
    if (LpUnit<T>::whole(u, lead, V)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cp_async16(dst + j * 32 + lane, row + e0 + j * 32 * VE);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + j * 32 * VE;
            if (e >= 0 && e + VE <= V) cp_async16(dst + j * 32 + lane, row + e);
        }
    }
}
// The words at the row's ends, which no copy brings, into their places.
template <typename T>
__device__ __forceinline__ void lp_ends(uint4* to, const T* row, int u, int lane, int V) {
    constexpr int VE = LpUnit<T>::VE;
    const int lead = LpUnit<T>::lead(row);
    if (LpUnit<T>::whole(u, lead, V)) return;
    const int e0 = LpUnit<T>::entry(u, 0, lane, lead);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = e0 + j * 32 * VE;
        if (e < 0 || e + VE > V) to[j * 32 + lane] = lp_word(row, e, V);
    }
}
__device__ __forceinline__ void lp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void lp_wait() {  // for the oldest of the stages
    asm volatile("cp.async.wait_group %0;" ::"n"(kLpStages - 1) : "memory");
}

// The top n of a row by one warp where the quick way does not do: few units, or many entries
// at its bound (a masked row, say).  The n-th largest of the lanes' largest entries: fewer
// than n lanes have entries above it, and of the entries that equal it the first n in order
// are enough.
template <typename T>
__device__ __noinline__ void lp_top_slow(const T* __restrict__ row, const T* LM, int V, int nunits, int n, int lane,
                                         float& bv, int& bi) {
    constexpr int VE = LpUnit<T>::VE;
    const int lead = LpUnit<T>::lead(row);
    const VId none = vid_empty();
    float best = -INFINITY;
#pragma unroll 4
    for (int u = 0; u < nunits; ++u) {
        float v = to_f32(LM[u * 32 + lane]);
        int id = lane, bid = lane;
        if (!__any_sync(kFull, v > __shfl_sync(kFull, best, 31))) continue;
        warp_sort_best_first(v, id);
        warp_merge_best_first(best, bid, v, id);
    }
    const float tau = __shfl_sync(kFull, best, n - 1);
    WarpTopK top;
    top.init(32);
    int equal = 0;
    for (int u = 0; u < nunits; ++u) {
        const float v = to_f32(LM[u * 32 + lane]);
        const bool above = __any_sync(kFull, v > tau), same = __any_sync(kFull, v >= tau);
        if (!above && (!same || equal >= n)) continue;
        for (int j = 0; j < 8; ++j) {
            const int e = LpUnit<T>::entry(u, j, lane, lead);
            const uint4 w = lp_word(row, e, V);
            int eq = 0;
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const bool in = e + q >= 0 && e + q < V;
                const float y = lp_at(w, q, static_cast<const T*>(nullptr));
                const bool is = in && y == tau;
                eq += is;
                const bool take = (in && y > tau) || (is && equal < n);
                if (__any_sync(kFull, take)) top.insert(take ? y : none.v, take ? e + q : none.id);
            }
            equal += __reduce_add_sync(kFull, eq);
        }
    }
    bv = top.v;
    bi = top.id;
}

// One row's results from its n_t shares, by the whole block: `own`, the thread's, or those at P
// (of several CTAs).
template <typename T>
__device__ __forceinline__ void lp_finish(const LpArgs& p, LpScratch& S, const T* __restrict__ row, const T* LM,
                                          const float4& own, const float4* P, int n_t, int i) {
    constexpr int VE = LpUnit<T>::VE, NT = kLpThreads, kWarps = kLpWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int V = p.V, nunits = p.nunits, top_n = p.top_n, lead = LpUnit<T>::lead(row);
    const int tok = p.token[i];
    const float xt = tok >= 0 ? to_f32(row[tok]) : 0.f;
    // ---- the row's reference, and the threads' largest entries in order
    float m = -INFINITY, best = -INFINITY;
    int id = lane;
    for (int u = tid; u < n_t; u += NT) {
        const float4 x = P ? P[u] : own;
        m = fmaxf(m, x.x);
        best = fmaxf(best, x.w);
    }
    if (top_n) warp_sort_best_first(best, id);
    m = redux_max(m);
    S.sorted[tid] = best;
    if (lane == 0) S.m[warp] = m;
    if (tid == 0) S.nl = S.nc = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, S.m[w]);
    // ---- Z and sum 2^w w (a NaN sum stays NaN)
    float z = 0.f, t = 0.f;
    for (int u = tid; u < n_t; u += NT) {
        const float4 x = P ? P[u] : own;
        if (x.y == 0.f) continue;
        const float d = fmaxf((x.x - m) * p.s2, kLpLow), f = tc::ex2(d);
        z = fmaf(f, x.y, z);
        t = fmaf(f, fmaf(d, x.y, x.z), t);
    }
    z = warp_sum(z);
    t = warp_sum(t);
    if (lane == 0) {
        S.z[warp] = z;
        S.t[warp] = t;
    }
    // ---- a bound from below on the row's n-th best value: the n-th largest of the threads'
    //      largest entries (each of those n has an entry that reaches it); the (unit, thread)
    //      pairs that reach it
    float tau = -INFINITY;
    if (top_n) {
        best = S.sorted[lane];
        for (int w = 1; w < kWarps; ++w) warp_merge_best_first(best, id, S.sorted[w * 32 + lane], lane);
        tau = __shfl_sync(kFull, best, top_n - 1);
#pragma unroll 4
        for (int x = tid * VE; x < nunits * 32; x += NT * VE) {
            const uint4 v = *reinterpret_cast<const uint4*>(LM + x);
#pragma unroll
            for (int q = 0; q < VE; ++q)
                if (lp_at(v, q, static_cast<const T*>(nullptr)) >= tau) {
                    const int at = atomicAdd(&S.nl, 1);
                    if (at < kLpLists) S.list[at] = x + q;
                }
        }
    }
    __syncthreads();
    z = t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        z += S.z[w];
        t += S.t[w];
    }
    int32_t* tt = p.top_token + (long long)i * top_n;
    float* tl = p.top_logprob + (long long)i * top_n;
    const bool bad = !(z > 0.f);  // NaN, +inf, or nothing above -inf
    const float LN2 = 0.6931471805599453f, lz = log2f(z);
    if (tid == 0) {
        p.logprob[i] = bad ? NAN : (tok >= 0 ? (xt - m) * p.inv_t - lz * LN2 : 0.f);
        if (p.entropy) p.entropy[i] = bad ? NAN : (lz - t / z) * LN2;
        p.status[i] = bad ? DDT_ERR_NONFINITE : DDT_OK;
    }
    if (bad && tid < top_n) {
        tt[tid] = -1;
        tl[tid] = NAN;
    }
    if (bad || top_n == 0) return;  // the same for the whole block
    // ---- their entries that reach it, each ranked by counting the better ones
    const int nl = S.nl;
    if (nl <= kLpLists) {
#pragma unroll 4
        for (int x = tid; x < nl * 8; x += NT) {
            const int l = S.list[x >> 3];
            const int e = LpUnit<T>::entry(l >> 5, x & 7, l & 31, lead);
            const uint4 v = lp_word(row, e, V);
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                const float y = lp_at(v, q, static_cast<const T*>(nullptr));
                if (y >= tau && e + q >= 0 && e + q < V) {
                    const int at = atomicAdd(&S.nc, 1);
                    if (at < kLpCand) {
                        S.cv[at] = y;
                        S.ci[at] = e + q;
                    }
                }
            }
        }
    }
    __syncthreads();
    const int nc = S.nc;
    if (nl <= kLpLists && nc <= kLpCand) {
        for (int x = tid; x < nc; x += NT) {
            const float v = S.cv[x];
            const int id = S.ci[x];
            int r = 0;
            for (int y = 0; y < nc; ++y) {
                const float o = S.cv[y];
                r += o > v || (o == v && S.ci[y] < id);
            }
            if (r < top_n) {
                tt[r] = id;
                tl[r] = (v - m) * p.inv_t - lz * LN2;
            }
        }
    } else if (warp == 0) {
        float bv;
        int bi;
        lp_top_slow<T>(row, LM, V, nunits, top_n, lane, bv, bi);
        if (lane < top_n) {
            tt[lane] = bi;
            tl[lane] = (bv - m) * p.inv_t - lz * LN2;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) k_token_logprobs(const T* __restrict__ logits, T* lane_max, const LpArgs p) {
    extern __shared__ __align__(16) uint4 s_ring[];  // [kLpWarps][kLpStages][256], largest entries (near)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int cl, rank;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int i = blockIdx.x / cl;
    if (!lp_asked(p, i)) {  // the whole cluster
        if (rank == 0) lp_padding(p, i, threadIdx.x);
        return;
    }
    const T* row = lp_row(p, logits, i);
    const int V = p.V, nunits = p.nunits, wid = rank * kLpWarps + warp, n_w = cl * kLpWarps;
    uint4* ring = s_ring + warp * kLpStages * 256;
    T* LM = p.near ? reinterpret_cast<T*>(s_ring + kLpWarps * kLpStages * 256) : lane_max + (long long)i * nunits * 32;
    int fu = wid, stage = 0;
    auto fetch = [&](int s) {
        if (fu < nunits) lp_fetch<T>(ring + s * 256, row, fu, lane, V);
        fu += n_w;
        lp_commit();
    };
#pragma unroll
    for (int s = 0; s < kLpStages; ++s) fetch(s);
    LpRun run;
    run.start();
    for (int u = wid; u < nunits; u += n_w) {
        uint4* at = ring + stage * 256;
        lp_wait();
        lp_ends<T>(at, row, u, lane, V);
        const float mt = lp_add<T>(run, at + lane, p.s2);
        fetch(stage);
        if (p.top_n) LM[u * 32 + lane] = from_f32<T>(mt);
        stage = stage + 1 == kLpStages ? 0 : stage + 1;
    }
    const float4 own = lp_share(run, p.s2);
    float4* P = nullptr;
    if (cl > 1) {  // the shares of all CTAs become visible to the cluster's first one
        P = p.part + (long long)i * n_w * 32;
        P[wid * 32 + lane] = own;
        tc::cluster_sync();
        if (rank) return;
    } else {
        __syncthreads();
    }
    // every copy has landed and been read: the ring becomes the scratch
    lp_finish<T>(p, *reinterpret_cast<LpScratch*>(s_ring), row, LM, own, P, n_w * 32, i);
}

template <typename T>
static cudaError_t lp_go(int B, int N, int V, int A, int top_n, float temperature, const void* logits,
                         const int32_t* node, const int32_t* token, float* logprob, float* entropy,
                         int32_t* top_token, float* top_logprob, int32_t* status, void* ws, cudaStream_t st) {
    const int nunits = lp_units(V, sizeof(T)), rows = B * A;
    unsigned char* w = static_cast<unsigned char*>(ws);
    LpArgs a{N, V, A, nunits, top_n, false, (float)(1.4426950408889634 / (double)temperature),
             (float)(1.0 / (double)temperature), node, token, reinterpret_cast<float4*>(w), logprob, entropy,
             top_token, top_logprob, status};
    T* lane_max = reinterpret_cast<T*>(w + kLpPartBytes);
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms > 256) sms = 256;
    constexpr int ring = kLpWarps * kLpStages * 4096;
    constexpr int room = 228 * 1024 / kLpCtas - 1024 - ring;  // a CTA
    static_assert(room >= 0 && sizeof(LpScratch) <= ring, "shared memory of an SM");
    // As many CTAs a row as are resident together.  Twice as many: 200 rows 22.7 instead of 17.5 us,
    // 450 rows 36.8 instead of 34.7.  (Walks pad their entries; two CTAs a row for 32 walks of up to 16
    // take 15.9 instead of 18.7 us if 2 are rows, but 22.0 instead of 19.6 if 8 are, 42 instead of 33
    // if all are.)
    int cl = 1;
    while (cl < 8 && rows * 2LL * cl <= (long long)kLpCtas * sms && cl * kLpWarps < nunits) cl *= 2;
    // the units' largest entries stay in shared memory where a row has one CTA and they leave its
    // six a place: 2000 rows of 151936 110 us, through the workspace 117 (its writes disturb the reads)
    const int maxima = top_n ? nunits * 32 * (int)sizeof(T) : 0;
    a.near = cl == 1 && maxima <= room;
    const cudaError_t e = cudaFuncSetAttribute(k_token_logprobs<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring + room);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(counted((unsigned)rows * cl));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = ring + (a.near ? maxima : 0);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cl;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_token_logprobs<T>, static_cast<const T*>(logits), lane_max, a);
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
