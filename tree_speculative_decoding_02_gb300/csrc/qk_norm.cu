// qk_norm.cu -- ddt_qk_norm_rope: the root-mean-square norm of every query and key head and the
// rotary embedding by position in one pass, from the projection's rows to the rows that the
// attention calls and the cache take.
//
// A row x of d channels with weights w: y = x / sqrt(mean(x^2) + eps) * (offset + w), then the
// pairs (i, i + rot/2) of the first rot channels turn by position * theta^(-2i/rot), as in
// ddt_rope_tree.  Everything in fp32, rounded once.
//
// A row is 16 channels a lane (d / 16 lanes): two runs of 8, the two halves of its rotation pairs,
// so a rotation needs no exchange and a bf16 run is one 16-byte load.  A CTA takes a few tokens of
// one layer; their cosines are formed once in shared memory for all heads, while the first rows are
// on their way.
// An angle is a fraction of a turn in 64-bit fixed point: frequency / 2 pi as a fraction of 2^64
// (from the host) times the position, modulo 2^64, is the reduced angle with no rounding but the
// table's, for any position; its upper half goes to sincospi.  No fp64, which is slow here.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace ddt {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // a CTA

struct NormFreq {
    unsigned long long f[128];  // theta^(-2i/rot) / (2 pi), in units of 2^-64
};

struct NormArgs {
    int B, N, Hq, Hkv, rot, tokens;  // tokens a CTA
    float eps, offset;
    long long qs[4], ks[4];  // strides of the inputs in elements: layer, request, row, head
    const void* q;
    const void* k;
    const void* qw;
    const void* kw;
    const int32_t* position;
    const int32_t* n_nodes;  // or null: all rows
    void* qo;
    void* ko;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_run(const T* p, float (&v)[8]) {
    if (VEC) {
        if (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);  // (may be what is written: not the read-only path)
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_run(T* p, const float (&v)[8]) {
    if (VEC) {
        if (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(v[i]);
    }
}

}  // namespace

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const NormArgs a, const __grid_constant__ NormFreq fr) {
    constexpr int LPR = D / 16, kRows = kThreads / LPR;  // lanes a row, rows at a time
    __shared__ float2 s_cs[kMaxTokens * D / 2];
    __shared__ int s_live[kMaxTokens];
    const int tid = threadIdx.x, half = a.rot / 2, heads = a.Hq + a.Hkv;
    const long long rows = (long long)a.B * a.N, first = (long long)blockIdx.x * a.tokens;
    const int l = blockIdx.y, nt = (int)min((long long)a.tokens, rows - first);
    const int c = tid % LPR;
    // this lane's two runs: of the rotated channels the halves of its pairs, of the others neighbours
    const bool turned = 16 * c < a.rot;
    const int lo = turned ? 8 * c : 16 * c, hi = turned ? half + 8 * c : 16 * c + 8;

    if (tid < nt) {
        const int b = (int)((first + tid) / a.N), n = (int)((first + tid) % a.N);
        const int nn = a.n_nodes ? a.n_nodes[b] : a.N;
        s_live[tid] = n < nn && nn <= a.N;
    }
    for (int e = tid; e < nt * half; e += kThreads) {
        const int t = e / half, i = e - t * half;
        const unsigned long long turn = (unsigned long long)(long long)a.position[first + t] * fr.f[i];
        float s, co;
        sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &co);  // half turns: 2^-31
        s_cs[e] = make_float2(co, s);
    }
    __syncthreads();
    const int items = nt * heads;
    const unsigned mask = ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);  // the lanes of a row, which agree throughout
    for (int it = tid / LPR; it < items; it += kRows) {
        const int t = it / heads, h = it - t * heads;
        const bool live = s_live[t];
        const long long tok = first + t;
        const int b = (int)(tok / a.N), n = (int)(tok - (long long)b * a.N);
        const bool isq = h < a.Hq;
        const T* x = isq ? static_cast<const T*>(a.q) + l * a.qs[0] + b * a.qs[1] + n * a.qs[2] + h * a.qs[3]
                         : static_cast<const T*>(a.k) + l * a.ks[0] + b * a.ks[1] + n * a.ks[2] + (h - a.Hq) * a.ks[3];
        T* y = isq ? static_cast<T*>(a.qo) + ((l * rows + tok) * a.Hq + h) * D
                   : static_cast<T*>(a.ko) + ((l * rows + tok) * a.Hkv + (h - a.Hq)) * D;
        const T* w = static_cast<const T*>(isq ? a.qw : a.kw) + (long long)l * D;
        if (!live) continue;
        float u[8], v[8], wu[8], wv[8];
        load_run<T, VEC>(x + lo, u);
        load_run<T, VEC>(x + hi, v);
        load_run<T, VEC>(w + lo, wu);
        load_run<T, VEC>(w + hi, wv);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = u[i] * r * (a.offset + wu[i]);
            v[i] = v[i] * r * (a.offset + wv[i]);
        }
        if (turned) {
            const float2* cs = s_cs + t * half + 8 * c;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 k = cs[i];
                const float p = u[i];
                u[i] = fmaf(p, k.x, -v[i] * k.y);
                v[i] = fmaf(v[i], k.x, p * k.y);
            }
        }
        store_run<T, VEC>(y + lo, u);
        store_run<T, VEC>(y + hi, v);
    }
}

template <typename T, int D>
static cudaError_t norm_go(int L, const NormArgs& a, const NormFreq& fr, bool vec, cudaStream_t st) {
    const long long rows = (long long)a.B * a.N;
    const dim3 grid((unsigned)((rows + a.tokens - 1) / a.tokens), L);
    if (vec) k_qk_norm_rope<T, D, true><<<counted(grid), kThreads, 0, st>>>(a, fr);
    else k_qk_norm_rope<T, D, false><<<counted(grid), kThreads, 0, st>>>(a, fr);
    return cudaGetLastError();
}
template <typename T>
static cudaError_t norm_d_go(int L, int d, const NormArgs& a, const NormFreq& fr, bool vec, cudaStream_t st) {
    return d == 64 ? norm_go<T, 64>(L, a, fr, vec, st) : (d == 128 ? norm_go<T, 128>(L, a, fr, vec, st) : norm_go<T, 256>(L, a, fr, vec, st));
}

cudaError_t launch_qk_norm_rope(int L, int B, int N, int Hq, int Hkv, int d, int rot, double theta, float eps, float offset,
                                ddt_dtype dtype, const void* q, const int64_t* q_stride, const void* k,
                                const int64_t* k_stride, const void* qw, const void* kw, const int32_t* position,
                                const int32_t* n_nodes, void* qo, void* ko, cudaStream_t st) {
    NormArgs a{};
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.rot = rot;
    a.eps = eps;
    a.offset = offset;
    a.q = q;
    a.k = k;
    a.qw = qw;
    a.kw = kw;
    a.position = position;
    a.n_nodes = n_nodes;
    a.qo = qo;
    a.ko = ko;
    const int esz = dtype == DDT_BF16 ? 2 : 4;
    uintptr_t bits = (uintptr_t)q | (uintptr_t)k | (uintptr_t)qw | (uintptr_t)kw | (uintptr_t)qo | (uintptr_t)ko;
    const int qn[4] = {L, B, N, Hq}, kn[4] = {L, B, N, Hkv};
    for (int i = 0; i < 4; ++i) {  // (the stride of a single entry says nothing)
        a.qs[i] = qn[i] > 1 ? q_stride[i] : 0;
        a.ks[i] = kn[i] > 1 ? k_stride[i] : 0;
        bits |= (uintptr_t)(a.qs[i] * esz) | (uintptr_t)(a.ks[i] * esz);
    }
    NormFreq fr{};
    for (int i = 0; i < rot / 2; ++i)
        fr.f[i] = (unsigned long long)(powl((long double)theta, -2.0L * i / rot) * (18446744073709551616.0L / 6.283185307179586476925L));
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    a.tokens = 1;
    while (a.tokens < kMaxTokens && a.tokens * (Hq + Hkv) * (d / 16) < kThreads && (long long)L * B * N >= 16LL * sms * a.tokens) a.tokens *= 2;
    return dtype == DDT_BF16 ? norm_d_go<__nv_bfloat16>(L, d, a, fr, (bits & 15) == 0, st) : norm_d_go<float>(L, d, a, fr, (bits & 15) == 0, st);
}

}  // namespace ddt
