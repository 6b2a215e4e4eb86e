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

// 8 channels as they lie in memory (which may be what is written later: not the read-only path)
template <typename T, bool VEC>
struct Run {
    static constexpr int W = 8 * (int)sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
                w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (sizeof(T) == 4) {
                    w[i % W] = reinterpret_cast<const uint32_t*>(p)[i];
                } else {
                    const uint32_t h = reinterpret_cast<const uint16_t*>(p)[i];
                    w[i / 2] = i % 2 ? w[i / 2] | h << 16 : h;
                }
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if (sizeof(T) == 4) return __uint_as_float(w[i % W]);
        return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

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
    __shared__ __align__(16) float2 s_cs[kMaxTokens * D / 2];
    __shared__ __align__(16) float s_w[2][D];  // offset + weight: of q, of k
    const int tid = threadIdx.x, half = a.rot / 2, heads = a.Hq + a.Hkv;
    const long long rows = (long long)a.B * a.N, first = (long long)blockIdx.x * a.tokens;
    const int l = blockIdx.y, nt = (int)min((long long)a.tokens, rows - first), items = nt * heads;
    const int c = tid % LPR;
    // this lane's two runs: of the rotated channels the halves of its pairs, of the others neighbours
    const bool turned = 16 * c < a.rot;
    const int lo = turned ? 8 * c : 16 * c, hi = turned ? half + 8 * c : 16 * c + 8;
    const unsigned mask = ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);  // the lanes of a row, which agree throughout

    // two rows are on their way while one is worked on
    Run<T, VEC> u[2], v[2];
    bool live[2];
    auto fetch = [&](int it, int s) {
        live[s] = false;
        if (it >= items) return;
        const int t = it / heads, h = it - t * heads;
        const long long tok = first + t;
        const int b = (int)(tok / a.N), n = (int)(tok - (long long)b * a.N);
        if (a.n_nodes) {
            const int nn = a.n_nodes[b];
            if (n >= nn || nn > a.N) return;
        }
        live[s] = true;
        const T* x = h < a.Hq ? static_cast<const T*>(a.q) + l * a.qs[0] + b * a.qs[1] + n * a.qs[2] + h * a.qs[3]
                              : static_cast<const T*>(a.k) + l * a.ks[0] + b * a.ks[1] + n * a.ks[2] + (h - a.Hq) * a.ks[3];
        u[s].load(x + lo);
        v[s].load(x + hi);
    };
    const int it0 = tid / LPR;
    fetch(it0, 0);
    fetch(it0 + kRows, 1);
    for (int e = tid; e < nt * half; e += kThreads) {
        const int t = e / half, i = e - t * half;
        const unsigned long long turn = (unsigned long long)(long long)a.position[first + t] * fr.f[i];
        float s, co;
        sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &co);  // half turns: 2^-31
        s_cs[e] = make_float2(co, s);
    }
    for (int e = tid; e < 2 * D; e += kThreads)
        s_w[e / D][e % D] = a.offset + to_f32(static_cast<const T*>(e < D ? a.qw : a.kw)[(long long)l * D + e % D]);
    __syncthreads();
    for (int it = it0; it < items; it += 2 * kRows) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int i0 = it + s * kRows, t = i0 / heads, h = i0 - t * heads;
            if (!live[s]) {
                fetch(i0 + 2 * kRows, s);
                continue;
            }
            const bool isq = h < a.Hq;
            T* y = isq ? static_cast<T*>(a.qo) + ((l * rows + first + t) * a.Hq + h) * D
                       : static_cast<T*>(a.ko) + ((l * rows + first + t) * a.Hkv + (h - a.Hq)) * D;
            float p[8], q[8], ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = u[s][i];
                q[i] = v[s][i];
                ss = fmaf(p[i], p[i], fmaf(q[i], q[i], ss));
            }
            fetch(i0 + 2 * kRows, s);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
            const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(s_w[!isq] + lo + i), z = *reinterpret_cast<const float4*>(s_w[!isq] + hi + i);
                p[i] *= r * x.x; p[i + 1] *= r * x.y; p[i + 2] *= r * x.z; p[i + 3] *= r * x.w;
                q[i] *= r * z.x; q[i + 1] *= r * z.y; q[i + 2] *= r * z.z; q[i + 3] *= r * z.w;
            }
            if (turned) {
                const float4* cs = reinterpret_cast<const float4*>(s_cs + t * half + 8 * c);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 k = cs[i / 2];
                    const float p0 = p[i], p1 = p[i + 1];
                    p[i] = fmaf(p0, k.x, -q[i] * k.y);
                    q[i] = fmaf(q[i], k.x, p0 * k.y);
                    p[i + 1] = fmaf(p1, k.z, -q[i + 1] * k.w);
                    q[i + 1] = fmaf(q[i + 1], k.z, p1 * k.w);
                }
            }
            store_run<T, VEC>(y + lo, p);
            store_run<T, VEC>(y + hi, q);
        }
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
    // frequency i as a product of two powers, 16 + 8 of them at most: a power takes the host some 50 ns
    NormFreq fr{};
    double near[16], far[8];
    for (int i = 0; i < 16 && i < rot / 2; ++i) near[i] = pow(theta, -2.0 * i / rot) * (18446744073709551616.0 / 6.283185307179586477);
    for (int i = 0; i < 8 && 16 * i < rot / 2; ++i) far[i] = pow(theta, -32.0 * i / rot);
    for (int i = 0; i < rot / 2; ++i) fr.f[i] = (unsigned long long)(near[i % 16] * far[i / 16]);
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    a.tokens = 1;
    while (a.tokens < kMaxTokens && (long long)L * B * N >= 8LL * sms * a.tokens) a.tokens *= 2;
    return dtype == DDT_BF16 ? norm_d_go<__nv_bfloat16>(L, d, a, fr, (bits & 15) == 0, st) : norm_d_go<float>(L, d, a, fr, (bits & 15) == 0, st);
}

}  // namespace ddt
