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
// (from the host, in fp64) times the position, modulo 2^64, is the reduced angle with no rounding but
// the table's; its upper half goes to sincospi.  No fp64 on the device, where it is slow.
//
// Bound by HBM: 16 layers of 32 x 65 tree rows (three quarters of them nodes), 24 + 4 heads of 256, bf16 (716 MB), 121 us,
// 5.9 TB/s; 169 with 64-bit divisions and half the instructions unpaired.  A row is a chain of a few hundred cycles (sum, four
// exchanges, root, products), and two rows a lane group are on their way meanwhile; three or four are no faster, and two
// chains side by side do not fit in the registers of four CTAs an SM.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 256;
// tokens a CTA at most: 4413 of 18 fp32 heads of 128 take 20.6 us with 8, 18.8 with 12; the batched rounds' bf16 rows 120.6 and 123.4
constexpr int max_tokens(int esz) { return esz == 2 ? 8 : 12; }

struct NormFreq {
    unsigned long long f[128];  // theta^(-2i/rot) / (2 pi), in units of 2^-64
};

struct NormArgs {
    int B, N, Hq, Hkv, rot, tokens;  // tokens a CTA
    int dt, dh;                      // the rows that a CTA takes at a time, as tokens and heads
    float eps, offset;
    long long qs[3], ks[3];  // strides of the inputs in elements: layer, request, row
    int q_head, k_head;      // and in bytes: head
    const void* q;
    const void* k;
    const void* qw;
    const void* kw;
    const int32_t* position;
    const int32_t* n_nodes;  // or null: all rows
    void* qo;
    void* ko;
};

// 8 channels as they lie in memory
template <typename T>
struct Run {
    static constexpr int W = 8 * (int)sizeof(T) / 4;
    uint32_t w[W];
    // VEC: from 16-byte words, else aligned to the elements (not by the read-only path: it may be written later)
    template <bool VEC>
    __device__ __forceinline__ void load(const void* p) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 u = static_cast<const uint4*>(p)[i / 4];
                w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (sizeof(T) == 4) {
                    w[i % W] = static_cast<const uint32_t*>(p)[i];
                } else {
                    const uint32_t h = static_cast<const uint16_t*>(p)[i];
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
__device__ __forceinline__ void copy16(uint4* to, const char* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_run(T* p, const F2 (&x)[4]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = f2_get(x[i]);
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
    }
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
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) k_qk_norm_rope(const NormArgs a, const __grid_constant__ NormFreq fr) {
    constexpr int LPR = D / 16, kMaxTokens = max_tokens(sizeof(T));  // lanes a row
    // four float4 a lane, lane after lane: a quarter warp reads 128 consecutive bytes
    __shared__ float4 s_cs[kMaxTokens * D / 4];  // [token][4][rot / 16]: two cosines, their sines
    __shared__ float4 s_w[2][4 * LPR];           // offset + weight: of q, of k
    // where a token's head 0 is in q, and would be in k, or null; the same of the outputs
    __shared__ const char* s_at[kMaxTokens][2];
    __shared__ char* s_to[kMaxTokens][2];
    const int tid = threadIdx.x, half = a.rot / 2, lanes = a.rot / 16, heads = a.Hq + a.Hkv;
    const unsigned rows = (unsigned)a.B * (unsigned)a.N, first = blockIdx.x * (unsigned)a.tokens;  // (fewer than 2^31)
    const int l = blockIdx.y, nt = (int)min((unsigned)a.tokens, rows - first);
    const int c = tid % LPR;
    // this lane's two runs: of the rotated channels the halves of its pairs, of the others too one in each half, so that
    // neighbouring lanes' runs lie together
    const bool turned = c < lanes;
    const int rest = (D - a.rot) / 2, lo = turned ? 8 * c : half + 8 * c, hi = lo + (turned ? half : rest);
    const unsigned mask = ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);  // the lanes of a row, which agree throughout

    if (tid < nt) {
        const unsigned tok = first + tid, b = tok / (unsigned)a.N, n = tok - b * (unsigned)a.N;
        const int nn = a.n_nodes ? a.n_nodes[b] : a.N;
        const bool live = (int)n < nn && nn <= a.N;
        s_at[tid][0] = live ? reinterpret_cast<const char*>(static_cast<const T*>(a.q) + l * a.qs[0] + b * a.qs[1] + n * a.qs[2]) : nullptr;
        s_at[tid][1] = live ? reinterpret_cast<const char*>(static_cast<const T*>(a.k) + l * a.ks[0] + b * a.ks[1] + n * a.ks[2]) -
                                  (long long)a.Hq * a.k_head
                            : nullptr;
        const long long row = (long long)l * rows + tok;
        s_to[tid][0] = reinterpret_cast<char*>(static_cast<T*>(a.qo) + row * a.Hq * D);
        s_to[tid][1] = reinterpret_cast<char*>(static_cast<T*>(a.ko) + (row * a.Hkv - a.Hq) * D);
    }
    __syncthreads();
    // a lane group's rows, kThreads / LPR apart: head h of token t is the next to be fetched
    int t = tid / LPR / heads, h = tid / LPR % heads;
    const int at_lo = lo * (int)sizeof(T), gap = (hi - lo) * (int)sizeof(T);
    // Two rows a lane group are on their way while one is worked on: bf16 words by asynchronous copies, every lane its own
    // (in registers 128 us, so 121; fp32, whose runs are two words each, 21 and 25 us for 4413 tokens of 18 heads of 128)
    constexpr bool kAsync = VEC && sizeof(T) == 2;
    __shared__ uint4 s_rows[kAsync ? 4 * kThreads : 1];
    uint4* const mine = s_rows + (kAsync ? tid : 0);
    Run<T> u[2], v[2];
    char* to[2];  // or null: no such row
    int of[2];    // its place among the cosines; and k's sign bit
    auto fetch = [&](int s) {
        to[s] = nullptr;
        if (t < nt) {
            const bool isk = h >= a.Hq;
            const char* x = s_at[t][isk];
            if (x) {
                x += h * (isk ? a.k_head : a.q_head) + at_lo;  // (a token's heads span less than 2^31 bytes)
                to[s] = s_to[t][isk] + (h * D * (int)sizeof(T) + at_lo);
                of[s] = (t * 4 * lanes + c) | (isk ? 1 << 31 : 0);
                if (kAsync) {
                    copy16(mine + 2 * s * kThreads, x);
                    copy16(mine + (2 * s + 1) * kThreads, x + gap);
                } else {
                    u[s].template load<VEC>(x);
                    v[s].template load<VEC>(x + gap);
                }
            }
        }
        if (kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
        t += a.dt;
        h += a.dh;
        if (h >= heads) {
            h -= heads;
            ++t;
        }
    };
    fetch(0);
    fetch(1);
    for (int e = tid; e < nt * half; e += kThreads) {
        const int t = e / half, i = e - t * half;
        const unsigned long long turn = (unsigned long long)(long long)a.position[first + t] * fr.f[i];
        float s, co;
        sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &co);  // half turns: 2^-31
        float* to = reinterpret_cast<float*>(s_cs + (t * 4 + i % 8 / 2) * lanes + i / 8) + i % 2;
        to[0] = co;
        to[2] = s;
    }
    for (int e = tid; e < 2 * D; e += kThreads) {
        // channel ch is the j-th of its lane: of the low run 0..7, of the high one 8..15
        const int x = e / D, ch = e % D, of = ch < a.rot ? ch : ch - a.rot, size = ch < a.rot ? half : rest;
        const int high = of >= size ? 8 : 0, k = (ch < a.rot ? 0 : lanes) + (high ? of - size : of) / 8, j = high + ch % 8;
        reinterpret_cast<float*>(s_w[x])[(j / 4 * LPR + k) * 4 + j % 4] =
            a.offset + to_f32(static_cast<const T*>(x ? a.kw : a.qw)[(long long)l * D + ch]);
    }
    __syncthreads();
    const int steps = (nt * heads + kThreads / LPR - 1) / (kThreads / LPR);
    for (int step = 0; step < steps; step += 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (kAsync) asm volatile("cp.async.wait_group 1;" ::: "memory");
            if (!to[s]) {
                fetch(s);
                continue;
            }
            T* const y = reinterpret_cast<T*>(to[s]);
            const bool isk = of[s] < 0;
            const float4* cs = s_cs + (of[s] & 0x7fffffff);
            if (kAsync) {
                u[s].template load<true>(mine + 2 * s * kThreads);
                v[s].template load<true>(mine + (2 * s + 1) * kThreads);
            }
            F2 p[4], q[4], sum = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = f2(u[s][2 * i], u[s][2 * i + 1]);
                q[i] = f2(v[s][2 * i], v[s][2 * i + 1]);
                sum = fma2(p[i], p[i], fma2(q[i], q[i], sum));
            }
            fetch(s);
            float ss = f2_get(sum).x + f2_get(sum).y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
            const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
            const F2 rr = f2(r, r);
            const float4* w = s_w[isk] + c;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = w[i * LPR], z = w[(2 + i) * LPR];
                p[2 * i] = p[2 * i] * (rr * f2(x.x, x.y));
                p[2 * i + 1] = p[2 * i + 1] * (rr * f2(x.z, x.w));
                q[2 * i] = q[2 * i] * (rr * f2(z.x, z.y));
                q[2 * i + 1] = q[2 * i + 1] * (rr * f2(z.z, z.w));
            }
            if (turned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 k = cs[i * lanes];
                    const F2 co = f2(k.x, k.y), si = f2(k.z, k.w), p0 = p[i];
                    p[i] = p0 * co - q[i] * si;
                    q[i] = fma2(q[i], co, p0 * si);
                }
            }
            store_run<T, VEC>(y, p);
            store_run<T, VEC>(reinterpret_cast<T*>(reinterpret_cast<char*>(y) + gap), q);
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
        const int64_t x = qn[i] > 1 ? q_stride[i] * esz : 0, y = kn[i] > 1 ? k_stride[i] * esz : 0;
        bits |= (uintptr_t)x | (uintptr_t)y;
        if (i == 3) {
            a.q_head = (int)x;
            a.k_head = (int)y;
        } else {
            a.qs[i] = x / esz;
            a.ks[i] = y / esz;
        }
    }
    // frequency i as a product of two powers, 16 + 8 of them at most: a power takes the host some 50 ns
    NormFreq fr{};
    double near[16], far[8];
    for (int i = 0; i < 16 && i < rot / 2; ++i) near[i] = pow(theta, -2.0 * i / rot) * (18446744073709551616.0 / 6.283185307179586477);
    for (int i = 0; i < 8 && 16 * i < rot / 2; ++i) far[i] = pow(theta, -32.0 * i / rot);
    for (int i = 0; i < rot / 2; ++i) fr.f[i] = (unsigned long long)(near[i % 16] * far[i / 16]);
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // tokens a CTA: the fewest steps in all, a CTA's start counted as two (rounds of the resident CTAs, and how
    // full a CTA's last step is)
    const int at_once = kThreads / (d / 16), resident = (dtype == DDT_BF16 ? 4 : 3) * sms;
    long long best = 0;
    for (int t = 1; t <= max_tokens(esz); ++t) {
        const long long ctas = ((long long)B * N + t - 1) / t * L;
        const long long steps = (ctas + resident - 1) / resident * (2 + ((long long)t * (Hq + Hkv) + at_once - 1) / at_once);
        if (t == 1 || steps < best) {
            best = steps;
            a.tokens = t;
        }
    }
    a.dt = kThreads / (d / 16) / (Hq + Hkv);
    a.dh = kThreads / (d / 16) % (Hq + Hkv);
    return dtype == DDT_BF16 ? norm_d_go<__nv_bfloat16>(L, d, a, fr, (bits & 15) == 0, st) : norm_d_go<float>(L, d, a, fr, (bits & 15) == 0, st);
}

}  // namespace ddt
