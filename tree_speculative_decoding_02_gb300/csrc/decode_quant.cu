// decode_quant.cu -- k_decode_quant's instances of calls that k_decode_finish joins, and the choice of one.
#include "decode_quant.cuh"

namespace ddt {

// those of clusters are in decode_quant_cluster.cu (two files, compiled side by side)
#define DDT_QUANT_EXTERN(T, D, HP, GH, QP, PP) \
    extern template cudaError_t quant_launch<T, D, HP, GH, QP, PP, true>(const DecodeParams&, const DecQuantArgs&, const CUtensorMap*, cudaStream_t);
DDT_QUANT_INSTANCES(DDT_QUANT_EXTERN)

namespace {

template <typename Tin, int D, int HP, int GH, int QP, int PP>
cudaError_t quant_go(DecodeParams& p, const DecQuantArgs& a, const CUtensorMap* maps, cudaStream_t st) {
    decode_clusters(p, DecodeSmall{1024., 896.}, QuantCfg<D, HP, GH, QP, PP>::kCtas);
    return p.cl ? quant_launch<Tin, D, HP, GH, QP, PP, true>(p, a, maps, st) : quant_launch<Tin, D, HP, GH, QP, PP, false>(p, a, maps, st);
}

template <int D>
cudaError_t quant_d_go(DecodeParams& p, ddt_dtype in, const DecQuantArgs& a, const CUtensorMap* maps, cudaStream_t st) {
    if (in == DDT_F32) return p.hbs == 8 ? quant_go<float, D, 8, 8, 6, 6>(p, a, maps, st) : quant_go<float, D, 16, 8, 6, 6>(p, a, maps, st);
    return p.G <= 2      ? quant_go<__nv_bfloat16, D, 8, 2, 2, 4>(p, a, maps, st)
           : p.G <= 4    ? quant_go<__nv_bfloat16, D, 8, 4, 2, 4>(p, a, maps, st)
           : p.hbs == 8  ? quant_go<__nv_bfloat16, D, 8, 8, 2, 4>(p, a, maps, st)
           : p.hbs == 16 ? quant_go<__nv_bfloat16, D, 16, 8, 2, 4>(p, a, maps, st)
                         : quant_go<__nv_bfloat16, D, 32, 8, 2, 4>(p, a, maps, st);
}

}  // namespace

// heads a block: the smallest of 8, 16 and 32 that holds the group (16 at most where the parts are six: N of P V)
int decode_quant_heads(int G, ddt_dtype in) { return G <= 8 ? 8 : (G <= 16 || in == DDT_F32 ? 16 : 32); }

// p.C: SMs on entry, CTAs on return
cudaError_t launch_decode_quant_tiles(DecodeParams& p, ddt_dtype in, cudaStream_t st) {
    EncodeTiledFn enc = decode_encode_fn();
    if (!enc) return cudaErrorNotSupported;
    DecQuantArgs a{p.page_rows % 128 == 0 ? 128 : (p.page_rows < 64 ? p.page_rows : 64)};
    CUtensorMap maps[2];
    const int row = p.d < 128 ? p.d : 128;
    const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.page_rows, (cuuint64_t)p.L * p.num_pages * p.Hkv};
    const cuuint64_t str[2] = {(cuuint64_t)p.d, (cuuint64_t)p.page_rows * p.d};
    const cuuint32_t box[3] = {(cuuint32_t)row, (cuuint32_t)a.sub, 1}, es[3] = {1, 1, 1};
    const void* base[2] = {p.k_pages, p.v_pages};
    for (int i = 0; i < 2; ++i)
        if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base[i]), dims, str, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    return p.d == 64 ? quant_d_go<64>(p, in, a, maps, st) : (p.d == 128 ? quant_d_go<128>(p, in, a, maps, st) : quant_d_go<256>(p, in, a, maps, st));
}

}  // namespace ddt
