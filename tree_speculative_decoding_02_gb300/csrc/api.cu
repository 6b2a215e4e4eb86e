// api.cu -- the extern "C" entry points of ddt.h: host-side argument checks, then
// stream-ordered kernel launches.  No device memory is allocated here and no host
// synchronisation happens; data errors found on the device go to the status words.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <initializer_list>

#include "ddt.h"
#include "kernels.h"

using namespace ddt;

namespace ddt {
static std::atomic<uint64_t> g_launches{0};
void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }
}  // namespace ddt

namespace {

inline ddt_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return DDT_OK;
    if (e == cudaErrorInvalidValue) return DDT_ERR_UNSUPPORTED;
    return DDT_ERR_CUDA;
}
inline bool dtype_ok(ddt_dtype t) { return t == DDT_F32 || t == DDT_BF16; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" {

const char* ddt_status_string(ddt_status s) {
    switch (s) {
        case DDT_OK: return "ok";
        case DDT_ERR_INVALID_ARG: return "invalid argument";
        case DDT_ERR_UNSUPPORTED: return "unsupported size or dtype combination";
        case DDT_ERR_CAPACITY: return "cache capacity exceeded";
        case DDT_ERR_CUDA: return "CUDA launch error";
        case DDT_ERR_TIMEOUT: return "bounded device wait gave up";
        case DDT_ERR_NONFINITE: return "non-finite logits";
        case DDT_ERR_TREE: return "malformed tree";
    }
    return "unknown status";
}

const char* ddt_version(void) { return "ddt 0.1 sm_103a"; }

uint64_t ddt_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

ddt_status ddt_wait_selftest(int32_t* status, ddt_stream_t stream) {
    if (!status) return DDT_ERR_INVALID_ARG;
    return launch_wait_selftest(status, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DDT_OK
                                                                                            : DDT_ERR_CUDA;
}

// ------------------------------------------------------------------------- build
size_t ddt_build_tree_workspace(int B, int D, int V, int top_k) {
    if (B < 1 || D < 1 || V < 1 || top_k < 1) return 0;
    return build_ws_bytes(B, D, V, top_k);
}

ddt_status ddt_build_tree(int B, int D, int V, int top_k, int budget, ddt_dtype dtype, const void* draft_logits,
                          const int32_t* root_token, const int32_t* prefix_len, int32_t* token, int32_t* parent,
                          int32_t* depth, int32_t* position, int32_t* n_nodes, uint32_t* anc, double* score,
                          int32_t* status, void* workspace, size_t ws_bytes, ddt_stream_t stream) {
    if (B < 1 || D < 1 || V < 1 || top_k < 1 || budget < 0 || !dtype_ok(dtype)) return DDT_ERR_INVALID_ARG;
    if (D > kMaxDepth || top_k > kMaxTopK || top_k > V || budget > kMaxBudget) return DDT_ERR_UNSUPPORTED;
    if (!draft_logits || !root_token || !prefix_len || !token || !parent || !depth || !position || !n_nodes ||
        !anc || !status || !workspace)
        return DDT_ERR_INVALID_ARG;
    if (ws_bytes < build_ws_bytes(B, D, V, top_k) || !aligned16(workspace)) return DDT_ERR_INVALID_ARG;
    if (build_tree_smem(D, top_k, budget) > 200 * 1024) return DDT_ERR_UNSUPPORTED;
    return from_cuda(launch_build_tree(B, D, V, top_k, budget, dtype, draft_logits, root_token, prefix_len, token,
                                       parent, depth, position, n_nodes, anc, score, status, workspace,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------------ attention
size_t ddt_tree_attn_workspace(int n_layers, int B, int N, int Hq, int Hkv, int d, int Pcap) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Pcap < 0) return 0;
    return attn_tc_ws_bytes(n_layers, B, N, Hq, Hkv, d, Pcap);
}

ddt_status ddt_tree_attn(int n_layers, int B, int N, int Hq, int Hkv, int d, int Pcap, ddt_dtype in_dtype,
                         ddt_dtype out_dtype, const void* q, const void* k_tree, const void* v_tree,
                         const void* k_cache, const void* v_cache, const int32_t* prefix_len, const int32_t* n_nodes,
                         const uint32_t* anc, float scale, void* o, int32_t* status, void* workspace,
                         size_t ws_bytes, ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Pcap < 0 || !dtype_ok(in_dtype) ||
        !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return DDT_ERR_INVALID_ARG;
    if (N > kMaxRows || (d != 64 && d != 128 && d != 256)) return DDT_ERR_UNSUPPORTED;
    if (!q || !k_tree || !v_tree || (Pcap > 0 && (!k_cache || !v_cache)) || !prefix_len || !n_nodes || !anc || !o ||
        !status)
        return DDT_ERR_INVALID_ARG;
    // bf16 with a compiled head size runs on the tensor cores; fp32 on the CUDA cores
    if (attn_tc_supported(d, in_dtype)) {
        if (!workspace || ws_bytes < attn_tc_ws_bytes(n_layers, B, N, Hq, Hkv, d, Pcap) || !aligned16(workspace))
            return DDT_ERR_INVALID_ARG;
        if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(o) ||
            (Pcap > 0 && (!aligned16(k_cache) || !aligned16(v_cache))))
            return DDT_ERR_INVALID_ARG;
        return from_cuda(launch_attn_tc(n_layers, B, N, Hq, Hkv, d, Pcap, out_dtype, q, k_tree, v_tree, k_cache,
                                        v_cache, prefix_len, n_nodes, anc, scale, o, status, workspace, ws_bytes,
                                        reinterpret_cast<cudaStream_t>(stream)));
    }
    return from_cuda(launch_attn_simt(n_layers, B, N, Hq, Hkv, d, Pcap, in_dtype, out_dtype, q, k_tree, v_tree,
                                      k_cache, v_cache, prefix_len, n_nodes, anc, scale, o, status,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

static bool page_rows_ok(int r) { return r >= 8 && r <= 4096 && (r >= 64 ? r % 64 == 0 : 64 % r == 0); }

size_t ddt_tree_attn_paged_workspace(int n_layers, int B, int N, int Hq, int Hkv, int d, int page_size,
                                     int max_pages) {
    if (!page_rows_ok(page_size) || max_pages < 1) return 0;
    return ddt_tree_attn_workspace(n_layers, B, N, Hq, Hkv, d, page_size * max_pages);
}

ddt_status ddt_tree_attn_paged(int n_layers, int B, int N, int Hq, int Hkv, int d, int page_size, int num_pages,
                               int max_pages, ddt_dtype in_dtype, ddt_dtype out_dtype, const void* q,
                               const void* k_tree, const void* v_tree, const void* k_pages, const void* v_pages,
                               const int32_t* block_table, const int32_t* prefix_len, const int32_t* n_nodes,
                               const uint32_t* anc, float scale, void* o, int32_t* status, void* workspace,
                               size_t ws_bytes, ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_pages < 1 || max_pages < 1 ||
        !dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (!page_rows_ok(page_size) || (long)page_size * max_pages > (1L << 30)) return DDT_ERR_UNSUPPORTED;
    if (N > kMaxRows || !attn_tc_supported(d, in_dtype)) return DDT_ERR_UNSUPPORTED;
    if (!q || !k_tree || !v_tree || !k_pages || !v_pages || !block_table || !prefix_len || !n_nodes || !anc || !o ||
        !status)
        return DDT_ERR_INVALID_ARG;
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    if (!workspace || ws_bytes < attn_tc_ws_bytes(n_layers, B, N, Hq, Hkv, d, page_size * max_pages) ||
        !aligned16(workspace))
        return DDT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(o) || !aligned16(k_pages) ||
        !aligned16(v_pages))
        return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_attn_tc_paged(n_layers, B, N, Hq, Hkv, d, pg, out_dtype, q, k_tree, v_tree, k_pages,
                                          v_pages, prefix_len, n_nodes, anc, scale, o, status, workspace, ws_bytes,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

ddt_status ddt_rope_tree(int n_layers, int B, int N, int Hq, int Hkv, int d, int rot_dim, double theta,
                         ddt_dtype dtype, const int32_t* position, const int32_t* n_nodes, void* q, void* k_tree,
                         ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || d < 2 || !dtype_ok(dtype)) return DDT_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim > d || rot_dim % 2 != 0 || !(theta > 1.0)) return DDT_ERR_INVALID_ARG;
    if (!position || !n_nodes || !k_tree) return DDT_ERR_INVALID_ARG;  // q NULL: rotate the keys only
    if (B > 65535) return DDT_ERR_UNSUPPORTED;
    return from_cuda(launch_rope_tree(n_layers, B, N, Hq, Hkv, d, rot_dim, theta, dtype, position, n_nodes, q, k_tree,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

// Rotary variants: q is taken before rotary embedding and rotated while the attention
// kernel stages it; the cos/sin table of every row's position goes to the end of the
// workspace (after the ddt_tree_attn(_paged)_workspace bytes).
static size_t rope_table_offset(size_t base) { return (base + 255) & ~(size_t)255; }

static ddt_status rope_args_ok(int d, ddt_dtype in_dtype, int rot_dim, double theta, const int32_t* position) {
    if (!position || rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0 || !(theta > 1.0)) return DDT_ERR_INVALID_ARG;
    if (in_dtype != DDT_BF16 || (d != 128 && d != 256)) return DDT_ERR_UNSUPPORTED;
    return DDT_OK;
}

ddt_status ddt_tree_attn_rope(int n_layers, int B, int N, int Hq, int Hkv, int d, int Pcap, ddt_dtype in_dtype,
                              ddt_dtype out_dtype, const void* q, const void* k_tree, const void* v_tree,
                              const void* k_cache, const void* v_cache, const int32_t* prefix_len,
                              const int32_t* n_nodes, const uint32_t* anc, const int32_t* position, int rot_dim,
                              double theta, float scale, void* o, int32_t* status, void* workspace, size_t ws_bytes,
                              ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Pcap < 0 || Hq % Hkv != 0 || !dtype_ok(in_dtype) ||
        !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (N > kMaxRows || B > 65535) return DDT_ERR_UNSUPPORTED;
    const ddt_status ra = rope_args_ok(d, in_dtype, rot_dim, theta, position);
    if (ra != DDT_OK) return ra;
    if (!q || !k_tree || !v_tree || (Pcap > 0 && (!k_cache || !v_cache)) || !prefix_len || !n_nodes || !anc || !o ||
        !status || !workspace || !aligned16(workspace))
        return DDT_ERR_INVALID_ARG;
    const size_t base = attn_tc_ws_bytes(n_layers, B, N, Hq, Hkv, d, Pcap);
    const size_t off = rope_table_offset(base);
    if (ws_bytes < off + sizeof(float) * (size_t)B * N * rot_dim) return DDT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(o) ||
        (Pcap > 0 && (!aligned16(k_cache) || !aligned16(v_cache))))
        return DDT_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float* table = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + off);
    cudaError_t e = launch_rope_table(B, N, rot_dim, theta, position, n_nodes, table, st);
    if (e != cudaSuccess) return from_cuda(e);
    const AttnRope rope{rot_dim, table};
    return from_cuda(launch_attn_tc(n_layers, B, N, Hq, Hkv, d, Pcap, out_dtype, q, k_tree, v_tree, k_cache, v_cache,
                                    prefix_len, n_nodes, anc, scale, o, status, workspace, base, st, &rope));
}

ddt_status ddt_tree_attn_paged_rope(int n_layers, int B, int N, int Hq, int Hkv, int d, int page_size, int num_pages,
                                    int max_pages, ddt_dtype in_dtype, ddt_dtype out_dtype, const void* q,
                                    const void* k_tree, const void* v_tree, const void* k_pages, const void* v_pages,
                                    const int32_t* block_table, const int32_t* prefix_len, const int32_t* n_nodes,
                                    const uint32_t* anc, const int32_t* position, int rot_dim, double theta,
                                    float scale, void* o, int32_t* status, void* workspace, size_t ws_bytes,
                                    ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_pages < 1 || max_pages < 1 ||
        !dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (!page_rows_ok(page_size) || (long)page_size * max_pages > (1L << 30)) return DDT_ERR_UNSUPPORTED;
    if (N > kMaxRows || B > 65535) return DDT_ERR_UNSUPPORTED;
    const ddt_status ra = rope_args_ok(d, in_dtype, rot_dim, theta, position);
    if (ra != DDT_OK) return ra;
    if (!q || !k_tree || !v_tree || !k_pages || !v_pages || !block_table || !prefix_len || !n_nodes || !anc || !o ||
        !status || !workspace || !aligned16(workspace))
        return DDT_ERR_INVALID_ARG;
    const size_t base = attn_tc_ws_bytes(n_layers, B, N, Hq, Hkv, d, page_size * max_pages);
    const size_t off = rope_table_offset(base);
    if (ws_bytes < off + sizeof(float) * (size_t)B * N * rot_dim) return DDT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(o) || !aligned16(k_pages) ||
        !aligned16(v_pages))
        return DDT_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float* table = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + off);
    cudaError_t e = launch_rope_table(B, N, rot_dim, theta, position, n_nodes, table, st);
    if (e != cudaSuccess) return from_cuda(e);
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    const AttnRope rope{rot_dim, table};
    return from_cuda(launch_attn_tc_paged(n_layers, B, N, Hq, Hkv, d, pg, out_dtype, q, k_tree, v_tree, k_pages,
                                          v_pages, prefix_len, n_nodes, anc, scale, o, status, workspace, base, st,
                                          &rope));
}

// ------------------------------------------------------------------------------ GDN
size_t ddt_tree_gdn_workspace(int n_layers, int B, int N, int Hk, int Hv, int dk, int dv) {
    (void)n_layers; (void)B; (void)N; (void)Hk; (void)Hv; (void)dk; (void)dv;
    return 256;
}

ddt_status ddt_tree_gdn(int n_layers, int B, int N, int Hk, int Hv, int dk, int dv, int conv_k, ddt_dtype in_dtype,
                        ddt_dtype out_dtype, const void* x, const void* conv_w, const void* conv_state,
                        const float* beta, const float* decay, const float* S, const int32_t* parent,
                        const int32_t* n_nodes, void* o, float* S_node_debug, int32_t* status, void* workspace,
                        size_t ws_bytes, ddt_stream_t stream) {
    (void)workspace; (void)ws_bytes;
    if (n_layers < 1 || B < 1 || N < 1 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || conv_k < 1 || !dtype_ok(in_dtype) ||
        !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    const bool dims = (dk == 32 && dv == 32) || (dk == 64 && dv == 64) || (dk == 128 && dv == 128) ||
                      (dk == 64 && dv == 128) || (dk == 128 && dv == 64);
    if (!dims || conv_k > 8 || N > kGdnMaxNodes || gdn_smem_bytes(N, dk, dv) > 227 * 1024) return DDT_ERR_UNSUPPORTED;
    if (!x || !conv_w || (conv_k > 1 && !conv_state) || !beta || !decay || !S || !parent || !n_nodes || !o ||
        !status || !aligned16(S))
        return DDT_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    // head size 128: dense part on the tensor cores (its TMA row loads want x and the conv
    // state 16-byte aligned); other sizes on the CUDA cores
    if (gdn_tc_supported(N, Hk, Hv, dk, dv, conv_k, in_dtype) && aligned16(x) && (conv_k == 1 || aligned16(conv_state)))
        e = launch_gdn_tc(n_layers, B, N, Hk, Hv, conv_k, in_dtype, out_dtype, x, conv_w, conv_state, beta, decay, S,
                          parent, n_nodes, o, status, st);
    else
        e = launch_gdn_tree(n_layers, B, N, Hk, Hv, dk, dv, conv_k, in_dtype, out_dtype, x, conv_w, conv_state, beta,
                            decay, S, parent, n_nodes, o, status, st);
    if (e == cudaSuccess && S_node_debug)
        e = launch_gdn_states(n_layers, B, N, Hk, Hv, dk, dv, conv_k, in_dtype, x, conv_w, conv_state, beta, decay,
                              S, parent, n_nodes, S_node_debug, st);
    return from_cuda(e);
}

// ----------------------------------------------------------------------------- walk
size_t ddt_walk_accept_workspace(int B, int N, int V) {
    if (B < 1 || N < 1 || V < 1) return 0;
    return walk_ws_bytes(B, N, V);
}

static ddt_status walk_accept(int B, int N, int V, int max_accept, ddt_dtype dtype, const void* target_logits,
                              int32_t* target_argmax, const int32_t* token, const int32_t* parent,
                              const int32_t* n_nodes, int32_t* acc_nodes, int32_t* acc_len, int32_t* bonus,
                              int32_t* emitted, int32_t* n_emitted, int32_t* status, void* workspace, size_t ws_bytes,
                              int flat, ddt_stream_t stream) {
    if (B < 1 || N < 1 || V < 1 || max_accept < 0 || !dtype_ok(dtype)) return DDT_ERR_INVALID_ARG;
    if (N > kMaxRows) return DDT_ERR_UNSUPPORTED;
    if (!target_argmax || !token || !parent || !n_nodes || !acc_nodes || !acc_len || !bonus || !emitted ||
        !n_emitted || !status)
        return DDT_ERR_INVALID_ARG;
    if (target_logits && (!workspace || ws_bytes < walk_ws_bytes(B, N, V) || !aligned16(workspace)))
        return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_walk(B, N, V, max_accept + 1, dtype, target_logits, target_argmax, token, parent, n_nodes,
                                 acc_nodes, acc_len, bonus, emitted, n_emitted, status, workspace, flat,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

ddt_status ddt_walk_accept(int B, int N, int V, int max_accept, ddt_dtype dtype, const void* target_logits,
                           int32_t* target_argmax, const int32_t* token, const int32_t* parent,
                           const int32_t* n_nodes, int32_t* acc_nodes, int32_t* acc_len, int32_t* bonus,
                           int32_t* emitted, int32_t* n_emitted, int32_t* status, void* workspace, size_t ws_bytes,
                           ddt_stream_t stream) {
    return walk_accept(B, N, V, max_accept, dtype, target_logits, target_argmax, token, parent, n_nodes, acc_nodes,
                       acc_len, bonus, emitted, n_emitted, status, workspace, ws_bytes, 0, stream);
}

ddt_status ddt_walk_accept_flat(int B, int N, int V, int max_accept, ddt_dtype dtype, const void* target_logits,
                                int32_t* target_argmax, const int32_t* token, const int32_t* parent,
                                const int32_t* n_nodes, int32_t* acc_nodes, int32_t* acc_len, int32_t* bonus,
                                int32_t* emitted, int32_t* n_emitted, int32_t* status, void* workspace,
                                size_t ws_bytes, ddt_stream_t stream) {
    return walk_accept(B, N, V, max_accept, dtype, target_logits, target_argmax, token, parent, n_nodes, acc_nodes,
                       acc_len, bonus, emitted, n_emitted, status, workspace, ws_bytes, 1, stream);
}

size_t ddt_walk_accept_sample_workspace(int B, int N, int V) {
    if (B < 1 || N < 1 || V < 1) return 0;
    return walk_sample_ws_bytes(B, N, V);
}

ddt_status ddt_walk_accept_sample(int B, int N, int V, int max_accept, int max_children, float temperature,
                                  ddt_dtype dtype, const void* target_logits, const float* uniforms,
                                  const int32_t* token, const int32_t* parent, const int32_t* n_nodes,
                                  int32_t* acc_nodes, int32_t* acc_len, int32_t* bonus, int32_t* emitted,
                                  int32_t* n_emitted, int32_t* status, void* workspace, size_t ws_bytes,
                                  ddt_stream_t stream) {
    if (B < 1 || N < 1 || V < 1 || max_accept < 0 || max_children < 1 || !dtype_ok(dtype)) return DDT_ERR_INVALID_ARG;
    // T > 0 with a finite fp32 reciprocal (the kernels scale by 1/T)
    if (!(temperature > 0.0f) || !(1.0f / temperature < INFINITY) || !(temperature < INFINITY))
        return DDT_ERR_INVALID_ARG;
    if (N > kMaxRows || B > 65535 || max_accept > kMaxAccept || max_children > kMaxTopK) return DDT_ERR_UNSUPPORTED;
    if (!target_logits || !uniforms || !token || !parent || !n_nodes || !acc_nodes || !acc_len || !bonus ||
        !emitted || !n_emitted || !status)
        return DDT_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < walk_sample_ws_bytes(B, N, V) || !aligned16(workspace)) return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_walk_sample(B, N, V, max_accept + 1, max_children, temperature, dtype, target_logits,
                                        uniforms, token, parent, n_nodes, acc_nodes, acc_len, bonus, emitted,
                                        n_emitted, status, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------------------- commit
ddt_status ddt_commit(int B, int N, int A, int n_attn_layers, int Hkv, int d, int Pcap, ddt_dtype kv_dtype,
                      const void* k_tree, const void* v_tree, void* k_cache, void* v_cache, int n_gdn_layers, int Hk,
                      int Hv, int dk, int dv, int conv_k, ddt_dtype x_dtype, const void* x, const void* conv_w,
                      const float* beta, const float* decay, float* S, void* conv_state, const int32_t* acc_nodes,
                      const int32_t* acc_len, int32_t* prefix_len, int32_t* src_row, int32_t* dst_pos,
                      int32_t* status, ddt_stream_t stream) {
    if (B < 1 || N < 1 || A < 1 || n_attn_layers < 0 || n_gdn_layers < 0) return DDT_ERR_INVALID_ARG;
    if (A > kMaxAccept + 1) return DDT_ERR_UNSUPPORTED;
    if (!acc_nodes || !acc_len || !prefix_len || !src_row || !dst_pos || !status) return DDT_ERR_INVALID_ARG;
    if (n_attn_layers > 0) {
        if (Hkv < 1 || d < 1 || Pcap < 1 || !dtype_ok(kv_dtype) || !k_tree || !v_tree || !k_cache || !v_cache)
            return DDT_ERR_INVALID_ARG;
    }
    if (n_gdn_layers > 0) {
        if (Hk < 1 || Hv < 1 || Hv % Hk != 0 || conv_k < 1 || conv_k > 8 || !dtype_ok(x_dtype) || !x || !conv_w ||
            !beta || !decay || !S || (conv_k > 1 && !conv_state) || !aligned16(S))
            return DDT_ERR_INVALID_ARG;
        const bool dims = (dk == 32 && dv == 32) || (dk == 64 && dv == 64) || (dk == 128 && dv == 128) ||
                          (dk == 64 && dv == 128) || (dk == 128 && dv == 64);
        if (!dims) return DDT_ERR_UNSUPPORTED;
    }
    return from_cuda(launch_commit(B, N, A, n_attn_layers, Hkv, d, Pcap, kv_dtype, k_tree, v_tree, k_cache, v_cache,
                                   n_gdn_layers, Hk, Hv, dk, dv, conv_k, x_dtype, x, conv_w, beta, decay, S,
                                   conv_state, acc_nodes, acc_len, prefix_len, src_row, dst_pos, status, nullptr,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

ddt_status ddt_commit_paged(int B, int N, int A, int n_attn_layers, int Hkv, int d, int page_size, int num_pages,
                            int max_pages, const int32_t* block_table, ddt_dtype kv_dtype, const void* k_tree,
                            const void* v_tree, void* k_pages, void* v_pages, int n_gdn_layers, int Hk, int Hv, int dk,
                            int dv, int conv_k, ddt_dtype x_dtype, const void* x, const void* conv_w,
                            const float* beta, const float* decay, float* S, void* conv_state,
                            const int32_t* acc_nodes, const int32_t* acc_len, int32_t* prefix_len, int32_t* src_row,
                            int32_t* dst_pos, int32_t* status, ddt_stream_t stream) {
    if (n_attn_layers < 1 || !block_table || num_pages < 1 || max_pages < 1) return DDT_ERR_INVALID_ARG;
    if (!page_rows_ok(page_size) || (long)page_size * max_pages > (1L << 30)) return DDT_ERR_UNSUPPORTED;
    if (B < 1 || N < 1 || A < 1 || n_gdn_layers < 0) return DDT_ERR_INVALID_ARG;
    if (A > kMaxAccept + 1) return DDT_ERR_UNSUPPORTED;
    if (!acc_nodes || !acc_len || !prefix_len || !src_row || !dst_pos || !status) return DDT_ERR_INVALID_ARG;
    if (Hkv < 1 || d < 1 || !dtype_ok(kv_dtype) || !k_tree || !v_tree || !k_pages || !v_pages)
        return DDT_ERR_INVALID_ARG;
    if (n_gdn_layers > 0) {
        if (Hk < 1 || Hv < 1 || Hv % Hk != 0 || conv_k < 1 || conv_k > 8 || !dtype_ok(x_dtype) || !x || !conv_w ||
            !beta || !decay || !S || (conv_k > 1 && !conv_state) || !aligned16(S))
            return DDT_ERR_INVALID_ARG;
        const bool dims = (dk == 32 && dv == 32) || (dk == 64 && dv == 64) || (dk == 128 && dv == 128) ||
                          (dk == 64 && dv == 128) || (dk == 128 && dv == 64);
        if (!dims) return DDT_ERR_UNSUPPORTED;
    }
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    return from_cuda(launch_commit(B, N, A, n_attn_layers, Hkv, d, page_size * max_pages, kv_dtype, k_tree, v_tree,
                                   k_pages, v_pages, n_gdn_layers, Hk, Hv, dk, dv, conv_k, x_dtype, x, conv_w, beta,
                                   decay, S, conv_state, acc_nodes, acc_len, prefix_len, src_row, dst_pos, status, &pg,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------- single-token decode
static bool paging_sizes_ok(int page_size, int num_pages, int max_pages) {
    return page_rows_ok(page_size) && (long)page_size * max_pages <= (1L << 30) && num_pages >= 1;
}

// Buffers that a call reads, or writes again, after it has begun to write the other.
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}
struct Span {
    const void* at;
    size_t bytes;
};
// one of the first n_out spans (what a call writes) meets another span; NULL meets none
static bool any_overlap(const Span* s, int n, int n_out) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (s[i].at && s[j].at && overlap(s[i].at, s[i].bytes, s[j].at, s[j].bytes)) return true;
    return false;
}

// the largest grid and plane counts the kernels index with 32 bits
static bool decode_sizes_ok(int n_layers, int B, int Hq, int Hkv, int num_pages) {
    const long most = 0x7fffffffL;
    return (long)n_layers * B <= most / Hq && (long)n_layers * num_pages <= most / Hkv && Hq / Hkv <= 1024;
}

size_t ddt_decode_attn_paged_workspace(int n_layers, int B, int Hq, int Hkv, int d, int page_size, int max_pages,
                                       ddt_dtype in_dtype, int want_weight) {
    if (n_layers < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1 || max_pages < 1 || !dtype_ok(in_dtype) ||
        !paging_sizes_ok(page_size, 1, max_pages))
        return 0;
    return decode_ws_bytes(n_layers, B, Hq, Hkv, d, page_size * max_pages, in_dtype, want_weight != 0);
}

ddt_status ddt_decode_attn_paged(int n_layers, int B, int Hq, int Hkv, int d, int page_size, int num_pages,
                                 int max_pages, ddt_dtype in_dtype, ddt_dtype out_dtype, const void* q,
                                 const void* k_new, const void* v_new, const void* k_pages, const void* v_pages,
                                 const int32_t* block_table, const int32_t* prefix_len, float scale, void* o,
                                 float* attn_weight, int32_t* status, void* workspace, size_t ws_bytes,
                                 ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_pages < 1 || max_pages < 1 ||
        !dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (!paging_sizes_ok(page_size, num_pages, max_pages) || !decode_sizes_ok(n_layers, B, Hq, Hkv, num_pages) ||
        (d != 64 && d != 128 && d != 256))
        return DDT_ERR_UNSUPPORTED;
    if (!q || !k_pages || !v_pages || !block_table || !prefix_len || !o || !status || !workspace || !k_new != !v_new)
        return DDT_ERR_INVALID_ARG;
    const size_t need = decode_ws_bytes(n_layers, B, Hq, Hkv, d, page_size * max_pages, in_dtype, attn_weight != nullptr);
    if (ws_bytes < need || !aligned16(workspace)) return DDT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) ||
        !aligned16(o) || !aligned16(attn_weight))
        return DDT_ERR_INVALID_ARG;
    const size_t n_lb = (size_t)n_layers * B, in = in_dtype == DDT_BF16 ? 2 : 4, n_new = n_lb * Hkv * d * in;
    const Span spans[] = {{o, n_lb * Hq * d * (out_dtype == DDT_BF16 ? 2 : 4)},
                          {attn_weight, n_lb * Hkv * page_size * max_pages * sizeof(float)},
                          {status, B * sizeof(int32_t)},
                          {workspace, need},
                          {q, n_lb * Hq * d * in},
                          {k_new, n_new},
                          {v_new, n_new},
                          {block_table, (size_t)B * max_pages * sizeof(int32_t)},
                          {prefix_len, B * sizeof(int32_t)}};
    if (any_overlap(spans, 9, 4)) return DDT_ERR_INVALID_ARG;
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    return from_cuda(launch_decode(n_layers, B, Hq, Hkv, d, pg, in_dtype, out_dtype, q, k_new, v_new, k_pages, v_pages,
                                   prefix_len, scale, o, attn_weight, status, workspace,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------------------ eviction
size_t ddt_evict_paged_workspace(int n_layers, int B, int Hkv, int page_size, int num_pages, int max_pages) {
    if (n_layers < 1 || B < 1 || Hkv < 1 || max_pages < 1 || !paging_sizes_ok(page_size, num_pages, max_pages)) return 0;
    return evict_ws_bytes(n_layers, B, Hkv, AttnPaging{page_size, num_pages, max_pages, nullptr});
}

ddt_status ddt_evict_paged(int n_layers, int B, int Hkv, int d, int page_size, int num_pages, int max_pages,
                           const int32_t* block_table, ddt_dtype kv_dtype, int keep, int n_sink, int n_recent,
                           void* k_pages, void* v_pages, const int32_t* seq_len, float* attn_weight, int32_t* row_pos,
                           int32_t* prefix_len, int32_t* n_placed, int32_t* status, void* workspace, size_t ws_bytes,
                           ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || Hkv < 1 || d < 1 || num_pages < 1 || max_pages < 1 || !dtype_ok(kv_dtype) || keep < 1 ||
        n_sink < 0 || n_recent < 0 || (long)n_sink + n_recent > keep)
        return DDT_ERR_INVALID_ARG;
    const long row_bytes = (long)d * (kv_dtype == DDT_BF16 ? 2 : 4);
    if (!paging_sizes_ok(page_size, num_pages, max_pages) || !decode_sizes_ok(n_layers, B, Hkv, Hkv, num_pages) ||
        row_bytes % 16 != 0 || row_bytes > 16384 || (long)num_pages * page_size > 0x7fffffffL)
        return DDT_ERR_UNSUPPORTED;
    if (!block_table || !k_pages || !v_pages || !seq_len || !attn_weight || !row_pos || !prefix_len || !n_placed ||
        !status || !workspace)
        return DDT_ERR_INVALID_ARG;
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    const size_t need = evict_ws_bytes(n_layers, B, Hkv, pg);
    if (ws_bytes < need || !aligned16(workspace) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(attn_weight) ||
        !aligned16(row_pos))
        return DDT_ERR_INVALID_ARG;
    const size_t n_b = (size_t)B * sizeof(int32_t), n_rows = (size_t)n_layers * B * Hkv * page_size * max_pages * 4;
    const Span spans[] = {{attn_weight, n_rows}, {row_pos, n_rows}, {prefix_len, n_b},       {n_placed, n_b},
                          {status, n_b},         {workspace, need}, {block_table, n_b * max_pages}, {seq_len, n_b}};
    if (any_overlap(spans, 8, 6)) return DDT_ERR_INVALID_ARG;
    const size_t n_pool = (size_t)n_layers * num_pages * Hkv * page_size * row_bytes;
    if (k_pages != v_pages && overlap(k_pages, n_pool, v_pages, n_pool)) return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_evict(n_layers, B, Hkv, (int)row_bytes, pg, keep, n_sink, n_recent, k_pages, v_pages, seq_len,
                                  attn_weight, row_pos, prefix_len, n_placed, status, workspace,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

// --------------------------------------------------------------------- log probabilities
size_t ddt_token_logprobs_workspace(int B, int A, int V, int top_n) {
    if (B < 1 || A < 1 || V < 1 || top_n < 0) return 0;
    return logprobs_ws_bytes(B, A, V, top_n);
}

ddt_status ddt_token_logprobs(int B, int N, int V, int A, int top_n, float temperature, ddt_dtype dtype,
                              const void* target_logits, const int32_t* node, const int32_t* token, float* logprob,
                              float* entropy, int32_t* top_token, float* top_logprob, int32_t* status, void* workspace,
                              size_t ws_bytes, ddt_stream_t stream) {
    if (B < 1 || N < 1 || V < 1 || A < 1 || top_n < 0 || !dtype_ok(dtype)) return DDT_ERR_INVALID_ARG;
    // T > 0 with log2(e) / T finite in fp32 (the kernels scale by it)
    if (!(temperature > 0.0f) || !((float)(1.4426950408889634 / (double)temperature) < INFINITY) ||
        !(temperature < INFINITY))
        return DDT_ERR_INVALID_ARG;
    if (!node && A != N) return DDT_ERR_INVALID_ARG;
    if (top_n > kMaxTopK || top_n > V || V > (1 << 30) || (long)B * A > 0x7fffffffL / (V / 1024 + 2))
        return DDT_ERR_UNSUPPORTED;
    if (!target_logits || !token || !logprob || !status || !workspace || (top_n > 0 && (!top_token || !top_logprob)))
        return DDT_ERR_INVALID_ARG;
    const size_t need = logprobs_ws_bytes(B, A, V, top_n), esz = dtype == DDT_BF16 ? 2 : 4;
    if (ws_bytes < need || !aligned16(workspace)) return DDT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(target_logits) % esz) return DDT_ERR_INVALID_ARG;
    const size_t n_a = (size_t)B * A * 4;
    const Span spans[] = {{logprob, n_a},
                          {entropy, n_a},
                          {top_token, n_a * top_n},
                          {top_logprob, n_a * top_n},
                          {status, n_a},
                          {workspace, need},
                          {target_logits, (size_t)B * N * V * esz},
                          {node, n_a},
                          {token, n_a}};
    if (any_overlap(spans, 9, 6)) return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_token_logprobs(B, N, V, A, top_n, temperature, dtype, target_logits, node, token, logprob,
                                           entropy, top_token, top_logprob, status, workspace,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ the 8-bit paged cache
// rows a scale: a power of two that divides a page
static bool scale_block_ok(int block, int page_size) { return block >= 8 && block <= 128 && (block & (block - 1)) == 0 && page_size % block == 0; }
// (a page of all heads is indexed with 32 bits)
static bool quant_page_ok(int Hkv, int page_size, int d) { return (long)Hkv * page_size <= 0x7fffffffL / d; }
static bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

ddt_status ddt_qk_norm_rope(int n_layers, int B, int N, int Hq, int Hkv, int d, int rot_dim, double theta, float eps,
                            float weight_offset, ddt_dtype dtype, const void* q, const int64_t* q_stride, const void* k,
                            const int64_t* k_stride, const void* q_weight, const void* k_weight, const int32_t* position,
                            const int32_t* n_nodes, void* q_out, void* k_out, ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || Hq < 1 || Hkv < 1 || !dtype_ok(dtype) || rot_dim < 0 || rot_dim > d ||
        !(theta > 1.0 && theta < INFINITY) || !(eps >= 0.0f && eps < INFINITY) || !(fabsf(weight_offset) < INFINITY))
        return DDT_ERR_INVALID_ARG;
    const long most = 0x7fffffffL;
    if (!head_dim_ok(d) || rot_dim % 16 != 0 || n_layers > 65535 || (long)B * N > most || (long)Hq + Hkv > (1 << 16))
        return DDT_ERR_UNSUPPORTED;
    if (!q || !k || !q_stride || !k_stride || !q_weight || !k_weight || !position || !q_out || !k_out) return DDT_ERR_INVALID_ARG;
    const int esz = dtype == DDT_BF16 ? 2 : 4;
    for (const void* p : {q, k, q_weight, k_weight, (const void*)q_out, (const void*)k_out})
        if (reinterpret_cast<uintptr_t>(p) % esz) return DDT_ERR_INVALID_ARG;
    // the spans of the inputs; in place only over rows that lie as the output's do
    const int64_t n[2][4] = {{n_layers, B, N, Hq}, {n_layers, B, N, Hkv}};
    const int64_t* stride[2] = {q_stride, k_stride};
    const void* in[2] = {q, k};
    void* out[2] = {q_out, k_out};
    size_t span[2], size[2];
    bool same[2];
    for (int x = 0; x < 2; ++x) {
        int64_t last = 0, dense = d;
        same[x] = in[x] == out[x];
        for (int i = 3; i >= 0; --i) {
            if (n[x][i] > 1 && stride[x][i] < 0) return DDT_ERR_INVALID_ARG;
            if (n[x][i] > 1 && stride[x][i] > (i == 3 ? (0x7fffffff / esz - d) / (Hq + Hkv) : (INT64_C(1) << 56) / n[x][i])) return DDT_ERR_UNSUPPORTED;
            if (n[x][i] > 1) last += (n[x][i] - 1) * stride[x][i];
            same[x] = same[x] && (n[x][i] == 1 || stride[x][i] == dense);
            dense *= n[x][i];
        }
        span[x] = (size_t)(last + d) * esz;
        size[x] = (size_t)dense * esz;
    }
    const size_t n_w = (size_t)n_layers * d * esz;
    const Span spans[] = {{q_out, size[0]},      {k_out, size[1]},      {same[0] ? nullptr : q, span[0]},
                          {same[1] ? nullptr : k, span[1]}, {q_weight, n_w}, {k_weight, n_w},
                          {position, (size_t)B * N * 4}, {n_nodes, (size_t)B * 4}};
    if (any_overlap(spans, 8, 2)) return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_qk_norm_rope(n_layers, B, N, Hq, Hkv, d, rot_dim, theta, eps, weight_offset, dtype, q, q_stride, k,
                                         k_stride, q_weight, k_weight, position, n_nodes, q_out, k_out,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

ddt_status ddt_append_paged_quant(int n_layers, int B, int N, int A, int Hkv, int d, int page_size, int num_pages,
                                  int max_pages, int block, ddt_dtype in_dtype, const void* k, const void* v,
                                  const int32_t* node, const int32_t* count, const int32_t* block_table,
                                  int32_t* prefix_len, int advance, void* k_pages, void* v_pages, uint8_t* k_scale,
                                  uint8_t* v_scale, int32_t* status, ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || N < 1 || A < 1 || Hkv < 1 || num_pages < 1 || max_pages < 1 || !dtype_ok(in_dtype) ||
        (!node && A > N))
        return DDT_ERR_INVALID_ARG;
    if (!paging_sizes_ok(page_size, num_pages, max_pages) || !decode_sizes_ok(n_layers, B, Hkv, Hkv, num_pages) ||
        !head_dim_ok(d) || !scale_block_ok(block, page_size) || !quant_page_ok(Hkv, page_size, d) || (node && A > kMaxRows) || A > (1 << 30) ||
        (long)n_layers * B > 65535 || Hkv > 32767)
        return DDT_ERR_UNSUPPORTED;
    if (!k || !v || !count || !block_table || !prefix_len || !k_pages || !v_pages || !k_scale || !v_scale || !status)
        return DDT_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages)) return DDT_ERR_INVALID_ARG;
    const size_t n_b = (size_t)B * 4, n_in = (size_t)n_layers * B * N * Hkv * d * (in_dtype == DDT_BF16 ? 2 : 4),
                 n_rows = (size_t)n_layers * num_pages * Hkv * page_size;
    const Span spans[] = {{k_pages, n_rows * d},     {v_pages, n_rows * d}, {k_scale, n_rows / block},
                          {v_scale, n_rows / block}, {status, n_b},         {prefix_len, n_b},
                          {k, n_in},                 {v, n_in},             {node, n_b * A},
                          {count, n_b},              {block_table, n_b * max_pages}};
    if (any_overlap(spans, 11, 6)) return DDT_ERR_INVALID_ARG;
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    return from_cuda(launch_append_quant(n_layers, B, N, A, Hkv, d, block, pg, in_dtype, k, v, node, count, prefix_len,
                                         advance, k_pages, v_pages, k_scale, v_scale, status,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

ddt_status ddt_read_paged_quant(int n_layers, int B, int Hkv, int d, int Pcap, int page_size, int num_pages, int max_pages,
                                int block, ddt_dtype out_dtype, const void* k_pages, const void* v_pages,
                                const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                                const int32_t* prefix_len, void* k_out, void* v_out, int32_t* status, ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || Hkv < 1 || Pcap < 1 || num_pages < 1 || max_pages < 1 || !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (!paging_sizes_ok(page_size, num_pages, max_pages) || !decode_sizes_ok(n_layers, B, Hkv, Hkv, num_pages) ||
        !head_dim_ok(d) || !scale_block_ok(block, page_size) || !quant_page_ok(Hkv, page_size, d) || Pcap > (1 << 30) || (long)n_layers * B > 65535 || Hkv > 32767)
        return DDT_ERR_UNSUPPORTED;
    if (!k_pages || !v_pages || !k_scale || !v_scale || !block_table || !prefix_len || !k_out || !v_out || !status)
        return DDT_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_out) || !aligned16(v_out)) return DDT_ERR_INVALID_ARG;
    const size_t n_b = (size_t)B * 4, n_out = (size_t)n_layers * B * Hkv * Pcap * d * (out_dtype == DDT_BF16 ? 2 : 4),
                 n_rows = (size_t)n_layers * num_pages * Hkv * page_size;
    const Span spans[] = {{k_out, n_out},      {v_out, n_out},            {status, n_b},
                          {k_pages, n_rows * d}, {v_pages, n_rows * d},   {k_scale, n_rows / block},
                          {v_scale, n_rows / block}, {block_table, n_b * max_pages}, {prefix_len, n_b}};
    if (any_overlap(spans, 9, 3)) return DDT_ERR_INVALID_ARG;
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    return from_cuda(launch_read_quant(n_layers, B, Hkv, d, block, Pcap, pg, out_dtype, k_pages, v_pages, k_scale, v_scale,
                                       prefix_len, k_out, v_out, status, reinterpret_cast<cudaStream_t>(stream)));
}

ddt_status ddt_chain_status(int n, int B, const int32_t* status, const int32_t* length, int32_t* length_out,
                            int32_t* status_out, ddt_stream_t stream) {
    if (n < 1 || B < 1 || !status || !length != !length_out || (!length_out && !status_out)) return DDT_ERR_INVALID_ARG;
    const size_t n_b = (size_t)B * 4;
    const Span spans[] = {{length_out, n_b}, {status_out, n_b}, {status, n_b * n}, {length, n_b}};
    if (any_overlap(spans, 4, 2)) return DDT_ERR_INVALID_ARG;
    return from_cuda(launch_chain_status(n, B, status, length, length_out, status_out, reinterpret_cast<cudaStream_t>(stream)));
}

size_t ddt_decode_attn_paged_quant_workspace(int n_layers, int B, int Hq, int Hkv, int d, ddt_dtype in_dtype) {
    if (n_layers < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1 || !dtype_ok(in_dtype)) return 0;
    return decode_quant_ws_bytes(n_layers, B, Hq, Hkv, d, in_dtype);
}

ddt_status ddt_decode_attn_paged_quant(int n_layers, int B, int Hq, int Hkv, int d, int page_size, int num_pages,
                                       int max_pages, int block, ddt_dtype in_dtype, ddt_dtype out_dtype, const void* q,
                                       const void* k_new, const void* v_new, const void* k_pages, const void* v_pages,
                                       const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table,
                                       const int32_t* prefix_len, float scale, void* o, int32_t* status, void* workspace,
                                       size_t ws_bytes, ddt_stream_t stream) {
    if (n_layers < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_pages < 1 || max_pages < 1 ||
        !dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return DDT_ERR_INVALID_ARG;
    if (!paging_sizes_ok(page_size, num_pages, max_pages) || !decode_sizes_ok(n_layers, B, Hq, Hkv, num_pages) ||
        !head_dim_ok(d) || !scale_block_ok(block, page_size) || !quant_page_ok(Hkv, page_size, d))
        return DDT_ERR_UNSUPPORTED;
    if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !prefix_len || !o || !status || !workspace ||
        !k_new != !v_new)
        return DDT_ERR_INVALID_ARG;
    const size_t need = decode_quant_ws_bytes(n_layers, B, Hq, Hkv, d, in_dtype);
    if (ws_bytes < need || !aligned16(workspace) || !aligned16(q) || !aligned16(k_new) || !aligned16(v_new) ||
        !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o))
        return DDT_ERR_INVALID_ARG;
    const size_t n_lb = (size_t)n_layers * B, in = in_dtype == DDT_BF16 ? 2 : 4, n_new = n_lb * Hkv * d * in,
                 n_rows = (size_t)n_layers * num_pages * Hkv * page_size;
    const Span spans[] = {{o, n_lb * Hq * d * (out_dtype == DDT_BF16 ? 2 : 4)},
                          {status, B * sizeof(int32_t)},
                          {workspace, need},
                          {q, n_lb * Hq * d * in},
                          {k_new, n_new},
                          {v_new, n_new},
                          {k_pages, n_rows * d},
                          {v_pages, n_rows * d},
                          {k_scale, n_rows / block},
                          {v_scale, n_rows / block},
                          {block_table, (size_t)B * max_pages * sizeof(int32_t)},
                          {prefix_len, B * sizeof(int32_t)}};
    if (any_overlap(spans, 12, 3)) return DDT_ERR_INVALID_ARG;
    const AttnPaging pg{page_size, num_pages, max_pages, block_table};
    return from_cuda(launch_decode_quant(n_layers, B, Hq, Hkv, d, block, pg, in_dtype, out_dtype, q, k_new, v_new, k_pages,
                                         v_pages, k_scale, v_scale, prefix_len, scale, o, status, workspace,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
