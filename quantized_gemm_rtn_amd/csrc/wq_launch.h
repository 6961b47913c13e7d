// Host-side launchers of the gfx950 kernels (internal; the public ABI is include/wq.h).
// Each returns the hipError_t of its launches; arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wq {

// Raises kernel `kern`'s dynamic-LDS limit to `bytes` on the current device, once:
// hipFuncSetAttribute costs tens of microseconds of host time per call, so the
// (kernel, device) pairs already raised are remembered (under a mutex).
hipError_t set_dynamic_lds(const void* kern, size_t bytes);

// Workspace carved up by the outlier split.
struct SplitWorkspace {
  uint32_t* hist;     // [2048] radix histogram
  uint32_t* state;    // [16]   select state: prefix, prefix mask, k remaining, count above
  uint32_t* cnt_gt;   // [N]    per row: keys above the threshold
  uint32_t* cnt_eq;   // [N]    per row: keys equal to the threshold
  uint32_t* take_eq;  // [N]    per row: equal keys that are selected
  uint32_t* mask;     // [N*K/32] selection bitmap
};
size_t split_workspace_bytes(int64_t N, int64_t K);
SplitWorkspace split_workspace_carve(void* base, int64_t N, int64_t K);

hipError_t launch_split(const float* W, int64_t N, int64_t K, int64_t sparse_k, int32_t* row_ptr,
                        int32_t* col, uint16_t* val, const SplitWorkspace& ws, hipStream_t stream);
hipError_t launch_fill_zero_i32(int32_t* p, int64_t n, hipStream_t stream);
// dst[r, i] = src[r, perm[i]] for a row-major [rows, K] matrix (K a multiple of 8)
hipError_t launch_gather_cols_f16(const uint16_t* src, int64_t rows, int64_t K, const int32_t* perm, uint16_t* dst,
                                  hipStream_t stream);
hipError_t launch_gather_cols_f32(const float* src, int64_t rows, int64_t K, const int32_t* perm, float* dst,
                                  hipStream_t stream);

// W4A8 with fp16 outlier channels (at most 16): workspace = xq | s_x | xo | w_hat of the outliers
size_t w4a8_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_act_int8(const uint16_t* x, int64_t M, int64_t K, const int32_t* outliers, int64_t n_out,
                           int8_t* xq, float* sx, uint16_t* xo, hipStream_t stream);
hipError_t launch_w4a8(const uint16_t* x, int64_t M, int64_t K, const int32_t* outliers, int64_t n_out,
                       const uint32_t* packed, const uint16_t* scales, const uint16_t* zeros, int64_t N, void* y,
                       int y_f32, void* workspace, hipStream_t stream);

// Root-mean-square norm of x + residual (may be null): fp16 output y, or (xq not null) the
// INT8 output of launch_act_int8 with sx and xo; h (may be null) takes the sum.
hipError_t launch_add_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t M,
                              int64_t K, float eps, const int32_t* outliers, int64_t n_out, uint16_t* h, uint16_t* y,
                              int8_t* xq, float* sx, uint16_t* xo, hipStream_t stream);
hipError_t launch_dequantize_act_int8(const int8_t* xq, const float* sx, const uint16_t* xo, const int32_t* outliers,
                                      int64_t n_out, int64_t M, int64_t K, uint16_t* out, hipStream_t stream);
// The W4A8 product of activations that are already INT8; wo: [N, 16] fp16 scratch.
hipError_t launch_w4a8_product(const int8_t* xq, const float* sx, const uint16_t* xo, int64_t M, int64_t K,
                               const int32_t* outliers, int64_t n_out, const uint32_t* packed, const uint16_t* scales,
                               const uint16_t* zeros, int64_t N, void* y, int y_f32, uint16_t* wo, hipStream_t stream);

// A batch's view of a 4-bit key/value cache: B sequences, whose new tokens are the rows
// seq_start[b] .. seq_start[b + 1] - 1 of the token-wise arrays and the last of ctx_len[b].
struct Kv4View {
  const int32_t* seq_start;   // [B + 1]
  const int32_t* ctx_len;     // [B]
  const int32_t* page_table;  // [B, max_pages]
  int64_t B, max_pages, num_pages, page_tokens, kv_heads;
};
struct KvCache;
KvCache kv4_cache_args(const Kv4View& c, int64_t T, int64_t head_dim);
hipError_t launch_kv4_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, int64_t T,
                             int64_t head_dim, int64_t max_new, const Kv4View& c, void* cache, hipStream_t stream);
hipError_t launch_kv4_read(const void* cache, int64_t T, int64_t head_dim, int64_t max_new, const Kv4View& c,
                           uint16_t* k, uint16_t* v, hipStream_t stream);
// at least the bytes launch_kv4_attention uses with the same sizes and any window
size_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t head_dim, int64_t max_q,
                                     int64_t max_ctx);
// what wq_kv4_attention_plan returns
int kv4_attention_plan(int64_t T, int64_t B, int64_t hq, int64_t hkv, int64_t head_dim, int64_t max_q, int64_t max_ctx,
                       int64_t window);
hipError_t launch_kv4_attention(const uint16_t* q, int64_t q_stride, int64_t T, int64_t hq, int64_t head_dim,
                                int64_t max_q, int64_t max_ctx, int64_t window, float scale, const void* cache,
                                const Kv4View& c, uint16_t* out, float* lse, void* workspace, hipStream_t stream);

hipError_t launch_quantize(const float* W, const uint32_t* mask, int64_t N, int64_t K, int64_t group, int bits,
                           uint8_t* codes, uint16_t* scales, uint16_t* zeros, hipStream_t stream);
hipError_t launch_pack(const uint8_t* codes, int64_t N, int64_t K, uint32_t* packed, hipStream_t stream);

// The up-projection of a low-rank branch, added to every output tile before its
// store: t [M, r] fp16 (the down-projection x . L1^T) and L2 [N, r] fp16; r = 0: none.
// With `row`, each row has a branch of its own: row[m] of the n that `up` [n, N, r] holds, or none
// (outside [0, n)); r is then a multiple of 8, and t's rows lie r rounded up to 32 apart, zeros beyond r.
struct LowRank {
  const uint16_t* t = nullptr;
  const uint16_t* up = nullptr;
  int64_t r = 0;
  const int32_t* row = nullptr;
  int64_t n = 0;
  int64_t t_stride() const { return (r + 31) / 32 * 32; }
};

// The down-projection t = fp16(x . L1^T) of a low-rank branch (r a multiple of 32),
// through fp32 partials of K chunks in `part` (lowrank_partial_bytes(M, K, r)).
size_t lowrank_partial_bytes(int64_t M, int64_t K, int64_t r);
hipError_t launch_lowrank_down(const uint16_t* x, int64_t M, int64_t K, const uint16_t* L1, int64_t r,
                               float* part, uint16_t* t, hipStream_t stream);

// The down-projections t[m] = fp16(scale[a] x[m] . L1_a^T) of the adapters a = row[m] that rows name, L1 [n, r, K],
// scale [n] (null: 1), t [M, r rounded up to 32].
struct Adapters {
  const uint16_t* L1;
  const float* scale;
  const int32_t* row;
  int64_t n;
};
size_t adapters_partial_bytes(int64_t M, int64_t K, int64_t r);  // of `part`: fp32 partials of K chunks
hipError_t launch_adapters_down(const uint16_t* x, int64_t M, int64_t K, const Adapters& ad, int64_t r, float* part,
                                uint16_t* t, hipStream_t stream);

// Softmax of each row's logits ([M, E] fp16, or fp32) and its k largest.
hipError_t launch_moe_route(const void* logits, int f32, int64_t M, int64_t E, int64_t k, int renormalize,
                            int32_t* experts, float* weights, hipStream_t stream);
// A mixture-of-experts layer for a few tokens: up [E, 2 I, H], down [E, H, I] in 4 bits.
size_t moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t k);
hipError_t launch_moe_experts(const uint16_t* x, int64_t M, int64_t H, const int32_t* experts, const float* weights,
                              int64_t k, int64_t E, const uint32_t* up, const uint16_t* up_s, const uint16_t* up_z,
                              int64_t I, const uint32_t* down, const uint16_t* down_s, const uint16_t* down_z, void* y,
                              int y_f32, void* workspace, hipStream_t stream);

// Weight format of a product: 4-bit codes (eight per word) or 3-bit codes (32 per
// three words, the layout of wq_pack_bits), with one (s, z) per 128 or per 64 input
// channels ([N, K/128] or [N, K/64] metadata).
struct WFormat {
  int bits = 4;
  bool g64 = false;
  bool plain() const { return bits == 4 && !g64; }
};

// mfma_only: never the single-row kernel (the MFMA decode kernels at every M)
bool gemv_fits(int64_t M, int64_t K, bool g64, bool adapters);  // whether the decode kernels take rows of K channels
hipError_t launch_gemv(const uint16_t* x, int64_t M, int64_t K, const uint32_t* packed,
                       const uint16_t* scales, const uint16_t* zeros, int64_t N, const int32_t* row_ptr,
                       const int32_t* col, const uint16_t* val, void* y, int y_f32, const LowRank& lr,
                       hipStream_t stream, WFormat f = WFormat{}, bool mfma_only = false);
// the same with the adapters that rows name (lr.row)
hipError_t launch_gemv_adapters(const uint16_t* x, int64_t M, int64_t K, const uint32_t* packed,
                                const uint16_t* scales, const uint16_t* zeros, int64_t N, const int32_t* row_ptr,
                                const int32_t* col, const uint16_t* val, void* y, int y_f32, const LowRank& lr,
                                hipStream_t stream);
// the same for the formats other than 4-bit with 128-channel groups (no low-rank branch)
hipError_t launch_gemv_fmt(const uint16_t* x, int64_t M, int64_t K, const uint32_t* packed,
                           const uint16_t* scales, const uint16_t* zeros, int64_t N, const int32_t* row_ptr,
                           const int32_t* col, const uint16_t* val, void* y, int y_f32, WFormat f,
                           hipStream_t stream);
// the single-row decode kernel (whole rows per wave, VALU dot products): for M = 1,
// K a multiple of 2048 up to 32768, 4-bit codes with 128-channel groups, 16-byte
// aligned scales and zeros
bool gemv_dot_supported(int64_t M, int64_t K, const uint16_t* scales, const uint16_t* zeros);
hipError_t launch_gemv_dot(const uint16_t* x, int64_t K, const uint32_t* packed, const uint16_t* scales,
                           const uint16_t* zeros, int64_t N, const int32_t* row_ptr, const int32_t* col,
                           const uint16_t* val, void* y, int y_f32, hipStream_t stream);
// packing of 3-bit codes: [N, K] bytes -> [N, 3K/32] words (K a multiple of 32)
hipError_t launch_pack3(const uint8_t* codes, int64_t N, int64_t K, uint32_t* packed, hipStream_t stream);
// The GEMM splits K through `workspace` (fp32 partials) when its tile grid alone
// cannot fill the GPU and the workspace holds gemm_workspace_bytes(M, N, K);
// otherwise it runs unsplit.
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
// ... of the plan one product takes (4-bit codes, 128-channel groups; a CSR term or
// not); at most gemm_workspace_bytes(M, N, K)
size_t gemm_plan_workspace_bytes(int64_t M, int64_t N, int64_t K, bool sparse);
// the dense GEMM's plan for M x N x K: blocks of its launch (split K included), K
// slices, whether it is gemm_big_kernel, and its tile width (256, or 128 for M <= 64
// where 256-wide tiles would leave compute units without a block)
struct GemmPlanInfo {
  int64_t blocks;
  int ksplit;
  bool big;
  int bn;
};
GemmPlanInfo gemm_plan_info(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm(const uint16_t* x, int64_t M, int64_t K, const uint32_t* packed,
                       const uint16_t* scales, const uint16_t* zeros, int64_t N, const int32_t* row_ptr,
                       const int32_t* col, const uint16_t* val, int64_t nnz, void* y, int y_f32, void* workspace,
                       size_t workspace_bytes, const LowRank& lr, hipStream_t stream, WFormat f = WFormat{});

}  // namespace wq
