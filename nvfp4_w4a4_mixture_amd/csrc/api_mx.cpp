// C ABI of the MXFP4 operators and the block norms.  Arguments are validated
// on the host before any HIP call, as in api.cpp.
#include <cstdint>

#include "api_check.h"
#include "launch.h"

namespace {

using moe::aligned;
using moe::check_device;
using moe::fail;
using moe::launched;
using moe::mx_padded;
using moe::round_up;

// A launch's work-items per grid dimension are a 32-bit count.
constexpr uint64_t kMaxThreads = (uint64_t)1 << 32;
constexpr uint64_t kMaxOperand = (uint64_t)1 << 32;  // bytes that 32-bit offsets reach
constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxInner = (int64_t)1 << 24;  // H and I of the experts
constexpr int64_t kMaxTiles = (int64_t)1 << 22;  // of one launch (the kernels count them in 32 bits)

bool dtype_ok(int32_t d) { return d == 0 || d == 1; }

// rows * padded columns of 4-bit elements fit one launch of 8 elements a thread
bool rows_fit(int64_t rows, int64_t cols) {
  return rows < kMaxDim && cols < kMaxDim &&
         (unsigned __int128)rows * (uint64_t)(mx_padded(cols) / 8) < (unsigned __int128)kMaxThreads - 4096;
}

moe_status check_rows(const char* fn, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, const void* x,
                      const void* codes, const void* scales) {
  if (!dtype_ok(dtype)) return fail(MOE_ERR_SHAPE, "%s: dtype must be 0 (BF16) or 1 (FP32)", fn);
  if (rows < 0 || cols <= 0 || cols % 32 != 0 || ld < cols)
    return fail(MOE_ERR_SHAPE, "%s: need rows >= 0, cols a positive multiple of 32, row stride >= cols", fn);
  if (!rows_fit(rows, cols)) return fail(MOE_ERR_SHAPE, "%s: too many elements for one call", fn);
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (ld % (dtype ? 4 : 8) != 0 || !aligned(x, 16) || !aligned(codes, 16))
    return fail(MOE_ERR_ALIGN, "%s: rows must start on 16-byte boundaries and codes be 16-byte aligned", fn);
  return MOE_OK;
}

moe_status check_weights(const char* fn, int64_t batch, int64_t N, int64_t K) {
  if (batch < 0 || N < 1 || K < 32 || K % 32 != 0)
    return fail(MOE_ERR_SHAPE, "%s: need batch >= 0, N >= 1, K a positive multiple of 32", fn);
  if (batch >= kMaxDim || N >= kMaxDim - 31 || K >= kMaxDim - 255)
    return fail(MOE_ERR_SHAPE, "%s: a size is out of range", fn);
  const unsigned __int128 blocks = (unsigned __int128)batch * (uint64_t)((N + 31) / 32 * 32) * (uint64_t)(mx_padded(K) / 32);
  if (blocks >= (unsigned __int128)kMaxThreads - 256) return fail(MOE_ERR_SHAPE, "%s: too many elements for one call", fn);
  return MOE_OK;
}

struct MxFfnWs {
  size_t h_codes, h_scales, total;
};

// `bits` of an element of h
MxFfnWs mx_ffn_ws(int64_t T, int64_t k, int64_t I, int bits) {
  MxFfnWs w{};
  size_t o = round_up((size_t)(T * k) * (size_t)(mx_padded(I) / 8 * bits), 256);
  w.h_scales = o;
  o = round_up(o + (size_t)(T * k) * (size_t)(mx_padded(I) / 32), 256);
  w.total = o;
  return w;
}

int ceil_log2(int64_t v) {
  int b = 0;
  while (((int64_t)1 << b) < v) ++b;
  return b;
}

}  // namespace

extern "C" {

moe_status mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                          uint8_t* scales, void* stream) {
  if (moe_status s = check_rows("mxfp4_quantize", rows, cols, ld, x_dtype, x, codes, scales)) return s;
  if (rows == 0) return MOE_OK;
  if (moe_status s = check_device()) return s;
  return launched(moe::launch_mx_quantize(x, x_dtype == 1, rows, cols, ld, codes, scales, (hipStream_t)stream),
                  "mxfp4_quantize");
}

moe_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            int32_t out_dtype, void* out, int64_t ld_out, void* stream) {
  if (moe_status s = check_rows("mxfp4_dequantize", rows, cols, ld_out, out_dtype, out, codes, scales)) return s;
  if (rows == 0) return MOE_OK;
  if (moe_status s = check_device()) return s;
  return launched(moe::launch_mx_dequantize(codes, scales, rows, cols, out_dtype == 1, out, ld_out, (hipStream_t)stream),
                  "mxfp4_dequantize");
}

moe_status mxfp4_quantize_weights(const uint16_t* w_bf16, int64_t batch, int64_t N, int64_t K, uint8_t* codes,
                                  uint8_t* scales, int32_t* max_scale, void* stream) {
  const char* fn = "mxfp4_quantize_weights";
  if (moe_status s = check_weights(fn, batch, N, K)) return s;
  if (batch == 0) return MOE_OK;
  if (!w_bf16 || !codes || !scales) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(w_bf16, 16) || !aligned(codes, 16) || !aligned(max_scale, 4))
    return fail(MOE_ERR_ALIGN, "%s: w and codes must be 16-byte, max_scale 4-byte aligned", fn);
  if (moe_status s = check_device()) return s;
  return launched(moe::launch_mx_quantize_weights(w_bf16, batch, N, K, codes, scales, max_scale, (hipStream_t)stream), fn);
}

static moe_status relayout(const char* fn, uint8_t* codes, uint8_t* scales, int64_t batch, int64_t N, int64_t K,
                           uint8_t* pcodes, uint8_t* pscales, int32_t* max_scale, bool pack, void* stream) {
  if (moe_status s = check_weights(fn, batch, N, K)) return s;
  if (batch == 0) return MOE_OK;
  if (!codes || !scales || !pcodes || !pscales) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(codes, 16) || !aligned(pcodes, 16) || !aligned(max_scale, 4))
    return fail(MOE_ERR_ALIGN, "%s: code arrays must be 16-byte, max_scale 4-byte aligned", fn);
  if (codes == pcodes || scales == pscales) return fail(MOE_ERR_SHAPE, "%s: the arrays must not overlap", fn);
  if (moe_status s = check_device()) return s;
  return launched(moe::launch_mx_relayout(codes, scales, batch, N, K, pcodes, pscales, max_scale, pack, (hipStream_t)stream),
                  fn);
}

moe_status mxfp4_pack_weights(const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t N, int64_t K,
                              uint8_t* packed_codes, uint8_t* packed_scales, int32_t* max_scale, void* stream) {
  return relayout("mxfp4_pack_weights", const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), batch, N, K,
                  packed_codes, packed_scales, max_scale, true, stream);
}

moe_status mxfp4_unpack_weights(const uint8_t* packed_codes, const uint8_t* packed_scales, int64_t batch, int64_t N,
                                int64_t K, uint8_t* codes, uint8_t* scales, void* stream) {
  return relayout("mxfp4_unpack_weights", codes, scales, batch, N, K, const_cast<uint8_t*>(packed_codes),
                  const_cast<uint8_t*>(packed_scales), nullptr, false, stream);
}

static moe_status check_linear(const char* fn, int64_t T, int64_t K, int64_t N, int64_t bytes_per_256) {
  if (T < 0) return fail(MOE_ERR_SHAPE, "%s: T must be >= 0 (got %lld)", fn, (long long)T);
  if (moe_status s = check_weights(fn, 1, N, K)) return s;
  if (T > 2097120) return fail(MOE_ERR_SHAPE, "%s: T must be at most 2097120", fn);
  if (N > ((int64_t)1 << 27) || ((T + 255) / 256) * ((N + 255) / 256) >= kMaxTiles)
    return fail(MOE_ERR_SHAPE, "%s: N or the result is too large for one call", fn);
  if ((uint64_t)T * (uint64_t)(mx_padded(K) / 256 * bytes_per_256) >= kMaxOperand)
    return fail(MOE_ERR_SHAPE, "%s: x codes must be under 4 GiB", fn);
  return MOE_OK;
}

// ---- MXFP8 activations

moe_status mxfp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                          uint8_t* scales, void* stream) {
  if (moe_status s = check_rows("mxfp8_quantize", rows, cols, ld, x_dtype, x, codes, scales)) return s;
  if (rows == 0) return MOE_OK;
  if (moe_status s = check_device()) return s;
  return launched(moe::launch_mx8_quantize(x, x_dtype == 1, rows, cols, ld, codes, scales, (hipStream_t)stream),
                  "mxfp8_quantize");
}

moe_status mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            int32_t out_dtype, void* out, int64_t ld_out, void* stream) {
  if (moe_status s = check_rows("mxfp8_dequantize", rows, cols, ld_out, out_dtype, out, codes, scales)) return s;
  if (rows == 0) return MOE_OK;
  if (moe_status s = check_device()) return s;
  return launched(moe::launch_mx8_dequantize(codes, scales, rows, cols, out_dtype == 1, out, ld_out, (hipStream_t)stream),
                  "mxfp8_dequantize");
}

size_t mxfp4_linear_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

moe_status mxfp4_linear(const uint8_t* x_codes, const uint8_t* x_scales, int64_t T, int64_t K,
                        const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int32_t out_dtype, void* y,
                        int64_t ldy, void*, size_t, void* stream) {
  const char* fn = "mxfp4_linear";
  if (!dtype_ok(out_dtype)) return fail(MOE_ERR_SHAPE, "%s: out_dtype must be 0 (BF16) or 1 (FP32)", fn);
  if (moe_status s = check_linear(fn, T, K, N, 128)) return s;
  if (ldy < N || ldy >= kMaxDim) return fail(MOE_ERR_SHAPE, "%s: ldy must be >= N and < 2^31", fn);
  if (T == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(y, out_dtype ? 4 : 2))
    return fail(MOE_ERR_ALIGN, "%s: code arrays must be 16-byte, scale arrays 4-byte aligned, y to its element", fn);
  if (moe_status s = check_device()) return s;
  moe::MxArgs a{};
  a.a_codes = x_codes;
  a.a_scales = x_scales;
  a.w_codes = w_codes;
  a.w_scales = w_scales;
  a.out = y;
  a.KK = (int32_t)(mx_padded(K) / 256);
  a.N = (int32_t)N;
  a.G = (int32_t)((N + 31) / 32);
  a.ldo = (int32_t)ldy;
  a.T = (int32_t)T;
  a.aux = (out_dtype ? moe::kMxOutF32 : 0) |
          (aligned(y, 16) && (ldy * (out_dtype ? 4 : 2)) % 16 == 0 ? moe::kMxOutVec : 0);
  return launched(moe::launch_mx_linear(a, (hipStream_t)stream), fn);
}

moe_status mxfp8_linear(const uint8_t* x_codes, const uint8_t* x_scales, int64_t T, int64_t K, const uint8_t* w_codes,
                        const uint8_t* w_scales, int64_t N, const uint16_t* bias, int32_t activation,
                        const void* residual, int32_t residual_dtype, int64_t ld_residual, int32_t out_dtype, void* y,
                        int64_t ldy, void* stream) {
  const char* fn = "mxfp8_linear";
  if (!dtype_ok(out_dtype)) return fail(MOE_ERR_SHAPE, "%s: out_dtype must be 0 (BF16) or 1 (FP32)", fn);
  if (activation < 0 || activation >= moe::kActCount) return fail(MOE_ERR_SHAPE, "%s: unknown activation", fn);
  if (moe_status s = check_linear(fn, T, K, N, 256)) return s;
  // four waves a tile of 256 x 64, and a grid of whole eights
  if (((uint64_t)T + 63) / 64 * (((uint64_t)N + 255) / 256) * 256 > kMaxThreads - 8 * 256)
    return fail(MOE_ERR_SHAPE, "%s: the result is too large for one call", fn);
  if (ldy < N || ldy >= kMaxDim) return fail(MOE_ERR_SHAPE, "%s: ldy must be >= N and < 2^31", fn);
  if (residual) {
    if (!dtype_ok(residual_dtype)) return fail(MOE_ERR_SHAPE, "%s: residual_dtype must be 0 (BF16) or 1 (FP32)", fn);
    if (ld_residual < N || ld_residual >= kMaxDim)
      return fail(MOE_ERR_SHAPE, "%s: ld_residual must be >= N and < 2^31", fn);
  }
  if (T == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(y, out_dtype ? 4 : 2) || !aligned(bias, 2) || !aligned(residual, residual_dtype ? 4 : 2))
    return fail(MOE_ERR_ALIGN, "%s: code arrays must be 16-byte, scale arrays 4-byte aligned, the others to their element", fn);
  if (residual == y && (residual_dtype != out_dtype || ld_residual != ldy))
    return fail(MOE_ERR_SHAPE, "%s: a residual that is y must have its type and stride", fn);
  if (moe_status s = check_device()) return s;
  moe::MxArgs a{};
  a.a_codes = x_codes;
  a.a_scales = x_scales;
  a.w_codes = w_codes;
  a.w_scales = w_scales;
  a.out = y;
  a.bias = bias;
  a.residual = residual;
  a.KK = (int32_t)(mx_padded(K) / 256);
  a.N = (int32_t)N;
  a.G = (int32_t)((N + 31) / 32);
  a.ldo = (int32_t)ldy;
  a.ldr = (int32_t)ld_residual;
  a.T = (int32_t)T;
  a.aux = (out_dtype ? moe::kMxOutF32 : 0) | (residual && residual_dtype ? moe::kMxResF32 : 0) |
          activation << moe::kMxActShift;
  return launched(moe::launch_mx8_linear(a, (hipStream_t)stream), fn);
}

static size_t ffn_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int bits) {
  if (T < 0 || k < 1 || E < 1 || H < 1 || I < 1 || T >= kMaxDim || k > 256 || I >= kMaxInner) return 0;
  return mx_ffn_ws(T, k, I, bits).total;
}
size_t mxfp4_ffn_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  return ffn_workspace_bytes(T, k, E, H, I, 4);
}
size_t mxfp8_ffn_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  return ffn_workspace_bytes(T, k, E, H, I, 8);
}

// Both formats' grouped FFN; `bits` of an element of x and h.
static moe_status grouped_ffn(const char* fn, int bits, const uint8_t* x_codes, const uint8_t* x_scales, int64_t T, int64_t H,
                             const uint8_t* w13_codes, const uint8_t* w13_scales, const uint8_t* w2_codes,
                             const uint8_t* w2_scales, const int32_t* w2_max_scale, int64_t E, int64_t I, int64_t k,
                             const int32_t* expert_offsets, const int32_t* sorted_pair_ids, const float* topk_w,
                             uint16_t* pair_out, float* pair_scale, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (T < 0) return fail(MOE_ERR_SHAPE, "%s: T must be >= 0 (got %lld)", fn, (long long)T);
  if (H <= 0 || H % 32 != 0) return fail(MOE_ERR_SHAPE, "%s: H must be a positive multiple of 32", fn);
  if (I <= 0 || I % 32 != 0) return fail(MOE_ERR_SHAPE, "%s: I must be a positive multiple of 32", fn);
  if (k < 1 || E < k || E > 256) return fail(MOE_ERR_SHAPE, "%s: need 1 <= k <= E <= 256", fn);
  if (H >= kMaxInner || I >= kMaxInner) return fail(MOE_ERR_SHAPE, "%s: H and I must be under 2^24", fn);
  if (T >= kMaxDim || T * k >= kMaxDim) return fail(MOE_ERR_SHAPE, "%s: T*k must be < 2^31", fn);
  if ((uint64_t)T * (uint64_t)(mx_padded(H) / 8 * bits) >= kMaxOperand)
    return fail(MOE_ERR_SHAPE, "%s: x codes must be under 4 GiB", fn);
  if ((uint64_t)(T * k) * (uint64_t)(mx_padded(I) / 8 * bits) >= kMaxOperand)
    return fail(MOE_ERR_SHAPE, "%s: h codes must be under 4 GiB", fn);
  if ((T * k / 128 + E) * (((2 * I > H ? 2 * I : H) + 255) / 256) >= kMaxTiles)
    return fail(MOE_ERR_SHAPE, "%s: too many tiles for one call", fn);
  if (T == 0) return MOE_OK;
  if (!x_codes || !x_scales || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !w2_max_scale ||
      !expert_offsets || !sorted_pair_ids || !topk_w || !pair_out || !pair_scale)
    return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(x_codes, 16) || !aligned(w13_codes, 16) || !aligned(w2_codes, 16) || !aligned(pair_out, 16) ||
      !aligned(x_scales, 4) || !aligned(w13_scales, 4) || !aligned(w2_scales, 4) || !aligned(pair_scale, 4) ||
      !aligned(w2_max_scale, 4) || !aligned(expert_offsets, 4) || !aligned(sorted_pair_ids, 4) || !aligned(topk_w, 4))
    return fail(MOE_ERR_ALIGN, "%s: code arrays and pair_out must be 16-byte, the other arrays 4-byte aligned", fn);
  const MxFfnWs L = mx_ffn_ws(T, k, I, bits);
  if (!workspace || workspace_bytes < L.total) return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes", fn, L.total);
  if (!aligned(workspace, 256)) return fail(MOE_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  if (moe_status s = check_device()) return s;

  unsigned char* ws = static_cast<unsigned char*>(workspace);
  moe::MxExperts x{};
  x.T = T;
  x.k = k;
  x.E = E;
  moe::MxArgs& a = x.gate_up;
  a.a_codes = x_codes;
  a.a_scales = x_scales;
  a.w_codes = w13_codes;
  a.w_scales = w13_scales;
  a.out = ws + L.h_codes;
  a.out_scales = ws + L.h_scales;
  a.offsets = expert_offsets;
  a.sorted = sorted_pair_ids;
  a.E = (int32_t)E;
  a.KK = (int32_t)(mx_padded(H) / 256);
  a.N = (int32_t)(2 * I);
  a.G = (int32_t)(2 * I / 32);
  a.ldo = (int32_t)(mx_padded(I) / 8 * bits);
  a.aux = (int32_t)k;
  moe::MxArgs& d = x.down;
  d.a_codes = ws + L.h_codes;
  d.a_scales = ws + L.h_scales;
  d.w_codes = w2_codes;
  d.w_scales = w2_scales;
  d.out = pair_out;
  d.out_scales = pair_scale;
  d.offsets = expert_offsets;
  d.sorted = sorted_pair_ids;
  d.E = (int32_t)E;
  d.topk_w = topk_w;
  d.w_max = w2_max_scale;
  d.KK = (int32_t)(mx_padded(I) / 256);
  d.N = (int32_t)H;
  d.G = (int32_t)(H / 32);
  d.ldo = (int32_t)H;
  d.aux = ceil_log2((bits == 8 ? 6 * 448 : 6 * 6) * I);
  return launched(bits == 8 ? moe::launch_mx8_experts(x, (hipStream_t)stream) : moe::launch_mx_experts(x, (hipStream_t)stream),
                  fn);
}

moe_status mxfp4_grouped_ffn(const uint8_t* x_codes, const uint8_t* x_scales, int64_t T, int64_t H,
                             const uint8_t* w13_codes, const uint8_t* w13_scales, const uint8_t* w2_codes,
                             const uint8_t* w2_scales, const int32_t* w2_max_scale, int64_t E, int64_t I, int64_t k,
                             const int32_t* expert_offsets, const int32_t* sorted_pair_ids, const float* topk_w,
                             uint16_t* pair_out, float* pair_scale, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return grouped_ffn("mxfp4_grouped_ffn", 4, x_codes, x_scales, T, H, w13_codes, w13_scales, w2_codes, w2_scales,
                     w2_max_scale, E, I, k, expert_offsets, sorted_pair_ids, topk_w, pair_out, pair_scale, workspace,
                     workspace_bytes, stream);
}

moe_status mxfp8_grouped_ffn(const uint8_t* x_codes, const uint8_t* x_scales, int64_t T, int64_t H,
                             const uint8_t* w13_codes, const uint8_t* w13_scales, const uint8_t* w2_codes,
                             const uint8_t* w2_scales, const int32_t* w2_max_scale, int64_t E, int64_t I, int64_t k,
                             const int32_t* expert_offsets, const int32_t* sorted_pair_ids, const float* topk_w,
                             uint16_t* pair_out, float* pair_scale, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return grouped_ffn("mxfp8_grouped_ffn", 8, x_codes, x_scales, T, H, w13_codes, w13_scales, w2_codes, w2_scales,
                     w2_max_scale, E, I, k, expert_offsets, sorted_pair_ids, topk_w, pair_out, pair_scale, workspace,
                     workspace_bytes, stream);
}

// ---- the whole layer for a few tokens

static bool layer_sizes_ok(int64_t T, int64_t H, int64_t E, int64_t k, int64_t I) {
  return T >= 0 && T <= moe::kLayerMaxTokens && H > 0 && H % 32 == 0 && H < kMaxInner && I > 0 && I % 32 == 0 &&
         I < kMaxInner && k >= 1 && E >= k && E <= 256;
}

size_t mxfp8_moe_layer_workspace_bytes(int64_t T, int64_t H, int64_t E, int64_t k, int64_t I) {
  return layer_sizes_ok(T, H, E, k, I) ? moe::mx_layer_workspace(T, E, k, H, I) : 0;
}

moe_status mxfp8_moe_layer(const uint16_t* x_bf16, int64_t T, int64_t H, int64_t ldx, const uint16_t* w_router_bf16,
                           const float* bias, int64_t E, int64_t k, float routed_scaling_factor,
                           const uint8_t* w13_codes, const uint8_t* w13_scales, const uint8_t* w2_codes,
                           const uint8_t* w2_scales, int64_t I, int32_t out_dtype, void* y, int32_t* topk_ids,
                           float* topk_w, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_moe_layer";
  if (!dtype_ok(out_dtype)) return fail(MOE_ERR_SHAPE, "%s: out_dtype must be 0 (BF16) or 1 (FP32)", fn);
  if (!layer_sizes_ok(T, H, E, k, I))
    return fail(MOE_ERR_SHAPE, "%s: need 0 <= T <= %lld, H and I positive multiples of 32 under 2^24, 1 <= k <= E <= 256", fn,
                (long long)moe::kLayerMaxTokens);
  if (ldx < H || ldx >= kMaxDim) return fail(MOE_ERR_SHAPE, "%s: ldx must be >= H and < 2^31", fn);
  if (!(routed_scaling_factor > 0.0f)) return fail(MOE_ERR_SHAPE, "%s: routed_scaling_factor must be > 0", fn);
  if (T == 0) return MOE_OK;
  if (!x_bf16 || !w_router_bf16 || !bias || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !y || !topk_ids || !topk_w)
    return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(w13_codes, 16) || !aligned(w2_codes, 16) || !aligned(y, 16) || !aligned(w13_scales, 4) || !aligned(w2_scales, 4) ||
      !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(x_bf16, 2) || !aligned(w_router_bf16, 2))
    return fail(MOE_ERR_ALIGN, "%s: code arrays and y must be 16-byte, scale arrays 4-byte aligned, the others to their element", fn);
  const size_t need = moe::mx_layer_workspace(T, E, k, H, I);
  if (!workspace || workspace_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes", fn, need);
  if (!aligned(workspace, 256)) return fail(MOE_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  if (moe_status s = check_device()) return s;
  moe::MxLayerArgs a{};
  a.x = x_bf16;
  a.w_router = w_router_bf16;
  a.bias = bias;
  a.w13_codes = w13_codes;
  a.w13_scales = w13_scales;
  a.w2_codes = w2_codes;
  a.w2_scales = w2_scales;
  a.y = y;
  a.topk_ids = topk_ids;
  a.topk_w = topk_w;
  a.ws = static_cast<uint8_t*>(workspace);
  a.ldx = (int32_t)ldx;
  a.T = (int32_t)T;
  a.E = (int32_t)E;
  a.k = (int32_t)k;
  a.H = (int32_t)H;
  a.I = (int32_t)I;
  a.rsf = routed_scaling_factor;
  a.y_f32 = out_dtype;
  return launched(moe::launch_mx_layer(a, (hipStream_t)stream), fn);
}


// ---- norms

static bool stride_ok(int64_t ld, int64_t H) { return ld >= H && ld < kMaxDim; }

static moe_status check_norm(const char* fn, int64_t T, int64_t H, float eps, const uint16_t* n, int64_t ldn,
                             const uint8_t* codes, const uint8_t* scales, bool norm_follows) {
  if (T < 0 || T >= kMaxDim / 2) return fail(MOE_ERR_SHAPE, "%s: T is out of range", fn);
  if (H < 1 || H > moe::norm_max_cols())
    return fail(MOE_ERR_SHAPE, "%s: H must be between 1 and %lld", fn, (long long)moe::norm_max_cols());
  if ((uint64_t)T * 256 >= kMaxThreads) return fail(MOE_ERR_SHAPE, "%s: too many rows for one call", fn);
  if (!(eps >= 0.0f)) return fail(MOE_ERR_SHAPE, "%s: eps must be >= 0", fn);
  if (codes && H % 32 != 0) return fail(MOE_ERR_SHAPE, "%s: H must be a multiple of 32 to quantize", fn);
  if (n && !stride_ok(ldn, H)) return fail(MOE_ERR_SHAPE, "%s: a row stride is smaller than H or over 2^31", fn);
  if (T > 0 && norm_follows && !n && !codes) return fail(MOE_ERR_NULL, "%s: neither n nor codes is given", fn);
  if (T > 0 && (codes != nullptr) != (scales != nullptr)) return fail(MOE_ERR_NULL, "%s: codes and scales go together", fn);
  if (!aligned(n, 2) || !aligned(codes, 4)) return fail(MOE_ERR_ALIGN, "%s: n must be 2-byte, codes 4-byte aligned", fn);
  return MOE_OK;
}

// The 8-bit forms always write codes (8 bytes a lane).
static moe_status check_mxfp8(const char* fn, int64_t T, const uint8_t* codes) {
  if (T > 0 && !codes) return fail(MOE_ERR_NULL, "%s: codes and scales are required", fn);
  if (!aligned(codes, 8)) return fail(MOE_ERR_ALIGN, "%s: codes must be 8-byte aligned", fn);
  return MOE_OK;
}

static moe_status norm_in(const char* fn, bool a8, const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const uint16_t* w, float eps,
                       uint16_t* n, int64_t ldn, uint8_t* codes, uint8_t* scales, void* stream) {
  if (moe_status s = check_norm(fn, T, H, eps, n, ldn, codes, scales, true)) return s;
  if (!stride_ok(ldx, H)) return fail(MOE_ERR_SHAPE, "%s: a row stride is smaller than H or over 2^31", fn);
  if (T == 0) return MOE_OK;
  if (!x || !w) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(x, 2) || !aligned(w, 2)) return fail(MOE_ERR_ALIGN, "%s: BF16 arrays must be 2-byte aligned", fn);
  if (moe_status s = check_device()) return s;
  moe::NormArgs a{};
  a.x = x;
  a.w = w;
  a.n = n;
  a.codes = codes;
  a.scales = scales;
  a.ldx = (int32_t)ldx;
  a.ldn = (int32_t)ldn;
  a.H = (uint32_t)H;
  a.Hp = (uint32_t)(codes ? mx_padded(H) : H);
  a.a8 = a8;
  a.eps = eps;
  return launched(moe::launch_norm(a, T, false, false, (hipStream_t)stream), fn);
}

moe_status moe_norm_in(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const uint16_t* w, float eps,
                       uint16_t* n, int64_t ldn, uint8_t* codes, uint8_t* scales, void* stream) {
  return norm_in("moe_norm_in", false, x, T, H, ldx, w, eps, n, ldn, codes, scales, stream);
}

moe_status moe_norm_in_mxfp8(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const uint16_t* w, float eps,
                             uint16_t* n, int64_t ldn, uint8_t* codes, uint8_t* scales, void* stream) {
  if (moe_status s = check_mxfp8("moe_norm_in_mxfp8", T, codes)) return s;
  return norm_in("moe_norm_in_mxfp8", true, x, T, H, ldx, w, eps, n, ldn, codes, scales, stream);
}

static moe_status norm_out(const char* fn, bool a8, const void* y, int32_t y_dtype, int64_t T, int64_t H, int64_t ldy, const uint16_t* r,
                        int64_t ldr, const uint16_t* w_post, const uint16_t* gate, int64_t gate_row_stride,
                        int64_t gate_col_stride, float residual_scale, const uint16_t* w_next, float eps,
                        uint16_t* r_out, int64_t ldro, uint16_t* n, int64_t ldn, uint8_t* codes, uint8_t* scales,
                        void* stream) {
  if (!dtype_ok(y_dtype)) return fail(MOE_ERR_SHAPE, "%s: y_dtype must be 0 (BF16) or 1 (FP32)", fn);
  if (moe_status s = check_norm(fn, T, H, eps, n, ldn, codes, scales, w_next != nullptr)) return s;
  if (!stride_ok(ldy, H) || !stride_ok(ldr, H) || !stride_ok(ldro, H))
    return fail(MOE_ERR_SHAPE, "%s: a row stride is smaller than H or over 2^31", fn);
  if (gate && (gate_row_stride < 0 || gate_row_stride >= kMaxDim || (gate_col_stride != 0 && gate_col_stride != 1)))
    return fail(MOE_ERR_SHAPE, "%s: gate strides must be >= 0 (rows) and 0 or 1 (columns)", fn);
  if (!w_next && (n || codes)) return fail(MOE_ERR_NULL, "%s: n and codes need w_next", fn);
  if (T == 0) return MOE_OK;
  if (!y || !r || !r_out) return fail(MOE_ERR_NULL, "%s: a required pointer is NULL", fn);
  if (!aligned(y, y_dtype ? 4 : 2) || !aligned(r, 2) || !aligned(r_out, 2) || !aligned(w_post, 2) ||
      !aligned(w_next, 2) || !aligned(gate, 2))
    return fail(MOE_ERR_ALIGN, "%s: arrays must be aligned to their element", fn);
  if (moe_status s = check_device()) return s;
  moe::NormArgs a{};
  a.x = y;
  a.r = r;
  a.w_post = w_post;
  a.gate = gate;
  a.w = w_next;
  a.r_out = r_out;
  a.n = n;
  a.codes = codes;
  a.scales = scales;
  a.ldx = (int32_t)ldy;
  a.ldr = (int32_t)ldr;
  a.ldro = (int32_t)ldro;
  a.ldn = (int32_t)ldn;
  a.gate_rs = (int32_t)gate_row_stride;
  a.H = (uint32_t)H;
  a.Hp = (uint32_t)(codes ? mx_padded(H) : H);
  a.a8 = a8;
  a.gate_row = gate_col_stride == 0;
  a.scale = residual_scale;
  a.eps = eps;
  return launched(moe::launch_norm(a, T, true, y_dtype == 1, (hipStream_t)stream), fn);
}

moe_status moe_norm_out(const void* y, int32_t y_dtype, int64_t T, int64_t H, int64_t ldy, const uint16_t* r,
                        int64_t ldr, const uint16_t* w_post, const uint16_t* gate, int64_t gate_row_stride,
                        int64_t gate_col_stride, float residual_scale, const uint16_t* w_next, float eps,
                        uint16_t* r_out, int64_t ldro, uint16_t* n, int64_t ldn, uint8_t* codes, uint8_t* scales,
                        void* stream) {
  return norm_out("moe_norm_out", false, y, y_dtype, T, H, ldy, r, ldr, w_post, gate, gate_row_stride, gate_col_stride,
                  residual_scale, w_next, eps, r_out, ldro, n, ldn, codes, scales, stream);
}

moe_status moe_norm_out_mxfp8(const void* y, int32_t y_dtype, int64_t T, int64_t H, int64_t ldy, const uint16_t* r,
                              int64_t ldr, const uint16_t* w_post, const uint16_t* gate, int64_t gate_row_stride,
                              int64_t gate_col_stride, float residual_scale, const uint16_t* w_next, float eps,
                              uint16_t* r_out, int64_t ldro, uint16_t* n, int64_t ldn, uint8_t* codes,
                              uint8_t* scales, void* stream) {
  if (moe_status s = check_mxfp8("moe_norm_out_mxfp8", T, codes)) return s;
  return norm_out("moe_norm_out_mxfp8", true, y, y_dtype, T, H, ldy, r, ldr, w_post, gate, gate_row_stride,
                  gate_col_stride, residual_scale, w_next, eps, r_out, ldro, n, ldn, codes, scales, stream);
}

}  // extern "C"
