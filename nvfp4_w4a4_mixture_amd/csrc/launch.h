// Internal launcher interface between the C-ABI host code (api.cpp) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>
#include <tuple>
#include <utility>
#include <vector>

namespace moe {

// Raise a kernel's dynamic LDS limit above the default 64 KiB (gfx950 has 160 KiB
// per CU), once per (kernel, device); later calls for the same pair return at once.
inline hipError_t set_max_dynamic_lds(const void* kernel, int bytes) {
  static std::mutex mu;
  static std::vector<std::pair<const void*, int>> done;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  for (const auto& d : done)
    if (d.first == kernel && d.second == dev) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.emplace_back(kernel, dev);
  return e;
}

// A launch without the configuration stack that <<< >>> goes through: 0.25 us
// less on the host, of some 2.5.
template <typename... P, typename... A>
inline hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t st, A... a) {
  std::tuple<P...> args(a...);
  return std::apply(
      [&](auto&... v) {
        void* p[] = {const_cast<void*>(static_cast<const void*>(&v))...};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, p, lds, st);
        if (e != hipSuccess) (void)hipGetLastError();  // reported here, not by the next call
        return e;
      },
      args);
}

// Arguments of one FFN stage (gate_up: A = x, B = w13; down: A = h, B = w2).
struct FfnArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  const float* a_gs;  // gate_up: x_gs [1]; down: h_gs [E]
  const float* b_gs;  // gate_up: w13_gs [E, 2]; down: w2_gs [E]
  const float* h_gs;  // gate_up: h_gs [E]
  int64_t K;          // reduction length (H or I)
  int64_t I;
  int64_t H;
  int k;
  const int32_t* offsets;
  const int32_t* sorted;
  const float* topk_w;
  // tiled schedule (workspace): per m-tile slot {expert, first pair row, rows, 0};
  // rows 0 marks a slot past the last m-tile
  const int32_t* tile_info;
  uint8_t* h_codes;  // gate_up output
  uint8_t* h_scales;
  uint16_t* pair_out;  // down outputs: FP16 [T*k, H], value = pair_out * pair_scale[row]
  float* pair_scale;   // [T*k] powers of two
  float* sq_part;   // [T*k, n_part] partial sums of f^2, or null
  int n_part;
};

hipError_t launch_quantize_bf16(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, const float* gs,
                                int64_t rows_per_gs, uint8_t* codes, uint8_t* scales, bool tiled_scales,
                                hipStream_t stream);
// canonical [rows, K/16] scales <-> tiled [rows/16, K/128, 16, 8] (rows % 16 == 0, K % 128 == 0)
hipError_t launch_relayout_scales(const uint8_t* src, int64_t rows, int64_t K, bool to_tiled, uint8_t* dst,
                                  hipStream_t st);
hipError_t launch_weight_global_scales(const uint16_t* w, int64_t batch, int64_t per_matrix, float* gs,
                                       hipStream_t stream);

size_t route_workspace_bytes(int64_t T, int64_t H, int64_t E, int64_t k);
hipError_t launch_route(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const uint16_t* wr, const float* bias,
                        int64_t E, int64_t k, float rsf, int32_t* topk_ids, float* topk_w, int32_t* counts,
                        int32_t* offsets, int32_t* sorted, void* workspace, const float* qgs, uint8_t* qcodes,
                        uint8_t* qscales, hipStream_t st);

int64_t ffn_max_tiles(int64_t T, int64_t k, int64_t E);
int ffn_sq_parts(int64_t H);
bool ffn_use_small(int64_t T);
int ffn_tiled_bm();
int ffn_tiled_hcols();
int ffn_tiled_bn();
// build_schedule: (re)build the tiled kernel's m-tile schedule in the workspace
// from expert_offsets before launching; a second stage of the same call may reuse it.
hipError_t launch_ffn_stage(int mode, FfnArgs a, int64_t T, int64_t E, bool build_schedule, hipStream_t st);
hipError_t launch_sq_reduce(const float* part, int64_t npairs, int n_part, float* out, hipStream_t st);

// y = sum_j pair_out[t*k + j] * pair_scale[t*k + j] (+ add[t] if add != null)
hipError_t launch_combine(const uint16_t* pair_out, const float* pair_scale, const float* add, int64_t T, int64_t k,
                          int64_t H, int out_dtype, void* y, hipStream_t st);
hipError_t launch_reap(const float* sq, const float* topk_w, const int32_t* offsets, const int32_t* sorted,
                       int64_t E, float* saliency, hipStream_t st);
hipError_t launch_combine_reap(const uint16_t* pair_out, const float* pair_scale, int64_t T, int64_t k, int64_t H, int out_dtype, void* y,
                               const float* sq, const float* topk_w, const int32_t* offsets, const int32_t* sorted,
                               int64_t E, float* saliency, hipStream_t st);
hipError_t launch_prune_select(const float* saliency, int64_t E, int64_t n_keep, int32_t* keep_ids, hipStream_t st);
hipError_t launch_gather_blocks(const void* src, int64_t n_src, int64_t bytes, const int32_t* ids, int64_t n_ids,
                                void* dst, hipStream_t st);

// BF16 shared expert: mode 0 = gate_up (a = x, writes h), 1 = down (a = h, writes out)
bool shared_use_small(int64_t T);
size_t shared_part_bytes(int64_t T, int64_t H, int64_t I);
hipError_t launch_shared_stage(int mode, const uint16_t* a, int64_t lda, const uint16_t* w, int64_t T, int64_t H,
                               int64_t I, uint16_t* h, float* out, float* part, hipStream_t st);

// dst = bf16((src * signs) . blockdiag(H_b) / sqrt(b)), row by row
int64_t hadamard_max_cols();
hipError_t launch_hadamard_rotate(const uint16_t* src, int64_t rows, int64_t cols, int64_t ld_src, const float* signs,
                                  int64_t b, uint16_t* dst, int64_t ld_dst, hipStream_t st);

// ---- MXFP4 (blocks of 32 E2M1 elements, E8M0 scales); rows are padded to whole column groups
constexpr int64_t mx_padded(int64_t cols) { return (cols + 255) / 256 * 256; }

// Arguments of an MXFP4 product.  104 bytes: a launch with up to 112 bytes of
// arguments was measured 0.8 us shorter on the host (2.9 against 3.7 us) than
// one with 128 or more, so the stages share fields and sizes are 32 bits.
struct MxArgs {
  const uint8_t* a_codes;   // activations [rows, KK * 128]
  const uint8_t* a_scales;  // [rows, KK * 8]
  const uint8_t* w_codes;   // packed weights (experts one after another)
  const uint8_t* w_scales;
  void* out;               // linear: BF16 or FP32 [T, ldo]; gate_up: h codes [T*k, ldo]; down: FP16 pair rows [T*k, ldo]
  void* out_scales;        // gate_up: h scale bytes [T*k, ldo / 16]; down: FP32 pair scales [T*k]
  const int32_t* offsets;  // experts: first pair of each, and their end [E + 1]
  const int32_t* sorted;   // experts: pairs by expert
  const float* topk_w;     // down: routing weights [T*k]
  const int32_t* w_max;    // down: largest weight scale byte per expert
  int32_t KK;              // column groups of 256 in the reduction
  int32_t N;               // weight rows (per expert)
  int32_t G;               // groups of 32 weight rows (per expert)
  int32_t ldo;             // elements (gate_up: bytes) of an output row
  int32_t T;               // linear: tokens
  int32_t E;               // experts: their number
  int32_t aux;             // gate_up: k; down: ceil(log2(36 I)); linear: bit 0 FP32 results, bit 1 rows on 16 bytes
};
static_assert(sizeof(MxArgs) <= 112, "see above");
constexpr int32_t kMxOutF32 = 1, kMxOutVec = 2;

// Both stages of the experts' FFN.
struct MxExperts {
  MxArgs gate_up, down;
  int64_t T, k, E;
};

hipError_t launch_mx_quantize(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                                void* out, int64_t ld, hipStream_t st);
hipError_t launch_mx_quantize_weights(const uint16_t* w, int64_t batch, int64_t N, int64_t K, uint8_t* codes,
                                      uint8_t* scales, int32_t* max_scale, hipStream_t st);
// canonical -> packed (pack) or back; max_scale (pack only) may be null
hipError_t launch_mx_relayout(uint8_t* codes, uint8_t* scales, int64_t batch, int64_t N, int64_t K, uint8_t* pcodes,
                              uint8_t* pscales, int32_t* max_scale, bool pack, hipStream_t st);
hipError_t launch_mx_linear(const MxArgs& a, hipStream_t st);
hipError_t launch_mx_experts(const MxExperts& x, hipStream_t st);

// Norms around a block; x is the row to norm (norm_in) or the block output y
// (norm_out).  As short as MxArgs, for the same reason.
struct NormArgs {
  const void* x;
  const uint16_t* r;
  const uint16_t* w_post;  // norm_out: null = no norm of y
  const uint16_t* gate;    // null = 1; element (t, c) at t * gate_rs + (gate_row ? 0 : c)
  const uint16_t* w;       // weight of the norm that follows; null = none
  uint16_t* r_out;
  uint16_t* n;     // null = only the codes
  uint8_t* codes;  // null = not quantised
  uint8_t* scales;
  int32_t ldx, ldr, ldro, ldn;
  int32_t gate_rs;
  uint32_t H : 16, Hp : 15, gate_row : 1;  // Hp: columns the row's lanes cover (padded when it is quantised)
  float scale, eps;
};
static_assert(sizeof(NormArgs) <= 112, "see MxArgs");
int64_t norm_max_cols();
hipError_t launch_norm(const NormArgs& a, int64_t T, bool post, bool y_f32, hipStream_t st);

}  // namespace moe
