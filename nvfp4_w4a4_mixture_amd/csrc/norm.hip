// RMS norms before and after a block, fused with the block's gate, residual
// scale and residual, and with the MXFP4 quantisation of what the next product
// reads.
#include "launch.h"
#include "mx_common.h"

namespace moe {

namespace {

// Sum over the row's waves, in a fixed order; every thread gets it.
template <int NW>
__device__ __forceinline__ float row_sum(float v, float* lds, int w) {
  v += __uint_as_float(lane_dpp<kLaneXor1>(__float_as_uint(v)));
  v += __uint_as_float(lane_dpp<kLaneXor2>(__float_as_uint(v)));
  v += __uint_as_float(lane_dpp<kLaneHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(lane_dpp<kLaneMirror>(__float_as_uint(v)));
  // each result holds one of a pair of 16 (32) lanes in both
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  if (NW == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[w] = v;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) s += lds[i];
  return s;
}

// 16 bytes at an address aligned to an element only: one access on gfx950 all
// the same, so rows of any length and stride move in 16-byte pieces.
typedef uint32_t u32x4_any2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef float float4_any4_t __attribute__((ext_vector_type(4), aligned(4)));

// Eight BF16 (FP32) elements at column c of a row of H, as they lie in memory;
// zero past H.  Only the row's last piece, if it is short, goes by elements.
__device__ __forceinline__ uint4 load8_bf16(const uint16_t* p, int c, int H) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (c + 8 <= H) {
    const u32x4_any2_t v = *reinterpret_cast<const u32x4_any2_t*>(p + c);
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  if (c < H) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) w[i >> 1] |= (uint32_t)p[c + i] << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ void load8_f32(const float* p, int c, int H, float* f) {
  if (c + 8 <= H) {
    const float4_any4_t u = *reinterpret_cast<const float4_any4_t*>(p + c), v = *reinterpret_cast<const float4_any4_t*>(p + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = u[i];
      f[4 + i] = v[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  if (c < H) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) f[i] = p[c + i];
  }
}
__device__ __forceinline__ void store8_bf16(uint16_t* p, int c, int H, const uint4& b) {
  const uint32_t d[4] = {b.x, b.y, b.z, b.w};
  if (c + 8 <= H) {
    const u32x4_any2_t v = {b.x, b.y, b.z, b.w};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any2_t*>(p + c));  // see store16_streaming
    return;
  }
  if (c < H) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) p[c + i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
  }
}

}  // namespace

// A workgroup is a row: NW waves, V chunks of 8 columns per lane; the row stays in registers
// between the passes.  POST: the row is y, and the first norm, gate, residual
// scale and residual give r'; otherwise the row is x itself.  Everything the
// row needs is loaded before the first sum, so that one memory latency covers
// it; the sums are FP32, in a fixed order, and results are rounded once, to
// BF16.  Memory bound: norm_out of 8192 x 6144 with FP32 y moves 503 MB in 82 us
// (6.1 TB/s; a copy with streaming stores reaches 6.05).  Loading the residual
// and the weights after the first sum took 99 us, cached stores 90.  Few rows
// are bound by one latency of memory and by the two sums: 2.0 us (norm_in) and
// 3.0 (norm_out) for one row of 6144, where sums through LDS shuffles and
// rounding in integer steps took 3.0 and 4.7.
template <int NW, int V, bool POST, bool YF32>
__global__ __launch_bounds__(64 * NW) void norm_kernel(NormArgs a) {
  __shared__ float lds[2][NW];
  const int w = threadIdx.x >> 6, t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int H = (int)a.H;
  const bool follow = !POST || a.w != nullptr;
  float x[V][8];
  uint4 rr[V], wp[V], wn[V], gg[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * 64 * NW + t) * 8;
    if constexpr (YF32) load8_f32(static_cast<const float*>(a.x) + row * a.ldx, c, H, x[v]);
    else unpack8(load8_bf16(static_cast<const uint16_t*>(a.x) + row * a.ldx, c, H), x[v]);
    if constexpr (POST) rr[v] = load8_bf16(a.r + row * a.ldr, c, H);
  }
  if constexpr (POST) {
    if (a.gate && !a.gate_row) {
#pragma unroll
      for (int v = 0; v < V; ++v) gg[v] = load8_bf16(a.gate + row * a.gate_rs, (v * 64 * NW + t) * 8, H);
    }
    if (a.w_post) {
#pragma unroll
      for (int v = 0; v < V; ++v) wp[v] = load8_bf16(a.w_post, (v * 64 * NW + t) * 8, H);
    }
  }
  if (follow) {
#pragma unroll
    for (int v = 0; v < V; ++v) wn[v] = load8_bf16(a.w, (v * 64 * NW + t) * 8, H);
  }
  if constexpr (POST) {
    const float g_row = a.gate && a.gate_row ? bf16_to_f32(a.gate[row * a.gate_rs]) : 1.0f;
    float inv = 1.0f;
    if (a.w_post) {
      float sq = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[v][i], x[v][i], sq);
      inv = rsqrtf(row_sum<NW>(sq, lds[0], w) / (float)H + a.eps);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float wv[8], rv[8], gv[8];
      unpack8(rr[v], rv);
      if (a.w_post) unpack8(wp[v], wv);
      if (a.gate && !a.gate_row) unpack8(gg[v], gv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z = x[v][i];
        if (a.w_post) z = z * inv * wv[i];
        if (a.gate) z *= a.gate_row ? g_row : gv[i];
        x[v][i] = fmaf(a.scale, z, rv[i]);
      }
      const uint4 o = pack8(x[v]);
      unpack8(o, x[v]);  // the next norm reads the residual that is kept
      store8_bf16(a.r_out + row * a.ldro, (v * 64 * NW + t) * 8, H, o);
    }
    if (!follow) return;
  }
  float sq = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(x[v][i], x[v][i], sq);
  const float inv = rsqrtf(row_sum<NW>(sq, lds[1], w) / (float)H + a.eps);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * 64 * NW + t) * 8;
    float wv[8], q[8];
    unpack8(wn[v], wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x[v][i] * inv * wv[i];
    const uint4 o = pack8(q);
    if (a.n) store8_bf16(a.n + row * a.ldn, c, H, o);
    if (a.codes) {  // H % 32 == 0: a quad of lanes holds one block
      uint32_t m = 0;
      unpack8(o, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c >= H) q[i] = 0.0f;  // the padding is zero whatever the norm is
        m = max(m, abs_bits(q[i]));
      }
      const uint32_t byte = mx_scale_byte(quad_max(m));
      if (c < (int)a.Hp) {
        reinterpret_cast<uint32_t*>(a.codes)[(row * (int)a.Hp + c) / 8] = mx_encode8(q, byte);
        if ((t & 3) == 0) a.scales[(row * (int)a.Hp + c) / 32] = (uint8_t)byte;
      }
    }
  }
}

namespace {

template <int NW, int V, bool POST>
hipError_t launch_norm_as(const NormArgs& a, int64_t T, bool y_f32, hipStream_t st) {
  const dim3 grid((unsigned)T), block(64 * NW);
  if constexpr (POST) {
    if (y_f32) return launch_kernel(norm_kernel<NW, V, POST, true>, grid, block, 0, st, a);
  }
  return launch_kernel(norm_kernel<NW, V, POST, false>, grid, block, 0, st, a);
}

// A wave alone needs no barrier and leaves fewer lanes idle, four waves finish a
// row sooner.  8192 rows of 1032: 8.5 us by one wave each, 10.8 by four (norm_out
// 24.5 and 28.2); 500 rows of 1999: 5.5 and 4.2 us.  From 2056 columns on four
// are as fast or faster at any number of rows; twelve take one row of 6144 in
// 1.8 (2.8) us against 2.0 (3.0), but 1024 rows in 4.8 (8.3) against 4.3 (7.2).
template <bool POST>
hipError_t launch_norm_shape(const NormArgs& a, int64_t T, bool y_f32, hipStream_t st) {
  const int cols = (int)a.Hp;
  if (cols <= 512) return launch_norm_as<1, 1, POST>(a, T, y_f32, st);
  if (cols <= 1024) return launch_norm_as<1, 2, POST>(a, T, y_f32, st);
  if (cols <= 1536 && T >= 2048) return launch_norm_as<1, 3, POST>(a, T, y_f32, st);
  if (cols <= 2047 && T >= 2048) return launch_norm_as<1, 4, POST>(a, T, y_f32, st);
  if (cols <= 2048) return launch_norm_as<4, 1, POST>(a, T, y_f32, st);
  if (cols <= 4096) return launch_norm_as<4, 2, POST>(a, T, y_f32, st);
  if (cols <= 6144) return launch_norm_as<4, 3, POST>(a, T, y_f32, st);
  if (cols <= 8192) return launch_norm_as<4, 4, POST>(a, T, y_f32, st);
  return launch_norm_as<4, 8, POST>(a, T, y_f32, st);
}

}  // namespace

int64_t norm_max_cols() { return 16384; }

hipError_t launch_norm(const NormArgs& a, int64_t T, bool post, bool y_f32, hipStream_t st) {
  return post ? launch_norm_shape<true>(a, T, y_f32, st) : launch_norm_shape<false>(a, T, false, st);
}

}  // namespace moe
