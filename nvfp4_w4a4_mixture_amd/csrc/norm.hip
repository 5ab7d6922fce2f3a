// RMS norms before and after a block, fused with the block's gate, residual
// scale and residual, and with the MXFP4 or MXFP8 quantisation of what the next
// product reads.
#include <type_traits>

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

// The same in FP64
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)lane_dpp<CTRL>((uint32_t)(b >> 32)) << 32 | lane_dpp<CTRL>((uint32_t)b));
}
template <int NW>
__device__ __forceinline__ double row_sum(double v, double* lds, int w) {
  v += dpp_f64<kLaneXor1>(v);
  v += dpp_f64<kLaneXor2>(v);
  v += dpp_f64<kLaneHalfMirror>(v);
  v += dpp_f64<kLaneMirror>(v);
  uint64_t b = __builtin_bit_cast(uint64_t, v);
  auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
  v = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  b = __builtin_bit_cast(uint64_t, v);
  hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
  v = __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  if (NW == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[w] = v;
  __syncthreads();
  double s = lds[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) s += lds[i];
  return s;
}

// Whether a value within `off` of f may round to another BF16 value than f does
__device__ __forceinline__ bool near_bf16_tie(float f, float off) {
  return fabsf(f - __uint_as_float((__float_as_uint(f) & 0xFFFF0000u) | 0x8000u)) <= off;
}
constexpr float kNormNoise = 0x1p-21f;  // relative, of the products of a result formed in FP32 (at most four roundings)

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
//
// A8 (the MXFP8 forms): results are all but always the exact ones, rounded to FP32
// and to BF16.  E4M3 has steps
// of up to an eighth of a value, so that the FP32 noise that moves one BF16 result
// in some 10^5 to its neighbour moves one element in 10^6 by such a step.  So the
// sums are FP64 (of FP32 sums of four squares: 10^-9 of a row's), and the eight results of a lane are formed again in FP64 if one of
// them lies within FP32's noise of a border: one group in some 500.
template <int NW, int V, bool POST, bool YF32, bool A8>
__global__ __launch_bounds__(64 * NW) void norm_kernel(NormArgs a) {
  using Sum = typename std::conditional<A8, double, float>::type;
  __shared__ Sum lds[2][NW];
  const int w = threadIdx.x >> 6, t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int H = (int)a.H;
  const bool follow = !POST || a.w != nullptr;
  auto square_sum = [](const float* v, Sum s) {  // of eight
    if constexpr (A8) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float g = fmaf(v[i], v[i], fmaf(v[i + 1], v[i + 1], fmaf(v[i + 2], v[i + 2], v[i + 3] * v[i + 3])));
        if (g > 1e-30f && g < 1e38f) {
          s += (double)g;
        } else {  // squares that leave FP32's range, NaN, or zeros
#pragma unroll
          for (int j = 0; j < 4; ++j) s = fma((double)v[i + j], (double)v[i + j], s);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
    }
    return s;
  };
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
    double inv64 = 1.0;
    if (a.w_post) {
      Sum sq = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) sq = square_sum(x[v], sq);
      if constexpr (A8) {
        inv64 = rsqrt(row_sum<NW>(sq, lds[0], w) * (1.0 / (double)H) + (double)a.eps);
        inv = (float)inv64;
      } else {
        inv = rsqrtf(row_sum<NW>(sq, lds[0], w) / (float)H + a.eps);
      }
    }
    const bool far = A8 && isinf(inv);  // rows under 2^-128 without an eps: FP32 cannot hold it
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float wv[8], rv[8], gv[8], f[8];
      unpack8(rr[v], rv);
      if (a.w_post) unpack8(wp[v], wv);
      if (a.gate && !a.gate_row) unpack8(gg[v], gv);
      bool close = far;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z = x[v][i];
        if (a.w_post) z = z * inv * wv[i];
        if (a.gate) z *= a.gate_row ? g_row : gv[i];
        f[i] = fmaf(a.scale, z, rv[i]);
        if constexpr (A8) close |= near_bf16_tie(f[i], kNormNoise * fabsf(a.scale * z) + kNormNoise * fabsf(f[i]));
      }
      if (A8 && close) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          double z = (double)x[v][i] * inv64;
          if (a.w_post) z *= (double)wv[i];
          if (a.gate) z *= (double)(a.gate_row ? g_row : gv[i]);
          f[i] = (float)fma(z, (double)a.scale, (double)rv[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = f[i];
      const uint4 o = pack8(x[v]);
      unpack8(o, x[v]);  // the next norm reads the residual that is kept
      store8_bf16(a.r_out + row * a.ldro, (v * 64 * NW + t) * 8, H, o);
    }
    if (!follow) return;
  }
  Sum sq = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) sq = square_sum(x[v], sq);
  float inv;
  double inv64 = 0.0;
  if constexpr (A8) {
    inv64 = rsqrt(row_sum<NW>(sq, lds[1], w) * (1.0 / (double)H) + (double)a.eps);
    inv = (float)inv64;
  } else {
    inv = rsqrtf(row_sum<NW>(sq, lds[1], w) / (float)H + a.eps);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * 64 * NW + t) * 8;
    float wv[8], q[8];
    unpack8(wn[v], wv);
    bool close = A8 && isinf(inv);  // as above
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = x[v][i] * inv * wv[i];
      if constexpr (A8) close |= ((__float_as_uint(q[i]) + 8u) & 0xFFF0u) == 0x8000u;  // 2^-20 to 2^-21 of it
    }
    if (A8 && close) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (float)((double)x[v][i] * inv64 * (double)wv[i]);
    }
    const uint4 o = pack8(q);
    if (a.n) store8_bf16(a.n + row * a.ldn, c, H, o);
    if (a.codes) {  // H % 32 == 0: a quad of lanes holds one block
      uint32_t m = 0;
      unpack8(o, q);
      if (c >= H) {  // the padding is zero whatever the norm is
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(q[i]));
      const uint32_t amax = quad_max(m), byte = A8 ? mx8_scale_byte(amax) : mx_scale_byte(amax);
      if (c < (int)a.Hp) {
        const int64_t at = (row * (int)a.Hp + c) / 8;
        if constexpr (A8) reinterpret_cast<uint2*>(a.codes)[at] = make_uint2(mx8_encode4(q, byte), mx8_encode4(q + 4, byte));
        else reinterpret_cast<uint32_t*>(a.codes)[at] = mx_encode8(q, byte);
        if ((t & 3) == 0) a.scales[at / 4] = (uint8_t)byte;
      }
    }
  }
}

namespace {

template <int NW, int V, bool POST, bool A8>
hipError_t launch_norm_as(const NormArgs& a, int64_t T, bool y_f32, hipStream_t st) {
  const dim3 grid((unsigned)T), block(64 * NW);
  if constexpr (POST) {
    if (y_f32) return launch_kernel(norm_kernel<NW, V, POST, true, A8>, grid, block, 0, st, a);
  }
  return launch_kernel(norm_kernel<NW, V, POST, false, A8>, grid, block, 0, st, a);
}

// A wave alone needs no barrier and leaves fewer lanes idle, four waves finish a
// row sooner.  8192 rows of 1032: 8.5 us by one wave each, 10.8 by four (norm_out
// 24.5 and 28.2); 500 rows of 1999: 5.5 and 4.2 us.  From 2056 columns on four
// are as fast or faster at any number of rows; twelve take one row of 6144 in
// 1.8 (2.8) us against 2.0 (3.0), but 1024 rows in 4.8 (8.3) against 4.3 (7.2).
template <bool POST, bool A8>
hipError_t launch_norm_shape(const NormArgs& a, int64_t T, bool y_f32, hipStream_t st) {
  const int cols = (int)a.Hp;
  if (cols <= 512) return launch_norm_as<1, 1, POST, A8>(a, T, y_f32, st);
  if (cols <= 1024) return launch_norm_as<1, 2, POST, A8>(a, T, y_f32, st);
  if (cols <= 1536 && T >= 2048) return launch_norm_as<1, 3, POST, A8>(a, T, y_f32, st);
  if (cols <= 2047 && T >= 2048) return launch_norm_as<1, 4, POST, A8>(a, T, y_f32, st);
  if (cols <= 2048) return launch_norm_as<4, 1, POST, A8>(a, T, y_f32, st);
  if (cols <= 4096) return launch_norm_as<4, 2, POST, A8>(a, T, y_f32, st);
  if (cols <= 6144) return launch_norm_as<4, 3, POST, A8>(a, T, y_f32, st);
  if (cols <= 8192) return launch_norm_as<4, 4, POST, A8>(a, T, y_f32, st);
  return launch_norm_as<4, 8, POST, A8>(a, T, y_f32, st);
}

// The MXFP8 forms do more arithmetic a row, so a row's waves share it further where
// they leave few lanes idle (norm_in / norm_out with FP32 y, 2000 rows of 2080, 2304
// and 2528 columns: 8.1 / 14.6, 8.1 / 15.0 and 8.3 / 15.6 us by four waves of two
// chunks, 7.4 / 13.7, 7.4 / 14.1 and 7.5 / 14.6 by five of one; 8192 rows of 2304 23.9 /
// 47.6 and 21.6 / 42.7, 16 rows 3.3 / 5.2 and 3.5 / 4.5), or where there are few long
// rows (16 of 5120: 3.9 / 6.0 by four waves of three, 3.5 / 5.2 by twelve; 256 of 6144
// 4.3 / 6.6 and 3.9 / 6.1; but 600 6.5 / 10.7 and 7.0 / 11.7, 8192 40 / 95 and 50 / 105,
// and 16 of 4096 3.9 / 4.8 by four waves of two and 3.5 / 5.0).
// A launch has less than 2^32 work-items, which the caller has checked for four waves a row.
template <bool POST>
hipError_t launch_norm8_shape(const NormArgs& a, int64_t T, bool y_f32, hipStream_t st) {
  const int cols = (int)a.Hp;
  if (cols > 2048 && cols <= 2560 && T * 320 < (int64_t)1 << 32) return launch_norm_as<5, 1, POST, true>(a, T, y_f32, st);
  if (cols > 4096 && cols <= 6144 && T <= 256) return launch_norm_as<12, 1, POST, true>(a, T, y_f32, st);
  return launch_norm_shape<POST, true>(a, T, y_f32, st);
}

}  // namespace

int64_t norm_max_cols() { return 16384; }

hipError_t launch_norm(const NormArgs& a, int64_t T, bool post, bool y_f32, hipStream_t st) {
  if (a.a8) return post ? launch_norm8_shape<true>(a, T, y_f32, st) : launch_norm8_shape<false>(a, T, false, st);
  return post ? launch_norm_shape<true, false>(a, T, y_f32, st) : launch_norm_shape<false, false>(a, T, false, st);
}

}  // namespace moe
