// MXFP4 quantisation of activations, its read-back, and the packing of weights.
#include "launch.h"
#include "mx_common.h"

namespace moe {

namespace {

// Eight consecutive elements as floats.
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

}  // namespace

// Four neighbouring lanes share one block of 32: each reads 8 elements (16 or
// 32 bytes), the block's amax is two exchanges within the quad, and each writes
// one dword of codes.  Columns past `cols` (up to the padded row) are zero
// blocks with scale byte 0.  Memory bound: 2 (4) + 17/32 bytes an element;
// 8192 x 6144 BF16 in 22 us (5.7 TB/s, what a copy reaches).  Four blocks of
// loads a thread were no faster there, and slower on a few rows (4.6 against
// 3.4 us for 16 x 6144).
template <typename X>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const X* __restrict__ x, uint32_t n, uint32_t cols,
                                                          int64_t ld, uint32_t chunks, uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;  // chunk of 8 elements of the padded rows
  if (i >= n) return;                                  // n % 32 == 0: a quad is in or out as one
  const uint32_t r = i / chunks, c = (i - r * chunks) * 8;
  float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (c < cols) load8(x + r * ld + c, f);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, abs_bits(f[k]));
  m = quad_max(m);
  const uint32_t byte = mx_scale_byte(m);
  codes[i] = mx_encode8(f, byte);
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

// The values that codes stand for, 8 elements a thread.  Memory bound: 8192 x
// 6144 to BF16 in 20 us (6.3 TB/s); four times 8 a thread take the same, decoding
// in integer steps took 23.  Streaming
// stores: quantising 8192 x 6144 BF16 and reading it back took 46 us with them
// and 54 us without.
template <bool F32>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, uint32_t n,
                                                            uint32_t chunks, uint32_t chunks_padded,
                                                            void* __restrict__ out, int64_t ld) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t r = i / chunks, c = i - r * chunks;
  const int64_t src = (int64_t)r * chunks_padded + c, at = r * ld + (int64_t)c * 8;
  const float s = mx_scale_value(scales[src >> 2]);
  float f[8];
  mx_decode8(codes[src], f);  // without the scale: the conversion has no byte 0 and no NaN
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= s;
  if (F32) {
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int k = 0; k < 8; k += 4)
      store16_streaming(p + k, __float_as_uint(f[k]), __float_as_uint(f[k + 1]), __float_as_uint(f[k + 2]),
                        __float_as_uint(f[k + 3]));
  } else {  // exact: two significant bits, and BF16 has FP32's exponents (down to 2^-133)
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (__float_as_uint(f[2 * k]) >> 16) | (__float_as_uint(f[2 * k + 1]) & 0xFFFF0000u);
    store16_streaming(static_cast<uint16_t*>(out) + at, w[0], w[1], w[2], w[3]);
  }
}

// MXFP8 of activations: as mx_quantize_kernel, but a chunk of 8 elements is 8
// bytes of codes.
template <typename X>
__global__ __launch_bounds__(256) void mx8_quantize_kernel(const X* __restrict__ x, uint32_t n, uint32_t cols,
                                                           int64_t ld, uint32_t chunks, uint2* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t r = i / chunks, c = (i - r * chunks) * 8;
  float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (c < cols) load8(x + r * ld + c, f);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, abs_bits(f[k]));
  m = quad_max(m);
  const uint32_t byte = mx8_scale_byte(m);
  codes[i] = make_uint2(mx8_encode4(f, byte), mx8_encode4(f + 4, byte));
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

template <bool F32>
__global__ __launch_bounds__(256) void mx8_dequantize_kernel(const uint2* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, uint32_t n,
                                                             uint32_t chunks, uint32_t chunks_padded,
                                                             void* __restrict__ out, int64_t ld) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t r = i / chunks, c = i - r * chunks;
  const int64_t src = (int64_t)r * chunks_padded + c, at = r * ld + (int64_t)c * 8;
  const float s = mx_scale_value(scales[src >> 2]);
  const uint2 d = codes[src];
  float f[8];
  mx8_decode4(d.x, f);
  mx8_decode4(d.y, f + 4);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= s;
  if (F32) {
    float* p = static_cast<float*>(out) + at;
#pragma unroll
    for (int k = 0; k < 8; k += 4)
      store16_streaming(p + k, __float_as_uint(f[k]), __float_as_uint(f[k + 1]), __float_as_uint(f[k + 2]),
                        __float_as_uint(f[k + 3]));
  } else {  // four significant bits: exact, but below 2^-130, whose values BF16's subnormals (steps of 2^-133) may round
    store16_streaming(static_cast<uint16_t*>(out) + at, bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                      bf16_pair(f[6], f[7]));
  }
}

// ---- weights: one thread per (row, block of 32) of the padded matrix, once per
// weight set.  The atomics bound the two kernels that give a largest byte, one a
// block on one word a matrix: 8 matrices of 4096 x 6144 take 71 ms, and 0.1 on the
// way back, which has none.

__device__ __forceinline__ bool mx_weight_slot(int64_t i, int64_t batch, int64_t G, int64_t KK, int64_t& b,
                                               int64_t& row, int64_t& blk) {
  const int64_t per = G * 32 * KK * 8;
  if (i >= batch * per) return false;
  b = i / per;
  const int64_t t = i - b * per;
  row = t / (KK * 8);
  blk = t - row * (KK * 8);
  return true;
}

__device__ __forceinline__ void mx_packed_offsets(int64_t b, int64_t row, int64_t blk, int64_t G, int64_t KK,
                                                  int64_t& code, int64_t& scale) {
  const int64_t tile = (b * G + (row >> 5)) * KK + (blk >> 3);
  const int s = (int)(blk & 3), lane = mx_packed_lane(row, blk);
  code = tile * kMxFragCodes + s * 1024 + lane * 16;
  scale = tile * kMxFragScales + lane * 4 + s;
}

__global__ __launch_bounds__(256) void mx_quantize_weights_kernel(const uint16_t* __restrict__ w, int64_t batch,
                                                                  int64_t N, int64_t K, int64_t G, int64_t KK,
                                                                  uint8_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales, int* max_scale) {
  int64_t b, row, blk;
  if (!mx_weight_slot((int64_t)blockIdx.x * 256 + threadIdx.x, batch, G, KK, b, row, blk)) return;
  uint4 c = make_uint4(0, 0, 0, 0);
  uint32_t byte = 0;
  if (row < N && blk * 32 < K) {
    float f[32];
    const uint16_t* src = w + (b * N + row) * K + blk * 32;
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) load8(src + 8 * q, f + 8 * q);
#pragma unroll
    for (int k = 0; k < 32; ++k) m = max(m, abs_bits(f[k]));
    byte = mx_scale_byte(m);
    c = make_uint4(mx_encode8(f, byte), mx_encode8(f + 8, byte), mx_encode8(f + 16, byte), mx_encode8(f + 24, byte));
    if (max_scale) atomicMax(max_scale + b, (int)byte);  // a maximum: the order does not matter
  }
  int64_t oc, os;
  mx_packed_offsets(b, row, blk, G, KK, oc, os);
  *reinterpret_cast<uint4*>(codes + oc) = c;
  scales[os] = (uint8_t)byte;
}

// canonical (row-major codes [batch, N, K/2], scales [batch, N, K/32]) <-> packed
template <bool PACK>
__global__ __launch_bounds__(256) void mx_relayout_kernel(uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                          int64_t batch, int64_t N, int64_t K, int64_t G, int64_t KK,
                                                          uint8_t* __restrict__ pcodes, uint8_t* __restrict__ pscales,
                                                          int* max_scale) {
  int64_t b, row, blk;
  if (!mx_weight_slot((int64_t)blockIdx.x * 256 + threadIdx.x, batch, G, KK, b, row, blk)) return;
  const bool in = row < N && blk * 32 < K;
  int64_t oc, os;
  mx_packed_offsets(b, row, blk, G, KK, oc, os);
  const int64_t at = (b * N + row) * (K / 32) + blk;
  if (PACK) {
    uint4 c = make_uint4(0, 0, 0, 0);
    uint32_t byte = 0;
    if (in) {
      c = reinterpret_cast<const uint4*>(codes)[at];
      byte = scales[at];
      if (max_scale) atomicMax(max_scale + b, (int)byte);
    }
    *reinterpret_cast<uint4*>(pcodes + oc) = c;
    pscales[os] = (uint8_t)byte;
  } else if (in) {
    reinterpret_cast<uint4*>(codes)[at] = *reinterpret_cast<const uint4*>(pcodes + oc);
    scales[at] = pscales[os];
  }
}

__global__ void mx_zero_ints_kernel(int* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

// rows * padded columns / 8 < 2^32 (checked by the caller)
hipError_t launch_mx_quantize(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t st) {
  const uint32_t chunks = (uint32_t)(mx_padded(cols) / 8), n = (uint32_t)(rows * chunks);
  const dim3 grid((unsigned)(((uint64_t)n + 255) / 256));
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (f32)
    return launch_kernel(mx_quantize_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(x), n,
                         (uint32_t)cols, ld, chunks, c, scales);
  return launch_kernel(mx_quantize_kernel<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(x), n,
                       (uint32_t)cols, ld, chunks, c, scales);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                                void* out, int64_t ld, hipStream_t st) {
  const uint32_t chunks = (uint32_t)(cols / 8), padded = (uint32_t)(mx_padded(cols) / 8), n = (uint32_t)(rows * chunks);
  auto* k = f32 ? mx_dequantize_kernel<true> : mx_dequantize_kernel<false>;
  return launch_kernel(k, dim3((n + 255) / 256), dim3(256), 0, st, reinterpret_cast<const uint32_t*>(codes), scales, n,
                       chunks, padded, out, ld);
}

// rows * padded columns / 8 < 2^32 (checked by the caller)
hipError_t launch_mx8_quantize(const void* x, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                               uint8_t* scales, hipStream_t st) {
  const uint32_t chunks = (uint32_t)(mx_padded(cols) / 8), n = (uint32_t)(rows * chunks);
  const dim3 grid((unsigned)(((uint64_t)n + 255) / 256));
  uint2* c = reinterpret_cast<uint2*>(codes);
  if (f32)
    return launch_kernel(mx8_quantize_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(x), n,
                         (uint32_t)cols, ld, chunks, c, scales);
  return launch_kernel(mx8_quantize_kernel<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(x), n,
                       (uint32_t)cols, ld, chunks, c, scales);
}

hipError_t launch_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool f32,
                                 void* out, int64_t ld, hipStream_t st) {
  const uint32_t chunks = (uint32_t)(cols / 8), padded = (uint32_t)(mx_padded(cols) / 8), n = (uint32_t)(rows * chunks);
  auto* k = f32 ? mx8_dequantize_kernel<true> : mx8_dequantize_kernel<false>;
  return launch_kernel(k, dim3((unsigned)(((uint64_t)n + 255) / 256)), dim3(256), 0, st, reinterpret_cast<const uint2*>(codes),
                       scales, n, chunks, padded, out, ld);
}

namespace {
struct WeightGrid {
  int64_t G, KK, n;
  WeightGrid(int64_t batch, int64_t N, int64_t K) : G((N + 31) / 32), KK(mx_padded(K) / 256), n(batch * G * 32 * KK * 8) {}
  dim3 grid() const { return dim3((unsigned)((n + 255) / 256)); }
};
void zero_max(int32_t* max_scale, int64_t batch, hipStream_t st) {
  if (max_scale)
    hipLaunchKernelGGL(mx_zero_ints_kernel, dim3((unsigned)((batch + 255) / 256)), dim3(256), 0, st, max_scale, batch);
}
}  // namespace

hipError_t launch_mx_quantize_weights(const uint16_t* w, int64_t batch, int64_t N, int64_t K, uint8_t* codes,
                                      uint8_t* scales, int32_t* max_scale, hipStream_t st) {
  const WeightGrid g(batch, N, K);
  zero_max(max_scale, batch, st);
  hipLaunchKernelGGL(mx_quantize_weights_kernel, g.grid(), dim3(256), 0, st, w, batch, N, K, g.G, g.KK, codes, scales,
                     max_scale);
  return hipGetLastError();
}

hipError_t launch_mx_relayout(uint8_t* codes, uint8_t* scales, int64_t batch, int64_t N, int64_t K, uint8_t* pcodes,
                              uint8_t* pscales, int32_t* max_scale, bool pack, hipStream_t st) {
  const WeightGrid g(batch, N, K);
  if (pack) {
    zero_max(max_scale, batch, st);
    hipLaunchKernelGGL(mx_relayout_kernel<true>, g.grid(), dim3(256), 0, st, codes, scales, batch, N, K, g.G, g.KK,
                       pcodes, pscales, max_scale);
  } else {
    hipLaunchKernelGGL(mx_relayout_kernel<false>, g.grid(), dim3(256), 0, st, codes, scales, batch, N, K, g.G, g.KK,
                       pcodes, pscales, max_scale);
  }
  return hipGetLastError();
}

}  // namespace moe
