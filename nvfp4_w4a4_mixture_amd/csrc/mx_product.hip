// Products of MXFP4 activations and packed MXFP4 weights on the scaled FP4
// MFMA: the dense y = x W^T, and the two stages of the routed experts' FFN.
#include "launch.h"
#include "mx_common.h"

namespace moe {

namespace {

enum { kLinear = 0, kGateUp = 1, kDown = 2 };

// Scale of a pair row: an exponent E with |w_p f| < 2^(E + 15) for every
// operand.  |f| <= I * 6^2 * 2^(bh - 127) * 2^(bw - 127) for the largest scale
// byte bh of the h row and bw of the expert's down weights, 36 I <= 2^lg, and
// |w_p| < 2^(ew + 1).  FP16's normal range reaches 29 binades below 2^15, so a
// loose bound costs no precision.  Clamped so that 2^E and 2^-E are normal.
__device__ __forceinline__ int pair_exponent(float wp, uint32_t bh, int bw, int lg) {
  const int ew = (int)((__float_as_uint(wp) >> 23) & 255u) - 127;
  const int e = ew + 1 + lg + (int)bh + bw - 254 - 15;
  return min(max(e, -126), 113);
}

__device__ __forceinline__ uint32_t max_byte(uint32_t d) {
  return max(max(d & 255u, (d >> 8) & 255u), max((d >> 16) & 255u, d >> 24));
}

}  // namespace

// Streaming product: few tokens per weight row, so the weights' bytes bound it.
// A workgroup takes R groups of 32 weight rows (gate_up: a gate group and the
// up group of the same h columns) and tiles of 32 tokens; its NW waves split
// the columns and load their fragments straight from memory to registers (a
// packed fragment is one contiguous kilobyte), and the partial sums meet in LDS
// in a fixed order.
template <int MODE, int R, int NW>
__global__ __launch_bounds__(NW * 64) void mx_stream_kernel(MxArgs a) {
  __shared__ float part[NW][R][16][64];
  __shared__ uint32_t hmax[NW][32];
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, n = l & 31, f = l >> 5;
  const int e = MODE == kLinear ? 0 : blockIdx.y;
  int64_t lo = 0, hi = a.T;
  if (MODE != kLinear) {
    lo = a.offsets[e];
    hi = a.offsets[e + 1];
  }
  int64_t g[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    g[i] = MODE == kGateUp ? (int64_t)blockIdx.x + i * (a.G / 2) : min((int64_t)blockIdx.x * R + i, a.G - 1);

  for (int64_t t0 = lo + (MODE == kLinear ? (int64_t)blockIdx.y * 32 : 0); t0 < hi; t0 += 32) {
    const int cnt = (int)min((int64_t)32, hi - t0);
    const int64_t pos = t0 + min(n, cnt - 1);  // lanes past the last token repeat it
    const int64_t arow = MODE == kGateUp ? a.sorted[pos] / a.k : pos;
    const uint8_t* xc = a.a_codes + arow * (a.KK * 128) + f * 64;
    const uint8_t* xs = a.a_scales + arow * (a.KK * 8) + f * 4;
    float16_t acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
    uint32_t bh = 0;
    for (int64_t c = w; c < a.KK; c += NW) {
      i32x4_t xf[4], wf[R][4];
      int ws[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t tile = ((int64_t)e * a.G + g[i]) * a.KK + c;
#pragma unroll
        for (int s = 0; s < 4; ++s)
          wf[i][s] = reinterpret_cast<const i32x4_t*>(a.w_codes + tile * kMxFragCodes)[s * 64 + l];
        ws[i] = reinterpret_cast<const int*>(a.w_scales + tile * kMxFragScales)[l];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) xf[s] = reinterpret_cast<const i32x4_t*>(xc + c * 128)[s];
      const int sx = *reinterpret_cast<const int*>(xs + c * 8);
      if (MODE == kDown) bh = max(bh, max_byte((uint32_t)sx));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        acc[i] = mx_mfma<0>(wf[i][0], xf[0], acc[i], ws[i], sx);
        acc[i] = mx_mfma<1>(wf[i][1], xf[1], acc[i], ws[i], sx);
        acc[i] = mx_mfma<2>(wf[i][2], xf[2], acc[i], ws[i], sx);
        acc[i] = mx_mfma<3>(wf[i][3], xf[3], acc[i], ws[i], sx);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) part[w][i][r][l] = acc[i][r];
    if (MODE == kDown) {
      bh = max(bh, (uint32_t)__shfl_xor((int)bh, 32));
      if (f == 0) hmax[w][n] = bh;
    }
    __syncthreads();
    // thread (tok, p): features 4 p .. 4 p + 3 of one token
    const int tok = tid >> 3, p = tid & 7;
    if (tid < 256 && tok < cnt) {
      float v[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float s = part[0][i][4 * (p & 3) + j][32 * (p >> 2) + tok];
#pragma unroll
          for (int q = 1; q < NW; ++q) s += part[q][i][4 * (p & 3) + j][32 * (p >> 2) + tok];
          v[i][j] = s;
        }
      const int64_t row = t0 + tok;
      if constexpr (MODE == kGateUp) {
        float h[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = silu(v[0][j]) * v[1][j];
          m = max(m, abs_bits(h[j]));
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        m = max(m, (uint32_t)__shfl_xor((int)m, 4));
        const uint32_t byte = mx_scale_byte(m);
        const int64_t blk = blockIdx.x;
        reinterpret_cast<uint16_t*>(a.h_codes + row * a.ldh)[blk * 8 + p] = (uint16_t)mx_encode8(h, byte);
        if (p == 0) a.h_scales[row * (a.ldh / 16) + blk] = (uint8_t)byte;
      } else {
        float wp = 1.0f, inv = 1.0f;
        int64_t out = row;
        if constexpr (MODE == kDown) {
          out = a.sorted[row];
          wp = a.topk_w[out];
          uint32_t b = hmax[0][tok];
#pragma unroll
          for (int q = 1; q < NW; ++q) b = max(b, hmax[q][tok]);
          const int E = pair_exponent(wp, b, a.w_max[e], a.lg36I);
          inv = __uint_as_float((uint32_t)(127 - E) << 23);
          if (blockIdx.x == 0 && p == 0) a.pair_scale[out] = __uint_as_float((uint32_t)(127 + E) << 23);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int64_t gi = (int64_t)blockIdx.x * R + i;
          if (gi >= a.G) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t col = gi * 32 + 4 * p + j;
            if (col >= a.N) continue;
            if constexpr (MODE == kDown)
              reinterpret_cast<_Float16*>(a.out)[out * a.ldo + col] = (_Float16)((wp * v[i][j]) * inv);
            else if (a.out_f32)
              static_cast<float*>(a.out)[out * a.ldo + col] = v[i][j];
            else
              static_cast<uint16_t*>(a.out)[out * a.ldo + col] = (uint16_t)bf16_bits_rne(v[i][j]);
          }
        }
      }
    }
    if (MODE == kLinear) break;
    __syncthreads();
  }
}

// Rows of h past I (a row is padded to a whole column group) are zero blocks.
__global__ __launch_bounds__(256) void mx_zero_pad_kernel(uint8_t* codes, uint8_t* scales, int64_t rows, int64_t ldh,
                                                          int64_t I) {
  const int64_t blocks = ldh / 16 - I / 32;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * blocks) return;
  const int64_t r = i / blocks, b = I / 32 + (i - r * blocks);
  *reinterpret_cast<uint4*>(codes + r * ldh + b * 16) = make_uint4(0, 0, 0, 0);
  scales[r * (ldh / 16) + b] = 0;
}

hipError_t launch_mx_linear(const MxArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((mx_stream_kernel<kLinear, 1, 8>), dim3((unsigned)a.G, (unsigned)((a.T + 31) / 32)), dim3(512), 0,
                     st, a);
  return hipGetLastError();
}

hipError_t launch_mx_gate_up(const MxArgs& a, int64_t E, hipStream_t st) {
  const int64_t I = a.N / 2, pad = a.ldh / 16 - I / 32, npairs = a.T * a.k;
  if (pad > 0)
    hipLaunchKernelGGL(mx_zero_pad_kernel, dim3((unsigned)((npairs * pad + 255) / 256)), dim3(256), 0, st, a.h_codes,
                       a.h_scales, npairs, a.ldh, I);
  hipLaunchKernelGGL((mx_stream_kernel<kGateUp, 2, 4>), dim3((unsigned)(a.G / 2), (unsigned)E), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_mx_down(const MxArgs& a, int64_t E, hipStream_t st) {
  hipLaunchKernelGGL((mx_stream_kernel<kDown, 2, 4>), dim3((unsigned)((a.G + 1) / 2), (unsigned)E), dim3(256), 0, st,
                     a);
  return hipGetLastError();
}

}  // namespace moe
