// Products of MXFP8 activations: the streaming kernel, and the shapes by sizes.
#include "mx_product.h"

namespace moe {

// Streaming product of 8-bit activations: few tokens per weight row, as
// mx_stream_kernel.  A workgroup takes 32 weight rows and up to 32 tokens; its
// eight waves split the columns and load their weight fragments straight from
// memory.  Their tokens' columns come as whole runs of 256 bytes and through LDS
// into fragments, one column group ahead: fetched as fragments, 32 rows of 16 bytes
// a load, they kept the memory pipes four times as long as the weights (16 x 6144 x
// 6144 10.2 us, so 7.0; 32 tokens 10.4 and 8.7; one token 6.5 either way, where the
// 4-bit product takes 4.6: twice the matrix instructions, and their operands to
// make).
//
// Activations go in as two operands (see mx8_part).  HALF: at most 16 tokens, so
// both fit the 32 columns of one: column n takes the large elements of token n %
// 16 if n < 16 and the rest if not, and the two columns' sums are added at the end.
template <bool HALF>
__global__ __launch_bounds__(512) void mx8_stream_kernel(MxArgs a) {
  constexpr int NW = 8, kRows = HALF ? 16 : 32, kParts = kRows / 4;  // tokens of a tile; loads of four rows
  constexpr int kPart = NW * 4 * 68 * 16, kStaged = NW * kRows * 256;
  __shared__ __align__(16) unsigned char smem[kPart > kStaged ? kPart : kStaged];
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int KK = (int)a.KK, tok_n = HALF ? n & 15 : n;
  const int t0 = (int)blockIdx.y * kRows, cnt = min(kRows, a.T - t0);
  const uint8_t* wc = a.w_codes + (int64_t)blockIdx.x * KK * kMxFragCodes;
  const uint8_t* ws = a.w_scales + (int64_t)blockIdx.x * KK * kMxFragScales;
  auto act_row = [&](int t) { return (uint32_t)(t0 + min(t, cnt - 1)); };  // rows past the last token repeat it
  uint32_t xoff[kParts];
#pragma unroll
  for (int i = 0; i < kParts; ++i) xoff[i] = act_row(4 * i + (l >> 4)) * (uint32_t)(KK * 256) + (uint32_t)(l & 15) * 16u;
  const uint8_t* xs = a.a_scales + (int64_t)act_row(tok_n) * (KK * 8) + f * 4;
  unsigned char* staged = smem + w * kRows * 256;  // the wave's own: 16-byte chunk c of row r at r * 256 + (c ^ (r & 15)) * 16
  struct Cols {
    i32x4_t x[kParts], w[4];
    int sw, sx;
  };
  // No branch stands before a load, so that the compiler can count those in flight (with one it waits for all of them)
  auto load = [&](int64_t c, Cols& d) {
    c = min(c, (int64_t)KK - 1);
#pragma unroll
    for (int i = 0; i < kParts; ++i) d.x[i] = *reinterpret_cast<const i32x4_t*>(a.a_codes + c * 256 + xoff[i]);
    d.sx = *reinterpret_cast<const int*>(xs + c * 8);
#pragma unroll
    for (int s = 0; s < 4; ++s) d.w[s] = reinterpret_cast<const i32x4_t*>(wc + c * kMxFragCodes)[s * 64 + l];
    d.sw = reinterpret_cast<const int*>(ws + c * kMxFragScales)[l];
  };
  float16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
  auto multiply = [&](Cols& d) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int r = 4 * i + (l >> 4);
      *reinterpret_cast<i32x4_t*>(staged + r * 256 + (((l & 15) ^ r) & 15) * 16) = d.x[i];
    }
    wave_lds_order();
    i32x8_t xf[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      xf[s] = join_halves(*reinterpret_cast<const i32x4_t*>(staged + tok_n * 256 + (((2 * s + f) ^ tok_n) & 15) * 16),
                          *reinterpret_cast<const i32x4_t*>(staged + tok_n * 256 + (((8 + 2 * s + f) ^ tok_n) & 15) * 16));
      if constexpr (HALF) xf[s] = mx8_part(xf[s], n >= 16);
    }
    wave_lds_order();
    acc = act_mfma<0, !HALF>(d.w[0], xf[0], acc, d.sw, d.sx);
    acc = act_mfma<1, !HALF>(d.w[1], xf[1], acc, d.sw, d.sx);
    acc = act_mfma<2, !HALF>(d.w[2], xf[2], acc, d.sw, d.sx);
    acc = act_mfma<3, !HALF>(d.w[3], xf[3], acc, d.sw, d.sx);
  };
  Cols d0, d1;
  load(w, d0);
  for (int c = w; c < KK; c += 2 * NW) {
    load(c + NW, d1);
    multiply(d0);
    if (c + NW >= KK) break;
    load(c + 2 * NW, d0);
    multiply(d1);
  }
  __syncthreads();  // the waves' sums take the place of their columns
  float4* part = reinterpret_cast<float4*>(smem);  // [NW][4 * 68]
#pragma unroll
  for (int q = 0; q < 4; ++q)
    part[w * 272 + q * 68 + f * 34 + n] = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
  __syncthreads();
  const int tok = tid >> 3, p = tid & 7, col = (int)blockIdx.x * 32 + 4 * p;  // features 4 p .. 4 p + 3 of one token
  if (tok >= cnt) return;
  float4 s = part[(p & 3) * 68 + (p >> 2) * 34 + tok];
#pragma unroll
  for (int k = 1; k < (HALF ? 2 : 1) * NW; ++k) {
    const float4 u = part[k % NW * 272 + (p & 3) * 68 + (p >> 2) * 34 + tok + (k < NW ? 0 : 16)];
    s.x += u.x;
    s.y += u.y;
    s.z += u.z;
    s.w += u.w;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
  const int64_t row = t0 + tok;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (col + q >= a.N) break;
    const float z = epilogue1(a, v[q], row, col + q);
    if (a.aux & kMxOutF32) static_cast<float*>(a.out)[row * a.ldo + col + q] = z;
    else static_cast<uint16_t*>(a.out)[row * a.ldo + col + q] = (uint16_t)bf16_pair(z, 0.0f);
  }
}

namespace {

// An 8-bit operand takes the matrix cores twice as long as a 4-bit one (a
// register-only loop of these products: 3.9 PFLOP/s on data, 4.8 on zeros), and a
// token's stage twice the LDS, so tiles are taller: weight rows are the cheaper
// side.  256 x 256 runs at 2.9 PFLOP/s of its loop (90% of the zeros' rate on
// zeros: the rest is power); stages of one MFMA step instead of two, with a ring
// twice as long, ran at 2.3, for their 32-byte runs of a token.  Waves of 128 x 64
// read two thirds of the LDS bytes of 64 x 128 and leave registers to spare, where
// those spilled.  Rings of eight stages for the small tile were no faster.
using Mx8_64x64 = MxTile<4, 2, 1, 1, 4, true>;
using Mx8_128x64 = MxTile<4, 2, 2, 1, 4, true>;
using Mx8_256x64 = MxTile<4, 4, 2, 2, 3, true>;
using Mx8_256x128 = MxTile<8, 4, 2, 2, 4, true>;
using Mx8_256x256 = MxTile<8, 2, 4, 2, 3, true>;

int64_t tiles(int64_t T, int64_t G, int64_t rows, int64_t tok) { return (G + rows / 32 - 1) / (rows / 32) * ((T + tok - 1) / tok); }

// The shape of a dense product with 16-bit results, both sides in us:
//   T x K x N            stream   64x64  128x64  256x64  256x128  256x256
//   1 x 6144 x 10240       10.0    10.5    12.0    18.9
//   1 x 6144 x 16384       12.7    11.4    12.3    19.7
//   1 x 4096 x 32768       17.3    13.2    12.8    15.7
//   32 x 6144 x 6144        8.1    10.6    12.4    16.4
//   32 x 6144 x 10240      16.1    11.3    13.3    20.4     22.4     34.6
//   64 x 6144 x 6144       14.7    11.8    14.6    20.2     22.4     35.0
//   64 x 6144 x 24576      48.5    27.0    20.9    26.4
//   128 x 6144 x 1024       7.9    11.3    14.7    20.2     28.9     36.6
//   509 x 6144 x 2048      30.7    12.8    16.1    21.6     31.5     55.2
//   512 x 6144 x 4096      59.7    25.3    19.0    25.8
//   512 x 6144 x 6144      88.2    36.7    32.6    26.4     34.5     58.2
//   1024 x 6144 x 6144             71.2    47.7    47.6     43.9     69.5
//   2048 x 2048 x 6144             50.4    34.2    29.1     35.6     33.3
//   8192 x 512 x 4096              38.2    34.7    29.0     32.3     30.5
//   8192 x 2048 x 6144            165.7   144.4   111.1    108.8     93.0
//   8192 x 6144 x 6144            467.5   390.7   284.2    246.8    225.6
// Streaming while its tiles of 32 x 32 fit the chip once; the smallest tile while
// its tiles do; the largest that still fills the chip; 256 x 128 where its tiles
// fill it just once.
Shape linear_shape(int64_t T, int64_t G, int64_t KK) {
  const int64_t cus = 256;
  if (tiles(T, G, 32, 32) <= cus) return kStream;
  if (tiles(T, G, 64, 64) <= cus) return k64x64;
  if (KK >= 8 && tiles(T, G, 256, 256) >= cus * 3 / 4) return k256x256;
  const int64_t n = tiles(T, G, 256, 128);
  if (n >= cus * 3 / 4 && n <= cus) return k256x128;
  return tiles(T, G, 256, 64) >= cus * 3 / 4 ? k256x64 : k128x64;
}

// FP32 results take two operands (see mx8_part), so the matrix cores bound them earlier:
//   T x K x N            stream   64x64  128x64  256x64  256x128  256x256
//   1 x 4096 x 32768       17.2    19.9    17.0    19.5
//   32 x 6144 x 10240      16.1    19.2    22.4    26.7     23.0     37.0
//   64 x 6144 x 6144       14.7    20.1    22.8    40.5     38.3     62.2
//   64 x 6144 x 10240      23.0    21.2    22.9    41.7
//   256 x 6144 x 6144      48.3            24.6    41.6     60.0    105.2
//   509 x 6144 x 2048      30.3    22.7    23.8    41.9
//   512 x 6144 x 4096      59.3    32.9    26.9    45.6
//   1024 x 6144 x 6144                     63.8    69.9     74.1    115.6
//   2048 x 6144 x 6144                    122.9   117.3    148.0    133.0
//   8192 x 2048 x 6144                    185.1   169.5    198.4    191.6
//   8192 x 6144 x 6144                    484.3   441.6    453.9    411.0
Shape linear_shape_exact(int64_t T, int64_t G) {
  if (T <= 32 || tiles(T, G, 32, 32) <= 512) return kStream;
  if (tiles(T, G, 64, 64) <= 256) return k64x64;
  return tiles(T, G, 256, 64) >= 512 ? k256x64 : k128x64;
}

// The shape of a stage of the experts' FFN; both stages in one shape, us:
//   E k H I, tokens         128x64  256x64  256x128  256x256
//   16 4 1024 512, 16         10.0    11.5     13.3     17.9
//   16 4 1024 512, 256        10.8    13.6     18.1     22.1
//   16 4 1024 512, 1024       20.4    19.2     19.4     28.0
//   16 4 1024 512, 8192      104.0    81.4     90.0     94.1
//   80 8 6144 2048, 16       164.1   159.9    171.6    202.8
//   80 8 6144 2048, 256      323.1   292.0    308.0    349.4
//   80 8 6144 2048, 1024     578.1   474.5    481.0    506.2
//   80 8 6144 2048, 2048     990.9   777.6    747.7    729.8
//   80 8 6144 2048, 8192      3275    2529     2358     2156
// (Few tokens through a small layer are streamed by mx_layer.hip's kernels.)
Shape experts_shape(int64_t pairs, int64_t E, int64_t rows, int64_t KK) {
  const int64_t some = pairs < E ? pairs : E;
  if ((pairs / 64 + some / 2) * ((rows + 255) / 256) < 256) return k128x64;
  return pairs >= 160 * E && KK >= 8 ? k256x256 : k256x64;
}

template <int MODE>
hipError_t launch_experts_stage(const MxArgs& a, const MxExperts& x, hipStream_t st) {
  const int64_t pairs = x.T * x.k;
  switch (experts_shape(pairs, x.E, a.N, a.KK)) {
    case k128x64: return launch_tiled<MODE, Mx8_128x64>(a, most_mtiles(pairs, x.E, 64), st);
    case k256x64: return launch_tiled<MODE, Mx8_256x64>(a, most_mtiles(pairs, x.E, 64), st);
    default: return launch_tiled<MODE, Mx8_256x256>(a, most_mtiles(pairs, x.E, 256), st);
  }
}

hipError_t launch_linear_stream(const MxArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.G, (unsigned)((a.T + 31) / 32));
  return launch_kernel(a.T <= 16 ? &mx8_stream_kernel<true> : &mx8_stream_kernel<false>, grid, dim3(512), 0, st, a);
}

}  // namespace

hipError_t launch_mx8_linear(const MxArgs& a, hipStream_t st) {
  const int64_t T = a.T;
  if (a.aux & kMxOutF32) {
    switch (linear_shape_exact(T, a.G)) {
      case kStream: return launch_linear_stream(a, st);
      case k64x64: return launch_tiled<kLinear, Mx8_64x64, true>(a, (T + 63) / 64, st);
      case k128x64: return launch_tiled<kLinear, Mx8_128x64, true>(a, (T + 63) / 64, st);
      default: return launch_tiled<kLinear, Mx8_256x64, true>(a, (T + 63) / 64, st);
    }
  }
  switch (linear_shape(T, a.G, a.KK)) {
    case kStream: return launch_linear_stream(a, st);
    case k64x64: return launch_tiled<kLinear, Mx8_64x64>(a, (T + 63) / 64, st);
    case k128x64: return launch_tiled<kLinear, Mx8_128x64>(a, (T + 63) / 64, st);
    case k256x64: return launch_tiled<kLinear, Mx8_256x64>(a, (T + 63) / 64, st);
    case k256x128: return launch_tiled<kLinear, Mx8_256x128>(a, (T + 127) / 128, st);
    default: return launch_tiled<kLinear, Mx8_256x256>(a, (T + 255) / 256, st);
  }
}

hipError_t launch_mx8_experts(const MxExperts& x, hipStream_t st) {
  if (hipError_t e = launch_experts_stage<kGateUp>(x.gate_up, x, st)) return e;
  return launch_experts_stage<kDown>(x.down, x, st);
}

}  // namespace moe
