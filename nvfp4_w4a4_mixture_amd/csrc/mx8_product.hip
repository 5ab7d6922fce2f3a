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
// Activations go in as two operands (see mx8_mfma).  HALF: at most 16 tokens, so
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
    acc = mx8_mfma<0, HALF>(d.w[0], xf[0], acc, d.sw, d.sx);
    acc = mx8_mfma<1, HALF>(d.w[1], xf[1], acc, d.sw, d.sx);
    acc = mx8_mfma<2, HALF>(d.w[2], xf[2], acc, d.sw, d.sx);
    acc = mx8_mfma<3, HALF>(d.w[3], xf[3], acc, d.sw, d.sx);
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
  const float4 s = add_waves<NW, HALF>(part, p, tok);
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
// register-only loop of these products: 3.9 PFLOP/s on data, 4.8 on zeros), it is
// multiplied twice (see mx8_mfma), and a token's stage takes twice the LDS, so
// tiles are taller: weight rows are the cheaper side, and a token's operand is
// parted once for all weight groups of a wave.  Waves of 128 x 64 read two thirds of
// the LDS bytes of 64 x 128 and leave registers to spare, where those spilled.  Rings
// of eight stages for the small tile were no faster, and neither were the reads of
// the next step before a step's products.
using Mx8_64x64 = MxTile<4, 2, 1, 1, 4, true>;
using Mx8_128x64 = MxTile<4, 2, 2, 1, 4, true>;
using Mx8_256x64 = MxTile<4, 4, 2, 2, 3, true>;
using Mx8_256x128 = MxTile<8, 4, 2, 2, 4, true>;
using Mx8_256x256 = MxTile<8, 2, 4, 2, 3, true>;

int64_t tiles(int64_t T, int64_t G, int64_t rows, int64_t tok) { return (G + rows / 32 - 1) / (rows / 32) * ((T + tok - 1) / tok); }

// Percentage of the products that are results, where tiles run one a CU in rounds of 256
int64_t useful(int64_t T, int64_t G, int64_t rows, int64_t tok) {
  return 100 * T * G * 32 / ((tiles(T, G, rows, tok) + 255) / 256 * 256 * rows * tok);
}

// The shape of a dense product, us (BF16 results; FP32 ones where they differ):
//   T x K x N             stream   64x64  128x64  256x64  256x128  256x256
//   1 x 6144 x 16384        12.8    17.7    20.8    23.6             35.4
//   1 x 6144 x 20480        16.4    24.5    21.1    23.6             35.4
//   8 x 6144 x 24576        18.4    24.9    21.5    24.0             36.0
//   1 x 4096 x 32768        17.1    18.7    16.3    18.1             26.9
//   1 x 6144 x 65536        40.6    45.0    35.5    32.9             39.2
//   1 x 6144 x 131072       92.9    97.6    80.1    76.6             85.8
//   16 x 6144 x 65536       43.7    45.6    38.1    32.9             40.6
//   16 x 6144 x 131072       122     104    83.4    78.0             86.2
//   32 x 6144 x 6144         8.3    17.0    20.4    23.5     22.0    35.4
//   32 x 6144 x 16384       16.9    18.6    22.0    24.2     23.4    35.6
//   24 x 6144 x 20480       22.2    25.0    21.5    24.2     22.7    35.8
//   64 x 6144 x 6144        14.1    18.5    21.0    38.0     36.1    60.2
//   64 x 6144 x 10240       22.5    19.5    21.6    38.7     36.8    60.8
//   64 x 6144 x 65536        120    64.1    46.5    51.8     45.8    68.3
//   64 x 6144 x 131072               169     118     102      105     138
//   128 x 6144 x 65536               129    87.8    80.9     74.6    76.3
//   256 x 6144 x 2048       14.8    18.9    21.4    38.3     56.3     103
//   256 x 6144 x 6144       42.4    28.9    23.5    39.7     56.6     104
//   509 x 6144 x 2048       29.6    20.7    22.6    39.2     56.4     104
//   512 x 6144 x 6144       83.2    43.5    41.3    44.6     61.3     105
//   1024 x 6144 x 6144       163    83.7    63.9    72.2     66.9     109
//   2048 x 2048 x 6144              56.5    49.6    46.3     53.6    47.8 (FP32 57.0)
//   2048 x 6144 x 6144               176     127     114      130     114 (FP32 123)
//   4096 x 6144 x 2048               125    86.4    79.5     73.1     114 (FP32 78.5 in 256x64 and 256x128)
//   4096 x 6144 x 6144               336     232     214      208     226 (FP32 218, 223, 243)
//   8192 x 512 x 4096                       40.2    37.5     40.4    37.0 (FP32 48.8, 63.8, 78.8)
//   8192 x 2048 x 6144                       187     164      162     142 (FP32 161, 182, 179)
//   8192 x 6144 x 6144                       485     417      403     362 (FP32 423, 425, 394)
// Streaming while its tiles of 32 x 32 fit the chip three times (up to 16 tokens,
// which take half the instructions) or twice; the smallest tile while its tiles fit
// it once.  Large tiles stand one a CU, so they need rounds that are nearly full of
// tiles, and tiles nearly full of tokens; short reductions and FP32 results (twice
// the epilogue, with nothing beside it) need two smaller tiles a CU instead.  Of
// those the taller one where they fit the chip twice over, or once if they hold at
// most 32 tokens: a wave then multiplies one group of two.
Shape linear_shape(int64_t T, int64_t G, int64_t KK, bool f32) {
  if (tiles(T, G, 32, 32) <= (T <= 16 ? 768 : 512)) return kStream;
  if (tiles(T, G, 64, 64) <= 256) return k64x64;
  const int64_t large = KK >= (f32 ? 16 : 4) ? useful(T, G, 256, 256) : 0, wide = KK >= 4 && !f32 ? useful(T, G, 256, 128) : 0;
  if (large >= (f32 ? 90 : 72) && 10 * large >= 9 * wide) return k256x256;
  if (wide >= 72) return k256x128;
  return tiles(T, G, 256, 64) >= (T <= 32 ? 256 : 512) ? k256x64 : k128x64;
}

// The shape of a stage of the experts' FFN, us of both stages with the other in 256x64:
//                             gate_up                      down
//   E k H I, tokens      128x64  256x64  256x256     128x64  256x64  256x256
//   80 8 6144 2048, 4       127     103      120       98.4     101      111
//   80 8 6144 2048, 16      191     188      223        191     187      209
//   80 8 6144 2048, 256     344     318      379        328     315      356
//   80 8 6144 2048, 2048   1148    1075     1147       1116    1078     1114
//   80 8 6144 2048, 8192   3988    3735     3653       3891    3741     3741
//   16 4 6144 2048, 64     73.0    83.7     91.1       69.5    70.1     85.5
//   16 4 6144 2048, 512     166     163      227        172     164      191
//   8 2 4096 1024, 512     41.4    44.2     86.4       43.4    44.6     52.4
//   8 2 4096 1024, 2048     105     112      113        112     108      124
//   8 2 4096 1024, 8192     346     333      357        346     331      354
//   16 4 1024 512, 256     15.0    18.3     27.4       16.2    18.0     23.1
//   16 4 1024 512, 8192     107     109      120        109     103      114
//   64 8 2048 768, 32      33.8    33.1     45.8       35.2    32.7     40.6
//   64 8 2048 768, 4096     289     263      277        283     260      275
// As above, by the number of tiles: the taller tile from some two and a half a CU on,
// or one a CU while experts have few pairs.  256x256 gains 2 to 3% in gate_up of the
// largest and loses elsewhere.
Shape experts_shape(int64_t pairs, int64_t E, int64_t rows) {
  const int64_t some = pairs < E ? pairs : E, n = (pairs / 64 + some / 2) * ((rows + 255) / 256);
  return n < (pairs <= 32 * E ? 256 : 600) ? k128x64 : k256x64;
}

template <int MODE>
hipError_t launch_experts_stage(const MxArgs& a, const MxExperts& x, hipStream_t st) {
  const int64_t pairs = x.T * x.k, most = most_mtiles(pairs, x.E, 64);
  if (experts_shape(pairs, x.E, a.N) == k128x64) return launch_tiled<MODE, Mx8_128x64>(a, most, st);
  return launch_tiled<MODE, Mx8_256x64>(a, most, st);
}

hipError_t launch_linear_stream(const MxArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.G, (unsigned)((a.T + 31) / 32));
  return launch_kernel(a.T <= 16 ? &mx8_stream_kernel<true> : &mx8_stream_kernel<false>, grid, dim3(512), 0, st, a);
}

}  // namespace

hipError_t launch_mx8_linear(const MxArgs& a, hipStream_t st) {
  const int64_t T = a.T;
  switch (linear_shape(T, a.G, a.KK, a.aux & kMxOutF32)) {
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
