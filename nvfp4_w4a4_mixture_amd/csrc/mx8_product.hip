// Products of MXFP8 activations: their shapes, by sizes.
#include "mx_product.h"

namespace moe {

namespace {

// An 8-bit operand takes the matrix cores twice as long as a 4-bit one (a
// register-only loop of these products: 3.9 PFLOP/s on data, 4.8 on zeros), and a
// token's stage twice the LDS, so tiles are taller: weight rows are the cheaper
// side.  256 x 256 runs at 2.9 PFLOP/s of its loop (90% of the zeros' rate on
// zeros: the rest is power); stages of one MFMA step instead of two, with a ring
// twice as long, ran at 2.3, for their 32-byte runs of a token.  Waves of 128 x 64
// read two thirds of the LDS bytes of 64 x 128 and leave registers to spare, where
// those spilled.  Rings of eight stages for the small tile were no faster.
using Mx8_128x64 = MxTile<4, 2, 2, 1, 4, true>;
using Mx8_256x64 = MxTile<4, 4, 2, 2, 3, true>;
using Mx8_256x128 = MxTile<8, 4, 2, 2, 4, true>;
using Mx8_256x256 = MxTile<8, 2, 4, 2, 3, true>;

int64_t tiles(int64_t T, int64_t G, int64_t rows, int64_t tok) { return (G + rows / 32 - 1) / (rows / 32) * ((T + tok - 1) / tok); }

// The shape of a dense product with 16-bit results, both sides in us:
//   T x K x N            stream  128x64  256x64  256x128  256x256
//   16 x 6144 x 6144       10.2    11.8    15.2     20.5     32.4
//   64 x 6144 x 6144       17.9    14.5    20.2     21.9     34.5
//   77 x 2080 x 1000        5.7     7.3    10.8     11.6     16.9
//   509 x 6144 x 2048      33.8    15.4    21.0     30.8     53.9
//   512 x 6144 x 6144      99.3    32.4    24.8     33.9     56.6
//   1024 x 6144 x 6144             51.7    43.0     37.2     66.0
//   2048 x 2048 x 6144             33.8    28.1     38.8     35.7
//   8192 x 512 x 4096              31.6    26.0     29.3     29.2
//   8192 x 2048 x 6144            146.8    99.0    103.0     94.8
//   8192 x 6144 x 6144            394.2   279.3    245.4    230.0
// Streaming while its tiles of 32 x 32 fit the chip once, or each CU fetches at
// most 32 rows of x a weight group; the largest tile that still fills the chip;
// 256 x 128 where its tiles fill it just once.
Shape linear_shape(int64_t T, int64_t G, int64_t KK) {
  const int64_t cus = 256;
  if (T <= 8 || (T <= 32 && T * G <= 32 * cus) || tiles(T, G, 32, 32) <= cus) return kStream;
  if (KK >= 8 && tiles(T, G, 256, 256) >= cus * 3 / 4) return k256x256;
  const int64_t n = tiles(T, G, 256, 128);
  if (n >= cus * 3 / 4 && n <= cus) return k256x128;
  return tiles(T, G, 256, 64) >= cus * 3 / 4 ? k256x64 : k128x64;
}

// FP32 results take two operands (see mx8_mfma), so the matrix cores bound them earlier:
//   T x K x N            stream  128x64  256x64  256x128  256x256
//   32 x 6144 x 10240      18.5    21.4    25.4     23.0     37.0
//   64 x 6144 x 6144       17.2    21.4    40.3     38.3     62.2
//   256 x 6144 x 6144      48.3    24.6    41.6     60.0    105.2
//   1024 x 6144 x 6144             63.8    69.9     74.1    115.6
//   2048 x 6144 x 6144            122.9   117.3    148.0    133.0
//   8192 x 2048 x 6144            185.1   169.5    198.4    191.6
//   8192 x 6144 x 6144            484.3   441.6    453.9    411.0
Shape linear_shape_exact(int64_t T, int64_t G) {
  if (T <= 32 || tiles(T, G, 32, 32) <= 512) return kStream;
  return tiles(T, G, 256, 64) >= 512 ? k256x64 : k128x64;
}

// The shape of a stage of the experts' FFN; both stages in one shape, us:
//   E k H I, tokens          stream  128x64  256x64  256x128  256x256
//   16 4 1024 512, 16           8.5     9.6    11.3     13.3     17.8
//   16 4 1024 512, 128         20.3    10.7    13.3     17.0     19.8
//   16 4 1024 512, 1024                20.3    19.1     19.4     28.0
//   16 4 1024 512, 8192                93.7    72.2     90.0     87.8
//   80 8 6144 2048, 16        168.3   165.1   157.7    171.6    199.4
//   80 8 6144 2048, 256       498.7   320.1   291.8    308.0    348.8
//   80 8 6144 2048, 1024              569.0   469.5    481.0    486.1
//   80 8 6144 2048, 2048              985.9   762.9    747.7    709.4
//   80 8 6144 2048, 8192               3227    2465     2358     2101
Shape experts_shape(int64_t pairs, int64_t E, int64_t rows, int64_t KK) {
  const int64_t some = pairs < E ? pairs : E;
  if (pairs <= 16 * E && some * (rows / 32) <= 2048) return kStream;
  if ((pairs / 64 + some / 2) * ((rows + 255) / 256) < 256) return k128x64;
  return pairs >= 160 * E && KK >= 8 ? k256x256 : k256x64;
}

template <int MODE>
hipError_t launch_experts_stage(const MxArgs& a, const MxExperts& x, hipStream_t st) {
  const int64_t pairs = x.T * x.k;
  switch (experts_shape(pairs, x.E, a.N, a.KK)) {
    case kStream: return launch_stream<MODE, true>(a, x.E, st);
    case k128x64: return launch_tiled<MODE, Mx8_128x64>(a, most_mtiles(pairs, x.E, 64), st);
    case k256x64: return launch_tiled<MODE, Mx8_256x64>(a, most_mtiles(pairs, x.E, 64), st);
    default: return launch_tiled<MODE, Mx8_256x256>(a, most_mtiles(pairs, x.E, 256), st);
  }
}

hipError_t launch_linear_stream(const MxArgs& a, hipStream_t st) {
  return a.T <= 16 ? launch_stream<kLinear, true, true>(a, 1, st) : launch_stream<kLinear, true>(a, 1, st);
}

}  // namespace

hipError_t launch_mx8_linear(const MxArgs& a, hipStream_t st) {
  const int64_t T = a.T;
  if (a.aux & kMxOutF32) {
    switch (linear_shape_exact(T, a.G)) {
      case kStream: return launch_linear_stream(a, st);
      case k128x64: return launch_tiled<kLinear, Mx8_128x64, true>(a, (T + 63) / 64, st);
      default: return launch_tiled<kLinear, Mx8_256x64, true>(a, (T + 63) / 64, st);
    }
  }
  switch (linear_shape(T, a.G, a.KK)) {
    case kStream: return launch_linear_stream(a, st);
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
