// Products of MXFP8 activations: their shapes, by sizes.
#include "mx_product.h"

namespace moe {

namespace {

// An 8-bit operand takes the matrix cores twice as long as a 4-bit one (a
// register-only loop: 3.5 to 4 PFLOP/s by card on random bits), and a token's
// stage twice the LDS.
using Mx8_128x64 = MxTile<4, 2, 2, 1, 4, true>;
using Mx8_128x128 = MxTile<4, 2, 2, 2, 3, true>;
using Mx8_256x128 = MxTile<8, 4, 2, 2, 4, true>;
using Mx8_256x256 = MxTile<8, 2, 4, 2, 3, true>;

Shape linear_shape(int64_t T, int64_t G, int64_t KK) {
  const int64_t cus = 256;
  auto tiles = [&](int64_t rows, int64_t tok) { return (G + rows / 32 - 1) / (rows / 32) * ((T + tok - 1) / tok); };
  if (T <= 8 || (T <= 32 && T * G <= 32 * cus) || tiles(32, 32) <= cus) return kStream;
  if (KK >= 16 && tiles(256, 256) >= cus * 3 / 4) return k256x256;
  if (tiles(256, 128) >= cus * 3 / 4) return k256x128;
  if (tiles(128, 128) >= cus / 2) return k128x128;
  return k128x64;
}

Shape experts_shape(int64_t pairs, int64_t E, int64_t rows, int64_t KK) {
  if (pairs <= 16 * E && (pairs < E ? pairs : E) * (rows / 32) <= 2048) return kStream;
  const int64_t tiles = (pairs / 128 + (pairs < E ? pairs : E) / 2) * ((rows + 255) / 256);
  if (pairs <= 32 * E || tiles < 256) return k128x64;
  return pairs < 128 * E || KK < 16 ? k256x128 : k256x256;
}

template <int MODE>
hipError_t launch_experts_stage(const MxArgs& a, Shape s, const MxExperts& x, hipStream_t st) {
  const int64_t pairs = x.T * x.k;
  switch (s) {
    case kStream: return launch_stream<MODE, true>(a, x.E, st);
    case k128x64: return launch_tiled<MODE, Mx8_128x64>(a, most_mtiles(pairs, x.E, 64), st);
    case k256x256: return launch_tiled<MODE, Mx8_256x256>(a, most_mtiles(pairs, x.E, 256), st);
    default: return launch_tiled<MODE, Mx8_256x128>(a, most_mtiles(pairs, x.E, 128), st);
  }
}

template <bool EXACT>
hipError_t launch_linear(const MxArgs& a, hipStream_t st) {
  const int64_t T = a.T;
  switch (linear_shape(T, a.G, a.KK)) {
    case kStream:
      return T <= 16 ? launch_stream<kLinear, true, true>(a, 1, st) : launch_stream<kLinear, true>(a, 1, st);
    case k128x64: return launch_tiled<kLinear, Mx8_128x64, EXACT>(a, (T + 63) / 64, st);
    case k128x128: return launch_tiled<kLinear, Mx8_128x128, EXACT>(a, (T + 127) / 128, st);
    case k256x128: return launch_tiled<kLinear, Mx8_256x128, EXACT>(a, (T + 127) / 128, st);
    default: return launch_tiled<kLinear, Mx8_256x256, EXACT>(a, (T + 255) / 256, st);
  }
}

}  // namespace

hipError_t launch_mx8_linear(const MxArgs& a, hipStream_t st) {
  return (a.aux & kMxOutF32) ? launch_linear<true>(a, st) : launch_linear<false>(a, st);
}

hipError_t launch_mx8_experts(const MxExperts& x, hipStream_t st) {
  const int64_t pairs = x.T * x.k;
  const Shape s0 = experts_shape(pairs, x.E, x.gate_up.N, x.gate_up.KK), s1 = experts_shape(pairs, x.E, x.down.N, x.down.KK);
  if (hipError_t e = launch_experts_stage<kGateUp>(x.gate_up, s0, x, st)) return e;
  return launch_experts_stage<kDown>(x.down, s1, x, st);
}

}  // namespace moe
