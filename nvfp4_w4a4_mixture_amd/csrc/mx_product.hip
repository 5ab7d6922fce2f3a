// Products of MXFP4 activations: their shapes, by sizes.
#include "mx_product.h"

namespace moe {

namespace {

// Weight rows by tokens.  The small tiles serve few tokens per expert, whose
// bound is the weight stream, and grids too small for the large ones: at 256 x
// 6144 x 6144 128 x 64 takes 11.8 us, 128 x 128 13.7 and 256 x 256 30; at 512
// tokens 22, 17 and 33.  256 x 128 (78 KB of LDS, two workgroups a CU) hides
// its epilogue and suits short reductions: 62 us at 8192 x 2048 x 6144, where
// 256 x 256 takes 65.  256 x 256 moves two thirds of its bytes per product: 154
// against 161 us at 8192 x 6144 x 6144.  Its eight waves of 64 x 128 measured
// the same as four of 128 x 128.
using Mx128x64 = MxTile<4, 2, 2, 1, 4>;
using Mx128x128 = MxTile<4, 2, 2, 2, 4>;
using Mx256x128 = MxTile<4, 2, 4, 2, 3>;
using Mx256x256 = MxTile<8, 4, 2, 4, 4>;

int shape_tokens(Shape s) { return s == k128x64 ? Mx128x64::kTok : s == k256x256 ? Mx256x256::kTok : Mx256x128::kTok; }

// The shape of a dense product.  The streaming kernel spreads over all CUs at
// any size, but a lane's pieces of x come from as many rows as there are tokens:
// at K = 6144 and 50,000 weight rows 1, 8, 16 and 32 tokens take 25, 26, 29 and
// 43 us, where a 128 x 64 tile takes 26 for up to 64; at 6144 rows (192 groups)
// they take 4.0 to 6.6 us and the tile, latency bound, 10.  They meet near tokens
// times groups of 32 * 256, each CU having 32 rows of x a group to fetch: on the two
// sides of it 32 tokens take 7.2 (streamed) and 9.6 us (tile), 16 take 10.4 and
// 11.1, 9 take 16.9 and 15.8; at 32 x 10,240 13.2 and 9.9.  Of the tiles the
// largest that still come to about one for each CU: fewer bytes a product; 256 x
// 256, with one workgroup a CU, from 4096 columns on, where its epilogue weighs
// less than what it saves: 4096 x K x 8192 takes 24.4 (K = 512), 47.6 (2048) and 69.0
// us (3584), by 256 x 128 21.6, 45.1 and 68.5; 8192 x K x 6144 110 and 154 us (K
// = 4096, 6144), by 256 x 128 111 and 161.
Shape linear_shape(int64_t T, int64_t G, int64_t KK) {
  const int64_t cus = 256;
  auto tiles = [&](int64_t rows, int64_t tok) { return (G + rows / 32 - 1) / (rows / 32) * ((T + tok - 1) / tok); };
  if (T <= 8 || (T <= 32 && T * G <= 32 * cus) || tiles(32, 32) <= cus) return kStream;
  if (KK >= 16 && tiles(256, 256) >= cus * 3 / 4) return k256x256;
  if (tiles(256, 128) >= cus * 3 / 4) return k256x128;
  if (tiles(128, 128) >= cus / 2) return k128x128;
  return k128x64;
}

// The shape of a stage of the experts' FFN over weights of `rows` rows; both
// sides measured on 80 experts of 6144 x 2048, top-8, us of gate_up (down):
//   mean pairs an expert      1.6        32         64         128        256        819
//   streaming             163 (87)   288 (144)  462 (222)
//   128 x 64              148 (75)   183 (101)  268 (121)  366 (182)  610 (312)
//   256 x 128             158 (79)   179 (101)  195 (109)  275 (146)  387 (218)  983 (597)
//   256 x 256             169 (93)   188 (112)  200 (121)  242 (148)  402 (243)  920 (632)
//   weights read          137 (69)   168 (84) from 32 on; operations 446 (223) at 819
// Small layers (16 experts of 1024 x 512) are latency bound: streaming takes
// 4.0 us at 16 pairs an expert where 128 x 64 takes 4.4; past that its second
// token tile costs more (10 experts of 4992 x 896, 29 pairs each: 20.0 against
// 11.5 us), and 128 x 64 stays ahead of 256 x 128 (6.4 against 8.9 us at 128)
// until the larger tiles fill the chip.
Shape experts_shape(int64_t pairs, int64_t E, int64_t rows, int64_t KK) {
  if (pairs <= 16 * E && (pairs < E ? pairs : E) * (rows / 32) <= 2048) return kStream;
  const int64_t tiles = (pairs / 128 + (pairs < E ? pairs : E) / 2) * ((rows + 255) / 256);
  if (pairs <= 32 * E || tiles < 256) return k128x64;
  return pairs < 128 * E || KK < 16 ? k256x128 : k256x256;
}

template <int MODE>
hipError_t launch_experts_stage(const MxArgs& a, Shape s, const MxExperts& x, hipStream_t st) {
  const int64_t mtiles = most_mtiles(x.T * x.k, x.E, shape_tokens(s));
  switch (s) {
    case kStream: return launch_stream<MODE, false>(a, x.E, st);
    case k128x64: return launch_tiled<MODE, Mx128x64>(a, mtiles, st);
    case k256x256: return launch_tiled<MODE, Mx256x256>(a, mtiles, st);
    default: return launch_tiled<MODE, Mx256x128>(a, mtiles, st);
  }
}

}  // namespace

hipError_t launch_mx_linear(const MxArgs& a, hipStream_t st) {
  const int64_t T = a.T;
  switch (linear_shape(T, a.G, a.KK)) {
    case kStream: return launch_stream<kLinear, false>(a, 1, st);
    case k128x64: return launch_tiled<kLinear, Mx128x64>(a, (T + 63) / 64, st);
    case k128x128: return launch_tiled<kLinear, Mx128x128>(a, (T + 127) / 128, st);
    case k256x128: return launch_tiled<kLinear, Mx256x128>(a, (T + 127) / 128, st);
    default: return launch_tiled<kLinear, Mx256x256>(a, (T + 255) / 256, st);
  }
}

hipError_t launch_mx_experts(const MxExperts& x, hipStream_t st) {
  const int64_t pairs = x.T * x.k;
  const Shape s0 = experts_shape(pairs, x.E, x.gate_up.N, x.gate_up.KK), s1 = experts_shape(pairs, x.E, x.down.N, x.down.KK);
  if (hipError_t e = launch_experts_stage<kGateUp>(x.gate_up, s0, x, st)) return e;
  return launch_experts_stage<kDown>(x.down, s1, x, st);
}

}  // namespace moe
