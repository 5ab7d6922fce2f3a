// Products of MXFP4 activations: the streaming kernel, and the shapes by sizes.
#include "mx_product.h"

namespace moe {

// Streaming product: few tokens per weight row, so the weights' bytes bound it.
// A workgroup takes R groups of 32 weight rows (gate_up: a gate group and the
// up group of the same h columns) and tiles of 32 tokens; its NW waves split
// the columns and load their fragments straight from memory to registers (a
// packed fragment is one contiguous kilobyte), and the partial sums meet in LDS
// in a fixed order.  One token, 6144 x 6144: 4.6 to 5.2 us, of which a launch
// takes about 2; 8 waves on 1 row group where 4 waves on 2 take 10.4 (too few
// workgroups), 16 waves or loads two groups ahead as many.  Token groups past
// the first would cost more here than in a tile: a lane's 16 bytes of x come
// from 32 different rows.
template <int MODE, int R, int NW>
__global__ __launch_bounds__(NW * 64) void mx_stream_kernel(MxArgs a) {
  __shared__ float4 part[NW][R][4 * 68];  // strides 68 and 34: 16 lanes of a reader take 16 different slots
  __shared__ uint32_t hmax[NW][32];
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int e = MODE == kLinear ? 0 : blockIdx.y;
  const int KK = (int)a.KK;
  int64_t lo = 0, hi = a.T;
  if (MODE != kLinear) {
    lo = a.offsets[e];
    hi = a.offsets[e + 1];
  }
  const uint8_t* wc[R];
  const uint8_t* ws[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int g = MODE == kGateUp ? (int)blockIdx.x + i * (a.G / 2) : min((int)blockIdx.x * R + i, a.G - 1);
    wc[i] = a.w_codes + ((int64_t)e * a.G + g) * a.KK * kMxFragCodes;
    ws[i] = a.w_scales + ((int64_t)e * a.G + g) * a.KK * kMxFragScales;
  }

  for (int64_t t0 = lo + (MODE == kLinear ? (int64_t)blockIdx.y * 32 : 0); t0 < hi; t0 += 32) {
    const int cnt = (int)min((int64_t)32, hi - t0);
    const int64_t pos = t0 + min(n, cnt - 1);  // lanes past the last token repeat it
    const int64_t arow = MODE == kGateUp ? a.sorted[pos] / a.aux : pos;
    const uint8_t* xc = a.a_codes + arow * (a.KK * 128) + f * 64;
    const uint8_t* xs = a.a_scales + arow * (a.KK * 8) + f * 4;
    // thread (tok, p) of the epilogue: features 4 p .. 4 p + 3 of one token; what it needs of the pair
    // is loaded here, under the products (two latencies less: down of a small layer 4.7 us, not 5.7)
    const int tok = tid >> 3, p = tid & 7;
    int pair = 0, wmax = 0;
    float wp = 0.0f;
    if constexpr (MODE == kDown) {
      pair = a.sorted[t0 + min(tok, cnt - 1)];
      wp = a.topk_w[pair];
      wmax = a.w_max[e];
    }
    float16_t acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
    uint32_t bh = 0;
    for (int64_t c = w; c < KK; c += NW) {
      i32x4_t wf[R][4], xf[4];
      int sw[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int s = 0; s < 4; ++s) wf[i][s] = reinterpret_cast<const i32x4_t*>(wc[i] + c * kMxFragCodes)[s * 64 + l];
        sw[i] = reinterpret_cast<const int*>(ws[i] + c * kMxFragScales)[l];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) xf[s] = reinterpret_cast<const i32x4_t*>(xc + c * 128)[s];
      const int sx = *reinterpret_cast<const int*>(xs + c * 8);
      if (MODE == kDown) bh = max(bh, max_byte((uint32_t)sx));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        acc[i] = mx_mfma<0>(wf[i][0], xf[0], acc[i], sw[i], sx);
        acc[i] = mx_mfma<1>(wf[i][1], xf[1], acc[i], sw[i], sx);
        acc[i] = mx_mfma<2>(wf[i][2], xf[2], acc[i], sw[i], sx);
        acc[i] = mx_mfma<3>(wf[i][3], xf[3], acc[i], sw[i], sx);
      }
    }
    if (MODE == kDown) {
      bh = max(bh, (uint32_t)__shfl_xor((int)bh, 32));
      if (f == 0) hmax[w][n] = bh;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part[w][i][q * 68 + f * 34 + n] = make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
    __syncthreads();
    if (tid < 256 && tok < cnt) {
      float v[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float4 s = part[0][i][(p & 3) * 68 + (p >> 2) * 34 + tok];
#pragma unroll
        for (int k = 1; k < NW; ++k) {
          const float4 u = part[k][i][(p & 3) * 68 + (p >> 2) * 34 + tok];
          s.x += u.x;
          s.y += u.y;
          s.z += u.z;
          s.w += u.w;
        }
        v[i][0] = s.x;
        v[i][1] = s.y;
        v[i][2] = s.z;
        v[i][3] = s.w;
      }
      const int64_t row = t0 + tok;
      if constexpr (MODE == kGateUp) {
        float h[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[q] = silu(v[0][q]) * v[1][q];
          m = max(m, abs_bits(h[q]));
        }
        m = quad_max(m);
        m = max(m, lane_dpp<kLaneHalfMirror>(m));
        const uint32_t byte = mx_scale_byte(m);
        const int64_t blk = blockIdx.x;
        reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.out) + row * a.ldo)[blk * 8 + p] = (uint16_t)mx_encode8(h, byte);
        if (p == 0) static_cast<uint8_t*>(a.out_scales)[row * (a.ldo / 16) + blk] = (uint8_t)byte;
        if (blk == 0) zero_h_pad<false>(a, row, p, 8);
      } else {
        float factor = 1.0f;
        int64_t out = row;
        if constexpr (MODE == kDown) {
          out = pair;
          uint32_t b = hmax[0][tok];
#pragma unroll
          for (int k = 1; k < NW; ++k) b = max(b, hmax[k][tok]);
          if (wmax == 255) wmax = finite_scale_max<8>(a, e, p);  // by the whole wave under the products: 0.2 us more
          const int E = pair_exponent(wp, b, wmax, a.aux);
          factor = wp * __uint_as_float((uint32_t)(127 - E) << 23);  // exact
          if (blockIdx.x == 0 && p == 0) static_cast<float*>(a.out_scales)[out] = __uint_as_float((uint32_t)(127 + E) << 23);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int col = ((int)blockIdx.x * R + i) * 32 + 4 * p;
          if (MODE == kDown) {  // N % 32 == 0 and the rows are aligned
            if (col < a.N)
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out * a.ldo + col) =
                  make_uint2(f16_pair(factor * v[i][0], factor * v[i][1]), f16_pair(factor * v[i][2], factor * v[i][3]));
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (col + q >= a.N) break;
              if (a.aux & kMxOutF32) static_cast<float*>(a.out)[out * a.ldo + col + q] = v[i][q];
              else static_cast<uint16_t*>(a.out)[out * a.ldo + col + q] = (uint16_t)bf16_pair(v[i][q], 0.0f);
            }
          }
        }
      }
    }
    if (MODE == kLinear) break;
    __syncthreads();
  }
}

namespace {

template <int MODE>
hipError_t launch_stream(const MxArgs& a, int64_t E, hipStream_t st) {
  if constexpr (MODE == kLinear)
    return launch_kernel(mx_stream_kernel<MODE, 1, 8>, dim3((unsigned)a.G, (unsigned)((a.T + 31) / 32)), dim3(512), 0, st,
                         a);
  else
    return launch_kernel(mx_stream_kernel<MODE, 2, 4>, dim3((unsigned)((a.G + 1) / 2), (unsigned)E), dim3(256), 0, st, a);
}

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
    case kStream: return launch_stream<MODE>(a, x.E, st);
    case k128x64: return launch_tiled<MODE, Mx128x64>(a, mtiles, st);
    case k256x256: return launch_tiled<MODE, Mx256x256>(a, mtiles, st);
    default: return launch_tiled<MODE, Mx256x128>(a, mtiles, st);
  }
}

}  // namespace

hipError_t launch_mx_linear(const MxArgs& a, hipStream_t st) {
  const int64_t T = a.T;
  switch (linear_shape(T, a.G, a.KK)) {
    case kStream: return launch_stream<kLinear>(a, 1, st);
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
