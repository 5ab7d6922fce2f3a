// Products of quantised activations and packed MXFP4 weights on the scaled
// MFMA: the dense y = x W^T, and the two stages of the routed experts' FFN.
//
// With few tokens the weights' bytes bound a product, with many the matrix
// cores.  A register-only loop of the 32x32x64 FP4 MFMA takes 32 cycles an
// instruction; on operands of random bits the card lowers its clock to some 1.6
// GHz under it (6.4 to 6.6 PFLOP/s by card; 9.8 on zeros).  The tiled kernel on
// 4096 x 16384 x 4096 reaches 4.6 PFLOP/s, 5.2 without its DMA, and 6.2 on zeros:
// in such long reductions what remains is mostly power, and a shape that moves
// fewer bytes per product wins over one that hides latencies better.  Short ones
// (the down stage's eight column groups) fill their ring and empty it for little.
//
// Activations are MXFP4, or MXFP8 (A8) under the same packed weights; then the
// FFN's h is MXFP8 too, and the dense product has an epilogue (bias, activation,
// residual).  Each format is instantiated by a source of its own, with the rules
// that choose its shapes.
#pragma once

#include "launch.h"
#include "mx_common.h"

namespace moe {

namespace {

template <int V>
struct Const {
  static constexpr int value = V;
};

enum { kLinear = 0, kGateUp = 1, kDown = 2 };

// Scale of a pair row: an exponent E with |w_p f| < 2^(E + 15) for every
// operand.  |f| <= I * 6^2 * 2^(bh - 127) * 2^(bw - 127) for the largest scale
// byte bh of the h row and bw of the expert's down weights, 36 I <= 2^lg, and
// |w_p| < 2^(ew + 1).  FP16's normal range reaches 29 binades below 2^15, so a
// loose bound costs no precision.  Clamped so that 2^E, 2^-E and w_p 2^-E are
// normal or zero (a row of zeros has a bound far below its weight).  FP16 and not
// FP32 because the rows are what the layer writes most of (805 MB for 8192 tokens
// of 8 x 6144) and its combine reads again; it rounds a row by 2.1e-4 in the
// 2-norm, which takes one BF16 result in some thirty to its neighbour.
__device__ __forceinline__ int pair_exponent(float wp, uint32_t bh, int bw, int lg) {
  const int ew = (int)((__float_as_uint(wp) >> 23) & 255u) - 127;
  const int e = ew + 1 + lg + (int)bh + bw - 254 - 15;
  return min(max(e, max(ew, 0) - 126), 113);
}

// bw for an expert whose weights hold NaN blocks, so that its largest byte is
// 255 and says nothing: the largest of its other scale bytes, which bounds the
// features that those blocks do not reach.  N lanes (8 or 64, in a row) read
// the expert's scales; weights without NaN never come here.
template <int N>
__device__ __forceinline__ int finite_scale_max(const MxArgs& a, int e, int lane) {
  const int64_t bytes = (int64_t)a.G * a.KK * kMxFragScales;
  const uint8_t* scales = a.w_scales + e * bytes;
  uint32_t m = 0;
  for (int64_t i = 4 * lane; i < bytes; i += 4 * N) {
    const uint32_t d = *reinterpret_cast<const uint32_t*>(scales + i);
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
      const uint32_t b = (d >> k) & 255u;
      m = b == 255u ? m : max(m, b);
    }
  }
  m = quad_max(m);
  m = max(m, lane_dpp<kLaneHalfMirror>(m));
#pragma unroll
  for (int x = 8; x < N; x *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, x));
  return (int)m;
}

// Two values rounded to nearest even in FP16, the first in the low half
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
}

__device__ __forceinline__ uint32_t max_byte(uint32_t d) {
  return max(max(d & 255u, (d >> 8) & 255u), max((d >> 16) & 255u, d >> 24));
}

// The blocks of h row `row` past I, up to its padded width, are zero; thread `p` of `n` takes every n-th.
template <bool A8>
__device__ __forceinline__ void zero_h_pad(const MxArgs& a, int64_t row, int p, int n) {
  constexpr int kBytes = A8 ? 32 : 16;  // of a block
  for (int b = a.G / 2 + p; b < a.ldo / kBytes; b += n) {
    uint4* c = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row * a.ldo + b * kBytes);
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) c[i] = make_uint4(0, 0, 0, 0);
    static_cast<uint8_t*>(a.out_scales)[row * (a.ldo / kBytes) + b] = 0;
  }
}

// An activation operand of one MFMA step, and the step on it.
template <bool A8>
struct ActFrag {
  typedef i32x4_t type;
};
template <>
struct ActFrag<true> {
  typedef i32x8_t type;
};
template <int S>
__device__ __forceinline__ float16_t act_mfma(i32x4_t w, const i32x4_t& x, float16_t c, int sw, int sx) {
  return mx_mfma<S>(w, x, c, sw, sx);
}
template <int S>
__device__ __forceinline__ float16_t act_mfma(i32x4_t w, const i32x8_t& x, float16_t c, int sw, int sx) {
  return mx8_mfma<S, false>(w, x, c, sw, sx);
}
// Sums that a tile's waves exchange through LDS: wave w's of features 4 p .. 4 p + 3 of
// column n are the float4 at w * STRIDE + (p & 3) * 68 + (p >> 2) * 34 + n.  Adds them over
// NW waves in order; HALF: and over the columns tok and tok + 16.  tok < 32, or 16.
constexpr int kWaveSums = 4 * 68;
template <int NW, bool HALF, int STRIDE = kWaveSums>
__device__ __forceinline__ float4 add_waves(const float4* part, int p, int tok) {
  static_assert(3 * 68 + 34 + 31 < kWaveSums, "the last column of the last features is the wave's own");
  const float4* own = part + (p & 3) * 68 + (p >> 2) * 34 + tok;
  float4 s = own[0];
#pragma unroll
  for (int k = 1; k < (HALF ? 2 : 1) * NW; ++k) {
    const float4 u = own[k % NW * STRIDE + (k < NW ? 0 : 16)];
    s.x += u.x;
    s.y += u.y;
    s.z += u.z;
    s.w += u.w;
  }
  return s;
}
__device__ __forceinline__ i32x8_t join_halves(i32x4_t a, i32x4_t b) {
  return i32x8_t{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// ---- the dense product's epilogue: act(z + bias) + residual, in FP32

// GELU by erf, z Phi(z), from the normal distribution's tail Phi(-a), a = |z|, so that
// nothing cancels: -a Phi(-a) for negative z, z - a Phi(-a) else.  Hastings' form (1955)
// of the tail, e^(-a^2/2) t P(t) with t = 1 / (1 + q a); P of degree 8 and q fitted for
// the least relative error on 0 <= a <= 16, 2.7e-8.  The exponent is formed in two
// parts, as its rounding alone would be 1e-5 of the result at a = 12.  At most 16 * 2^-24 of
// the result, 5 over all BF16 arguments.  By the library's erfc 8192 x 512 x 4096 took 78 us, so
// 61, by 0.5 z (1 + erf), which loses a result of -5 to 4%, 60.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 16.0f), t = __builtin_amdgcn_rcpf(fmaf(a, 0.3479999899864197f, 1.0f));
  float p = -0.028869353234767914f;
  p = fmaf(p, t, 0.1446346640586853f);
  p = fmaf(p, t, -0.2620934247970581f);
  p = fmaf(p, t, 0.1703842133283615f);
  p = fmaf(p, t, -0.028765540570020676f);
  p = fmaf(p, t, 0.10794074088335037f);
  p = fmaf(p, t, 0.11882702261209488f);
  p = fmaf(p, t, 0.13912083208560944f);
  p = fmaf(p, t, 0.1388208419084549f);
  constexpr float kHigh = -0.7213475108146667f, kLow = -9.629815167500055e-09f;  // -log2(e) / 2
  const float s = a * a, e = s * kHigh, rest = fmaf(fmaf(a, a, -s), kHigh, fmaf(s, kLow, fmaf(s, kHigh, -e)));
  const float x = __builtin_amdgcn_exp2f(e), tail = t * p * fmaf(x * 0.69314718055994531f, rest, x);
  return fmaf(-a, tail, z < 0.0f ? 0.0f : z);  // past 16 the tail is 0; NaN stays
}
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;  // NaN stays
    case kActSilu: return silu(z);
    case kActGelu: return gelu(z);
    case kActGeluTanh: {  // 0.5 (1 + tanh(u)) = 1 / (1 + e^-2u)
      const float u = 0.79788456080286536f * fmaf(0.044715f * z * z, z, z);
      return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-2.88539008177792681f * u));
    }
    default: return z;
  }
}

// One element, of row `row` and column `col`
__device__ __forceinline__ float epilogue1(const MxArgs& a, float z, int64_t row, int col) {
  if (a.bias) z += bf16_to_f32(a.bias[col]);
  z = activate(a.aux >> kMxActShift, z);
  if (a.residual) {
    const int64_t at = row * a.ldr + col;
    z += (a.aux & kMxResF32) ? static_cast<const float*>(a.residual)[at]
                             : bf16_to_f32(static_cast<const uint16_t*>(a.residual)[at]);
  }
  return z;
}

// 16 bytes at an address aligned to an element only (one access on gfx950 all the same)
typedef uint32_t mx_u32x4_any2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef float mx_float4_any4_t __attribute__((ext_vector_type(4), aligned(4)));

// Eight values of BF16 (FP32) elements from p on, of which n are there
__device__ __forceinline__ void epilogue_load8(const uint16_t* p, int n, float* v) {
  if (n >= 8) {
    const mx_u32x4_any2_t u = *reinterpret_cast<const mx_u32x4_any2_t*>(p);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[2 * r] = bf16_to_f32(u[r] & 0xFFFFu);
      v[2 * r + 1] = __uint_as_float(u[r] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = r < n ? bf16_to_f32(p[r]) : 0.0f;
  }
}
__device__ __forceinline__ void epilogue_load8(const float* p, int n, float* v) {
  if (n >= 8) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const mx_float4_any4_t u = *reinterpret_cast<const mx_float4_any4_t*>(p + 4 * q);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * q + r] = u[r];
    }
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = r < n ? p[r] : 0.0f;
  }
}
__device__ __forceinline__ void epilogue_residual8(const MxArgs& a, int64_t row, int col, float* v) {
  const int64_t at = row * a.ldr + col;
  if (a.aux & kMxResF32) epilogue_load8(static_cast<const float*>(a.residual) + at, a.N - col, v);
  else epilogue_load8(static_cast<const uint16_t*>(a.residual) + at, a.N - col, v);
}
// Columns col .. col + 7 of row `row`, those that there are
__device__ __forceinline__ void epilogue_store8(const MxArgs& a, int64_t row, int col, const float* v) {
  const int64_t at = row * a.ldo + col;
  if (a.aux & kMxOutF32) {
    float* p = static_cast<float*>(a.out) + at;
    if (col + 8 <= a.N) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const mx_float4_any4_t u = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        __builtin_nontemporal_store(u, reinterpret_cast<mx_float4_any4_t*>(p + 4 * q));  // see store16_streaming
      }
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (col + r < a.N) p[r] = v[r];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(a.out) + at;
    const mx_u32x4_any2_t u = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    if (col + 8 <= a.N) {
      __builtin_nontemporal_store(u, reinterpret_cast<mx_u32x4_any2_t*>(p));
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (col + r < a.N) p[r] = (uint16_t)(u[r >> 1] >> (16 * (r & 1)));
    }
  }
}

}  // namespace

// Tiled product: four waves share a tile of kSlots * 32 weight rows by kTok
// tokens through LDS.  A stage is half a column group (128 columns, two MFMA
// steps); a ring of four stages is filled by global -> LDS DMA three stages
// ahead.  Weights arrive in fragment order, so a wave reads them back as they
// lie.  A token's 64 bytes of a stage are four 16-byte chunks, stored exchanged
// by mx_swizzle(row), so that the lanes of one LDS cycle touch all banks (8-bit
// activations: 128 bytes, eight chunks, mx8_swizzle).
// Scale dwords (a whole column group's) come by DMA too: the loop then has no
// load that the compiler would wait for, and every wait is one written here.
//
// Wave (wm, wx) of WM x (4 / WM) holds GW weight groups by GX token groups of
// 32 in accumulators.  The fragments of the next MFMA step are read while the
// current one multiplies; the barrier that hands over a stage stands between
// its two steps, so that the second covers the first reads of the next stage.
template <int NW, int WM, int GW_, int GX_, int RING_, bool A8_ = false>
struct MxTile {
  static constexpr bool kA8 = A8_;
  static constexpr int kXRow = A8_ ? 128 : 64;  // bytes of a token's stage
  static constexpr int kWM = WM, GW = GW_, GX = GX_;
  static constexpr int kWX = NW / WM;
  static constexpr int kSlots = WM * GW;       // weight groups of a tile
  static constexpr int kTok = kWX * GX * 32;   // tokens of a tile
  static constexpr int kWaves = NW;
  static constexpr int kRing = RING_;
  static constexpr int kWBytes = kSlots * 2048;
  static constexpr int kStage = kWBytes + kTok * kXRow;
  static constexpr int kUnits = kSlots + kTok / 32;  // scale dwords: 256 bytes a group of 32 rows
  static constexpr int kLds = kRing * kStage + 2 * kUnits * 256;
  // epilogue: a row of 16-bit results in LDS, offset by 16 bytes against bank conflicts; then the output rows
  static constexpr int kOutRow = kSlots * 64 + 16;
  static_assert(kTok * (kOutRow + 4) <= kLds, "the epilogue's tile fits the ring");
  // DMA instructions per wave: weights and tokens of a stage, scales of a column group
  static constexpr int kWDma = 2 * kSlots / NW, kXDma = kTok * kXRow / 1024 / NW, kSDma = (kUnits + NW - 1) / NW;
};

// Exchange of the four chunks of LDS row r (64 bytes): distinct for the rows that share a bank
// group, both over 8 rows (128 bytes a cycle) and over 16.
__device__ __forceinline__ int mx_swizzle(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }
// The same for the eight chunks of a row of 128 bytes
__device__ __forceinline__ int mx8_swizzle(int r) { return ((r >> 1) & 7) ^ ((r & 1) << 2); }

// The m-tiles of up to 256 experts, TOK pairs each, found by every wave for
// itself: lane l counts those of experts 4 l .. 4 l + 3, and a scan gives each
// lane's first.  It costs a tile 0.3 us (10 us of the 1.6 ms of 8192 tokens, 80
// experts, top-8) and saves a launch of 3 us before the first stage.  One m-tile
// an expert without the scan, for so few tokens that an expert's pairs fit one,
// was no faster: 16 tokens of that layer took 185 us against 179, 2 took 52
// against 50, 64 249 against 239, 8 the same.
template <int TOK>
struct ExpertTiles {
  int off[5], end;  // the lane's offsets; tiles up to the end of its experts
  __device__ __forceinline__ int tiles(int i) const { return (off[i + 1] - off[i] + TOK - 1) / TOK; }
  __device__ __forceinline__ void count(const int32_t* offsets, int E, int l) {
#pragma unroll
    for (int i = 0; i < 5; ++i) off[i] = offsets[min(4 * l + i, E)];
    end = tiles(0) + tiles(1) + tiles(2) + tiles(3);
    // within rows of 16 lanes, then the last lanes' sums on to the rows after them
    end += __builtin_amdgcn_update_dpp(0, end, 0x111, 0xF, 0xF, false);  // from 1 lane before
    end += __builtin_amdgcn_update_dpp(0, end, 0x112, 0xF, 0xF, false);  // 2
    end += __builtin_amdgcn_update_dpp(0, end, 0x114, 0xF, 0xF, false);  // 4
    end += __builtin_amdgcn_update_dpp(0, end, 0x118, 0xF, 0xF, false);  // 8
    end += __builtin_amdgcn_update_dpp(0, end, 0x142, 0xA, 0xF, false);  // lane 15 of row 0 (2) to row 1 (3)
    end += __builtin_amdgcn_update_dpp(0, end, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  }
  __device__ __forceinline__ int total() const { return __builtin_amdgcn_readlane(end, 63); }
  // {expert, its first m-tile, its first pair, its pairs} of m-tile m < total()
  __device__ __forceinline__ int4 find(int m) const {
    const int lane = __builtin_ctzll(__ballot(end > m));
    int o[5], n[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) o[i] = __builtin_amdgcn_readlane(off[i], lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = (o[i + 1] - o[i] + TOK - 1) / TOK;
    int y = __builtin_amdgcn_readlane(end, lane) - n[0] - n[1] - n[2] - n[3], i = 0, lo = o[0], hi = o[1];
#pragma unroll
    for (int k = 1; k < 4; ++k)
      if (m >= y + n[k - 1] && i == k - 1) {
        y += n[k - 1];
        i = k;
        lo = o[k];
        hi = o[k + 1];
      }
    return make_int4(4 * lane + i, y, lo, hi - lo);
  }
};

template <int MODE, class S>
__global__ __launch_bounds__(S::kWaves * 64, 2) void mx_tiled_kernel(MxArgs a) {
  constexpr bool A8 = S::kA8;
  constexpr int kGroup = A8 ? 256 : 128;  // bytes of a column group of an activation row
  constexpr int NW = S::kWaves, WM = S::kWM, GW = S::GW, GX = S::GX, RING = S::kRing;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, l = tid & 63, n = l & 31, f = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w % WM, wx = w / WM;

  // ---- which tile: each XCD takes one contiguous run of the tile order (under 2^24 tiles)
  const int nw = MODE == kGateUp ? (a.G / 2 + S::kSlots / 2 - 1) / (S::kSlots / 2) : (a.G + S::kSlots - 1) / S::kSlots;
  ExpertTiles<S::kTok> experts;
  if (MODE != kLinear) experts.count(a.offsets, a.E, l);
  const int mtiles = MODE == kLinear ? (a.T + S::kTok - 1) / S::kTok : experts.total();
  const int total = mtiles * nw, chunk = (total + 7) / 8, slot = blockIdx.x >> 3;
  const int at = (int)(blockIdx.x & 7) * chunk + slot;
  if (slot >= chunk || at >= total) return;
  int e = 0, rows = a.T, span = mtiles, q = at;
  int64_t first = 0;
  if (MODE != kLinear) {
    const int4 t = experts.find(at / nw);
    e = t.x;
    q = at - t.y * nw;
    first = t.z;
    rows = t.w;
    span = (rows + S::kTok - 1) / S::kTok;
  }
  // blocks of up to four token tiles by all weight tiles, tokens fastest
  const int blk = q / (4 * nw), rem = q - blk * 4 * nw, tc = min(4, span - 4 * blk), wt = rem / tc;
  const int t0 = (4 * blk + rem - wt * tc) * S::kTok, cnt = min(S::kTok, rows - t0);
  first += t0;

  // weight group of slot s (of kSlots)
  auto group = [&](int s) -> int {
    if (MODE == kGateUp) {  // a wave holds gate groups and the up groups of the same h columns
      const int half = a.G / 2, hb = wt * (S::kSlots / 2) + (s / GW) * (GW / 2) + s % (GW / 2);
      return min(hb, half - 1) + (s % GW >= GW / 2 ? half : 0);
    }
    return min(wt * S::kSlots + s, a.G - 1);
  };

  auto act_row = [&](int t) -> int64_t {  // activation row of the tile's token t (rows past the end repeat the last)
    const int64_t pos = first + min(t, cnt - 1);
    return MODE == kGateUp ? a.sorted[pos] / a.aux : pos;
  };

  // ---- DMA sources: this wave's share of the weight pieces, token rows and scales
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  const uint8_t* wsrc[S::kWDma];
  uint32_t xoff[S::kXDma];
  const uint8_t* ssrc[S::kSDma];
  uint32_t soff[S::kSDma], sstep[S::kSDma];
#pragma unroll
  for (int i = 0; i < S::kWDma; ++i) {
    const int piece = w * S::kWDma + i;  // (slot, piece of the stage)
    wsrc[i] = a.w_codes + ((int64_t)e * a.G + group(piece >> 1)) * a.KK * kMxFragCodes + (piece & 1) * 1024;
  }
#pragma unroll
  for (int i = 0; i < S::kXDma; ++i) {
    if constexpr (A8) {
      const int r = (w * S::kXDma + i) * 8 + (l >> 3), q = (l & 7) ^ mx8_swizzle(r);  // q = 4 piece + 2 block + half
      xoff[i] = (uint32_t)(act_row(r) * (a.KK * kGroup)) + (uint32_t)((q & 2) * 64 + (q >> 2) * 32 + (q & 1) * 16);
    } else {
      const int r = (w * S::kXDma + i) * 16 + (l >> 2), q = (l & 3) ^ mx_swizzle(r);  // q = 2 half + piece
      xoff[i] = (uint32_t)(act_row(r) * (a.KK * kGroup)) + (uint32_t)((4 * (q >> 1) + (q & 1)) * 16);
    }
  }
#pragma unroll
  for (int i = 0; i < S::kSDma; ++i) {
    const int u = min(w * S::kSDma + i, S::kUnits - 1);
    if (u < S::kSlots) {
      ssrc[i] = a.w_scales + ((int64_t)e * a.G + group(u)) * a.KK * kMxFragScales;
      soff[i] = (uint32_t)l * 4u;
      sstep[i] = kMxFragScales;
    } else {
      ssrc[i] = a.a_scales;
      soff[i] = (uint32_t)(act_row((u - S::kSlots) * 32 + n) * (a.KK * 8)) + (uint32_t)f * 4u;
      sstep[i] = 8;
    }
  }
  // Part `part` of 2 GW parts of a stage's DMA (the first with the scales of its column group if it is the first half).
  auto dma = [&](int st, int part) {
    const int64_t c = st >> 1;
    const uint32_t buf = __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)(st % RING) * (uint32_t)S::kStage);
    if (part == 0 && (st & 1) == 0) {
      const uint32_t sb = __builtin_amdgcn_readfirstlane(
          lds0 + (uint32_t)(S::kRing * S::kStage) + ((uint32_t)c & 1u) * (uint32_t)(S::kUnits * 256));
#pragma unroll
      for (int i = 0; i < S::kSDma; ++i)
        dma4_async(ssrc[i] + c * sstep[i], soff[i], sb + (uint32_t)min(w * S::kSDma + i, S::kUnits - 1) * 256u);
    }
    constexpr int kAll = S::kWDma + S::kXDma;
#pragma unroll
    for (int i = 0; i < S::kWDma; ++i)
      if (i * 2 * GW / kAll == part)
        dma16_async(wsrc[i] + c * kMxFragCodes + (st & 1) * 2048, (uint32_t)l * 16u,
                    buf + (uint32_t)((w * S::kWDma + i) * 1024));
    const uint8_t* xc = a.a_codes + c * kGroup + (st & 1) * (A8 ? 64 : 32);
#pragma unroll
    for (int i = 0; i < S::kXDma; ++i)
      if ((S::kWDma + i) * 2 * GW / kAll == part)
        dma16_async(xc, xoff[i], buf + (uint32_t)(S::kWBytes + (w * S::kXDma + i) * 1024));
  };

  // ---- fragments and scales from LDS
  struct Frags {
    i32x4_t w[GW];
    typename ActFrag<A8>::type x[GX];
  };
  struct Scales {
    int w[GW], x[GX];
  };
  const int xlane = (wx * GX * 32 + n) * S::kXRow, sw_n = A8 ? mx8_swizzle(n) : mx_swizzle(n);  // a wave's token groups are 32 rows apart
  // Fragment r of piece p of stage st: the token fragments (lx of them), then the GW weight fragments.
  auto read = [&](int st, int p, int r, int lx, Frags& fr) {
    const unsigned char* buf = smem + (st % RING) * S::kStage;
    if (r < lx) {
      const unsigned char* row = buf + S::kWBytes + xlane + r * (32 * S::kXRow);
      if constexpr (A8)
        fr.x[r] = join_halves(*reinterpret_cast<const i32x4_t*>(row + ((4 * p + f) ^ sw_n) * 16),
                              *reinterpret_cast<const i32x4_t*>(row + ((4 * p + 2 + f) ^ sw_n) * 16));
      else fr.x[r] = *reinterpret_cast<const i32x4_t*>(row + ((2 * f + p) ^ sw_n) * 16);
    } else
      fr.w[r - lx] = *reinterpret_cast<const i32x4_t*>(buf + (wm * GW * 2 + p) * 1024 + l * 16 + (r - lx) * 2048);
  };
  auto read_scales = [&](int c, int lx, Scales& s) {
    if (lx == 0) return;
    const unsigned char* buf = smem + S::kRing * S::kStage + (c & 1) * (S::kUnits * 256) + l * 4;
#pragma unroll
    for (int i = 0; i < GW; ++i) s.w[i] = *reinterpret_cast<const int*>(buf + (wm * GW + i) * 256);
#pragma unroll
    for (int i = 0; i < lx; ++i) s.x[i] = *reinterpret_cast<const int*>(buf + (S::kSlots + wx * GX + i) * 256);
  };

  // what the epilogue needs of the pairs, loaded ahead of the products
  int pair[GX];
  float pair_w[GX];
  if constexpr (MODE == kDown) {
#pragma unroll
    for (int j = 0; j < GX; ++j) {
      pair[j] = a.sorted[first + min((wx * GX + j) * 32 + n, cnt - 1)];
      pair_w[j] = a.topk_w[pair[j]];
    }
  }
  float16_t acc[GW][GX];
#pragma unroll
  for (int i = 0; i < GW; ++i)
#pragma unroll
    for (int j = 0; j < GX; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  uint32_t bh[GX];
#pragma unroll
  for (int j = 0; j < GX; ++j) bh[j] = 0;

  // One MFMA step on `fr`, reading `nx` = piece np of stage nst under it and
  // issuing half `half` (0, 1; 2 = none) of the DMA of stage dst.  Reads and DMA
  // are dealt out between the products, which leave the issue slots free: the
  // LDS takes 8 cycles for a fragment of one wave and the memory pipe 16 for a
  // 1 KB DMA, so that waves that issue theirs in a burst wait for each other
  // with the matrix cores idle.  The last quarter of a step has no reads: a
  // barrier may follow, and waits for them.  The steps hold no branches:
  // products have no side effects, and the compiler would move them past a
  // branch to where their result is used.  Token groups past the end are left out
  // (live of GX remain): a wave with none only does its share of the DMA, and
  // its SIMD is the other wave's.
  auto step = [&](auto live, auto sel, auto half, const Frags& fr, const Scales& sc, Frags& nx, int nst, int np, int dst) {
    constexpr int LX = decltype(live)::value, kHalf = decltype(half)::value;
    constexpr int kReads = GW + LX, kSpan = 3 * GW * LX / 4;
    if constexpr (LX == 0) {
      if constexpr (kHalf < 2) {
#pragma unroll
        for (int i = 0; i < GW; ++i) dma(dst, kHalf * GW + i);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < GW; ++i) {
#pragma unroll
      for (int j = 0; j < LX; ++j) {
        acc[i][j] = act_mfma<decltype(sel)::value>(fr.w[i], fr.x[j], acc[i][j], sc.w[i], sc.x[j]);
#pragma unroll
        for (int k = 0; k < kReads; ++k)
          if (k * kSpan / kReads == i * LX + j) read(nst, np, k, LX, nx);
        if constexpr (kHalf < 2)
          if (j == LX / 2) dma(dst, kHalf * GW + i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  Frags f0, f1;
  Scales sc;
  // DMA instructions of a stage; an even one has kSDma more, its column group's scales
  constexpr int kPlain = S::kWDma + S::kXDma;
  // Column group c; t of the groups after it count, later ones are as many as
  // it takes (t >= (RING + 1) / 2).  The DMA of the stage RING ahead of one is
  // issued in two halves, in the two steps after its hand-over: here those of
  // the hand-overs before, inside and at the end of this group, as far as there
  // are such stages.  A hand-over waits until the next stage is in LDS, leaving
  // the later ones (up to RING - 2) in flight, and until no wave reads the
  // present one any more.
  auto group_cols = [&](auto live, int c, auto after) {
    constexpr int t = decltype(after)::value;
    constexpr bool kD0 = 2 * t + 2 >= RING, kD1 = 2 * t + 1 >= RING, kD2 = 2 * t >= RING;
    constexpr int n1 = 2 * t < RING - 2 ? 2 * t : RING - 2, w1 = n1 * kPlain + (n1 + 1) / 2 * S::kSDma;
    constexpr int m2 = t > 0 ? 2 * t - 1 : 0, n2 = m2 < RING - 2 ? m2 : RING - 2, w2 = n2 * kPlain + n2 / 2 * S::kSDma;
    const int st = 2 * c;
    if (MODE == kDown) {
#pragma unroll
      for (int j = 0; j < decltype(live)::value; ++j) bh[j] = max(bh[j], max_byte((uint32_t)sc.x[j]));
    }
    step(live, Const<0>(), Const<(kD0 ? 1 : 2)>(), f0, sc, f1, st, 1, st - 1 + RING);
    wait_vmcnt<w1>();
    barrier_after_lds();
    step(live, Const<1>(), Const<(kD1 ? 0 : 2)>(), f1, sc, f0, st + 1, 0, st + RING);
    step(live, Const<2>(), Const<(kD1 ? 1 : 2)>(), f0, sc, f1, st + 1, 1, st + RING);
    Scales last;  // the fourth step's bytes
#pragma unroll
    for (int i = 0; i < GW; ++i) last.w[i] = (int)((uint32_t)sc.w[i] >> 24);
#pragma unroll
    for (int j = 0; j < decltype(live)::value; ++j) last.x[j] = (int)((uint32_t)sc.x[j] >> 24);
    wait_vmcnt<w2>();
    barrier_after_lds();
    // past the last group these read buffers that are not used
    read_scales(c + 1, decltype(live)::value, sc);
    step(live, Const<0>(), Const<(kD2 ? 0 : 2)>(), f1, last, f0, st + 2, 0, st + 1 + RING);
  };
  const int KK = (int)a.KK;
  constexpr int kLong = (RING + 1) / 2;
#pragma unroll
  for (int st = 0; st < RING; ++st)
    if (st < 2 * KK) {
#pragma unroll
      for (int p = 0; p < (st == RING - 1 ? GW : 2 * GW); ++p) dma(st, p);  // the last one's second half: first step
    }
  // the first stage is in LDS; of the RING - 1 later ones all but the half-issued last may be in flight
  if (2 * KK >= RING) wait_vmcnt<(RING - 2) * kPlain + (RING - 2) / 2 * S::kSDma>();
  else wait_vmcnt<0>();
  barrier_after_lds();
  auto tail = [&](auto self, auto live, auto after) {
    constexpr int t = decltype(after)::value;
    if (KK > t) group_cols(live, KK - 1 - t, after);
    if constexpr (t > 0) self(self, live, Const<t - 1>());
  };
  auto all_cols = [&](auto live) {
    constexpr int LX = decltype(live)::value;
    read_scales(0, LX, sc);
    if constexpr (LX > 0) {
#pragma unroll
      for (int k = 0; k < GW + LX; ++k) read(0, 0, k, LX, f0);
    }
    for (int c = 0; c + kLong < KK; ++c) group_cols(live, c, Const<kLong>());
    tail(tail, live, Const<kLong - 1>());
  };
  const int groups = (cnt - wx * GX * 32 + 31) / 32;  // of this wave's tokens
  if (groups >= GX) all_cols(Const<GX>());
  else if (GX > 3 && groups == 3) all_cols(Const<(GX > 3 ? 3 : 0)>());
  else if (GX > 2 && groups == 2) all_cols(Const<(GX > 2 ? 2 : 0)>());
  else if (GX > 1 && groups == 1) all_cols(Const<(GX > 1 ? 1 : 0)>());
  else all_cols(Const<0>());

  // ---- epilogue of the dense product of 8-bit activations: FP32 results go through LDS (the ring is no longer needed),
  // as many token groups at a time as it holds, so that bias, residual and result move in runs of whole rows
  if constexpr (MODE == kLinear && A8) {
    constexpr int kCols = S::kSlots * 32, kRow = kCols + 4;  // floats; 16 bytes more against bank conflicts
    constexpr int JP = S::kWX * GX * 32 * kRow * 4 <= S::kLds ? GX : GX / 2;
    static_assert(S::kWX * JP * 32 * kRow * 4 <= S::kLds && GX % JP == 0, "a pass fits the ring");
    constexpr int kLanes = kCols / 8, kRows = NW * 64 / kLanes;
    constexpr int kAll = S::kWX * JP * 32, kAhead = kAll / kRows < 4 ? kAll / kRows : 4;  // rows of a pass; rows a thread takes at a time
    static_assert(kAll % (kRows * kAhead) == 0, "whole steps");
    const int c8 = tid % kLanes * 8, col = wt * kCols + c8, act = a.aux >> kMxActShift;
    float* tile = reinterpret_cast<float*>(smem);
    float bias[8];
    if (a.bias && col < a.N) epilogue_load8(a.bias + col, a.N - col, bias);
#pragma unroll
    for (int j0 = 0; j0 < GX; j0 += JP) {
      auto token = [&](int r) { return (r / (32 * JP) * GX + j0) * 32 + r % (32 * JP); };
      float res[kAhead][8];
      auto load = [&](int r0) {  // residuals of rows r0, r0 + kRows, ...
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (a.residual && col < a.N && token(r0 + k * kRows) < cnt) epilogue_residual8(a, first + token(r0 + k * kRows), col, res[k]);
      };
      if (j0 > 0) barrier_after_lds();
      load(tid / kLanes);  // the first ones under the way through LDS
#pragma unroll
      for (int j = 0; j < JP; ++j)
#pragma unroll
        for (int i = 0; i < GW; ++i) {
          float4* p = reinterpret_cast<float4*>(tile + ((wx * JP + j) * 32 + n) * kRow + (wm * GW + i) * 32 + f * 16);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            p[q] = make_float4(acc[i][j0 + j][4 * q], acc[i][j0 + j][4 * q + 1], acc[i][j0 + j][4 * q + 2], acc[i][j0 + j][4 * q + 3]);
        }
      barrier_after_lds();
      if (col < a.N) {
#pragma unroll 1
        for (int r0 = tid / kLanes; r0 < kAll; r0 += kRows * kAhead) {
          if (r0 >= kRows) load(r0);
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * kRows, tok = token(r);
            if (tok >= cnt) continue;
            const float4 u = *reinterpret_cast<const float4*>(tile + r * kRow + c8), w4 = *reinterpret_cast<const float4*>(tile + r * kRow + c8 + 4);
            float v[8] = {u.x, u.y, u.z, u.w, w4.x, w4.y, w4.z, w4.w};
            if (a.bias) {
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] += bias[q];
            }
            if (act != kActNone) {
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] = activate(act, v[q]);
            }
            if (a.residual) {
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] += res[k][q];
            }
            epilogue_store8(a, first + tok, col, v);
          }
        }
      }
    }
    return;
  }

  int* out_row = reinterpret_cast<int*>(smem + S::kTok * S::kOutRow);
  int wmax = 0;
  if constexpr (MODE == kDown) {
    wmax = a.w_max[e];
    if (wmax == 255) wmax = finite_scale_max<64>(a, e, l);
  }
  // ---- epilogue: a lane holds 16 consecutive features (half f of a group) of token n
#pragma unroll
  for (int j = 0; j < GX; ++j) {
    const int tok = (wx * GX + j) * 32 + n;
    const int64_t row = first + tok;
    const bool in = tok < cnt;
    if constexpr (MODE == kGateUp) {
#pragma unroll
      for (int i = 0; i < GW / 2; ++i) {
        float h[16];
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          h[r] = silu(acc[i][j][r]) * acc[i + GW / 2][j][r];
          m = max(m, abs_bits(h[r]));
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        const uint32_t byte = A8 ? mx8_scale_byte(m) : mx_scale_byte(m);
        const int hb = wt * (S::kSlots / 2) + wm * (GW / 2) + i;
        if (in && hb < a.G / 2) {
          uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.ldo;
          if constexpr (A8)
            *reinterpret_cast<uint4*>(out + hb * 32 + f * 16) =
                make_uint4(mx8_encode4(h, byte), mx8_encode4(h + 4, byte), mx8_encode4(h + 8, byte), mx8_encode4(h + 12, byte));
          else *reinterpret_cast<uint2*>(out + hb * 16 + f * 8) = make_uint2(mx_encode8(h, byte), mx_encode8(h + 8, byte));
          if (f == 0) static_cast<uint8_t*>(a.out_scales)[row * (a.ldo / (A8 ? 32 : 16)) + hb] = (uint8_t)byte;
        }
      }
      if (wt == 0 && wm == 0 && in) zero_h_pad<A8>(a, row, f, 2);
    } else if (MODE == kLinear && (a.aux & kMxOutF32)) {
      if (!in) continue;
#pragma unroll
      for (int i = 0; i < GW; ++i) {
        const int col = (wt * S::kSlots + wm * GW + i) * 32 + f * 16;
        float* p = static_cast<float*>(a.out) + row * a.ldo + col;
        if ((a.aux & kMxOutVec) && col + 16 <= a.N) {
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            store16_streaming(p + r, __float_as_uint(acc[i][j][r]), __float_as_uint(acc[i][j][r + 1]),
                              __float_as_uint(acc[i][j][r + 2]), __float_as_uint(acc[i][j][r + 3]));
        } else {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (col + r < a.N) p[r] = acc[i][j][r];
        }
      }
    } else {
      // 16-bit results go through LDS (the ring is no longer needed), so that
      // every row leaves as one run of kSlots * 64 bytes
      float factor = 1.0f;
      if constexpr (MODE == kDown) {
        const uint32_t b = max(bh[j], (uint32_t)__shfl_xor((int)bh[j], 32));
        if (in) {
          const int E = pair_exponent(pair_w[j], b, wmax, a.aux);
          factor = pair_w[j] * __uint_as_float((uint32_t)(127 - E) << 23);  // exact
          if (wm == 0 && f == 0) {
            out_row[tok] = pair[j];
            if (wt == 0) static_cast<float*>(a.out_scales)[pair[j]] = __uint_as_float((uint32_t)(127 + E) << 23);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < GW; ++i) {
        uint32_t v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = MODE == kDown ? f16_pair(factor * acc[i][j][2 * r], factor * acc[i][j][2 * r + 1])
                               : bf16_pair(acc[i][j][2 * r], acc[i][j][2 * r + 1]);
        uint4* p = reinterpret_cast<uint4*>(smem + tok * S::kOutRow + (wm * GW + i) * 64 + f * 32);
        p[0] = make_uint4(v[0], v[1], v[2], v[3]);
        p[1] = make_uint4(v[4], v[5], v[6], v[7]);
      }
    }
  }
  if (MODE == kGateUp || (MODE == kLinear && (a.aux & kMxOutF32))) return;
  barrier_after_lds();
  constexpr int kLanes = S::kSlots * 4, kRows = 64 / kLanes;  // lanes that write a row, rows a wave writes at a time
  const int col = wt * S::kSlots * 32 + (l % kLanes) * 8;
  if (col >= a.N) return;
  for (int t = w * kRows + l / kLanes; t < cnt; t += NW * kRows) {
    const uint4 v = *reinterpret_cast<const uint4*>(smem + t * S::kOutRow + (l % kLanes) * 16);
    uint16_t* p = static_cast<uint16_t*>(a.out) + (MODE == kDown ? (int64_t)out_row[t] : first + t) * a.ldo + col;
    if (MODE == kDown || ((a.aux & kMxOutVec) && col + 8 <= a.N)) {
      store16_streaming(p, v.x, v.y, v.z, v.w);
    } else {
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (col + r < a.N) p[r] = (uint16_t)(d[r >> 1] >> (16 * (r & 1)));
    }
  }
}

namespace {

// max_mtiles: an upper bound on the m-tiles (for experts the kernel counts them)
template <int MODE, class S>
hipError_t launch_tiled(const MxArgs& a, int64_t max_mtiles, hipStream_t st) {
  auto* k = &mx_tiled_kernel<MODE, S>;
  if (hipError_t e = set_max_dynamic_lds(reinterpret_cast<const void*>(k), S::kLds)) return e;
  const int64_t rows = MODE == kGateUp ? a.G / 2 : a.G, per = MODE == kGateUp ? S::kSlots / 2 : S::kSlots;
  const int64_t grid = (max_mtiles * ((rows + per - 1) / per) + 7) / 8 * 8;
  return launch_kernel(k, dim3((unsigned)grid), dim3(64 * S::kWaves), S::kLds, st, a);
}

enum Shape { kStream, k64x64, k128x64, k128x128, k256x64, k256x128, k256x256 };

// m-tiles of `tok` pairs that E experts can have at most
inline int64_t most_mtiles(int64_t pairs, int64_t E, int64_t tok) { return pairs / tok + (pairs < E ? pairs : E); }

}  // namespace

}  // namespace moe
