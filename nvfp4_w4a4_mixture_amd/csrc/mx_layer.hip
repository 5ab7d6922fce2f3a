// The whole routed-expert layer for up to 32 tokens, in three kernels: the
// router's scores with the quantisation of x; gate_up with the selection; down
// with the combine.  With many scores a fourth, before gate_up, ranks them.
//
//   z[t, e] = x[t] . W_r[e] in FP64, s = sigmoid(z)
//   the k experts of a token: largest s + bias first, ties to the lower index
//   w[t, e] = rsf * s / (sum of the k s)
//   y[t] = sum over e of w[t, e] * W2[e] . q(silu(W_gate[e] . q(x[t])) * (W_up[e] . q(x[t])))
//
// With so few tokens the touched experts' weights bound it (and launches, where
// the layer is small), so the tokens are the 32 columns of one MFMA tile whatever
// they chose: no permutation of pairs is needed, columns of tokens that did not
// choose an expert are left out of its results, and the sum over the experts stays
// in FP32 accumulators, in a fixed order.  No atomic decides an order.
#include "launch.h"
#include "mx_common.h"
#include "mx_product.h"

namespace moe {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kMaxTok = (int)kLayerMaxTokens;
constexpr int kMaxParts = 4;
constexpr int64_t kRankWork = 1 << 15;  // comparisons past which the ranking is a kernel of its own
constexpr int kRankScores = 1024;       // the most scores of no more: T * E <= sqrt(32 * kRankWork)

// Workgroups that share 32 features of y: as many as leave each a CU, and each of
// its waves four column groups of products.  With one workgroup H = 2048 used 64 of
// 256 CUs: 32 tokens of 64 experts, I = 1408: 52.5 us in one, 40.3 in four; 16 of
// 256, H = 4096, I = 1024: 60.8 and 55.4 in two; with two column groups a wave it
// loses (1 of 256: 24.7 and 25.3).
__host__ __device__ inline int64_t down_parts(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  const int64_t items = (T * k < E ? T * k : E) * ((I + 255) / 256), cus = 256 / (H / 32), n = items / 32 < cus ? items / 32 : cus;
  return n < 1 ? 1 : n > kMaxParts ? kMaxParts : n;
}

// Everything between the kernels: keys (the order of the scores) and sigmoids of
// all experts, the chosen sigmoids by slot, all experts' ranks, x and h in MXFP8,
// the parts' sums and their counts.  Up to 16 tokens x and h are kept as the two
// operands that they are multiplied as (see mx8_mfma), the large elements and the
// rest, which are the halves of one operand's 32 columns: one instruction
// multiplies both.  Past 16 they are kept whole and parted at the product (kept as
// two, 32 tokens of 80 experts took 205 us instead of 170: twice the bytes of x
// through the L1, which every tile reads anew).
// x lies in the order of the fragments, [operand, KK, step, block of two, half,
// column, 16] and scale bytes [KK, half, column, 4], so that a load of a wave is a
// whole run; h in rows, of which a wave reads the few that chose its expert.
struct LayerWs {
  size_t key, sig, chosen, slot, x_codes, x_scales, h_codes, h_scales, parts, arrived, total;
  __host__ __device__ LayerWs(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
    const size_t Hp = (size_t)((H + 255) / 256 * 256), Ip = (size_t)((I + 255) / 256 * 256), t = (size_t)T, p = t * (size_t)k;
    size_t o = 0;
    auto take = [&](size_t bytes) {
      const size_t at = o;
      o += (bytes + 255) / 256 * 256;
      return at;
    };
    key = take(t * (size_t)E * 8);
    sig = take(t * (size_t)E * 8);
    chosen = take(p * 8);
    slot = take(t * (size_t)E * 2);
    x_codes = take(Hp * 32);
    x_scales = take(Hp);
    h_codes = take(p * Ip * (T <= 16 ? 2 : 1));
    h_scales = take(p * Ip / 32);
    const size_t n = (size_t)down_parts(T, E, k, H, I), groups = (size_t)(H / 32);
    parts = take(n > 1 ? n * groups * kMaxTok * 32 * 4 : 0);
    arrived = take(n > 1 ? groups * 4 : 0);
    total = o;
  }
};

typedef uint32_t u32x4_any2_t __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ u32x4_any2_t load8(const uint16_t* p) { return *reinterpret_cast<const u32x4_any2_t*>(p); }
__device__ __forceinline__ float element(const u32x4_any2_t& v, int i) {
  return __uint_as_float((i & 1) ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
}

}  // namespace

// Workgroup (e, g), e < E: the scores of expert e for TT tokens; those after them
// quantise x.  A product of two BF16 values is exact in FP64; the sum's order is
// fixed: each thread's columns, then lanes, then waves.  After the exchanges lane
// group t of 64 / TT lanes holds token t.  Up to four tokens a workgroup: with 16
// in one the conversions to FP64 took 14 us (80 experts of 6144).
template <int TT>
__global__ __launch_bounds__(kScoreThreads) void mx_layer_score_kernel(MxLayerArgs a) {
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if (down_parts(a.T, a.E, a.k, a.H, a.I) > 1 && blockIdx.y == 0)  // zero before the down kernel counts
    for (int i = (int)blockIdx.x * kScoreThreads + tid; i < a.H / 32; i += (int)gridDim.x * kScoreThreads)
      reinterpret_cast<uint32_t*>(a.ws + ws.arrived)[i] = 0;
  if ((int)blockIdx.x >= a.E) {
    const int chunks = (a.H + 255) / 256 * 32;  // of 8 columns, of a padded row
    const int i = (((int)blockIdx.x - a.E) * (int)gridDim.y + (int)blockIdx.y) * kScoreThreads + tid;
    if (i >= a.T * chunks) return;  // whole quads
    const int t = i / chunks, c = (i - t * chunks) * 8;
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t m = 0;
    if (c < a.H) {
      const u32x4_any2_t v = load8(a.x + (int64_t)t * a.ldx + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = element(v, j);
        m = max(m, abs_bits(f[j]));
      }
    }
    const uint32_t byte = mx8_scale_byte(quad_max(m));
    const int cg = c >> 8, u = (c >> 7) & 1, st = (c >> 5) & 3, half = (c >> 4) & 1;
    const uint32_t d[2] = {mx8_encode4(f, byte), mx8_encode4(f + 4, byte)};
    uint8_t* xc = a.ws + ws.x_codes + (int64_t)(((cg * 4 + st) * 2 + u) * 2 + half) * 512 + t * 16 + (c & 15);
    uint8_t* xs = a.ws + ws.x_scales + ((int64_t)(cg * 2 + u) * 32 + t) * 4 + st;
    if ((tid & 3) == 0) xs[0] = (uint8_t)byte;
    if (a.T > 16) {
      *reinterpret_cast<uint2*>(xc) = make_uint2(d[0], d[1]);
      return;
    }
    const uint32_t large[2] = {mx8_large(d[0]), mx8_large(d[1])};
    *reinterpret_cast<uint2*>(xc) = make_uint2(large[0], large[1]);
    *reinterpret_cast<uint2*>(xc + 256) = make_uint2(d[0] ^ large[0], d[1] ^ large[1]);
    if ((tid & 3) == 0) xs[64] = (uint8_t)byte;
    return;
  }
  __shared__ double red[kScoreThreads / 64][TT];
  const int e = blockIdx.x, t0 = (int)blockIdx.y * TT;
  const uint16_t* xr[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xr[t] = a.x + (int64_t)min(t0 + t, a.T - 1) * a.ldx;
  const uint16_t* wr = a.w_router + (int64_t)e * a.H;
  double acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0;
#pragma unroll 3
  for (int c = tid * 8; c < a.H; c += kScoreThreads * 8) {
    const u32x4_any2_t wv = load8(wr + c);
    u32x4_any2_t xv[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xv[t] = load8(xr[t] + c);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = __builtin_fma((double)element(xv[t], j), (double)element(wv, j), acc[t]);
  }
  int m = 32;
#pragma unroll
  for (int n = TT / 2; n > 0; n /= 2, m /= 2) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool up = (lane & m) != 0;
      const double keep = up ? acc[i + n] : acc[i], give = up ? acc[i] : acc[i + n];
      acc[i] = keep + __shfl_xor(give, m);
    }
  }
  for (; m > 0; m /= 2) acc[0] += __shfl_xor(acc[0], m);
  if (lane % (64 / TT) == 0) red[w][lane / (64 / TT)] = acc[0];
  __syncthreads();
  if (tid >= TT || t0 + tid >= a.T) return;
  double z = red[0][tid];
#pragma unroll
  for (int i = 1; i < kScoreThreads / 64; ++i) z += red[i][tid];
  const double s = 1.0 / (1.0 + exp(-z));
  const int at = (t0 + tid) * a.E + e;
  reinterpret_cast<double*>(a.ws + ws.sig)[at] = s;
  reinterpret_cast<long long*>(a.ws + ws.key)[at] = score_key(s + (double)a.bias[e]);
}

// The number of experts that come before expert o of a token: of larger key, or of
// the same and lower index.  The keys' upper halves decide unless two are alike.
// Lane i of the NL that share an expert takes every NL-th comparison.
template <int NL>
__device__ __forceinline__ int rank_of(const int* high, const long long* key, int E, int o, int i) {
  const int mine = high[o];
  int r = 0, same = 0;
#pragma unroll 8
  for (int q = i; q < E; q += NL) {
    r += (int)(high[q] > mine);
    same += (int)(high[q] == mine);
  }
#pragma unroll
  for (int m = 1; m < NL; m *= 2) {
    r += __shfl_xor(r, m);
    same += __shfl_xor(same, m);
  }
  if (same > 1) {
    const long long whole = key[o];
    r = 0;
    for (int q = 0; q < E; ++q) r += (int)(key[q] > whole) | ((int)(key[q] == whole) & (int)(q < o));
  }
  return r;
}

// Workgroup t ranks token t's experts.
__global__ __launch_bounds__(1024) void mx_layer_rank_kernel(MxLayerArgs a) {
  __shared__ int high[256];
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const int tid = threadIdx.x, o = tid >> 2, at = (int)blockIdx.x * a.E;
  const long long* key = reinterpret_cast<const long long*>(a.ws + ws.key) + at;
  if (tid < a.E) high[tid] = (int)(key[tid] >> 32);
  __syncthreads();
  if (o >= a.E) return;  // whole groups of four lanes
  const int r = rank_of<4>(high, key, a.E, o, tid & 3);
  if ((tid & 3) == 0) reinterpret_cast<uint16_t*>(a.ws + ws.slot)[at + o] = (uint16_t)r;
}

// The 32 h columns of one group of one expert (a tile) for the tokens that chose
// it, as mx8_stream_kernel.  A token chose an expert if fewer than k rank before
// it, and that number is its slot: found here from the token's keys, so that no
// kernel stands between the scores and the weights.
//
// Every workgroup lists the touched experts and takes every gridDim.x-th of their
// tiles, a column group ahead across tiles too.  RANK: it ranks all scores itself,
// T * E * E comparisons; with many (kRankWork) a kernel before it does.  The layer in
// us with the ranking here, and with the kernel (H = 2048, I = 768, top-8):
//   T x E   1 x 128 16.5 K  2 x 128 33 K  8 x 64 33 K  32 x 32 33 K  16 x 48 37 K  12 x 64 49 K  4 x 128 66 K  16 x 64 66 K
//   here         18.2          23.2         32.0          34.8          34.8          34.5          29.1          36.4
//   kernel       18.3          23.9         32.6          34.3          35.0          34.4          27.8          35.0
// (1 x 256, 66 K: H = 1024 17.2 and 17.1, H = 256 15.8 and 16.3.)  16 x 256: 124 and 63.
//
// Bounds: the weights' bytes.  16 tokens of 80 experts, H = 6144, I = 2048, 28
// touched: 374 MB in 70 us (5.4 TB/s), after 5 of the ranking (ranked here 76).
// One token, 8 touched: 20 us (5.4 TB/s).
template <bool RANK, bool HALF>
__global__ __launch_bounds__(256, 2) void mx_layer_gate_up_kernel(MxLayerArgs a) {
  constexpr int NW = 4;
  __shared__ float4 part[NW][2][4 * 68];
  __shared__ int high[RANK ? kRankScores : 1];
  __shared__ uint16_t slot[RANK ? kRankScores : kMaxTok * 256], listed[256];
  __shared__ uint32_t mask[8];
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int col_tok = HALF ? n & 15 : n, groups = a.I / 32, KK = (a.H + 255) / 256, G = a.I / 16, all = a.T * a.E;
  const long long* key = reinterpret_cast<const long long*>(a.ws + ws.key);
  if (tid < 8) mask[tid] = 0;
  if constexpr (RANK)
    for (int i = tid; i < all; i += 256) high[i] = (int)(key[i] >> 32);
  __syncthreads();
  for (int i = tid; i < all; i += 256) {
    const int t = i / a.E, o = i - t * a.E;
    const int r = RANK ? rank_of<1>(high + t * a.E, key + t * a.E, a.E, o, 0) : reinterpret_cast<const uint16_t*>(a.ws + ws.slot)[i];
    slot[i] = (uint16_t)r;
    if (r < a.k) atomicOr(&mask[o >> 5], 1u << (o & 31));
  }
  __syncthreads();
  int before = 0, touched = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < (tid >> 5)) before += __popc(mask[i]);
    touched += __popc(mask[i]);
  }
  if ((mask[tid >> 5] >> (tid & 31)) & 1) listed[before + __popc(mask[tid >> 5] & ((1u << (tid & 31)) - 1u))] = (uint16_t)tid;
  const int tiles = touched * groups;
  __syncthreads();
  struct Cols {
    i32x8_t x[4];
    i32x4_t w[2][4];
    int sw[2], sx;
  };
  // No branch stands before a load, so that the compiler can count those in
  // flight: past the end they repeat what is there, and columns of tokens that did
  // not choose the expert, whose sums nobody reads, all take the first one's place.
  auto load = [&](int t, int c, Cols& d) {
    t = min(t, tiles - 1);
    c = min(c, KK - 1);
    const int i = t / groups, e = listed[i], g = t - i * groups;
    const bool chosen = col_tok < a.T && slot[min(col_tok, a.T - 1) * a.E + e] < a.k;
    const int place = f * 32 + (chosen ? n : 0);
    const uint8_t* xc = a.ws + ws.x_codes + (int64_t)c * 8192 + place * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint8_t* p = xc + s * 2048;
      d.x[s] = join_halves(*reinterpret_cast<const i32x4_t*>(p), *reinterpret_cast<const i32x4_t*>(p + 1024));
    }
    d.sx = *reinterpret_cast<const int*>(a.ws + ws.x_scales + (int64_t)c * 256 + place * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = ((int64_t)e * G + g + i * (G / 2)) * KK + c;
#pragma unroll
      for (int s = 0; s < 4; ++s) d.w[i][s] = reinterpret_cast<const i32x4_t*>(a.w13_codes + at * kMxFragCodes)[s * 64 + l];
      d.sw[i] = reinterpret_cast<const int*>(a.w13_scales + at * kMxFragScales)[l];
    }
  };
  float16_t acc[2];
  auto multiply = [&](int c, const Cols& d) {
    if (c >= KK) return;
    acc[0] = mx8_mfma<0, HALF>(d.w[0][0], d.x[0], acc[0], d.sw[0], d.sx);
    acc[1] = mx8_mfma<0, HALF>(d.w[1][0], d.x[0], acc[1], d.sw[1], d.sx);
    acc[0] = mx8_mfma<1, HALF>(d.w[0][1], d.x[1], acc[0], d.sw[0], d.sx);
    acc[1] = mx8_mfma<1, HALF>(d.w[1][1], d.x[1], acc[1], d.sw[1], d.sx);
    acc[0] = mx8_mfma<2, HALF>(d.w[0][2], d.x[2], acc[0], d.sw[0], d.sx);
    acc[1] = mx8_mfma<2, HALF>(d.w[1][2], d.x[2], acc[1], d.sw[1], d.sx);
    acc[0] = mx8_mfma<3, HALF>(d.w[0][3], d.x[3], acc[0], d.sw[0], d.sx);
    acc[1] = mx8_mfma<3, HALF>(d.w[1][3], d.x[3], acc[1], d.sw[1], d.sx);
  };
  // The tile's sums, h and its quantisation
  auto finish = [&](int t) {
    const int e = listed[t / groups], blk = t % groups;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part[w][i][q * 68 + f * 34 + n] = make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
    __syncthreads();
    const int tok = tid >> 3, p = tid & 7;  // features 4 p .. 4 p + 3 of one token
    const int r = tok < a.T ? slot[tok * a.E + e] : a.E;
    if (blk == 0 && p == 0 && r < a.k) {
      a.topk_ids[tok * a.k + r] = e;
      reinterpret_cast<double*>(a.ws + ws.chosen)[tok * a.k + r] = reinterpret_cast<const double*>(a.ws + ws.sig)[tok * a.E + e];
    }
    if (r < a.k) {  // eight lanes together
      float v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 s = add_waves<NW, HALF, 2 * kWaveSums>(part[0][i], p, tok);
        v[i][0] = s.x;
        v[i][1] = s.y;
        v[i][2] = s.z;
        v[i][3] = s.w;
      }
      float h[4];
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[q] = silu(v[0][q]) * v[1][q];
        m = max(m, abs_bits(h[q]));
      }
      m = quad_max(m);
      m = max(m, lane_dpp<kLaneHalfMirror>(m));
      const uint32_t byte = mx8_scale_byte(m), d = mx8_encode4(h, byte), large = HALF ? mx8_large(d) : d;
      const int Ip = (a.I + 255) / 256 * 256;
      const int64_t row = tok * a.k + r, rest = (int64_t)a.T * a.k * Ip;  // from a large element to what is left of it
      uint8_t* hc = a.ws + ws.h_codes + row * Ip;
      uint8_t* hs = a.ws + ws.h_scales + row * (Ip / 32);
      reinterpret_cast<uint32_t*>(hc)[blk * 8 + p] = large;
      if (HALF) reinterpret_cast<uint32_t*>(hc + rest)[blk * 8 + p] = d ^ large;
      if (p == 0) hs[blk] = (uint8_t)byte;
      if (blk == 0) {  // the padding past I is zero
        for (int b = a.I / 32 + p; b < Ip / 32; b += 8) {
#pragma unroll
          for (int q = 0; q < (HALF ? 4 : 2); ++q) reinterpret_cast<uint4*>(hc + (q >> 1) * rest)[2 * b + (q & 1)] = make_uint4(0, 0, 0, 0);
          hs[b] = 0;
        }
      }
    }
    __syncthreads();  // part is free
  };
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  };
  // every wave takes as many steps a tile (the last of some past KK: nothing), so that all meet in finish
  int t = blockIdx.x, c = w;
  if (t >= tiles) return;
  Cols d0, d1;
  load(t, c, d0);
  clear();
  auto step = [&](Cols& now, Cols& next) {  // false: the last tile is done
    const bool last = c - w + NW >= KK;
    const int nt = last ? t + (int)gridDim.x : t, nc = last ? w : c + NW;
    load(nt, nc, next);
    multiply(c, now);
    if (last) {
      finish(t);
      clear();
    }
    t = nt;
    c = nc;
    return nt < tiles;
  };
  while (step(d0, d1) && step(d1, d0)) {
  }
}

namespace {

// LDS of the down kernel: the chosen sigmoids (later the waves' sums), the pairs'
// weights and experts, the pair of each (touched expert, token), the touched experts
struct DownLds {
  int weight, id, pair, expert, total;
  __host__ __device__ DownLds(int T, int E, int k) {
    const int pairs = T * k, touched = pairs < E ? pairs : E;
    weight = pairs * 8 > 8 * 4 * 68 * 16 ? pairs * 8 : 8 * 4 * 68 * 16;
    id = weight + pairs * 4;
    pair = id + (pairs * 2 + 3) / 4 * 4;
    expert = pair + touched * kMaxTok * 2;
    total = expert + (touched * 2 + 3) / 4 * 4;
  }
};

}  // namespace

// Workgroup g: 32 features of y for all tokens.  Its waves take the column groups
// of the touched experts in turn, each product's FP32 result is added to the
// wave's sum under the token's weight, and the waves' sums meet in LDS.  Where H
// gives few workgroups, gridDim.y share the products.
//
// 16 tokens of 80 experts, H = 6144, I = 2048, 28 touched: 187 MB in 49 us (3.8
// TB/s).  A row of h is read by all H / 32 groups, and with both operands that is
// twice the weights' bytes through the L1; four workgroups a group took 47, two
// column groups ahead 52.
template <bool F32, bool HALF>
__global__ __launch_bounds__(512) void mx_layer_down_kernel(MxLayerArgs a) {
  constexpr int NW = 8;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t mask[8];
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const DownLds lds(a.T, a.E, a.k);
  float4* part = reinterpret_cast<float4*>(smem);  // [NW][4 * 68]
  double* chosen = reinterpret_cast<double*>(smem);
  float* weight = reinterpret_cast<float*>(smem + lds.weight);
  uint16_t* id = reinterpret_cast<uint16_t*>(smem + lds.id);
  int16_t* pair_of = reinterpret_cast<int16_t*>(smem + lds.pair);
  uint16_t* expert = reinterpret_cast<uint16_t*>(smem + lds.expert);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int pairs = a.T * a.k, most = min(pairs, a.E), col_tok = HALF ? n & 15 : n;
  if (tid < 8) mask[tid] = 0;
  for (int p = tid; p < pairs; p += 64 * NW) {
    id[p] = (uint16_t)a.topk_ids[p];
    chosen[p] = reinterpret_cast<const double*>(a.ws + ws.chosen)[p];
  }
  for (int i = tid; i < most * kMaxTok / 2; i += 64 * NW) reinterpret_cast<int*>(pair_of)[i] = -1;
  __syncthreads();
  for (int p = tid; p < pairs; p += 64 * NW) {
    atomicOr(&mask[id[p] >> 5], 1u << (id[p] & 31));
    const int t = p / a.k;
    double sum = 0.0;
    for (int j = 0; j < a.k; ++j) sum += chosen[t * a.k + j];
    weight[p] = (float)((double)a.rsf * chosen[p] / sum);
    if (blockIdx.x == 0 && blockIdx.y == 0) a.topk_w[p] = weight[p];
  }
  __syncthreads();
  int before[8], touched = 0;  // touched experts below each word of the mask
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    before[i] = touched;
    touched += __popc(mask[i]);
  }
  for (int p = tid; p < pairs; p += 64 * NW) {
    const int e = id[p];
    int i = __popc(mask[e >> 5] & ((1u << (e & 31)) - 1u));
#pragma unroll
    for (int q = 0; q < 8; ++q) i += (e >> 5) == q ? before[q] : 0;
    expert[i] = (uint16_t)e;  // every pair of the expert writes the same
    pair_of[i * kMaxTok + p / a.k] = (int16_t)p;
  }
  __syncthreads();

  const int KK = (a.I + 255) / 256, G = a.H / 32, g = blockIdx.x, all = touched * KK;
  const int parts = gridDim.y, each = (all + parts - 1) / parts, first = (int)blockIdx.y * each, items = min(all, first + each);
  const int64_t rest = (int64_t)pairs * KK * 256;  // from a large element of h to what is left of it
  struct Item {
    i32x4_t w[4];
    i32x8_t h[4];
    int sw, sh, p;
  };
  auto load = [&](int it, Item& d) {  // no branch before a load, as in gate_up
    it = min(it, all - 1);
    const int i = it / KK, c = it - i * KK;
    const int64_t at = ((int64_t)expert[i] * G + g) * KK + c;
    d.p = pair_of[i * kMaxTok + col_tok];
    const int64_t row = ((int64_t)max(d.p, 0) * KK + c) * 256;
    const uint8_t* hc = a.ws + ws.h_codes + row + f * 16 + (HALF && n >= 16 ? rest : 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint8_t* q = hc + s * 32;
      d.h[s] = join_halves(*reinterpret_cast<const i32x4_t*>(q), *reinterpret_cast<const i32x4_t*>(q + 128));
    }
    d.sh = *reinterpret_cast<const int*>(a.ws + ws.h_scales + row / 32 + f * 4);
#pragma unroll
    for (int s = 0; s < 4; ++s) d.w[s] = reinterpret_cast<const i32x4_t*>(a.w2_codes + at * kMxFragCodes)[s * 64 + l];
    d.sw = reinterpret_cast<const int*>(a.w2_scales + at * kMxFragScales)[l];
  };
  float16_t sum;
#pragma unroll
  for (int r = 0; r < 16; ++r) sum[r] = 0.0f;
  auto multiply = [&](const Item& d) {
    float16_t v;
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = 0.0f;
    v = mx8_mfma<0, HALF>(d.w[0], d.h[0], v, d.sw, d.sh);
    v = mx8_mfma<1, HALF>(d.w[1], d.h[1], v, d.sw, d.sh);
    v = mx8_mfma<2, HALF>(d.w[2], d.h[2], v, d.sw, d.sh);
    v = mx8_mfma<3, HALF>(d.w[3], d.h[3], v, d.sw, d.sh);
    const float wp = weight[max(d.p, 0)];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float with = fmaf(wp, v[r], sum[r]);
      sum[r] = d.p >= 0 ? with : sum[r];
    }
  };
  Item d0, d1;  // one ahead
  load(first + w, d0);
  for (int it = first + w; it < items; it += 2 * NW) {
    load(it + NW, d1);
    __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
    multiply(d0);
    if (it + NW >= items) break;
    load(it + 2 * NW, d0);
    __builtin_amdgcn_sched_barrier(0);
    multiply(d1);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    part[w * 272 + q * 68 + f * 34 + n] = make_float4(sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]);
  __syncthreads();
  const int tok = tid >> 3, p = tid & 7;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (tok < a.T) s = add_waves<NW, HALF>(part, p, tok);
  else if (parts == 1) return;
  if (parts > 1) {
    // The parts' sums meet in the workspace, and who comes last adds them, in the
    // parts' order.  They are written through the caches and waited for before the
    // count, so that nothing else has to be written back (a fence at the agent's
    // scope for it took 80 us).
    float* sums = reinterpret_cast<float*>(a.ws + ws.parts) + ((int64_t)g * parts * kMaxTok + tok) * 32 + 4 * p;
    if (tok < a.T) {
      const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        __hip_atomic_store(sums + (int64_t)blockIdx.y * kMaxTok * 32 + q, v[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) mask[0] = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.ws + ws.arrived) + g, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (mask[0] != (uint32_t)parts - 1 || tok >= a.T) return;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < parts; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] += __hip_atomic_load(sums + (int64_t)i * kMaxTok * 32 + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s = make_float4(v[0], v[1], v[2], v[3]);
  }
  const int64_t out = (int64_t)tok * a.H + g * 32 + 4 * p;
  if (F32) *reinterpret_cast<float4*>(static_cast<float*>(a.y) + out) = s;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + out) = make_uint2(bf16_pair(s.x, s.y), bf16_pair(s.z, s.w));
}

size_t mx_layer_workspace(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) { return LayerWs(T, E, k, H, I).total; }

hipError_t launch_mx_layer(const MxLayerArgs& a, hipStream_t st) {
  const int TT = a.T <= 1 ? 1 : a.T <= 2 ? 2 : 4, groups = (a.T + TT - 1) / TT;
  const int quant = (a.T * ((a.H + 255) / 256 * 32) + kScoreThreads - 1) / kScoreThreads;
  const dim3 grid((unsigned)(a.E + (quant + groups - 1) / groups), (unsigned)groups), block(kScoreThreads);
  auto* score = TT == 1 ? &mx_layer_score_kernel<1> : TT == 2 ? &mx_layer_score_kernel<2> : &mx_layer_score_kernel<4>;
  if (hipError_t e = launch_kernel(score, grid, block, 0, st, a)) return e;

  const bool half = a.T <= 16, rank = (int64_t)a.T * a.E * a.E <= kRankWork;
  if (!rank)
    if (hipError_t e = launch_kernel(&mx_layer_rank_kernel, dim3((unsigned)a.T), dim3(1024), 0, st, a)) return e;
  auto* gate_up = half ? (rank ? &mx_layer_gate_up_kernel<true, true> : &mx_layer_gate_up_kernel<false, true>)
                       : (rank ? &mx_layer_gate_up_kernel<true, false> : &mx_layer_gate_up_kernel<false, false>);
  const int64_t most = (int64_t)(a.T * a.k < a.E ? a.T * a.k : a.E) * (a.I / 32);
  if (hipError_t e = launch_kernel(gate_up, dim3((unsigned)(most < 512 ? most : 512)), dim3(256), 0, st, a)) return e;

  auto* down = half ? (a.y_f32 ? &mx_layer_down_kernel<true, true> : &mx_layer_down_kernel<false, true>)
                    : (a.y_f32 ? &mx_layer_down_kernel<true, false> : &mx_layer_down_kernel<false, false>);
  if (hipError_t e = set_max_dynamic_lds(reinterpret_cast<const void*>(down), DownLds(kMaxTok, 256, 256).total)) return e;
  return launch_kernel(down, dim3((unsigned)(a.H / 32), (unsigned)down_parts(a.T, a.E, a.k, a.H, a.I)), dim3(512), (size_t)DownLds(a.T, a.E, a.k).total, st, a);
}

}  // namespace moe
