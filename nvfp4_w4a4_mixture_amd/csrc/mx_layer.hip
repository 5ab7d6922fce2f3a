// The whole routed-expert layer for up to 32 tokens, in three kernels: the
// router's scores with the quantisation of x; gate_up with the selection; down
// with the combine.
//
//   z[t, e] = x[t] . W_r[e] in FP64, s = sigmoid(z)
//   the k experts of a token: largest s + bias first, ties to the lower index
//   w[t, e] = rsf * s / (sum of the k s)
//   y[t] = sum over e of w[t, e] * W2[e] . q(silu(W_gate[e] . q(x[t])) * (W_up[e] . q(x[t])))
//
// With so few tokens the touched experts' weights bound it (and launches, where
// the layer is small), so the tokens are the 32 columns of one MFMA tile whatever
// they chose: no permutation of pairs is needed, columns that did not choose an
// expert are multiplied as zeros and left out of the sums, and the sum over the
// experts stays in FP32 accumulators, in the order of the experts.  A kernel's
// end is the only synchronisation; no atomics decide an order.
#include "launch.h"
#include "mx_common.h"
#include "mx_product.h"

namespace moe {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kMaxTok = (int)kLayerMaxTokens;
constexpr int kSparse = 512;  // scores that a workgroup of the sparse gate_up ranks

// Everything between the kernels: keys (the order of the scores) and sigmoids of
// all experts, the chosen sigmoids by slot, x and h in MXFP8.
struct LayerWs {
  size_t key, sig, chosen, x_codes, x_scales, h_codes, h_scales, total;
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
    x_codes = take(t * Hp);
    x_scales = take(t * Hp / 32);
    h_codes = take(p * Ip);
    h_scales = take(p * Ip / 32);
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
    reinterpret_cast<uint2*>(a.ws + ws.x_codes)[i] = make_uint2(mx8_encode4(f, byte), mx8_encode4(f + 4, byte));
    if ((tid & 3) == 0) (a.ws + ws.x_scales)[i >> 2] = (uint8_t)byte;
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

// Workgroup (g, i): the 32 h columns of group g of one expert for the tokens that
// chose it, as mx_stream_kernel's gate_up.  A token chose an expert if fewer than k
// rank before it, and that number is its slot: found here from the token's keys,
// so that no kernel stands between the scores and the weights.  SPARSE (few pairs
// beside the experts): i counts the touched experts, which every workgroup finds
// from all ranks; else i is the expert, and those that nobody chose end at once.
// HALF: up to 16 tokens, both operands of a token in one (see mx_stream_kernel).
template <bool SPARSE, bool HALF>
__global__ __launch_bounds__(256) void mx_layer_gate_up_kernel(MxLayerArgs a) {
  constexpr int NW = 4;
  __shared__ float4 part[NW][2][4 * 68];
  __shared__ int rank[kMaxTok];
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int blk = blockIdx.x, col_tok = HALF ? n & 15 : n;
  const long long* key = reinterpret_cast<const long long*>(a.ws + ws.key);
  if (tid < kMaxTok) rank[tid] = tid < a.T ? 0 : a.E;
  int e = blockIdx.y;
  if constexpr (SPARSE) {  // T * E <= kSparse scores
    __shared__ long long keys[kSparse];
    __shared__ uint16_t slot[kSparse];
    __shared__ uint32_t mask[8];
    if (tid < 8) mask[tid] = 0;
    for (int i = tid; i < a.T * a.E; i += 256) keys[i] = key[i];
    __syncthreads();
    for (int i = tid; i < a.T * a.E; i += 256) {
      const int t = i / a.E, o = i - t * a.E;
      const long long mine = keys[i], *row = keys + t * a.E;
      int r = 0;
#pragma unroll 8
      for (int q = 0; q < a.E; ++q) r += (int)(row[q] > mine) | ((int)(row[q] == mine) & (int)(q < o));
      slot[i] = (uint16_t)r;
      if (r < a.k) atomicOr(&mask[o >> 5], 1u << (o & 31));
    }
    __syncthreads();
    int left = blockIdx.y;  // of the touched experts below the one sought
    e = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = mask[i];
      const int c = __popc(m);
      if (e < 0 && left < c) {
        for (; left > 0; --left) m &= m - 1;
        e = 32 * i + __builtin_ctz(m);
      }
      left -= c;
    }
    if (e < 0) return;
    if (tid < a.T) rank[tid] = slot[tid * a.E + e];
    __syncthreads();
  } else {
    __syncthreads();
    for (int i = tid; i < a.T * a.E; i += 256) {
      const int t = i / a.E, o = i - t * a.E;
      const long long mine = key[t * a.E + e], other = key[i];
      if (other > mine || (other == mine && o < e)) atomicAdd(&rank[t], 1);  // a count: the order does not matter
    }
    __syncthreads();
  }
  const bool chosen = rank[col_tok] < a.k;
  if (__ballot(chosen) == 0) return;  // the same in every wave
  if (blk == 0 && tid < a.T && rank[tid] < a.k) {
    const int p = tid * a.k + rank[tid];
    a.topk_ids[p] = e;
    reinterpret_cast<double*>(a.ws + ws.chosen)[p] = reinterpret_cast<const double*>(a.ws + ws.sig)[tid * a.E + e];
  }

  const int KK = (a.H + 255) / 256, G = a.I / 16;
  const uint8_t* wc[2];
  const uint8_t* wsc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t g = (int64_t)e * G + blk + i * (G / 2);
    wc[i] = a.w13_codes + g * KK * kMxFragCodes;
    wsc[i] = a.w13_scales + g * KK * kMxFragScales;
  }
  const uint8_t* xc = a.ws + ws.x_codes + (int64_t)col_tok * KK * 256 + f * 16;
  const uint8_t* xs = a.ws + ws.x_scales + (int64_t)col_tok * KK * 8 + f * 4;
  struct Cols {
    i32x8_t x[4];
    i32x4_t w[2][4];
    int sw[2], sx;
  };
  auto load = [&](int c, Cols& d) {
    d.sx = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) d.x[s] = i32x8_t{0, 0, 0, 0, 0, 0, 0, 0};
    if (chosen) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        d.x[s] = join_halves(*reinterpret_cast<const i32x4_t*>(xc + c * 256 + 32 * s),
                             *reinterpret_cast<const i32x4_t*>(xc + c * 256 + 128 + 32 * s));
      d.sx = *reinterpret_cast<const int*>(xs + c * 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int s = 0; s < 4; ++s) d.w[i][s] = reinterpret_cast<const i32x4_t*>(wc[i] + (int64_t)c * kMxFragCodes)[s * 64 + l];
      d.sw[i] = reinterpret_cast<const int*>(wsc[i] + (int64_t)c * kMxFragScales)[l];
    }
  };
  float16_t acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  auto multiply = [&](Cols& d) {
    if constexpr (HALF) {
#pragma unroll
      for (int s = 0; s < 4; ++s) d.x[s] = mx8_part(d.x[s], n >= 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      acc[i] = act_mfma<0, !HALF>(d.w[i][0], d.x[0], acc[i], d.sw[i], d.sx);
      acc[i] = act_mfma<1, !HALF>(d.w[i][1], d.x[1], acc[i], d.sw[i], d.sx);
      acc[i] = act_mfma<2, !HALF>(d.w[i][2], d.x[2], acc[i], d.sw[i], d.sx);
      acc[i] = act_mfma<3, !HALF>(d.w[i][3], d.x[3], acc[i], d.sw[i], d.sx);
    }
  };
  Cols d0, d1;  // one column group ahead
  if (w < KK) load(w, d0);
  for (int c = w; c < KK; c += 2 * NW) {
    if (c + NW < KK) load(c + NW, d1);
    multiply(d0);
    if (c + NW < KK) {
      if (c + 2 * NW < KK) load(c + 2 * NW, d0);
      multiply(d1);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      part[w][i][q * 68 + f * 34 + n] = make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
  __syncthreads();
  const int tok = tid >> 3, p = tid & 7;  // features 4 p .. 4 p + 3 of one token
  if (rank[tok] >= a.k) return;           // eight lanes together
  float v[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float4 s = part[0][i][(p & 3) * 68 + (p >> 2) * 34 + tok];
#pragma unroll
    for (int k = 1; k < (HALF ? 2 : 1) * NW; ++k) {
      const float4 u = part[k % NW][i][(p & 3) * 68 + (p >> 2) * 34 + tok + (k < NW ? 0 : 16)];
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
  float h[4];
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    h[q] = silu(v[0][q]) * v[1][q];
    m = max(m, abs_bits(h[q]));
  }
  m = quad_max(m);
  m = max(m, lane_dpp<kLaneHalfMirror>(m));
  const uint32_t byte = mx8_scale_byte(m);
  const int Ip = (a.I + 255) / 256 * 256;
  const int64_t row = tok * a.k + rank[tok];
  uint8_t* hc = a.ws + ws.h_codes + row * Ip;
  uint8_t* hs = a.ws + ws.h_scales + row * (Ip / 32);
  reinterpret_cast<uint32_t*>(hc)[blk * 8 + p] = mx8_encode4(h, byte);
  if (p == 0) hs[blk] = (uint8_t)byte;
  if (blk == 0) {  // the padding past I is zero
    for (int b = a.I / 32 + p; b < Ip / 32; b += 8) {
      reinterpret_cast<uint4*>(hc)[2 * b] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(hc)[2 * b + 1] = make_uint4(0, 0, 0, 0);
      hs[b] = 0;
    }
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
// wave's sum under the token's weight, and the waves' sums meet in LDS.
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
    if (blockIdx.x == 0) a.topk_w[p] = weight[p];
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

  const int KK = (a.I + 255) / 256, G = a.H / 32, g = blockIdx.x, items = touched * KK;
  struct Item {
    i32x4_t w[4];
    i32x8_t h[4];
    int sw, sh, p;
  };
  auto load = [&](int it, Item& d) {
    const int i = it / KK, c = it - i * KK;
    const int64_t at = ((int64_t)expert[i] * G + g) * KK + c;
    d.p = pair_of[i * kMaxTok + col_tok];
    d.sh = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) d.h[s] = i32x8_t{0, 0, 0, 0, 0, 0, 0, 0};
    if (d.p >= 0) {
      const uint8_t* hc = a.ws + ws.h_codes + ((int64_t)d.p * KK + c) * 256 + f * 16;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        d.h[s] = join_halves(*reinterpret_cast<const i32x4_t*>(hc + 32 * s), *reinterpret_cast<const i32x4_t*>(hc + 128 + 32 * s));
      d.sh = *reinterpret_cast<const int*>(a.ws + ws.h_scales + ((int64_t)d.p * KK + c) * 8 + f * 4);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) d.w[s] = reinterpret_cast<const i32x4_t*>(a.w2_codes + at * kMxFragCodes)[s * 64 + l];
    d.sw = reinterpret_cast<const int*>(a.w2_scales + at * kMxFragScales)[l];
  };
  float16_t sum;
#pragma unroll
  for (int r = 0; r < 16; ++r) sum[r] = 0.0f;
  auto multiply = [&](Item& d) {
    if constexpr (HALF) {
#pragma unroll
      for (int s = 0; s < 4; ++s) d.h[s] = mx8_part(d.h[s], n >= 16);
    }
    float16_t v;
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = 0.0f;
    v = act_mfma<0, !HALF>(d.w[0], d.h[0], v, d.sw, d.sh);
    v = act_mfma<1, !HALF>(d.w[1], d.h[1], v, d.sw, d.sh);
    v = act_mfma<2, !HALF>(d.w[2], d.h[2], v, d.sw, d.sh);
    v = act_mfma<3, !HALF>(d.w[3], d.h[3], v, d.sw, d.sh);
    if (d.p >= 0) {
      const float wp = weight[d.p];
#pragma unroll
      for (int r = 0; r < 16; ++r) sum[r] = fmaf(wp, v[r], sum[r]);
    }
  };
  Item d0, d1;  // one ahead
  if (w < items) load(w, d0);
  for (int it = w; it < items; it += 2 * NW) {
    if (it + NW < items) load(it + NW, d1);
    multiply(d0);
    if (it + NW < items) {
      if (it + 2 * NW < items) load(it + 2 * NW, d0);
      multiply(d1);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    part[w * 272 + q * 68 + f * 34 + n] = make_float4(sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]);
  __syncthreads();
  const int tok = tid >> 3, p = tid & 7;
  if (tok >= a.T) return;
  float4 s = part[(p & 3) * 68 + (p >> 2) * 34 + tok];
#pragma unroll
  for (int k = 1; k < (HALF ? 2 : 1) * NW; ++k) {
    const float4 u = part[(k % NW) * 272 + (p & 3) * 68 + (p >> 2) * 34 + tok + (k < NW ? 0 : 16)];
    s.x += u.x;
    s.y += u.y;
    s.z += u.z;
    s.w += u.w;
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

  const bool half = a.T <= 16, sparse = a.T * a.k * 4 <= a.E && a.T * a.E <= kSparse;
  auto* gate_up = half ? (sparse ? &mx_layer_gate_up_kernel<true, true> : &mx_layer_gate_up_kernel<false, true>)
                       : (sparse ? &mx_layer_gate_up_kernel<true, false> : &mx_layer_gate_up_kernel<false, false>);
  const dim3 tiles((unsigned)(a.I / 32), (unsigned)(sparse ? a.T * a.k : a.E));
  if (hipError_t e = launch_kernel(gate_up, tiles, dim3(256), 0, st, a)) return e;

  auto* down = half ? (a.y_f32 ? &mx_layer_down_kernel<true, true> : &mx_layer_down_kernel<false, true>)
                    : (a.y_f32 ? &mx_layer_down_kernel<true, false> : &mx_layer_down_kernel<false, false>);
  const int most = DownLds(kMaxTok, 256, 256).total;
  if (hipError_t e = set_max_dynamic_lds(reinterpret_cast<const void*>(down), most)) return e;
  return launch_kernel(down, dim3((unsigned)(a.H / 32)), dim3(512), (size_t)DownLds(a.T, a.E, a.k).total, st, a);
}

}  // namespace moe
