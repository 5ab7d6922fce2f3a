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

constexpr int kScoreThreads = 512;
constexpr int kMaxTok = (int)kLayerMaxTokens;

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

// Workgroup e < E: the scores of expert e for all tokens; those after it quantise
// x.  A product of two BF16 values is exact in FP64; the sum's order is fixed:
// each thread's columns, then lanes, then waves.  TT: tokens rounded up to a power
// of two; after the exchanges lane group t of 64 / TT lanes holds token t.
template <int TT>
__global__ __launch_bounds__(kScoreThreads) void mx_layer_score_kernel(MxLayerArgs a) {
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if ((int)blockIdx.x >= a.E) {
    const int chunks = (a.H + 255) / 256 * 32;  // of 8 columns, of a padded row
    const int i = ((int)blockIdx.x - a.E) * kScoreThreads + tid;
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
  const int e = blockIdx.x;
  double acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0;
  for (int c = tid * 8; c < a.H; c += kScoreThreads * 8) {
    const u32x4_any2_t wv = load8(a.w_router + (int64_t)e * a.H + c);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const u32x4_any2_t xv = load8(a.x + (int64_t)min(t, a.T - 1) * a.ldx + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t] = __builtin_fma((double)element(xv, j), (double)element(wv, j), acc[t]);
    }
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
  if (tid >= a.T) return;
  double z = red[0][tid];
#pragma unroll
  for (int i = 1; i < kScoreThreads / 64; ++i) z += red[i][tid];
  const double s = 1.0 / (1.0 + exp(-z));
  reinterpret_cast<double*>(a.ws + ws.sig)[tid * a.E + e] = s;
  reinterpret_cast<long long*>(a.ws + ws.key)[tid * a.E + e] = score_key(s + (double)a.bias[e]);
}

// Workgroup (g, e): the 32 h columns of group g of expert e for the tokens that
// chose it, as mx_stream_kernel's gate_up.  A token chose e if fewer than k
// experts rank before it, and that number is its slot: found here from the
// token's keys, so that no kernel stands between the scores and the weights.
__global__ __launch_bounds__(256) void mx_layer_gate_up_kernel(MxLayerArgs a) {
  constexpr int NW = 4;
  __shared__ float4 part[NW][2][4 * 68];
  __shared__ int rank[kMaxTok];
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int e = blockIdx.y, blk = blockIdx.x;
  if (tid < kMaxTok) rank[tid] = tid < a.T ? 0 : a.E;
  __syncthreads();
  const long long* key = reinterpret_cast<const long long*>(a.ws + ws.key);
  for (int i = tid; i < a.T * a.E; i += 256) {
    const int t = i / a.E, o = i - t * a.E;
    const long long mine = key[t * a.E + e], other = key[i];
    if (other > mine || (other == mine && o < e)) atomicAdd(&rank[t], 1);  // a count: the order does not matter
  }
  __syncthreads();
  const bool chosen = rank[n] < a.k;
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
  const uint8_t* xc = a.ws + ws.x_codes + (int64_t)n * KK * 256 + f * 16;
  const uint8_t* xs = a.ws + ws.x_scales + (int64_t)n * KK * 8 + f * 4;
  float16_t acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  for (int64_t c = w; c < KK; c += NW) {
    i32x4_t wf[2][4];
    int sw[2], sx = 0;
    i32x8_t xf[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int s = 0; s < 4; ++s) wf[i][s] = reinterpret_cast<const i32x4_t*>(wc[i] + c * kMxFragCodes)[s * 64 + l];
      sw[i] = reinterpret_cast<const int*>(wsc[i] + c * kMxFragScales)[l];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) xf[s] = i32x8_t{0, 0, 0, 0, 0, 0, 0, 0};
    if (chosen) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        xf[s] = join_halves(*reinterpret_cast<const i32x4_t*>(xc + c * 256 + 32 * s),
                            *reinterpret_cast<const i32x4_t*>(xc + c * 256 + 128 + 32 * s));
      sx = *reinterpret_cast<const int*>(xs + c * 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      acc[i] = act_mfma<0, true>(wf[i][0], xf[0], acc[i], sw[i], sx);
      acc[i] = act_mfma<1, true>(wf[i][1], xf[1], acc[i], sw[i], sx);
      acc[i] = act_mfma<2, true>(wf[i][2], xf[2], acc[i], sw[i], sx);
      acc[i] = act_mfma<3, true>(wf[i][3], xf[3], acc[i], sw[i], sx);
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

// LDS of the down kernel: the waves' sums, then the pair of each (touched expert,
// token), the pairs' weights, the touched experts
struct DownLds {
  int pair, weight, expert, total;
  __host__ __device__ DownLds(int T, int E, int k) {
    const int pairs = T * k, touched = pairs < E ? pairs : E;
    pair = 8 * 4 * 68 * 16;
    weight = pair + touched * kMaxTok * 2;
    expert = weight + pairs * 4;
    total = expert + (touched * 2 + 3) / 4 * 4;
  }
};

}  // namespace

// Workgroup g: 32 features of y for all tokens.  Its waves take the column groups
// of the touched experts in turn, each product's FP32 result is added to the
// wave's sum under the token's weight, and the waves' sums meet in LDS.
template <bool F32>
__global__ __launch_bounds__(512) void mx_layer_down_kernel(MxLayerArgs a) {
  constexpr int NW = 8;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t mask[8];
  const LayerWs ws(a.T, a.E, a.k, a.H, a.I);
  const DownLds lds(a.T, a.E, a.k);
  float4* part = reinterpret_cast<float4*>(smem);  // [NW][4 * 68]
  int16_t* pair_of = reinterpret_cast<int16_t*>(smem + lds.pair);
  float* weight = reinterpret_cast<float*>(smem + lds.weight);
  uint16_t* expert = reinterpret_cast<uint16_t*>(smem + lds.expert);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, n = l & 31, f = l >> 5;
  const int pairs = a.T * a.k;
  if (tid < 8) mask[tid] = 0;
  __syncthreads();
  const double* chosen = reinterpret_cast<const double*>(a.ws + ws.chosen);
  for (int p = tid; p < pairs; p += 64 * NW) {
    const int e = a.topk_ids[p], t = p / a.k;
    atomicOr(&mask[e >> 5], 1u << (e & 31));
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
  auto index = [&](int e) {
    int b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) b = (e >> 5) == i ? before[i] : b;
    return b + __popc(mask[e >> 5] & ((1u << (e & 31)) - 1u));
  };
  if (tid < a.E && ((mask[tid >> 5] >> (tid & 31)) & 1)) expert[index(tid)] = (uint16_t)tid;
  for (int i = tid; i < touched * kMaxTok; i += 64 * NW) pair_of[i] = -1;
  __syncthreads();
  for (int p = tid; p < pairs; p += 64 * NW) pair_of[index(a.topk_ids[p]) * kMaxTok + p / a.k] = (int16_t)p;
  __syncthreads();

  const int KK = (a.I + 255) / 256, G = a.H / 32, g = blockIdx.x;
  float16_t sum;
#pragma unroll
  for (int r = 0; r < 16; ++r) sum[r] = 0.0f;
  for (int it = w; it < touched * KK; it += NW) {
    const int i = it / KK, c = it - i * KK;
    const int64_t at = ((int64_t)expert[i] * G + g) * KK + c;
    const int p = pair_of[i * kMaxTok + n];
    i32x4_t wf[4];
    i32x8_t hf[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) wf[s] = reinterpret_cast<const i32x4_t*>(a.w2_codes + at * kMxFragCodes)[s * 64 + l];
    const int sw = reinterpret_cast<const int*>(a.w2_scales + at * kMxFragScales)[l];
    int sh = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) hf[s] = i32x8_t{0, 0, 0, 0, 0, 0, 0, 0};
    float wp = 0.0f;
    if (p >= 0) {
      const uint8_t* hc = a.ws + ws.h_codes + ((int64_t)p * KK + c) * 256 + f * 16;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        hf[s] = join_halves(*reinterpret_cast<const i32x4_t*>(hc + 32 * s), *reinterpret_cast<const i32x4_t*>(hc + 128 + 32 * s));
      sh = *reinterpret_cast<const int*>(a.ws + ws.h_scales + ((int64_t)p * KK + c) * 8 + f * 4);
      wp = weight[p];
    }
    float16_t v;
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = 0.0f;
    v = act_mfma<0, true>(wf[0], hf[0], v, sw, sh);
    v = act_mfma<1, true>(wf[1], hf[1], v, sw, sh);
    v = act_mfma<2, true>(wf[2], hf[2], v, sw, sh);
    v = act_mfma<3, true>(wf[3], hf[3], v, sw, sh);
    if (p >= 0) {
#pragma unroll
      for (int r = 0; r < 16; ++r) sum[r] = fmaf(wp, v[r], sum[r]);
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
  for (int k = 1; k < NW; ++k) {
    const float4 u = part[k * 272 + (p & 3) * 68 + (p >> 2) * 34 + tok];
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
  const unsigned quant = (unsigned)((a.T * ((a.H + 255) / 256 * 32) + kScoreThreads - 1) / kScoreThreads);
  const dim3 grid((unsigned)a.E + quant), block(kScoreThreads);
  hipError_t e;
  if (a.T <= 1) e = launch_kernel(mx_layer_score_kernel<1>, grid, block, 0, st, a);
  else if (a.T <= 2) e = launch_kernel(mx_layer_score_kernel<2>, grid, block, 0, st, a);
  else if (a.T <= 4) e = launch_kernel(mx_layer_score_kernel<4>, grid, block, 0, st, a);
  else if (a.T <= 8) e = launch_kernel(mx_layer_score_kernel<8>, grid, block, 0, st, a);
  else if (a.T <= 16) e = launch_kernel(mx_layer_score_kernel<16>, grid, block, 0, st, a);
  else e = launch_kernel(mx_layer_score_kernel<32>, grid, block, 0, st, a);
  if (e != hipSuccess) return e;
  if ((e = launch_kernel(mx_layer_gate_up_kernel, dim3((unsigned)(a.I / 32), (unsigned)a.E), dim3(256), 0, st, a)) != hipSuccess)
    return e;
  auto* down = a.y_f32 ? &mx_layer_down_kernel<true> : &mx_layer_down_kernel<false>;
  const DownLds lds(a.T, a.E, a.k);
  if ((e = set_max_dynamic_lds(reinterpret_cast<const void*>(down), DownLds(kMaxTok, 256, 256).total)) != hipSuccess) return e;
  return launch_kernel(down, dim3((unsigned)(a.H / 32)), dim3(512), (size_t)lds.total, st, a);
}

}  // namespace moe
