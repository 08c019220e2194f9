// Routing of tokens to experts, and the combination of a token's experts.
//
// Routing: the k best of E logits per token, then a counting sort of the T k
// choices by expert.  The sort uses no atomics and no scratch memory: for each
// expert one block reads all choices (from the L2; 256 KiB for 8192 tokens of 8),
// counts those of lower experts, which gives the expert's first row, and ranks
// its own in token order.  That is E times the reading that a histogram in two
// launches would do, and one launch less.
//
// Combination: bound by HBM, T (k + 2) rows.
#include "../../include/prune24_experts.h"
#include "p24_api_internal.hpp"
#include "p24_f8.hpp"

namespace p24 {

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  const float* bias;
  int* experts;
  float* weights;
  int* offsets;
  int* tokens;
  int* positions;
  int T, E, k;
  int score, normalize;
  float scale;
};

// Keys whose unsigned order is the order of the scores: NaN above +inf, -0 as +0.  No score has key 0.
__device__ __forceinline__ uint32_t score_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t score_key(double v) {
  if (v != v) return ~0ull;
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// Reductions over the G lanes of a token, 16 or all 64, the result in each: quads, mirrored halves and
// rows of 16, then the wave's four rows.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int SWAP1 = 0xB1, SWAP2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140;   // quad_perm 1 0 3 2, 2 3 0 1, ..
template <int G, typename F>
__device__ __forceinline__ uint32_t reduce(uint32_t v, F&& f) {
  static_assert(G == 16 || G == 64, "a row of lanes, or a wave");
  v = f(v, dpp<SWAP1>(v));
  v = f(v, dpp<SWAP2>(v));
  v = f(v, dpp<HALF_MIRROR>(v));
  v = f(v, dpp<MIRROR>(v));
  if constexpr (G == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return reduce<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t min_of(uint32_t v) {
  return reduce<G>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int G>
__device__ __forceinline__ uint64_t max_of(uint64_t v) {
  const uint32_t hi = max_of<G>((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | max_of<G>((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
template <int G>
__device__ __forceinline__ float sum_of(float v) {
  return __uint_as_float(reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__device__ __forceinline__ float logit_at(const uint16_t* row, int e) { return __uint_as_float((uint32_t)row[e] << 16); }
__device__ __forceinline__ float logit_at(const float* row, int e) { return row[e]; }

// One token on G lanes, V experts each (4 G c + 4 lane + [0, 4) for c < V / 4).  Slot j's expert and weight
// end up in lane j % G, entry j / G.
template <typename T, typename Key, int G, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int (&expert)[2], float (&weight)[2]) {
  constexpr bool WIDE = sizeof(Key) == 8;   // sigmoid and bias
  const int lane = threadIdx.x % G;
  const T* row = (const T*)a.logits + t * a.ldl;
  Key key[V];
  float l[WIDE ? 1 : V];
#pragma unroll
  for (int c = 0; c < V / 4; ++c) {
    const int e = 4 * G * c + 4 * lane;
    float x[4], b[4];
    load_row<4>(row + e, a.E - e, x);
    if constexpr (WIDE) load_row<4>(a.bias + e, a.E - e, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool open = e + i < a.E && x[i] != -INFINITY;
      if constexpr (WIDE) {
        key[4 * c + i] = open ? score_key(1.0 / (1.0 + exp(-(double)x[i])) + (double)b[i]) : 0;
      } else {
        key[4 * c + i] = open ? score_key(x[i]) : 0;
        l[4 * c + i] = open ? x[i] : -INFINITY;
      }
    }
    if constexpr (WIDE) __builtin_amdgcn_sched_barrier(0);   // four exponentials at a time: their registers
  }
  expert[0] = expert[1] = -1;
  int first = -1;    // the best expert
  for (int j = 0; j < a.k; ++j) {
    Key best = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (key[v] > best) {     // the lower of equals
        best = key[v];
        at = v;
      }
    }
    const int mine = 4 * G * (at / 4) + 4 * lane + at % 4;
    const Key top = max_of<G>(best);
    if (top == 0) break;       // of all the token's lanes alike
    const int e = (int)min_of<G>(best == top ? (uint32_t)mine : 0xFFFFFFFFu);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (4 * G * (v / 4) + 4 * lane + v % 4 == e) key[v] = 0;
    if (j == 0) first = e;
    if (lane == j % G) {
      if (j < G) expert[0] = e;
      else expert[1] = e;
    }
  }
  // weights, from the logits themselves
  float w[2] = {0.0f, 0.0f};
  float all = 0.0f;
  if (a.score == P24_SCORE_SOFTMAX) {
    const float top = first >= 0 ? logit_at(row, first) : 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) w[s] = expf(logit_at(row, expert[s]) - top);
    if constexpr (!WIDE) {
      if (!a.normalize) {
#pragma unroll
        for (int v = 0; v < V; ++v) all += expf(l[v] - top);   // closed ones: exp(-inf)
        all = sum_of<G>(all);
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) w[s] = 1.0f / (1.0f + expf(-logit_at(row, expert[s])));
    all = 1.0f;
  }
  if (a.normalize) all = sum_of<G>(w[0] + w[1]);
#pragma unroll
  for (int s = 0; s < 2; ++s) weight[s] = expert[s] >= 0 ? w[s] / all * a.scale : 0.0f;
}

template <typename T, typename Key, int G, int V>
__global__ __launch_bounds__(256) void k_route_top(const RouteArgs a) {
  const int t = blockIdx.x * (256 / G) + threadIdx.x / G, lane = threadIdx.x % G;
  if (t >= a.T) return;
  int e[2];
  float w[2];
  route_token<T, Key, G, V>(a, t, e, w);
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (G * s + lane < a.k) {
      a.experts[(int64_t)t * a.k + G * s + lane] = e[s];
      a.weights[(int64_t)t * a.k + G * s + lane] = w[s];
    }
}

// A few tokens in one block: T k <= 512 choices, each ranked against all others in LDS.
constexpr int FEW = 512;
template <typename T, typename Key, int G, int V>
__global__ __launch_bounds__(512) void k_route_few(const RouteArgs a) {
  __shared__ __attribute__((aligned(16))) int id[FEW];     // slots without an expert rank last
  const int n = a.T * a.k, lane = threadIdx.x % G;
  for (int i = n + threadIdx.x; i < FEW; i += blockDim.x) id[i] = INT32_MAX;
  for (int t = threadIdx.x / G; t < a.T; t += blockDim.x / G) {
    int e[2];
    float w[2];
    route_token<T, Key, G, V>(a, t, e, w);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (G * s + lane < a.k) {
        const int i = t * a.k + G * s + lane;
        a.experts[i] = e[s];
        a.weights[i] = w[s];
        id[i] = e[s] < 0 ? INT32_MAX : e[s];
      }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int mine = id[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += id[j] < mine || (id[j] == mine && j < i);
    a.positions[i] = mine == INT32_MAX ? -1 : rank;
    a.tokens[rank] = mine == INT32_MAX ? -1 : i / a.k;
  }
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
    int below = 0;
    for (int j = 0; j < n; ++j) below += id[j] < e;
    a.offsets[e] = below;
  }
}

// Block e of E + 1: expert e's offset and rows; the last one the slots without an expert.  The block's 16
// waves each take a run of the choices in order, 256 at a time (four a lane); a lane keeps which of
// its first 64 are the expert's, and reads those past them again.
__global__ __launch_bounds__(1024) void k_route_sort(const RouteArgs a) {
  constexpr int WAVES = 16, KEPT = 16;
  __shared__ int below_of[WAVES], mine_of[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool rest = (int)blockIdx.x == a.E;
  const int target = rest ? -1 : (int)blockIdx.x;
  const int n = a.T * a.k;
  const int rounds = ((n + 255) / 256 + WAVES - 1) / WAVES;      // of a wave
  const int first = wave * rounds * 256;
  auto matches = [&](int r, int& below) {
    const int i = first + r * 256 + 4 * lane;
    int id[4] = {-2, -2, -2, -2};
    if (i + 4 <= n) {
      const int4 v = *reinterpret_cast<const int4*>(a.experts + i);
      id[0] = v.x;
      id[1] = v.y;
      id[2] = v.z;
      id[3] = v.w;
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < n) id[u] = a.experts[i + u];
    }
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      m |= (uint32_t)(id[u] == target) << u;
      below += rest ? id[u] >= 0 : (id[u] >= 0 && id[u] < target);
    }
    return m;
  };
  int below = 0, mine = 0;
  uint64_t kept = 0;
#pragma unroll 4
  for (int r = 0; r < rounds; ++r) {
    const uint32_t m = matches(r, below);
    mine += __popc(m);
    if (r < KEPT) kept |= (uint64_t)m << (4 * r);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    below += __shfl_xor(below, o);
    mine += __shfl_xor(mine, o);
  }
  if (lane == 0) {
    below_of[wave] = below;
    mine_of[wave] = mine;
  }
  __syncthreads();
  int start = 0, before = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    start += below_of[w];
    before += w < wave ? mine_of[w] : 0;
  }
  if (threadIdx.x == 0) a.offsets[blockIdx.x] = start;
  int row = start + before;
  for (int r = 0; r < rounds && mine; ++r) {
    int unused = 0;
    const uint32_t m = r < KEPT ? (uint32_t)(kept >> (4 * r)) & 15u : matches(r, unused);
    uint64_t who[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) who[u] = __ballot(m >> u & 1);
    const uint64_t ahead = (1ull << lane) - 1;
    int at = row;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      at += __popcll(who[u] & ahead);
      row += __popcll(who[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (m >> u & 1) {
        const int i = first + r * 256 + 4 * lane + u;
        a.tokens[at] = rest ? -1 : i / a.k;
        a.positions[i] = rest ? -1 : at;
        ++at;
      }
    }
  }
}

template <typename T, typename Key, int G, int V>
static p24_status launch_route(const RouteArgs& a, hipStream_t st) {
  if ((int64_t)a.T * a.k <= FEW) {
    const int threads = a.T >= 16 || a.E > 256 ? 512 : 256;
    hipLaunchKernelGGL((k_route_few<T, Key, G, V>), dim3(1), dim3(threads), 0, st, a);
    return launch_status();
  }
  hipLaunchKernelGGL((k_route_top<T, Key, G, V>), dim3((unsigned)(((int64_t)a.T * G + 255) / 256)), dim3(256), 0, st, a);
  const p24_status s = launch_status();
  if (s != P24_OK) return s;
  hipLaunchKernelGGL(k_route_sort, dim3((unsigned)a.E + 1), dim3(1024), 0, st, a);
  return launch_status();
}

template <typename T, typename Key>
static p24_status route_by_experts(const RouteArgs& a, hipStream_t st) {
  if (a.E <= 64) return launch_route<T, Key, 16, 4>(a, st);
  if (a.E <= 128) return launch_route<T, Key, 16, 8>(a, st);
  if (a.E <= 256) return launch_route<T, Key, 16, 16>(a, st);
  return launch_route<T, Key, 64, 16>(a, st);
}

struct CombineArgs {
  const void* Z;
  const int* positions;
  const float* weights;
  const void* residual;
  void* y;
  int64_t ldz, ldr, ldy;
  int T, k, width, rows;
};

// A token's row in parts of 256 chunks of 16 bytes of Z, or (ONE) a token per wave where that holds it.
template <typename ZT, typename OutT, bool ONE>
__global__ __launch_bounds__(256) void k_combine(const CombineArgs a) {
  constexpr int V = 16 / sizeof(ZT), U = 4;
  const int t = ONE ? __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + threadIdx.x / 64) : blockIdx.x;
  const int c = (ONE ? threadIdx.x % 64 : blockIdx.y * 256 + threadIdx.x) * V;
  if (t >= a.T || c >= a.width) return;
  const int* p = a.positions + (int64_t)t * a.k;
  const float* w = a.weights + (int64_t)t * a.k;
  float r[V];
  if (a.residual) load_row<V>((const OutT*)a.residual + t * a.ldr + c, a.width - c, r);
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += U) {
    float z[U][V];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = j0 + u < a.k ? p[j0 + u] : -1;
      on[u] = (uint32_t)at < (uint32_t)a.rows;
      if (on[u]) load_row<V>((const ZT*)a.Z + at * a.ldz + c, a.width - c, z[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on[u]) {
        const float f = w[j0 + u];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = fmaf(f, z[u][i], sum[i]);
      }
  }
  if (a.residual)
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += r[i];
  store_row<V>((OutT*)a.y + t * a.ldy + c, a.width - c, sum);
}

template <typename ZT, typename OutT>
static p24_status launch_combine(const CombineArgs& a, hipStream_t st) {
  constexpr int V = 16 / sizeof(ZT);
  const int chunks = (a.width + V - 1) / V;
  if (chunks <= 64) {
    hipLaunchKernelGGL((k_combine<ZT, OutT, true>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((k_combine<ZT, OutT, false>), dim3((unsigned)a.T, (unsigned)((chunks + 255) / 256)), dim3(256), 0, st, a);
  }
  return launch_status();
}

static bool float_type(int32_t d) { return d == P24_F32 || d == P24_BF16; }
static size_t float_bytes(int32_t d) { return d == P24_F32 ? 4 : 2; }

}  // namespace p24

using namespace p24;

extern "C" P24_API p24_status experts_route(const void* logits, int32_t l_dtype, int64_t ldl, int64_t T, int64_t E,
                                            int64_t k, int32_t score, const float* bias, int32_t normalize, float scale,
                                            int32_t* experts, float* weights, int32_t* offsets, int32_t* tokens,
                                            int32_t* positions, void* stream) {
  if (!float_type(l_dtype)) return P24_ERR_DTYPE;
  if (T < 0 || E < 1 || k < 1 || k > E || ldl < E || !(scale - scale == 0.0f)) return P24_ERR_SHAPE;
  if (score != P24_SCORE_SOFTMAX && score != P24_SCORE_SIGMOID) return P24_ERR_UNSUPPORTED;
  if (bias && score != P24_SCORE_SIGMOID) return P24_ERR_UNSUPPORTED;
  if (E > P24_EXPERTS_MAX || k > P24_EXPERTS_K_MAX || T > (1 << 18)) return P24_ERR_UNSUPPORTED;
  if (!offsets || (T && (!logits || !experts || !weights || !tokens || !positions))) return P24_ERR_NULL;
  if (!aligned(offsets, 4) || !aligned(logits, float_bytes(l_dtype)) || !aligned(weights, 4) || !aligned(tokens, 4) ||
      !aligned(positions, 4) || !aligned(experts, 16) || (bias && !aligned(bias, 4)))
    return P24_ERR_ALIGN;
  RouteArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.bias = bias;
  a.experts = experts;
  a.weights = weights;
  a.offsets = offsets;
  a.tokens = tokens;
  a.positions = positions;
  a.T = (int)T;
  a.E = (int)E;
  a.k = (int)k;
  a.score = score;
  a.normalize = normalize != 0;
  a.scale = scale;
  const hipStream_t st = (hipStream_t)stream;
  if (l_dtype == P24_F32) return bias ? route_by_experts<float, uint64_t>(a, st) : route_by_experts<float, uint32_t>(a, st);
  return bias ? route_by_experts<uint16_t, uint64_t>(a, st) : route_by_experts<uint16_t, uint32_t>(a, st);
}

extern "C" P24_API p24_status experts_combine(const void* Z, int32_t z_dtype, int64_t ldz, int64_t rows,
                                              const int32_t* positions, const float* weights, int64_t T, int64_t k,
                                              int64_t width, const void* residual, int64_t ldr, void* y, int32_t y_dtype,
                                              int64_t ldy, void* stream) {
  if (!float_type(z_dtype) || !float_type(y_dtype)) return P24_ERR_DTYPE;
  if (T < 0 || rows < 0 || rows > INT32_MAX || k < 1 || width < 1 || width > P24_ROW_MAX || ldz < width || ldy < width ||
      (residual && ldr < width))
    return P24_ERR_SHAPE;
  if (k > P24_EXPERTS_K_MAX || T >= (1 << 22)) return P24_ERR_UNSUPPORTED;
  if (T == 0) return P24_OK;
  if ((!Z && rows) || !positions || !weights || !y) return P24_ERR_NULL;
  const size_t ze = float_bytes(z_dtype), ye = float_bytes(y_dtype);
  if (!aligned(Z, ze) || !aligned(y, ye) || (residual && !aligned(residual, ye)) || !aligned(positions, 4) ||
      !aligned(weights, 4))
    return P24_ERR_ALIGN;
  CombineArgs a{};
  a.Z = Z;
  a.positions = positions;
  a.weights = weights;
  a.residual = residual;
  a.y = y;
  a.ldz = ldz;
  a.ldr = ldr;
  a.ldy = ldy;
  a.T = (int)T;
  a.k = (int)k;
  a.width = (int)width;
  a.rows = (int)rows;
  const hipStream_t st = (hipStream_t)stream;
  if (z_dtype == P24_F32)
    return y_dtype == P24_F32 ? launch_combine<float, float>(a, st) : launch_combine<float, uint16_t>(a, st);
  return y_dtype == P24_F32 ? launch_combine<uint16_t, float>(a, st) : launch_combine<uint16_t, uint16_t>(a, st);
}
