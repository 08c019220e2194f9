// Routing of tokens to experts, and the combination of a token's experts.
//
// Routing: the k best of E logits per token, then a counting sort of the T k
// choices by expert, without atomics on memory.  Which of 32 tokens chose an expert
// is one word, whose bits count the expert's rows and rank them in token order.
// The first launch picks and leaves the counts of each 32 tokens; in the second
// every group adds up the counts ahead of it (from the L2: T / 32 x E) and places
// its rows.  Past 16384 tokens (of 256 experts) a launch between them sums the counts once for all;
// up to 64 tokens one launch does everything.
// Bound by instructions: about 90 for each choice of four tokens.  8192 tokens, 8 of 256 experts with a bias: 16 us,
// 10 to pick and 6 to place; one token, 8 of 128: 5.5, a launch.
//
// Combination: bound by HBM, T (k + 2) rows.  4096 tokens of 8 rows of 4096 bf16: 65 us, 5.1 TB/s.
#include <type_traits>

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
  int* counts;       // groups of 32 tokens x E, and a row of sums
  int T, E, k;
  int score, normalize;
  float scale;
  bool added;       // k_route_place sums the counts
};

// Keys whose unsigned order is the order of the scores: NaN above +inf, -0 as +0.  No score has key 0.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return v != v ? 0xFFFFFFFFu : k;
}
__device__ __forceinline__ uint64_t score_key(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  const uint64_t k = u >> 63 ? ~u : u | 1ull << 63;
  return v != v ? ~0ull : k;
}

// The score of a key.
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Reductions over the 16 lanes of a token, the result in each: quads, then mirrored halves and rows.
constexpr int G = 16;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int SWAP1 = 0xB1, SWAP2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140;   // quad_perm 1 0 3 2, 2 3 0 1, ..
template <typename F>
__device__ __forceinline__ uint32_t reduce(uint32_t v, F&& f) {
  v = f(v, dpp<SWAP1>(v));
  v = f(v, dpp<SWAP2>(v));
  v = f(v, dpp<HALF_MIRROR>(v));
  return f(v, dpp<MIRROR>(v));
}
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t min_of(uint32_t v) {
  return reduce(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ uint64_t max_of(uint64_t v) {
  const uint32_t hi = max_of((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | max_of((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
__device__ __forceinline__ float sum_of(float v) {
  return __uint_as_float(reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__device__ __forceinline__ float logit_at(const uint16_t* row, int e) { return __uint_as_float((uint32_t)row[e] << 16); }
__device__ __forceinline__ float logit_at(const float* row, int e) { return row[e]; }

// What ranks an expert with a bias: in 64 bits, or (T float) to within 2^-22 of max(1, |score|): the exponent's
// roundings, |x| 2^-23 of exp(x), weigh |x| s (1 - s) < 1/4 in the sigmoid s, exp2 and the reciprocal one ulp each.
template <typename T>
__device__ __forceinline__ T biased_score(float logit, float bias) {
  if constexpr (sizeof(T) == 8) return 1.0 / (1.0 + exp(-(double)logit)) + (double)bias;
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(logit * -1.44269504088896341f)) + bias;
}

// The k best keys of one token on 16 lanes, V experts each (64 c + 4 lane + [0, 4) for c < V / 4): slot j's expert
// and key end up in lane j % 16, entry j / 16; `first` is the best's key.  Key 0 is no expert.  With CHECK the k + 1 best are
// picked, and the result says what cannot be told apart: NEAR two neighbours among them, EDGE the last and the one behind it.
enum { NEAR = 1, EDGE = 2 };
template <int V, bool CHECK, typename Key>
__device__ __forceinline__ int pick(Key (&key)[V], int k, int (&expert)[2], Key (&chosen)[2], Key& first) {
  const int lane = threadIdx.x % G;
  expert[0] = expert[1] = -1;
  chosen[0] = chosen[1] = first = 0;
  int unsure = 0;
  float last = 0.0f;
  for (int j = 0; j < k + (CHECK ? 2 : 0); ++j) {
    Key best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    const Key top = max_of(best);
    if (top == 0) break;       // of all the token's lanes alike
    if constexpr (CHECK) {
      const float score = key_score(top);
      if (j > 0 && !(last - score > 0x1p-20f * fmaxf(1.0f, fmaxf(fabsf(last), fabsf(score))))) unsure |= j <= k ? NEAR : EDGE;
      last = score;
      if (j > k) break;
    }
    int at = V;                // the lane's lowest expert of that key
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == top ? v : at;
    const uint32_t mine = at < V ? (uint32_t)(64 * (at / 4) + 4 * lane + at % 4) : 0xFFFFFFFFu;
    const uint32_t e = min_of(mine);
    at = mine == e ? at : V;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = at == v ? 0 : key[v];
    if (j == 0) first = top;
    if (lane == j % G) {
      if (j < G) {
        expert[0] = (int)e;
        chosen[0] = top;
      } else if (j < 2 * G) {
        expert[1] = (int)e;
        chosen[1] = top;
      }
    }
  }
  return unsure;
}

// Lane j's expert and key, j < 16, into descending order of the keys (ties: the lower expert); -1 is no expert.
__device__ __forceinline__ int in_order(int expert, uint64_t key) {
  const int lane = threadIdx.x % G;
  int rank = 0, out = -1;
  for (int i = 0; i < G; ++i) {
    const int e = __shfl(expert, i, G);
    const uint64_t k = (uint64_t)(uint32_t)__shfl((int)(key >> 32), i, G) << 32 | (uint32_t)__shfl((int)key, i, G);
    rank += e >= 0 && (k > key || (k == key && e < expert));
  }
  if (expert < 0) rank = G;
  for (int i = 0; i < G; ++i) {
    const int e = __shfl(expert, i, G), r = __shfl(rank, i, G);
    out = r == lane ? e : out;
  }
  return out;
}

// One token: its slots' experts and weights, in the lanes of pick.  BIAS: sigmoid and bias.  64-bit exponentials of all
// scores take as long as all the rest (8192 tokens of 256 experts: 14.3 us, 10.8 this way), so 32 bits pick one
// expert more than asked for; where those cannot tell two of them apart, one token in some hundreds, 64 bits put
// them in order, and only where the edge of what was picked is unsure too, everything is done in 64.
template <typename T, bool BIAS, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int (&expert)[2], float (&weight)[2]) {
  const int lane = threadIdx.x % G;
  const T* row = (const T*)a.logits + t * a.ldl;
  float l[V];
#pragma unroll
  for (int c = 0; c < V / 4; ++c) {
    const int e = 4 * G * c + 4 * lane;
    float x[4];
    load_row<4>(row + e, a.E - e, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) l[4 * c + i] = e + i < a.E ? x[i] : -INFINITY;
  }
  float at[2] = {0.0f, 0.0f}, top = 0.0f;    // the chosen logits, and the largest (softmax)
  auto biased = [&](auto KEY, auto CHECK) {
    typedef decltype(KEY) Key;
    typedef std::conditional_t<sizeof(Key) == 8, double, float> Score;
    Key key[V];
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const int e = 4 * G * c + 4 * lane;
      float b[4];
      load_row<4>(a.bias + e, a.E - e, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Key score = score_key(biased_score<Score>(l[4 * c + i], b[i]));     // of all: a branch for each would wait for each
        key[4 * c + i] = l[4 * c + i] == -INFINITY ? 0 : score;
      }
      __builtin_amdgcn_sched_barrier(0);   // four exponentials at a time: their registers
    }
    Key chosen[2], first;
    return pick<V, decltype(CHECK)::value>(key, a.k, expert, chosen, first);
  };
  if constexpr (BIAS) {
    const int unsure = biased(uint32_t{}, std::true_type{});
    if (unsure & NEAR) {
      if (a.k < G && !(unsure & EDGE)) {
        const int e = max(expert[0], 0);
        const uint64_t key = score_key(biased_score<double>(logit_at(row, e), a.bias[e]));
        expert[0] = in_order(expert[0], key);
      } else {
        biased(uint64_t{}, std::false_type{});
      }
    }
    if (lane >= a.k) expert[0] = -1;      // the one more
    if (lane + G >= a.k) expert[1] = -1;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) at[s] = logit_at(row, expert[s]);
  } else {
    uint32_t key[V], chosen[2], first;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t score = score_key(l[v]);
      key[v] = l[v] == -INFINITY ? 0 : score;
    }
    pick<V, false>(key, a.k, expert, chosen, first);
    at[0] = key_score(chosen[0]);
    at[1] = key_score(chosen[1]);
    top = key_score(first);
  }
  // weights, from the logits themselves
  float w[2] = {0.0f, 0.0f};
  float all = 1.0f;
  if (a.score == P24_SCORE_SOFTMAX) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) w[s] = expf(at[s] - top);
    if (!a.normalize) {
      all = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float p = expf(l[v] - top);
        all += l[v] == -INFINITY ? 0.0f : p;
      }
      all = sum_of(all);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) w[s] = 1.0f / (1.0f + expf(-at[s]));
  }
  if (a.normalize) all = sum_of(w[0] + w[1]);
  // Sigmoids leave fp32 where their quotients do not: all of them 0 below -88.7.  With a sum this small all logits l lie
  // below -2, and exp(l - max) / (1 + exp(l)) are the sigmoids over exp(max), none of which counts and is lost.
  // (Below -709.78 exp(-l) leaves 64 bits too: there the formula's quotient is 0 / 0.)
  if (a.normalize && a.score == P24_SCORE_SIGMOID && all < 0.119f) {
    const float low = fmaxf(expert[0] >= 0 ? at[0] : -INFINITY, expert[1] >= 0 ? at[1] : -INFINITY);
    const float most = key_score(max_of(score_key(low)));
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (expert[s] >= 0) w[s] = most > -709.78271f ? expf(at[s] - most) / (1.0f + expf(at[s])) : 0.0f;
    all = sum_of(w[0] + w[1]);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) weight[s] = expert[s] >= 0 ? w[s] / all * a.scale : 0.0f;
}

constexpr int GROUP = 32;       // tokens whose choices are counted together
constexpr int FEW = 64;         // tokens that one block takes
constexpr int SLOTS = P24_EXPERTS_MAX;

// base[e] = rows of lower experts + ahead(e), from the experts' rows total(e); the sums alone to `offsets`, if
// given.  All threads of the block.  Returns the number of rows in all.
template <typename Total, typename Ahead>
__device__ __forceinline__ int scan_experts(int* base, Total total, Ahead ahead, int E, int* offsets) {
  __shared__ int waves[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, count = blockDim.x >> 6;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x, mine = e < E ? total(e) : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int other = __shfl_up(upto, o);
      upto += lane >= o ? other : 0;
    }
    if (lane == 63) waves[wave] = upto;
    __syncthreads();
    int before = carry, sum = 0;
    for (int w = 0; w < count; ++w) {
      before += w < wave ? waves[w] : 0;
      sum += waves[w];
    }
    if (e < E) {
      base[e] = before + upto - mine + ahead(e);
      if (offsets) offsets[e] = before + upto - mine;
    }
    carry += sum;
    __syncthreads();
  }
  if (offsets && threadIdx.x == 0) offsets[E] = carry;
  return carry;
}

// The rows of tokens t0 on, one bit each of `chosen`, from the experts' bases; `experts`: their choices.
template <typename Word>
__device__ __forceinline__ void place_rows(const RouteArgs& a, int t0, const int* experts, const Word* chosen,
                                           const int* base) {
  const int n = min(a.T - t0, (int)sizeof(Word) * 8) * a.k;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t slot = (int64_t)t0 * a.k + i;
    const int e = experts[i], t = i / a.k;
    int at = -1;
    if (e >= 0) {
      at = base[e] + __popcll(chosen[e] & (((Word)1 << t) - 1));
      a.tokens[at] = t0 + t;
    }
    a.positions[slot] = at;
  }
}
// Rows from `rows` on have no token.
__device__ __forceinline__ void no_tokens(const RouteArgs& a, int rows, int thread, int threads) {
  for (int i = rows + thread; i < a.T * a.k; i += threads) a.tokens[i] = -1;
}

// Picks the experts of tokens t0 on and sets their bits (LDS; the order does not matter).
template <typename T, bool BIAS, int V, typename Word>
__device__ __forceinline__ void pick_group(const RouteArgs& a, int t0, Word* chosen, int* copy = nullptr) {
  const int lane = threadIdx.x % G;
  for (int t = threadIdx.x / G; t < min(a.T - t0, (int)sizeof(Word) * 8); t += blockDim.x / G) {
    int e[2];
    float w[2];
    route_token<T, BIAS, V>(a, t0 + t, e, w);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (G * s + lane < a.k) {
        const int64_t i = (int64_t)(t0 + t) * a.k + G * s + lane;
        a.experts[i] = e[s];
        a.weights[i] = w[s];
        if (copy) copy[t * a.k + G * s + lane] = e[s];
        if (e[s] >= 0) atomicOr(&chosen[e[s]], (Word)1 << t);
      }
  }
}

// ADDED: every block adds up all groups' counts itself; a group's lie in one byte each then, rows of whole words.  That is groups^2
// words from the L2, for a launch less: 16384 tokens of 256 experts 22.0 us, 24.1 with the launch (64 experts 13.0, 18.0), of
// 1024 experts 69, 57.  The sums have 16 bits.
__host__ __device__ __forceinline__ int count_words(int E) { return (E + 3) / 4; }
static bool route_adds(int64_t groups, int E) {
  return groups * GROUP < 65536 && groups * groups * count_words(E) <= 1 << 24;
}

// 32 tokens a block: picks, and counts the rows.
template <typename T, bool BIAS, int V>
__global__ __launch_bounds__(512) void k_route_pick(const RouteArgs a) {
  __shared__ unsigned chosen[SLOTS];
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) chosen[e] = 0;
  __syncthreads();
  pick_group<T, BIAS, V>(a, blockIdx.x * GROUP, chosen);
  __syncthreads();
  if (!a.added) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.E + e] = __popc(chosen[e]);
    return;
  }
  for (int w = threadIdx.x; w < count_words(a.E); w += blockDim.x) {
    unsigned c = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) c |= 4 * w + u < a.E ? __popc(chosen[4 * w + u]) << (8 * u) : 0;
    reinterpret_cast<unsigned*>(a.counts)[(int64_t)blockIdx.x * count_words(a.E) + w] = c;
  }
}

// 64 tokens at most, in one block.
template <typename T, bool BIAS, int V>
__global__ __launch_bounds__(512) void k_route_few(const RouteArgs a) {
  __shared__ unsigned long long chosen[SLOTS];
  __shared__ int base[SLOTS], experts[FEW * P24_EXPERTS_K_MAX];
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) chosen[e] = 0;
  __syncthreads();
  pick_group<T, BIAS, V>(a, 0, chosen, experts);
  __syncthreads();
  const int rows = scan_experts(base, [&](int e) { return __popcll(chosen[e]); }, [](int) { return 0; }, a.E, a.offsets);
  place_rows(a, 0, experts, chosen, base);
  no_tokens(a, rows, threadIdx.x, blockDim.x);
}

// The counts of 64 experts a block: each group's become those of the groups ahead of it, their sums the last row.
// The block's 16 waves take a run of groups each.
__global__ __launch_bounds__(1024) void k_route_sum(const RouteArgs a, int groups) {
  constexpr int WAVES = 16;
  __shared__ int part[WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x * 64 + lane;
  const int run = (groups + WAVES - 1) / WAVES, g0 = min(wave * run, groups), g1 = min(g0 + run, groups);
  int* const col = a.counts + e;
  int sum = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int g = g0; g < g1; ++g) sum += col[(int64_t)g * a.E];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (e >= a.E) return;
  int before = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) before += w < wave ? part[w][lane] : 0;
#pragma unroll 8
  for (int g = g0; g < g1; ++g) {
    const int c = col[(int64_t)g * a.E];
    col[(int64_t)g * a.E] = before;
    before += c;
  }
  if (wave == WAVES - 1) col[(int64_t)groups * a.E] = before;
}

// The rows of 32 tokens a block.  SUMMED: k_route_sum has run.
template <bool SUMMED>
__global__ __launch_bounds__(1024) void k_route_place(const RouteArgs a) {
  __shared__ unsigned chosen[SLOTS];
  __shared__ int base[SLOTS];
  __shared__ unsigned all[2][SLOTS / 4], lower[2][SLOTS / 4];
  __shared__ int total[SUMMED ? SLOTS : 1], ahead[SUMMED ? SLOTS : 1];
  const int t0 = blockIdx.x * GROUP, groups = gridDim.x, E = a.E, words = count_words(E);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    chosen[e] = 0;
    if constexpr (SUMMED) {
      total[e] = a.counts[(int64_t)groups * E + e];
      ahead[e] = a.counts[(int64_t)blockIdx.x * E + e];
    }
  }
  if constexpr (!SUMMED)
    for (int w = threadIdx.x; w < words; w += blockDim.x) all[0][w] = all[1][w] = lower[0][w] = lower[1][w] = 0;
  __syncthreads();
  const int n = min(a.T - t0, GROUP) * a.k;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = a.experts[(int64_t)t0 * a.k + i];
    if (e >= 0) atomicOr(&chosen[e], 1u << (i / a.k));
  }
  if constexpr (!SUMMED) {
    // the groups' counts, four experts a word, several runs of groups side by side; two sums of 16 bits a word,
    // whose parts meet in LDS (whole numbers: any order)
    const int width = words <= 16 ? 16 : words <= 32 ? 32 : words <= 64 ? 64 : words <= 128 ? 128 : 256;
    const int parts = 1024 / width, part = threadIdx.x / width, w = threadIdx.x % width;
    if (w < words && part < groups) {
      const unsigned* const col = reinterpret_cast<const unsigned*>(a.counts) + w;
      unsigned sum[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll 8
      for (int g = part; g < groups; g += parts) {
        const unsigned c = col[g * words], even = c & 0x00FF00FF, odd = (c >> 8) & 0x00FF00FF;
        sum[0] += even;
        sum[1] += odd;
        before[0] += g < (int)blockIdx.x ? even : 0;
        before[1] += g < (int)blockIdx.x ? odd : 0;
      }
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        atomicAdd(&all[o][w], sum[o]);
        atomicAdd(&lower[o][w], before[o]);
      }
    }
  }
  __syncthreads();
  const int rows = scan_experts(
      base, [&](int e) { return SUMMED ? total[e] : (int)(all[e & 1][e / 4] >> (8 * (e & 2)) & 0xFFFF); },
      [&](int e) { return SUMMED ? ahead[e] : (int)(lower[e & 1][e / 4] >> (8 * (e & 2)) & 0xFFFF); }, E,
      blockIdx.x == 0 ? a.offsets : nullptr);
  place_rows(a, t0, a.experts + (int64_t)t0 * a.k, chosen, base);
  no_tokens(a, rows, blockIdx.x * 1024 + threadIdx.x, groups * 1024);
}

static int64_t route_groups(int64_t T) { return (T + GROUP - 1) / GROUP; }

template <typename T, bool BIAS, int V>
static p24_status launch_route(RouteArgs a, hipStream_t st) {
  if (a.T <= FEW) {
    hipLaunchKernelGGL((k_route_few<T, BIAS, V>), dim3(1), dim3(a.T <= 16 ? 256 : 512), 0, st, a);
    return launch_status();
  }
  const unsigned groups = (unsigned)route_groups(a.T);
  a.added = route_adds(groups, a.E);
  hipLaunchKernelGGL((k_route_pick<T, BIAS, V>), dim3(groups), dim3(512), 0, st, a);
  p24_status s = launch_status();
  if (s != P24_OK) return s;
  if (a.added) {
    hipLaunchKernelGGL(k_route_place<false>, dim3(groups), dim3(1024), 0, st, a);
    return launch_status();
  }
  hipLaunchKernelGGL(k_route_sum, dim3((unsigned)(a.E + 63) / 64), dim3(1024), 0, st, a, (int)groups);
  s = launch_status();
  if (s != P24_OK) return s;
  hipLaunchKernelGGL(k_route_place<true>, dim3(groups), dim3(1024), 0, st, a);
  return launch_status();
}

template <typename T, bool BIAS>
static p24_status route_by_experts(const RouteArgs& a, hipStream_t st) {
  if (a.E <= 64) return launch_route<T, BIAS, 4>(a, st);
  if (a.E <= 128) return launch_route<T, BIAS, 8>(a, st);
  if (a.E <= 256) return launch_route<T, BIAS, 16>(a, st);
  if (a.E <= 512) return launch_route<T, BIAS, 32>(a, st);
  return launch_route<T, BIAS, 64>(a, st);
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

extern "C" P24_API size_t experts_route_workspace(int64_t T, int64_t E) {
  return T <= FEW || E < 1 ? 0 : (size_t)(route_groups(T) + 1) * (size_t)E * 4;
}

extern "C" P24_API p24_status experts_route(const void* logits, int32_t l_dtype, int64_t ldl, int64_t T, int64_t E,
                                            int64_t k, int32_t score, const float* bias, int32_t normalize, float scale,
                                            int32_t* experts, float* weights, int32_t* offsets, int32_t* tokens,
                                            int32_t* positions, void* ws, size_t ws_bytes, void* stream) {
  if (!float_type(l_dtype)) return P24_ERR_DTYPE;
  if (T < 0 || E < 1 || k < 1 || k > E || ldl < E || !(scale - scale == 0.0f)) return P24_ERR_SHAPE;
  if (score != P24_SCORE_SOFTMAX && score != P24_SCORE_SIGMOID) return P24_ERR_UNSUPPORTED;
  if (bias && score != P24_SCORE_SIGMOID) return P24_ERR_UNSUPPORTED;
  if (E > P24_EXPERTS_MAX || k > P24_EXPERTS_K_MAX || T > (1 << 18)) return P24_ERR_UNSUPPORTED;
  if (!offsets || (T && (!logits || !experts || !weights || !tokens || !positions))) return P24_ERR_NULL;
  if (!aligned(offsets, 4) || !aligned(logits, float_bytes(l_dtype)) || !aligned(weights, 4) || !aligned(tokens, 4) ||
      !aligned(positions, 4) || !aligned(experts, 4) || (bias && !aligned(bias, 4)))
    return P24_ERR_ALIGN;
  const size_t need = experts_route_workspace(T, E);
  if (need && !ws) return P24_ERR_NULL;
  if (need && !aligned(ws, 4)) return P24_ERR_ALIGN;
  if (ws_bytes < need) return P24_ERR_WORKSPACE;
  RouteArgs a{};
  a.counts = (int*)ws;
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
  if (l_dtype == P24_F32) return bias ? route_by_experts<float, true>(a, st) : route_by_experts<float, false>(a, st);
  return bias ? route_by_experts<uint16_t, true>(a, st) : route_by_experts<uint16_t, false>(a, st);
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
