// The small kernels around the head's scores: the lists of wanted words before the product, what its partials
// say of each row after it (log probabilities, entropy, best words; the distillation's loss), and the places that the
// distillation's gradient has at the listed words. A block of 256 threads for each row (a row has up to 256 listed words, and
// 505 to 1010 partials of a vocabulary of 129280), a warp for each of many rows in the search for the best words, a thread
// for each listed word where the gradient's places are written.
#include <type_traits>

#include "mm16_small.cuh"

namespace ds4 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCandidates = 128;
static_assert(kCandidates >= kMmTop, "the k best fit among the candidates");
static_assert(kMmListed <= kThreads, "a thread for each listed word");

// A block's sum or maximum, in a fixed order; every thread has the result. Two scratch rows take turns: a third call comes
// after the barrier of the second.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float (&s)[2][kWarps], int& turn, float v) {
  v = MAX ? warp_max(v) : warp_sum(v);
  float(&mine)[kWarps] = s[turn & 1];
  ++turn;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = mine[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) r = MAX ? fmaxf(r, mine[i]) : r + mine[i];
  return r;
}

// A word's place in ascending order is the number of words before it; then, for each tile of the vocabulary, the first of
// them that is not below the tile's first word.
__global__ void __launch_bounds__(kThreads) sort_words_kernel(const int* words, int n, int vocab, int tile, int tiles, int2* want, uint16_t* first) {
  __shared__ int key[kThreads], sorted[kThreads];
  begin();
  const int64_t t = blockIdx.x;
  const int j = threadIdx.x;
  int w = INT32_MAX;
  if (j < n) {
    w = words[t * n + j];
    if (w < 0 || w >= vocab) w = INT32_MAX;
    key[j] = w;
  }
  __syncthreads();
  if (j < n) {
    int before = 0;
    for (int i = 0; i < n; ++i) before += key[i] < w || (key[i] == w && i < j);
    sorted[before] = w;
    want[t * n + before] = make_int2(w, j);
  }
  __syncthreads();
  for (int i = j; i < tiles; i += kThreads) {
    const int from = i * tile;
    int lo = 0, left = n;
    while (left > 0) {
      const int half = left >> 1;
      if (sorted[lo + half] < from)
        lo += half + 1, left -= half + 1;
      else
        left = half;
    }
    first[t * tiles + i] = (uint16_t)lo;
  }
}

// The G threads (a block or a warp) that work on one row, and what they do together; every thread has the results.
template <int G>
struct Team;
template <>
struct Team<32> {
  static constexpr int kRows = kThreads / 32;  // rows of a block
  __device__ __forceinline__ int id() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int row() const { return threadIdx.x >> 5; }
  __device__ __forceinline__ float max(float v) { return warp_max(v); }
  __device__ __forceinline__ float sum(float v) { return warp_sum(v); }
  __device__ __forceinline__ int count(int v) { return __reduce_add_sync(0xffffffffu, v); }
  __device__ __forceinline__ int votes(bool v) { return __popc(__ballot_sync(0xffffffffu, v)); }
  __device__ __forceinline__ bool any(bool v) { return __any_sync(0xffffffffu, v); }
  __device__ __forceinline__ void sync() { __syncwarp(); }
};
template <>
struct Team<kThreads> {
  static constexpr int kRows = 1;
  float (&f)[2][kWarps];
  int (&n)[2][kWarps];
  int turn = 0;
  __device__ __forceinline__ int id() const { return threadIdx.x; }
  __device__ __forceinline__ int row() const { return 0; }
  __device__ __forceinline__ float max(float v) { return block_reduce<true>(f, turn, v); }
  __device__ __forceinline__ float sum(float v) { return block_reduce<false>(f, turn, v); }
  __device__ __forceinline__ int count(int v) {
    v = __reduce_add_sync(0xffffffffu, v);
    int(&mine)[kWarps] = n[turn & 1];
    ++turn;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
    __syncthreads();
    int r = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) r += mine[i];
    return r;
  }
  __device__ __forceinline__ int votes(bool v) { return __syncthreads_count(v); }
  __device__ __forceinline__ bool any(bool v) { return __syncthreads_or(v); }
  __device__ __forceinline__ void sync() { __syncthreads(); }
};

// The teacher's probabilities of one row: softmax(logit / T) over the entries in the vocabulary, item(j) = (there, logit), j <
// n. No entries, or none that is above -inf, leave `taught` false; a NaN among them makes every p NaN.
struct Teacher {
  float top, sum;
  bool taught;
  __device__ __forceinline__ float p(float logit, float inv_t) const { return expf((logit - top) * inv_t) / sum; }
};
template <class T, class There>
__device__ __forceinline__ Teacher teach(T& team, const There& there, const float* logits, int n, float inv_t, int g) {
  Teacher r;
  float m = -INFINITY;
  bool bad = false;
  for (int j = team.id(); j < n; j += g)
    if (there(j)) m = fmaxf(m, logits[j]), bad |= logits[j] != logits[j];
  bad = team.any(bad);
  r.top = team.max(m);
  r.taught = bad || r.top > -INFINITY;
  float s = 0.f;
  for (int j = team.id(); j < n; j += g)
    if (there(j) && r.top > -INFINITY) s += expf((logits[j] - r.top) * inv_t);
  r.sum = team.sum(s);
  if (bad) r.sum = NAN;
  return r;
}

// ---- the k best of n items with distinct keys. A key orders first by value, then by the lower index: the float's bits,
// turned so that they order as unsigned numbers, above the index's complement. 0 stands for nothing (a NaN).
__device__ __forceinline__ unsigned long long key_of(float v, int i) {
  if (v != v) return 0;
  v += 0.f;  // (-0 is +0)
  const uint32_t b = __float_as_uint(v);
  return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(unsigned long long k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int index_of(unsigned long long k) { return (int)~(uint32_t)k; }

// Shared memory of a team's selections.
template <int G>
struct Picks {
  static constexpr int kKept = G == kThreads ? 4096 : 1;  // keys that are not fetched again (a warp has registers)
  unsigned long long keys[kKept], cand[kCandidates], list[2][kMmTop];
  int count;
};

// Leaves the k largest keys of item(0..n-1) (all, if there are fewer) in `list` in their order, and returns their number.
// The k-th largest of the threads' largest values, found bit by bit from the top, is reached by at least k items and as a
// rule by few more: those are ranked by counting. Where more than kCandidates reach it (equal values) the k-th largest key
// itself is found, bit by bit over all items (for all rows and sizes at first: 2048 rows,
// 20 best, 68 us instead of 64). What item() reads may not be `list`.
// A warp's threads hold up to HELD items each in registers, unrolled. A block (HELD 0) keeps them in shared memory under
// rolled loops: with few rows it runs its code once, and the product has driven that out of the caches (one row, 8 best of
// 129280: a call 188 us with unrolled loops, 185 so; 256 rows of 32000 words, d 4096: 93 us, 80).
template <int HELD, int G, class Item>
__device__ __forceinline__ int best_of(Team<G>& team, Picks<G>& p, int n, int k, unsigned long long* list, const Item& item) {
  unsigned long long mine[HELD ? HELD : 1];
  const bool held = HELD && n <= HELD * G;
  unsigned long long most = 0;
  if (held) {
#pragma unroll
    for (int u = 0; u < HELD; ++u) {
      const int i = team.id() + u * G;
      mine[u] = i < n ? item(i) : 0;
      most = mine[u] > most ? mine[u] : most;
    }
  } else {
#pragma unroll 2
    for (int i = team.id(); i < n; i += G) {
      const unsigned long long q = item(i);
      if (i < p.kKept) p.keys[i] = q;  // (read by the same thread only)
      most = q > most ? q : most;
    }
  }
  const auto each = [&](const auto& fn) {
    if (held) {
#pragma unroll
      for (int u = 0; u < HELD; ++u) fn(mine[u]);
    } else {
#pragma unroll 1
      for (int i = team.id(); i < n; i += G) fn(i < p.kKept ? p.keys[i] : item(i));
    }
  };
  const auto reach = [&](unsigned long long least) {
    int c = 0;
    each([&](unsigned long long q) { c += q >= least; });
    return team.count(c);
  };
  const uint32_t top = (uint32_t)(most >> 32);
  uint32_t reached = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t to = reached | 1u << bit;
    const int c = team.votes(top >= to);
    if (c >= k) reached = to;
    if (c == k) break;
  }
  unsigned long long least = reached ? (unsigned long long)reached << 32 : 1;
  if (reach(least) > kCandidates) {
    least = 0;  // (there are k at least: kCandidates are more)
#pragma unroll 1
    for (int bit = 63; bit >= 0; --bit) {
      const unsigned long long to = least | 1ull << bit;
      const int c = reach(to);
      if (c >= k) least = to;
      if (c == k) break;
    }
  }
  if (team.id() == 0) p.count = 0;
  team.sync();
  each([&](unsigned long long q) {
    if (q >= least) p.cand[atomicAdd(&p.count, 1)] = q;
  });
  team.sync();
  const int got = p.count;
  for (int i = team.id(); i < got; i += G) {
    const unsigned long long q = p.cand[i];
    int ahead = 0;
#pragma unroll 4
    for (int j = 0; j < got; ++j) ahead += p.cand[j] > q;
    if (ahead < k) list[ahead] = q;
  }
  team.sync();
  return min(got, k);
}

// Joins the partials (max, sum, spread), whole sets of words each: M = max m_i, S = sum s_i r_i, U = sum (u_i + (m_i - M) s_i) r_i
// with r_i = exp((m_i - M) / T): lse = M / T + log S, entropy = log S - U / (T S).
// (A set without a number has m_i = NaN: it adds its sum, 0 or NaN, and is nothing to the search.)
// The k best words lie in the k tiles with the largest maxima (a word of any other tile has k words ahead of it, one in
// each of these), and there in the k chunks of 32 words with the largest: three selections of k.
template <int G>
__device__ __forceinline__ void score_join(const MmScores& a, Team<G> team, Picks<G>& picks) {
  const int64_t t = blockIdx.x * (int64_t)Team<G>::kRows + team.row();
  if (t >= a.rows) return;  // (whole teams)
  const int id = team.id();
  const float c = a.inv_t;
  const float2* part = a.part + t;
  const int64_t rows = a.rows;
  // (a thread joins its partials one after the other, then the team's threads theirs)
  float m = -INFINITY, s = 0.f, u = 0.f;
  const auto shift = [&](float from, float to) { return from == to ? 0.f : fmaxf(from - to, -1e30f); };
#pragma unroll 4
  for (int i = id; i < a.parts; i += G) {
    const float2 q = part[i * rows];
    const float e = a.entropy ? a.ent[i * rows + t] : 0.f;
    const float top = fmaxf(m, q.x), d0 = shift(m, top), d1 = shift(q.x, top), r0 = expf(d0 * c), r1 = expf(d1 * c);
    u = (u + d0 * s) * r0 + (e + d1 * q.y) * r1;
    s = s * r0 + q.y * r1;
    m = top;
  }
  {
    const float top = team.max(m), d = shift(m, top), r = expf(d * c);
    u = team.sum((u + d * s) * r);
    s = team.sum(s * r);
    m = top;
  }
  const float log_s = logf(s);
  if (id == 0) {
    if (a.lse) a.lse[t] = m * c + log_s;
    if (a.entropy) {
      const float h = log_s - u * c / s;
      a.entropy[t] = h < 0.f ? 0.f : h;
    }
  }
  const int* words = a.words + t * a.n;
  float* logprob = a.logprob + t * a.n;
  const float* zwant = a.zwant + t * a.n;
  const auto there = [&](int j) { return words[j] >= 0 && words[j] < a.vocab; };
  const auto logp = [&](int j) { return there(j) ? (zwant[j] - m) * c - log_s : 0.f; };
  for (int j = id; j < a.n; j += G) {
    logprob[j] = logp(j);
    if (!there(j) && words[j] != -1) atomicOr(a.err, 1);
  }
  if (a.loss) {
    const float* teacher = a.teacher + t * a.n;
    const Teacher of = teach(team, there, teacher, a.n, c, G);
    const float log_sum = logf(of.sum);
    float sum = 0.f;
    for (int j = id; j < a.n; j += G) {
      const float p = there(j) && of.taught ? of.p(teacher[j], c) : 0.f;
      if (p != 0.f) sum += p * ((teacher[j] - of.top) * c - log_sum - logp(j));
    }
    sum = team.sum(sum);
    if (id == 0) a.loss[t] = sum;
  }
  if (a.top_k == 0) return;
  // The k best tiles, their k best chunks, these chunks' k best words; few rows have no tiles.
  const int per_tile = a.tile / kMmStatChunk, chunks = (a.vocab + kMmStatChunk - 1) / kMmStatChunk;
  int found = per_tile == 1 ? chunks : a.parts;
  const auto pick = [&](auto held, int step) {
    const unsigned long long* from = picks.list[step & 1];  // (of the step before)
    const int each = step == 0 || (step == 1 && per_tile == 1) ? 1 : step == 1 ? per_tile : kMmStatChunk;
    found = best_of<decltype(held)::value>(team, picks, found * each, a.top_k, picks.list[(step + 1) & 1], [&](int i) -> unsigned long long {
      const int at = each == 1 ? i : index_of(from[i / each]) * each + i % each;
      if (at >= (step == 0 ? a.parts : step == 1 ? chunks : a.vocab)) return 0;
      return key_of(step == 0 ? part[at * rows].x : (step == 1 ? a.chunk_max : a.logits)[at * rows + t], at);
    });
  };
  if (G == kThreads) {
#pragma unroll 1
    for (int step = per_tile == 1 ? 1 : 0; step < 3; ++step) pick(std::integral_constant<int, 0>(), step);
  } else {
    pick(std::integral_constant<int, 16>(), 0);
    pick(std::integral_constant<int, 16>(), 1);
    pick(std::integral_constant<int, 32>(), 2);
  }
  for (int j = id; j < a.top_k; j += G) {
    const unsigned long long mine = j < found ? picks.list[1][j] : 0;
    a.top_index[t * a.top_k + j] = mine ? index_of(mine) : -1;
    a.top_logprob[t * a.top_k + j] = mine ? (value_of(mine) - m) * c - log_s : NAN;
  }
}

__global__ void __launch_bounds__(kThreads) score_join_block_kernel(const MmScores a) {
  __shared__ float f[2][kWarps];
  __shared__ int n[2][kWarps];
  __shared__ Picks<kThreads> picks;
  begin();
  score_join<kThreads>(a, Team<kThreads>{f, n}, picks);
}
__global__ void __launch_bounds__(kThreads) score_join_warp_kernel(const MmScores a) {
  __shared__ Picks<32> picks[kWarps];
  begin();
  score_join<32>(a, Team<32>{}, picks[threadIdx.x >> 5]);
}

__global__ void __launch_bounds__(kThreads) distill_prepare_kernel(const int* ids, const float* teacher, const float* logq,
                                                                   const float* dloss, int n, int vocab, float inv_t, float* g, float* at) {
  __shared__ float f[2][kWarps];
  __shared__ int c[2][kWarps];
  __shared__ int all[kThreads];
  __shared__ float p_of[kThreads];
  begin();
  const int64_t t = blockIdx.x;
  const int j = threadIdx.x, id = j < n ? ids[t * n + j] : -1;
  const bool there = id >= 0 && id < vocab;
  Team<kThreads> team{f, c};
  const Teacher of = teach(team, [&](int) { return there; }, teacher + t * n, n, inv_t, kThreads);
  if (j == 0) g[t] = of.taught ? dloss[t] * inv_t : 0.f;
  all[j] = id;
  p_of[j] = there && of.taught ? of.p(teacher[t * n + j], inv_t) : 0.f;
  __syncthreads();
  if (!there) return;
  float p = 0.f;
  int first = n;
  for (int i = 0; i < n; ++i)  // (a word named twice has the sum of its entries, in their order, and the first one's log q)
    if (all[i] == id) p += p_of[i], first = min(first, i);
  at[t * n + j] = expf(logq[t * n + first]) - p;
}

__global__ void __launch_bounds__(kThreads) distill_scatter_kernel(const int* ids, const float* at, const float* g, const float* gs,
                                                                   int n, int rows, int word0, int words, void* dz, int64_t lddz,
                                                                   int f16) {
  begin();
  const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (i >= (int64_t)rows * n) return;
  const int id = ids[i] - word0;
  if (ids[i] < 0 || id < 0 || id >= words) return;
  const int t = (int)(i / n);
  const float gw = g[t] / *gs * kMmGradOne;
  st16(dz, id * lddz + t, gw == 0.f ? 0.f : at[i] * gw, f16);
}

}  // namespace

cudaError_t mm_sort_words(const int* words, int n, int vocab, int rows, int tile, int2* want, uint16_t* first, cudaStream_t s) {
  return launch(sort_words_kernel, dim3(rows), kThreads, s, words, n, vocab, tile, (vocab + tile - 1) / tile, want, first);
}

// A warp for each row where there are best words to find and rows enough to fill the SMs with warps: it needs no barriers (a call
// of 2048 rows of 129280 words, d 64, 20 best: 281 us, with a block for each 307; 1024 rows, 8 best: 149 both; but the join of 512
// rows of 32000 words, 8 best: 28 us, 20 by blocks). Up to 28 best words: the k-th largest of a warp's 32 values is then passed by
// 32 log(32 / (32 - k)) = 67 items on average, at 31 by 111 and from 32 on by more than the candidates hold in most rows, and above
// 32 there is no k-th (2048 rows of 129280 words, 33 best: 972 us, by blocks 335; 64 best 1902, 386; 151936 words, 32 best 494, 372).
constexpr int kWarpTop = 28;
cudaError_t mm_score_join(const MmScores& a, cudaStream_t s) {
  if (a.top_k && a.top_k <= kWarpTop && a.rows >= 1024) return launch(score_join_warp_kernel, dim3((a.rows + kWarps - 1) / kWarps), kThreads, s, a);
  return launch(score_join_block_kernel, dim3(a.rows), kThreads, s, a);
}

cudaError_t mm_distill_prepare(const int* ids, const float* teacher, const float* logq, const float* dloss, int n, int vocab,
                               int rows, float inv_t, float* g, float* at, cudaStream_t s) {
  return launch(distill_prepare_kernel, dim3(rows), kThreads, s, ids, teacher, logq, dloss, n, vocab, inv_t, g, at);
}

cudaError_t mm_distill_scatter(const int* ids, const float* at, const float* g, const float* gs, int n, int rows, int word0,
                               int words, void* dz, int64_t lddz, int f16, cudaStream_t s) {
  const int64_t blocks = ((int64_t)rows * n + kThreads - 1) / kThreads;
  return launch(distill_scatter_kernel, dim3((unsigned)blocks), kThreads, s, ids, at, g, gs, n, rows, word0, words, dz, lddz, f16);
}

}  // namespace ds4
