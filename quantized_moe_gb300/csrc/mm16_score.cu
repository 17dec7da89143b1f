// The small kernels around the head's scores: the lists of wanted words before the product, what its partials
// say of each row after it (log probabilities, entropy, best words; the distillation's loss), and the places that the
// distillation's gradient has at the listed words. One block of 256 threads for each row throughout: a row has up to 256
// listed words, and 505 tiles of a vocabulary of 129280 (4040 where few tokens have tiles of 32 words).
#include "mm16_small.cuh"

namespace ds4 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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

// The teacher's probabilities of one row, thread j's entry: softmax(logit / T) over the entries in the vocabulary. No
// entries, or none that is above -inf, leave `taught` false; a NaN among them makes every p NaN.
struct Teacher {
  float top, sum;
  bool taught;
};
__device__ __forceinline__ Teacher teach(float (&s)[2][kWarps], int& turn, bool there, float logit, float inv_t) {
  Teacher r;
  const bool bad = __syncthreads_or(there && logit != logit);
  r.top = block_reduce<true>(s, turn, there ? logit : -INFINITY);
  r.taught = bad || r.top > -INFINITY;
  r.sum = block_reduce<false>(s, turn, there && r.top > -INFINITY ? expf((logit - r.top) * inv_t) : 0.f);
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

// Leaves the k largest keys of item(0..n-1) (all, if there are fewer) in `list`, in any order, and returns their number. The
// k-th largest key is found bit by bit from the top, counting the items that reach a candidate; it ends as soon as
// exactly k do. Called by all threads; list and count are shared.
template <int HELD, class Item>
__device__ __forceinline__ int best_of(int n, int k, unsigned long long* list, int* count, const Item& item) {
  unsigned long long mine[HELD];  // a thread's items stay in registers up to that many
  const bool held = n <= HELD * kThreads;
  if (held) {
#pragma unroll
    for (int u = 0; u < HELD; ++u) {
      const int i = threadIdx.x + u * kThreads;
      mine[u] = i < n ? item(i) : 0;
    }
  }
  const auto reach = [&](unsigned long long least) {  // of a thread's own
    int c = 0;
    if (held) {
#pragma unroll
      for (int u = 0; u < HELD; ++u) c += mine[u] >= least;
    } else {
      for (int i = threadIdx.x; i < n; i += kThreads) c += item(i) >= least;
    }
    return c;
  };
  __shared__ int sums[2][kWarps];
  unsigned long long least = 1;
  if (n > k) {
    unsigned long long found = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const unsigned long long to = found | 1ull << bit;
      const int c = __reduce_add_sync(0xffffffffu, reach(to));
      if ((threadIdx.x & 31) == 0) sums[bit & 1][threadIdx.x >> 5] = c;
      __syncthreads();
      int total = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) total += sums[bit & 1][i];
      if (total >= k) found = to;
      if (total == k) break;
    }
    least = found > 1 ? found : 1;
  }
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  if (held) {
#pragma unroll
    for (int u = 0; u < HELD; ++u)
      if (mine[u] >= least) list[atomicAdd(count, 1)] = mine[u];
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const unsigned long long q = item(i);
      if (q >= least) list[atomicAdd(count, 1)] = q;
    }
  }
  __syncthreads();
  const int got = *count;
  __syncthreads();
  return got;
}

// Joins the tiles' (max, sum, spread) as M = max m_i, S = sum s_i r_i, U = sum (u_i + (m_i - M) s_i) r_i
// with r_i = exp((m_i - M) / T): lse = M / T + log S, entropy = log S - U / (T S).
// The k best words lie in the k tiles with the largest maxima (a word of any other tile has k words ahead of it, one in
// each of these), and there in the k chunks of 32 words with the largest: three selections of k.
__global__ void __launch_bounds__(kThreads) score_join_kernel(const MmScores a) {
  __shared__ float red[2][kWarps];
  __shared__ unsigned long long list[2][kMmTop];
  __shared__ int count;
  begin();
  const int64_t t = blockIdx.x;
  const int j = threadIdx.x;
  int turn = 0;
  const float c = a.inv_t;
  float m = -INFINITY;
  for (int i = j; i < a.tiles; i += kThreads) m = fmaxf(m, a.part[(int64_t)i * a.rows + t].x);
  m = block_reduce<true>(red, turn, m);
  float s = 0.f, u = 0.f;
  for (int i = j; i < a.tiles; i += kThreads) {
    const float2 q = a.part[(int64_t)i * a.rows + t];
    const float d = q.x == m ? 0.f : fmaxf(q.x - m, -1e30f), r = q.x == m ? 1.f : expf(d * c);
    s += q.y * r;
    u += (a.ent[(int64_t)i * a.rows + t] + d * q.y) * r;
  }
  s = block_reduce<false>(red, turn, s), u = block_reduce<false>(red, turn, u);
  const float log_s = logf(s);
  if (j == 0) {
    if (a.lse) a.lse[t] = m * c + log_s;
    if (a.entropy) {
      const float h = log_s - u * c / s;
      a.entropy[t] = h < 0.f ? 0.f : h;
    }
  }
  const int word = j < a.n ? a.words[t * a.n + j] : -1;
  const bool there = word >= 0 && word < a.vocab;
  float logp = 0.f;
  if (there) logp = (a.zwant[t * a.n + j] - m) * c - log_s;
  if (j < a.n) a.logprob[t * a.n + j] = logp;
  if (!there && word != -1) atomicOr(a.err, 1);
  if (a.loss) {
    const float logit = there ? a.teacher[t * a.n + j] : -INFINITY;
    const Teacher of = teach(red, turn, there, logit, c);
    const float p = there && of.taught ? expf((logit - of.top) * c) / of.sum : 0.f;
    const float sum = block_reduce<false>(red, turn, p != 0.f ? p * ((logit - of.top) * c - logf(of.sum) - logp) : 0.f);
    if (j == 0) a.loss[t] = sum;
  }
  if (a.top_k == 0) return;
  constexpr int kChunks = kMmStatTile / kMmStatChunk;
  const auto tile_max = [&](int i) { return key_of(a.part[(int64_t)i * a.rows + t].x, i); };
  const int chunks = (a.vocab + kMmStatChunk - 1) / kMmStatChunk;
  int n_chunks;
  if (a.tile == kMmStatChunk) {
    n_chunks = best_of<16>(a.tiles, a.top_k, list[1], &count, tile_max);
  } else {
    const int n_tiles = best_of<2>(a.tiles, a.top_k, list[0], &count, tile_max);
    n_chunks = best_of<2>(n_tiles * kChunks, a.top_k, list[1], &count, [&](int i) {
      const int chunk = index_of(list[0][i / kChunks]) * kChunks + i % kChunks;
      return chunk < chunks ? key_of(a.chunk_max[(int64_t)chunk * a.rows + t], chunk) : 0ull;
    });
  }
  const int n_words = best_of<8>(n_chunks * kMmStatChunk, a.top_k, list[0], &count, [&](int i) {
    const int w = index_of(list[1][i / kMmStatChunk]) * kMmStatChunk + i % kMmStatChunk;
    return w < a.vocab ? key_of(a.logits[(int64_t)w * a.rows + t], w) : 0ull;
  });
  if (j < a.top_k) {
    if (j < n_words) {
      const unsigned long long mine = list[0][j];
      int ahead = 0;
      for (int i = 0; i < n_words; ++i) ahead += list[0][i] > mine;
      a.top_index[t * a.top_k + ahead] = index_of(mine);
      a.top_logprob[t * a.top_k + ahead] = (value_of(mine) - m) * c - log_s;
    } else {
      a.top_index[t * a.top_k + j] = -1;
      a.top_logprob[t * a.top_k + j] = NAN;
    }
  }
}

__global__ void __launch_bounds__(kThreads) distill_prepare_kernel(const int* ids, const float* teacher, const float* logq,
                                                                   const float* dloss, int n, int vocab, float inv_t, float* g, float* at) {
  __shared__ float red[2][kWarps];
  __shared__ int all[kThreads];
  __shared__ float p_of[kThreads];
  begin();
  const int64_t t = blockIdx.x;
  const int j = threadIdx.x, id = j < n ? ids[t * n + j] : -1;
  const bool there = id >= 0 && id < vocab;
  const float logit = there ? teacher[t * n + j] : -INFINITY;
  int turn = 0;
  const Teacher of = teach(red, turn, there, logit, inv_t);
  if (j == 0) g[t] = of.taught ? dloss[t] * inv_t : 0.f;
  all[j] = id;
  p_of[j] = there && of.taught ? expf((logit - of.top) * inv_t) / of.sum : 0.f;
  __syncthreads();
  if (!there) return;
  float p = 0.f;
  for (int i = 0; i < n; ++i)  // (a word named twice has the sum of its entries, in their order)
    if (all[i] == id) p += p_of[i];
  at[t * n + j] = expf(logq[t * n + j]) - p;
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

// In stream order, not as a programmatic dependent launch: blocks that wait for the product would all settle on the SMs that
// it leaves first (2048 rows: 1340 us instead of 345, a block for eight rows).
cudaError_t mm_score_join(const MmScores& a, cudaStream_t s) {
  score_join_kernel<<<a.rows, kThreads, 0, s>>>(a);
  return cudaGetLastError();
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
