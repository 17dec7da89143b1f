// The small kernels around the head's scores: the lists of wanted words before the product, what its partials
// say of each row after it (log probabilities, entropy, best words; the distillation's loss), and the places that the
// distillation's gradient has at the listed words.
#include "mm16_small.cuh"

namespace ds4 {
namespace {

// One warp per row: a word's place in ascending order is the number of words before it (n is a few hundred at most).
__global__ void __launch_bounds__(256) sort_words_kernel(const int* words, int n, int vocab, int rows, int2* want) {
  begin();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= rows) return;
  const int* mine = words + (int64_t)t * n;
  for (int j = lane; j < n; j += 32) {
    const auto key = [&](int i) {
      const int w = mine[i];
      return w >= 0 && w < vocab ? w : INT32_MAX;
    };
    const int w = key(j);
    int before = 0;
    for (int i = 0; i < n; ++i) {
      const int v = key(i);
      before += v < w || (v == w && i < j);
    }
    want[(int64_t)t * n + before] = make_int2(w, j);
  }
}

// The teacher's probabilities of one row: softmax(logit / T) over the entries in the vocabulary. 0 entries (or none that is
// above -inf) leave `taught` false; a NaN among them makes the sum NaN.
struct Teacher {
  float top, sum, inv_t;
  bool taught;
  __device__ __forceinline__ void start(const int* ids, const float* logits, int n, int vocab, float it, int lane) {
    inv_t = it;
    float m = -INFINITY;
    int bad = 0;
    for (int j = lane; j < n; j += 32) {
      if (ids[j] < 0 || ids[j] >= vocab) continue;
      m = fmaxf(m, logits[j]);
      bad |= logits[j] != logits[j];
    }
    top = warp_max(m);
    bad = __any_sync(0xffffffffu, bad);
    float s = 0.f;
    for (int j = lane; j < n; j += 32)
      if (ids[j] >= 0 && ids[j] < vocab && top > -INFINITY) s += expf((logits[j] - top) * it);
    sum = bad ? NAN : warp_sum(s);
    taught = bad || top > -INFINITY;
  }
  __device__ __forceinline__ float p(float logit) const { return expf((logit - top) * inv_t) / sum; }
  __device__ __forceinline__ float log_p(float logit) const { return (logit - top) * inv_t - logf(sum); }
};

// One row's best words in order, spread over a warp: places lane and lane + 32.
struct Best {
  float v[2];
  int id[2];
  __device__ __forceinline__ float value(int at) const { return __shfl_sync(0xffffffffu, at < 32 ? v[0] : v[1], at & 31); }
  __device__ __forceinline__ int word(int at) const { return __shfl_sync(0xffffffffu, at < 32 ? id[0] : id[1], at & 31); }
};
__device__ __forceinline__ bool ahead(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// One warp per row. Joins the tiles' (max, sum, spread) as M = max m_i, S = sum s_i r_i, U = sum (u_i + (m_i - M) s_i) r_i
// with r_i = exp((m_i - M) / T): lse = M / T + log S, entropy = log S - U / (T S).
// The k best words lie in the k tiles with the largest maxima (a word of any other tile has k words ahead of it, one in
// each of these): those tiles are taken in order and their logits put into a sorted list, a word at a time, unless they do
// not beat its last one.
__global__ void __launch_bounds__(256) score_join_kernel(const MmScores a) {
  begin();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= a.rows) return;
  const float c = a.inv_t;
  float m = -INFINITY;
  for (int i = lane; i < a.tiles; i += 32) m = fmaxf(m, a.part[(int64_t)i * a.rows + t].x);
  m = warp_max(m);
  float s = 0.f, u = 0.f;
  for (int i = lane; i < a.tiles; i += 32) {
    const float2 q = a.part[(int64_t)i * a.rows + t];
    const float d = q.x == m ? 0.f : fmaxf(q.x - m, -1e30f), r = q.x == m ? 1.f : expf(d * c);
    s += q.y * r;
    u += (a.ent[(int64_t)i * a.rows + t] + d * q.y) * r;
  }
  s = warp_sum(s), u = warp_sum(u);
  const float log_s = logf(s);
  if (lane == 0) {
    if (a.lse) a.lse[t] = m * c + log_s;
    if (a.entropy) {
      const float h = log_s - u * c / s;
      a.entropy[t] = h < 0.f ? 0.f : h;
    }
  }
  const int* words = a.words + (int64_t)t * a.n;
  int outside = 0;
  if (a.loss) {
    const float* teacher = a.teacher + (int64_t)t * a.n;
    Teacher of;
    of.start(words, teacher, a.n, a.vocab, c, lane);
    float sum = 0.f;
    for (int j = lane; j < a.n; j += 32) {
      const bool there = words[j] >= 0 && words[j] < a.vocab;
      const float lq = there ? (a.zwant[(int64_t)t * a.n + j] - m) * c - log_s : 0.f;
      outside |= !there && words[j] != -1;
      a.logprob[(int64_t)t * a.n + j] = lq;
      const float p = there && of.taught ? of.p(teacher[j]) : 0.f;
      if (p != 0.f) sum += p * (of.log_p(teacher[j]) - lq);
    }
    sum = warp_sum(sum);
    if (lane == 0) a.loss[t] = sum;
  } else {
    for (int j = lane; j < a.n; j += 32) {
      const bool there = words[j] >= 0 && words[j] < a.vocab;
      outside |= !there && words[j] != -1;
      a.logprob[(int64_t)t * a.n + j] = there ? (a.zwant[(int64_t)t * a.n + j] - m) * c - log_s : 0.f;
    }
  }
  if (outside) atomicOr(a.err, 1);
  if (a.top_k == 0) return;
  Best best;
  best.v[0] = best.v[1] = -INFINITY, best.id[0] = best.id[1] = INT32_MAX;
  float last_v = INFINITY;  // the tile taken last
  int last_i = -1;
  for (int k = 0; k < min(a.top_k, a.tiles); ++k) {
    float tv = -INFINITY;
    int ti = INT32_MAX;
    for (int i = lane; i < a.tiles; i += 32) {
      const float v = a.part[(int64_t)i * a.rows + t].x;
      if (ahead(last_v, last_i, v, i) && ahead(v, i, tv, ti)) tv = v, ti = i;
    }
    const float wv = warp_max(tv);
    const int wi = __reduce_min_sync(0xffffffffu, tv == wv ? ti : INT32_MAX);
    last_v = wv, last_i = wi;
    for (int w0 = wi * kMmStatTile; w0 < min((wi + 1) * kMmStatTile, a.vocab); w0 += 32) {
      const int w = w0 + lane;
      const float v = w < a.vocab ? a.logits[(int64_t)w * a.rows + t] : NAN;
      float cut_v = best.value(a.top_k - 1);
      int cut_i = best.word(a.top_k - 1);
      unsigned left = __ballot_sync(0xffffffffu, v == v && ahead(v, w, cut_v, cut_i));
      while (left) {
        const int from = __ffs(left) - 1;
        left &= left - 1;
        const float nv = __shfl_sync(0xffffffffu, v, from);
        const int ni = w0 + from;
        if (!ahead(nv, ni, cut_v, cut_i)) continue;
        // its place: the words of the list that are ahead of it; those behind move one on
        const int place = __popc(__ballot_sync(0xffffffffu, ahead(best.v[0], best.id[0], nv, ni))) +
                          __popc(__ballot_sync(0xffffffffu, ahead(best.v[1], best.id[1], nv, ni)));
        float up0 = __shfl_up_sync(0xffffffffu, best.v[0], 1), up1 = __shfl_up_sync(0xffffffffu, best.v[1], 1);
        int ui0 = __shfl_up_sync(0xffffffffu, best.id[0], 1), ui1 = __shfl_up_sync(0xffffffffu, best.id[1], 1);
        const float over_v = __shfl_sync(0xffffffffu, best.v[0], 31);
        const int over_i = __shfl_sync(0xffffffffu, best.id[0], 31);
        if (lane == 0) up1 = over_v, ui1 = over_i;
        if (lane > place) best.v[0] = up0, best.id[0] = ui0;
        if (lane + 32 > place) best.v[1] = up1, best.id[1] = ui1;
        if (lane == place) best.v[0] = nv, best.id[0] = ni;
        if (lane + 32 == place) best.v[1] = nv, best.id[1] = ni;
        cut_v = best.value(a.top_k - 1);
        cut_i = best.word(a.top_k - 1);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    if (j >= a.top_k) break;
    const bool found = best.id[h] != INT32_MAX;
    a.top_index[(int64_t)t * a.top_k + j] = found ? best.id[h] : -1;
    a.top_logprob[(int64_t)t * a.top_k + j] = found ? (best.v[h] - m) * c - log_s : NAN;
  }
}

// One warp per row.
__global__ void __launch_bounds__(256) distill_prepare_kernel(const int* ids, const float* teacher, const float* logq,
                                                              const float* dloss, int n, int vocab, int rows, float inv_t,
                                                              float* g, float* at) {
  begin();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= rows) return;
  ids += (int64_t)t * n, teacher += (int64_t)t * n;
  Teacher of;
  of.start(ids, teacher, n, vocab, inv_t, lane);
  if (lane == 0) g[t] = of.taught ? dloss[t] * inv_t : 0.f;
  for (int j = lane; j < n; j += 32) {
    const int id = ids[j];
    float p = 0.f;
    if (id >= 0 && id < vocab && of.taught)
      for (int i = 0; i < n; ++i)  // (a word named twice has the sum of its entries, in their order)
        if (ids[i] == id) p += of.p(teacher[i]);
    at[(int64_t)t * n + j] = expf(logq[(int64_t)t * n + j]) - p;
  }
}

__global__ void __launch_bounds__(256) distill_scatter_kernel(const int* ids, const float* at, const float* g, const float* gs,
                                                              int n, int rows, int word0, int words, void* dz, int64_t lddz,
                                                              int f16) {
  begin();
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (i >= (int64_t)rows * n) return;
  const int id = ids[i] - word0;
  if (ids[i] < 0 || id < 0 || id >= words) return;
  const int t = (int)(i / n);
  const float gw = g[t] / *gs * kMmGradOne;
  st16(dz, id * lddz + t, gw == 0.f ? 0.f : at[i] * gw, f16);
}

}  // namespace

cudaError_t mm_sort_words(const int* words, int n, int vocab, int rows, int2* want, cudaStream_t s) {
  return launch(sort_words_kernel, dim3((rows + 7) / 8), 256, s, words, n, vocab, rows, want);
}

cudaError_t mm_score_join(const MmScores& a, cudaStream_t s) { return launch(score_join_kernel, dim3((a.rows + 7) / 8), 256, s, a); }

cudaError_t mm_distill_prepare(const int* ids, const float* teacher, const float* logq, const float* dloss, int n, int vocab,
                               int rows, float inv_t, float* g, float* at, cudaStream_t s) {
  return launch(distill_prepare_kernel, dim3((rows + 7) / 8), 256, s, ids, teacher, logq, dloss, n, vocab, rows, inv_t, g, at);
}

cudaError_t mm_distill_scatter(const int* ids, const float* at, const float* g, const float* gs, int n, int rows, int word0,
                               int words, void* dz, int64_t lddz, int f16, cudaStream_t s) {
  const int64_t blocks = ((int64_t)rows * n + 255) / 256;
  return launch(distill_scatter_kernel, dim3((unsigned)blocks), 256, s, ids, at, g, gs, n, rows, word0, words, dz, lddz, f16);
}

}  // namespace ds4
