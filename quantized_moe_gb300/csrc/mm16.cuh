// Products of 16-bit matrices (bf16 or fp16, fp32 accumulation) and their epilogues: the shared
// description of one product and the per-element epilogue arithmetic.
//
// Every product of the 16-bit operators is written as
//   out[c][l] = sum_r A(l, r) B(c, r),   l < lanes (contiguous in the output), c < cols, r < red,
// where A and B are row-major matrices read along either index:
//   y  = x W^T    lanes = output features (A = W, r contiguous), cols = rows of x (B = x, r contiguous)
//   dx = dy W     lanes = input features (A = W, l contiguous),  cols = rows (B = dy, r contiguous)
//   dW = dy^T x   lanes = input features (A = x, l contiguous),  cols = output features (B = dy, c contiguous)
// and, of the cross entropy over a vocabulary with weights W, where dz is kept transposed ([v][t]):
//   z          lanes = tokens (A = x, r contiguous), cols = words (B = W, r contiguous): a thread owns a
//              token, so that its softmax needs no exchange between threads. Scores of few tokens have them the
//              other way round: no lane is idle, and all of shared memory holds W on its way
//   dx = dz W  lanes = features (A = W, l contiguous), cols = tokens (B = dz, c contiguous)
//   dW = dz x  lanes = features (A = x, l contiguous), cols = words (B = dz, r contiguous)
// and, of the gated block with weights W = [gate; up] ([2 n][k]):
//   h          lanes = 16 gate features, the same 16 up features, the next 16 gate features, ... (A = W, r
//              contiguous), cols = rows of x: the 32 lanes of one warp of the epilogue hold both factors of its
//              16 results
#pragma once

#include "common.cuh"

namespace ds4 {

enum MmRag : int {
  MM_DENSE = 0,
  MM_RAG_COLS = 1,  // group g owns columns offsets[g] .. offsets[g+1]-1; A moves by its group stride
  MM_RAG_RED = 2    // group g owns that range of the reduction; the output moves by its group stride
};
enum MmEpi : int {
  MM_EPI_STORE = 0,     // out = act(v + bias) + residual, or v * scale + what is there
  MM_EPI_STATS = 1,     // per lane: max and sum of exponentials over the tile's columns; the label's value
  MM_EPI_SOFTGRAD = 2,  // out = (exp(v / T - lse) - [column is the label]) * g; its rows have room for whole, aligned pieces of
                        // eight, and the lanes behind the last token get zeros
  MM_EPI_GLU = 3,       // out = act(gate) * up; lanes are the features of out, A has twice as many rows
  MM_EPI_SCORE = 4,     // per lane: as STATS of v / T, and the entropy's sum; the logits of listed words; the logits
  MM_EPI_SCORE_FEW = 5  // the same of few tokens: lanes are words, columns (up to kMmFewRows) tokens, a tile 32 words
};
enum MmAct : int { MM_ACT_NONE = 0, MM_ACT_RELU = 1, MM_ACT_SILU = 2, MM_ACT_GELU = 3 };

struct MmOperand {
  const void* p;
  int64_t ld;            // elements from one row to the next
  int64_t group_stride;  // A only: elements from one group's matrix to the next
  int red_major;         // 1: the reduction index is the contiguous one
};

struct MmEpiArgs {
  void* out;
  int64_t ld, group_stride;  // elements
  int out_f32;               // out is fp32 (else the operands' type)
  int accumulate;            // out += v (out's own type; read in fp32)
  const float* acc_in;       // [cols][acc_ld] fp32 added to v, or null
  int64_t acc_ld;
  const float* scale;        // device scalar that multiplies the final sum, or null
  const void* bias;          // [lanes] or null
  const void* residual;      // [cols][ldr] or null
  int64_t ldr;
  void* z;                   // [cols][ldz] or null: v + bias, rounded
  int64_t ldz;
  int act;
  // cross entropy: lanes are tokens, columns a piece of the vocabulary from word0
  int word0, vocab, ignore;
  const int* labels;
  const float* lse;
  const float* g;        // dloss
  const float* gscale;   // device scalar: max |g|
  float2* part;          // [column tiles][lanes] (max, sum)
  float* zlab;           // [lanes] the label's logit
  float inv_t;           // 1 / T
  // scores, of tokens against the vocabulary in tiles of so many words (mm_score_tile)
  int tile;
  float* ent;            // [tiles][tokens] sum of (v - max) exp((v - max) / T), or null
  const int2* want;      // [tokens][n_want] (word, place), ascending; words that there are not come last
  const uint16_t* first; // [tokens][tiles] the first entry of want in or behind a tile
  const int* words;      // the caller's [tokens][n_want] instead of both: one, of few tokens up to kMmDirect of them
  int n_want;
  float* zwant;          // [tokens][n_want] the listed words' logits, by place
  float* logits;         // [vocab][tokens], or null
  float* chunk_max;      // [vocab / kMmStatChunk][tokens]; with logits
};

struct MmProblem {
  MmOperand a, b;
  int lanes, cols, red;
  int groups;          // 1 when dense
  const int* offsets;  // device [groups + 1], null when dense
  int rag, epi, f16;
  MmEpiArgs e;
  int* err;            // error word (bit 2 and a site bit: a pipeline wait gave up)
  int may_spread;      // the result need not have the bits of an unsplit sum: wide tiles may share out a long reduction
};

// Loads of what earlier launches wrote are plain ones throughout, never through the non-coherent path: a launch may
// start before those are complete (programmatic dependent launch) and must not meet lines cached before.
__device__ __forceinline__ float ld16(const void* p, int64_t i, int f16) {
  return f16 ? __half2float(static_cast<const __half*>(p)[i]) : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void st16(void* p, int64_t i, float v, int f16) {
  if (f16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// The normal distribution beyond u >= 0 is exp(-u^2 / 2) M(u). M falls from 1/2 like 1 / u: a polynomial in
// t = 1 / (1 + p u) without a constant term (the form of C. Hastings, Approximations for Digital Computers, 1955),
// fitted here for the smallest relative error over 0..14.5: 1e-7, with the arithmetic in fp32 5e-7. gelu and its slope are
// taken from it on both sides of zero: 1 + erf(z / sqrt 2) would cancel in the negative tail, where 16 bits still
// resolve the result (4 % off at z = -5). erfc would not, at a price (4096 x 4096 x 256: 56 us; erf and this form 40).
constexpr float kGaussFar = 40.f;  // exp(-u^2 / 2) is 0 from here on, and u may be infinite or NaN
__device__ __forceinline__ float gauss_mills(float u) {
  const float t = __fdividef(1.f, 1.f + 0.305f * u);
  float m = 0.03663887083530426f;
  m = m * t - 0.15274609625339508f;
  m = m * t + 0.18531492352485657f;
  m = m * t - 0.03762068599462509f;
  m = m * t + 0.1208404004573822f;
  m = m * t + 0.10347369313240051f;
  m = m * t + 0.12245868146419525f;
  m = m * t + 0.12164024263620377f;
  return m * t;
}
__device__ __forceinline__ float mm_gelu(float z) {
  const float u = fminf(fabsf(z), kGaussFar), away = u * (__expf(-0.5f * u * u) * gauss_mills(u));
  return z > 0.f ? z - away : z == z ? -away : z;
}

__device__ __forceinline__ float mm_relu(float z) { return z > 0.f ? z : z == z ? 0.f : z; }  // (NaN stays NaN)
// silu with the hardware exponential and division: a few units of 2^-22, and 0 instead of a value below 2^-118.
__device__ __forceinline__ float mm_silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }
// dy * act'(z). z is what its type kept of an fp32 value, so that it may be infinite where the forward was finite: the
// slope's limits are 0 and 1 there. z times a slope's factor that has run to 0 is taken at +-256, where that factor is
// already 0 in fp32 (infinity times 0 would be NaN). NaN stays NaN; a place that relu closes passes nothing, whatever lies
// in dy.
__device__ __forceinline__ float mm_act_back(float dy, float z, int act) {
  if (act == MM_ACT_RELU) return z > 0.f ? dy : z == z ? 0.f : z;
  if (act == MM_ACT_SILU) {
    const float near = z > 256.f ? 256.f : z < -256.f ? -256.f : z;  // (NaN stays)
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return dy * (s * (1.f + near * (1.f - s)));
  }
  const float u = fminf(fabsf(z), kGaussFar), f = __expf(-0.5f * u * u) * (gauss_mills(u) - u * 0.39894228040143268f);
  return z > 0.f ? dy * (1.f - f) : z == z ? dy * f : z;
}

// The gated block: h = act(g) u, and from z as its type kept it act(g) (silu at -inf is its limit 0) and
// dh u act'(g). Where the slope is 0 nothing passes, whatever dh and u hold.
__device__ __forceinline__ float mm_act(float z, int act) {
  return act == MM_ACT_SILU ? mm_silu(z) : act == MM_ACT_GELU ? mm_gelu(z) : act == MM_ACT_RELU ? mm_relu(z) : z;
}
__device__ __forceinline__ float mm_act_kept(float z, int act) { return mm_act(act == MM_ACT_SILU && z < -256.f ? -256.f : z, act); }
__device__ __forceinline__ float mm_glu_dgate(float dh, float g, float u, int act) {
  if (act == MM_ACT_NONE) return dh * u;
  const float slope = mm_act_back(1.f, g, act);
  return slope == 0.f ? 0.f : dh * u * slope;
}

// dz of the cross entropy is kept in 16 bits as (exp(z - lse) - [label]) * (g / max |g|) * 2^13. The
// division makes the label's term of a mean's gradient, -1 + p, a value just below a power of two,
// which 8 bits hold to about p (kept with g folded in, every label's term carried the same rounding
// error of up to 2^-9: the gradients were 1.6 times as far off as now); 2^13 keeps p down to 2^-27
// a normal fp16 number.
constexpr float kMmGradOne = 8192.f;

// Whether the TMA unit can address a matrix: 16-byte aligned start and row distances.
inline bool mm_aligned(const MmOperand& o) {
  return (uintptr_t)o.p % 16 == 0 && o.ld % 8 == 0 && o.group_stride % 8 == 0 && o.ld < (int64_t)1 << 36 && o.group_stride < (int64_t)1 << 36;
}
// Words of one softmax partial: part[] has ceil(vocab / kMmStatTile) rows of one entry per token.
constexpr int kMmStatTile = 256;
constexpr int kMmStatChunk = 32;  // words of one chunk's maximum
constexpr int kMmFewRows = 32;    // tokens of MM_EPI_SCORE_FEW

// Sets kernel attributes on the current device (once per device).
cudaError_t mm_prepare();
// An estimate of a dense product's time (columns of a tile times stages of the reduction, by rounds over the SMs).
int64_t mm_cost(int lanes, int cols, int red, bool b_red);
// Words of a tile of scores. Up to 128 rows a call is one pass over W, for which smaller tiles leave more of it in flight (64
// rows of 129280 words, d 4096: 168 us, in tiles of 256 178); beyond, on pairs of CTAs, tiles of 128 would load x
// once more for every word (333 rows of 32003 words, d 1000: 42 us, 33).
inline int mm_score_tile(int rows, bool few) { return few ? kMmStatChunk : rows <= 128 ? 128 : kMmStatTile; }
// Softmax partials of each of few tokens: one for every epilogue warp.
int mm_few_parts(int vocab);
constexpr int kMmFewParts = 1024;  // at most
// Launches one product. Nothing to do (no lanes or columns) is not an error.
cudaError_t mm_launch(const MmProblem& p, cudaStream_t s);

// dz = dy * act'(z) rounded to 16 bits (dz null: not stored) and, when part is not null, its unrounded
// column sums over chunks of rows, part[chunk][n]; then db = the sum over the chunks in order.
int mm_colsum_chunks(int rows);
cudaError_t mm_act_grad(const void* dy, int64_t lddy, const void* z, int64_t ldz, void* dz, int64_t lddz, float* part,
                        void* db, int rows, int n, int act, int f16, cudaStream_t s);
// Joins the softmax partials of each token: lse, loss, and bit 0 of *err for labels outside the vocabulary.
cudaError_t mm_softmax_join(const float2* part, int tiles, const float* zlab, const int* labels, int ignore, int vocab,
                            int rows, float* loss, float* lse, int* err, cudaStream_t s);
// gs[0] = max |g| over the rows with a label (labels null: all) and a finite g (1 where that is 0), gs[1] = gs[0] / kMmGradOne.
cudaError_t mm_grad_scale(const float* g, const int* labels, int ignore, int vocab, int rows, float* gs, cudaStream_t s);

// The gated block's dz = [dh * up * act'(gate), dh * act(gate)] rounded to 16 bits, from z = [gate, up] ([rows][2 n]), of
// the rows that have a group (offsets null: all).
cudaError_t mm_glu_grad(const void* dh, int64_t lddh, const void* z, int64_t ldz, void* dz, int64_t lddz, const int* offsets,
                        int groups, int rows, int n, int act, int f16, cudaStream_t s);

// Sorts each row's n words for the scores' epilogue (MmEpiArgs::want, first): a word outside the vocabulary comes last.
constexpr int kMmListed = 256, kMmTop = 64;  // most given words, and best words, of a row
constexpr int kMmDirect = 4;  // given words of few tokens that need no sorting: 4 us of a launch
cudaError_t mm_sort_words(const int* words, int n, int vocab, int rows, int tile, int2* want, uint16_t* first, cudaStream_t s);
// What the scores' partials say of each row (temperature T = 1 / inv_t).
struct MmScores {
  const float2* part;
  const float* ent;
  int parts, rows, vocab;
  int tile;             // words of a partial; kMmStatChunk: partials are not of tiles (few rows)
  float inv_t;
  const float* zwant;   // [rows][n] logits of the listed words
  const int* words;     // [rows][n]
  int n;
  float* lse;           // [rows], or null
  int* err;             // bit 0: a word other than -1 outside the vocabulary
  // log probabilities
  float* logprob;       // [rows][n]
  float* entropy;       // [rows], or null
  const float* logits;  // [vocab][rows]
  const float* chunk_max;
  int top_k;
  int* top_index;       // [rows][top_k]
  float* top_logprob;
  // distillation: logprob is log q of the listed words
  const float* teacher;  // [rows][n] logits
  float* loss;           // [rows]
};
cudaError_t mm_score_join(const MmScores& a, cudaStream_t s);
// The distillation's gradient at the listed words: g[t] = dloss[t] / T of the rows with a teacher, else 0, and
// at[t][j] = exp(log q_j) - the teacher's probability of that word (all its entries together).
cudaError_t mm_distill_prepare(const int* ids, const float* teacher, const float* logq, const float* dloss, int n, int vocab,
                               int rows, float inv_t, float* g, float* at, cudaStream_t s);
// ... and its way into a piece of dz ([words][lddz], from word0): the listed words' places are overwritten.
cudaError_t mm_distill_scatter(const int* ids, const float* at, const float* g, const float* gs, int n, int rows, int word0,
                               int words, void* dz, int64_t lddz, int f16, cudaStream_t s);

}  // namespace ds4
