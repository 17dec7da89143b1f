// The small kernels beside the 16-bit products: dz = dy * act'(z) with the column sums of db, the
// join of the softmax partials, and the scale that dz of the cross entropy carries.
#include "mm16.cuh"

namespace ds4 {
namespace {

constexpr int kMaxChunks = 256;

// Column sums run over chunks of at least 16 rows: one block computes a strip of 64 columns of one
// chunk with four rows of threads, adds these through shared memory and writes one partial per
// column; the second kernel adds the chunks in order. The order of every sum is fixed.
__global__ void __launch_bounds__(256) act_grad_kernel(const void* __restrict__ dy, int64_t lddy,
                                                       const void* __restrict__ z, int64_t ldz, void* __restrict__ dz,
                                                       int64_t lddz, float* __restrict__ part, int rows, int n,
                                                       int act, int f16, int chunk_rows) {
  __shared__ float s[4][64];
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + tx;
  const int r0 = blockIdx.y * chunk_rows, r1 = min(r0 + chunk_rows, rows);
  float sum = 0.f;
  if (c < n)
    for (int r = r0 + ty; r < r1; r += 4) {
      float v = ld16(dy, (int64_t)r * lddy + c, f16);
      if (act != MM_ACT_NONE) v *= mm_act_slope(ld16(z, (int64_t)r * ldz + c, f16), act);
      if (dz) st16(dz, (int64_t)r * lddz + c, v, f16);
      sum += v;
    }
  if (!part) return;
  s[ty][tx] = sum;
  __syncthreads();
  if (ty == 0 && c < n) part[(int64_t)blockIdx.y * n + c] = (s[0][tx] + s[1][tx]) + (s[2][tx] + s[3][tx]);
}

__global__ void colsum_join_kernel(const float* __restrict__ part, int chunks, int n, void* __restrict__ db, int f16) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= n) return;
  float v = 0.f;
  for (int i = 0; i < chunks; ++i) v += part[(int64_t)i * n + c];
  st16(db, c, v, f16);
}

// One warp per token: the tiles' (max, sum) are joined as (M, S) with M = max m_i and
// S = sum s_i exp(m_i - M); lse = M + log S.
__global__ void __launch_bounds__(256) softmax_join_kernel(const float2* __restrict__ part, int tiles,
                                                           const float* __restrict__ zlab,
                                                           const int* __restrict__ labels, int ignore, int vocab,
                                                           int rows, float* __restrict__ loss,
                                                           float* __restrict__ lse, int* err) {
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= rows) return;
  float m = -INFINITY;
  for (int i = lane; i < tiles; i += 32) m = fmaxf(m, part[(int64_t)i * rows + t].x);
  m = warp_max(m);
  float sum = 0.f;
  for (int i = lane; i < tiles; i += 32) {
    const float2 q = part[(int64_t)i * rows + t];
    sum += q.y * expf(q.x - m);
  }
  sum = warp_sum(sum);
  if (lane == 0) {
    const float l = m + logf(sum);
    const int lab = labels[t];
    const bool out = lab < 0 || lab >= vocab;
    if (out && lab != ignore) atomicOr(err, 1);
    lse[t] = l;
    loss[t] = out || lab == ignore ? 0.f : l - zlab[t];
  }
}

__global__ void __launch_bounds__(1024) grad_scale_kernel(const float* __restrict__ g, const int* __restrict__ labels,
                                                          int ignore, int vocab, int rows, float* __restrict__ gs) {
  __shared__ float s[32];
  float m = 0.f;
  for (int i = threadIdx.x; i < rows; i += 1024) {
    const int lab = labels[i];
    if (lab != ignore && lab >= 0 && lab < vocab) m = fmaxf(m, fabsf(g[i]));
  }
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = warp_max(s[threadIdx.x]);
    if (threadIdx.x == 0) {
      if (!(m > 0.f) || !isfinite(m)) m = 1.f;
      gs[0] = m;
      gs[1] = m * (1.f / kMmGradOne);
    }
  }
}

}  // namespace

int mm_colsum_chunks(int rows) {
  const int c = (rows + 15) / 16;
  return c < 1 ? 1 : c > kMaxChunks ? kMaxChunks : c;
}

cudaError_t mm_act_grad(const void* dy, int64_t lddy, const void* z, int64_t ldz, void* dz, int64_t lddz, float* part,
                        void* db, int rows, int n, int act, int f16, cudaStream_t s) {
  const int chunks = mm_colsum_chunks(rows);
  act_grad_kernel<<<dim3((n + 63) / 64, chunks), 256, 0, s>>>(dy, lddy, z, ldz, dz, lddz, part, rows, n, act, f16,
                                                              (rows + chunks - 1) / chunks);
  if (part) colsum_join_kernel<<<(n + 127) / 128, 128, 0, s>>>(part, chunks, n, db, f16);
  return cudaGetLastError();
}

cudaError_t mm_softmax_join(const float2* part, int tiles, const float* zlab, const int* labels, int ignore, int vocab,
                            int rows, float* loss, float* lse, int* err, cudaStream_t s) {
  softmax_join_kernel<<<(rows + 7) / 8, 256, 0, s>>>(part, tiles, zlab, labels, ignore, vocab, rows, loss, lse, err);
  return cudaGetLastError();
}

cudaError_t mm_grad_scale(const float* g, const int* labels, int ignore, int vocab, int rows, float* gs,
                          cudaStream_t s) {
  grad_scale_kernel<<<1, 1024, 0, s>>>(g, labels, ignore, vocab, rows, gs);
  return cudaGetLastError();
}

}  // namespace ds4
