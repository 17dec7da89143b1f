// The small kernels beside the 16-bit products: dz = dy * act'(z) with the column sums of db, the
// gated block's dz, the join of the softmax partials, and the scale that dz of the cross entropy carries.
#include "mm16_small.cuh"

namespace ds4 {
namespace {

constexpr int kMaxChunks = 128;

// dz = dy * act'(z), and the column sums of dz (unrounded, fp32). A block takes 256 columns of one chunk of rows: each of
// its eight warps walks every eighth row with one 16-byte load per operand (eight columns a thread), then the warps'
// sums are added in order through shared memory, one partial per column and chunk. The second kernel adds the chunks
// in order, 8 rows of threads per column. The order of every sum is fixed. dz itself is rounded to 16 bits, because the
// tensor cores multiply such operands: the gradients' error is 1.4 times that of a result rounded once. HBM bound: dy, z and dz cross it once
// (elements that cannot be moved 8 at a time go one by one).
template <bool VEC, int ACT>
__global__ void __launch_bounds__(256) act_grad_kernel(const void* dy, int64_t lddy,
                                                       const void* z, int64_t ldz, void* dz,
                                                       int64_t lddz, float* part, int rows, int n,
                                                       int f16, int chunk_rows) {
  __shared__ float s[8][256 + 8];
  begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + lane * 8;
  const int r0 = blockIdx.y * chunk_rows, r1 = min(r0 + chunk_rows, rows);
  float sum[8] = {};
  if (c < n) {
    for (int r = r0 + warp; r < r1; r += 16) {  // two rows in flight
      Eight hy[2], hz[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rk = r + 8 * k;
        const uint16_t* py = static_cast<const uint16_t*>(dy) + (int64_t)rk * lddy + c;
        const uint16_t* pz = static_cast<const uint16_t*>(z) + (int64_t)rk * ldz + c;
        if (VEC) {
          hy[k].piece() = rk < r1 ? *reinterpret_cast<const uint4*>(py) : make_uint4(0, 0, 0, 0);
          if (ACT != MM_ACT_NONE) hz[k].piece() = rk < r1 ? *reinterpret_cast<const uint4*>(pz) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            hy[k].h[i] = rk < r1 && c + i < n ? py[i] : (uint16_t)0;
            if (ACT != MM_ACT_NONE) hz[k].h[i] = rk < r1 && c + i < n ? pz[i] : (uint16_t)0;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rk = r + 8 * k;
        if (rk >= r1) break;
        Eight out;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float g = ld16(hy[k].h, i, f16);
          if (ACT != MM_ACT_NONE) g = mm_act_back(g, ld16(hz[k].h, i, f16), ACT);
          sum[i] += g;
          st16(out.h, i, g, f16);
        }
        if (dz) {
          uint16_t* pd = static_cast<uint16_t*>(dz) + (int64_t)rk * lddz + c;
          if (VEC) {
            *reinterpret_cast<uint4*>(pd) = out.piece();
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < n) pd[i] = out.h[i];
          }
        }
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[warp][lane * 8 + i] = sum[i];
  __syncthreads();
  const int cc = blockIdx.x * 256 + threadIdx.x;
  if (cc < n) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += s[w][threadIdx.x];
    part[(int64_t)blockIdx.y * n + cc] = v;
  }
}

// The gated block's dz: for h = act(g) u, dg = dh u act'(g) and du = dh act(g), each rounded to 16 bits because the
// tensor cores multiply such operands. A thread takes eight neighbouring features of a row; dh, z and dz cross HBM once.
template <bool VEC, int ACT>
__global__ void __launch_bounds__(256) glu_grad_kernel(const void* dh, int64_t lddh, const void* z, int64_t ldz, void* dz,
                                                       int64_t lddz, const int* offsets, int groups, int rows, int n, int f16) {
  begin();
  const int units = (n + 7) / 8;
  int lo = 0, hi = rows;
  if (offsets) lo = min(max(*offsets, 0), rows), hi = min(max(*(offsets + groups), 0), rows);
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < (int64_t)rows * units; i += gridDim.x * (int64_t)256) {
    const int r = (int)(i / units), c = (int)(i - (int64_t)r * units) * 8;
    if (r < lo || r >= hi) continue;
    const uint16_t* ph = static_cast<const uint16_t*>(dh) + r * lddh + c;
    const uint16_t* pz = static_cast<const uint16_t*>(z) + r * ldz + c;
    uint16_t* pd = static_cast<uint16_t*>(dz) + r * lddz + c;
    Eight h, g, u, dg, du;
    if (VEC) {
      h.piece() = *reinterpret_cast<const uint4*>(ph);
      g.piece() = *reinterpret_cast<const uint4*>(pz);
      u.piece() = *reinterpret_cast<const uint4*>(pz + n);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool there = c + k < n;
        h.h[k] = there ? ph[k] : (uint16_t)0, g.h[k] = there ? pz[k] : (uint16_t)0, u.h[k] = there ? pz[n + k] : (uint16_t)0;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float dhv = ld16(h.h, k, f16), gv = ld16(g.h, k, f16), uv = ld16(u.h, k, f16);
      st16(dg.h, k, mm_glu_dgate(dhv, gv, uv, ACT), f16);
      st16(du.h, k, dhv * mm_act_kept(gv, ACT), f16);
    }
    if (VEC) {
      *reinterpret_cast<uint4*>(pd) = dg.piece();
      *reinterpret_cast<uint4*>(pd + n) = du.piece();
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < n) pd[k] = dg.h[k], pd[n + k] = du.h[k];
    }
  }
}

__global__ void __launch_bounds__(256) colsum_join_kernel(const float* part, int chunks, int n,
                                                          void* db, int f16) {
  __shared__ float s[8][32];
  begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int i = warp; i < chunks; i += 8) v += part[(int64_t)i * n + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < n) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += s[w][lane];
    st16(db, c, v, f16);
  }
}

// One warp per token: the tiles' (max, sum) are joined as (M, S) with M = max m_i and
// S = sum s_i exp(m_i - M); lse = M + log S. A tile at the maximum adds its sum as it is, so that a row whose every logit is
// -inf has S = 0 and lse = -inf (exp(-inf + inf) would be NaN); a tile with NaN logits has a sum of NaN.
__global__ void __launch_bounds__(256) softmax_join_kernel(const float2* part, int tiles,
                                                           const float* zlab,
                                                           const int* labels, int ignore, int vocab,
                                                           int rows, float* loss,
                                                           float* lse, int* err) {
  begin();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= rows) return;
  float m = -INFINITY;
  for (int i = lane; i < tiles; i += 32) m = fmaxf(m, part[(int64_t)i * rows + t].x);
  m = warp_max(m);
  float sum = 0.f;
  for (int i = lane; i < tiles; i += 32) {
    const float2 q = part[(int64_t)i * rows + t];
    sum += q.x == m ? q.y : q.y * expf(q.x - m);
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

// The scale of dz: the largest |g| of the rows with a label. A row whose g is not finite keeps that to itself: its dz is
// not finite under any scale, and the scale of the others may not depend on it (an fp16 dz would overflow).
__global__ void __launch_bounds__(1024) grad_scale_kernel(const float* g, const int* labels,
                                                          int ignore, int vocab, int rows, float* gs) {
  __shared__ float s[32];
  begin();
  float m = 0.f;
  for (int i = threadIdx.x; i < rows; i += 1024) {
    const int lab = labels ? labels[i] : 0;
    if (!labels || (lab != ignore && lab >= 0 && lab < vocab)) m = fmaxf(m, isfinite(g[i]) ? fabsf(g[i]) : 0.f);
  }
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = warp_max(s[threadIdx.x]);
    if (threadIdx.x == 0) {
      if (m == 0.f) m = 1.f;
      gs[0] = m;
      gs[1] = m * (1.f / kMmGradOne);
    }
  }
}

}  // namespace

int mm_colsum_chunks(int rows) {
  const int c = (rows + 31) / 32;
  return c < 1 ? 1 : c > kMaxChunks ? kMaxChunks : c;
}

cudaError_t mm_act_grad(const void* dy, int64_t lddy, const void* z, int64_t ldz, void* dz, int64_t lddz, float* part,
                        void* db, int rows, int n, int act, int f16, cudaStream_t s) {
  const int chunks = mm_colsum_chunks(rows), chunk_rows = (rows + chunks - 1) / chunks;
  const auto vec = [](const void* p, int64_t ld) { return !p || ((uintptr_t)p % 16 == 0 && ld % 8 == 0); };
  const dim3 grid((n + 255) / 256, chunks);
  const bool wide = n % 8 == 0 && vec(dy, lddy) && (act == MM_ACT_NONE || vec(z, ldz)) && vec(dz, lddz);
  const auto run = [&](auto kernel) { return launch(kernel, grid, 256, s, dy, lddy, z, ldz, dz, lddz, part, rows, n, f16, chunk_rows); };
  cudaError_t e;
  switch (act) {  // (one kernel for each: all activations in one overflow the instruction cache, 4096 x 2048 silu 27 us instead of 12)
    case MM_ACT_RELU: e = run(wide ? act_grad_kernel<true, MM_ACT_RELU> : act_grad_kernel<false, MM_ACT_RELU>); break;
    case MM_ACT_SILU: e = run(wide ? act_grad_kernel<true, MM_ACT_SILU> : act_grad_kernel<false, MM_ACT_SILU>); break;
    case MM_ACT_GELU: e = run(wide ? act_grad_kernel<true, MM_ACT_GELU> : act_grad_kernel<false, MM_ACT_GELU>); break;
    default: e = run(wide ? act_grad_kernel<true, MM_ACT_NONE> : act_grad_kernel<false, MM_ACT_NONE>);
  }
  if (e == cudaSuccess && part) e = launch(colsum_join_kernel, dim3((n + 31) / 32), 256, s, part, chunks, n, db, f16);
  return e;
}

cudaError_t mm_glu_grad(const void* dh, int64_t lddh, const void* z, int64_t ldz, void* dz, int64_t lddz, const int* offsets,
                        int groups, int rows, int n, int act, int f16, cudaStream_t s) {
  const auto vec = [](const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; };
  const bool wide = n % 8 == 0 && vec(dh, lddh) && vec(z, ldz) && vec(dz, lddz);
  const int units = (n + 7) / 8;
  const int64_t blocks = ((int64_t)rows * units + 255) / 256;
  const dim3 grid((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20));
  const auto run = [&](auto kernel) { return launch(kernel, grid, 256, s, dh, lddh, z, ldz, dz, lddz, offsets, groups, rows, n, f16); };
  switch (act) {
    case MM_ACT_RELU: return run(wide ? glu_grad_kernel<true, MM_ACT_RELU> : glu_grad_kernel<false, MM_ACT_RELU>);
    case MM_ACT_SILU: return run(wide ? glu_grad_kernel<true, MM_ACT_SILU> : glu_grad_kernel<false, MM_ACT_SILU>);
    case MM_ACT_GELU: return run(wide ? glu_grad_kernel<true, MM_ACT_GELU> : glu_grad_kernel<false, MM_ACT_GELU>);
    default: return run(wide ? glu_grad_kernel<true, MM_ACT_NONE> : glu_grad_kernel<false, MM_ACT_NONE>);
  }
}

cudaError_t mm_softmax_join(const float2* part, int tiles, const float* zlab, const int* labels, int ignore, int vocab,
                            int rows, float* loss, float* lse, int* err, cudaStream_t s) {
  return launch(softmax_join_kernel, dim3((rows + 7) / 8), 256, s, part, tiles, zlab, labels, ignore, vocab, rows, loss, lse, err);
}

cudaError_t mm_grad_scale(const float* g, const int* labels, int ignore, int vocab, int rows, float* gs,
                          cudaStream_t s) {
  return launch(grad_scale_kernel, dim3(1), 1024, s, g, labels, ignore, vocab, rows, gs);
}

}  // namespace ds4
