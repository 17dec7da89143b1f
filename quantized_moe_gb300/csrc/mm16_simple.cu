// The plain form of the 16-bit products on the FMA pipe: a 64 x 64 output tile per block, 4 x 4
// per thread, operands staged through shared memory as fp32 in steps of 16 of the reduction. Reads
// any strides and both index orders, and runs every epilogue. One thread does 16 FMAs per 8
// shared-memory words, so shared memory, not the FMA pipe, bounds it.
#include "mm16.cuh"

namespace ds4 {
namespace {

constexpr int T = 64, RK = 16;

__global__ void __launch_bounds__(256) mm_simple_kernel(const MmProblem p, int lane_tiles) {
  __shared__ float As[RK][T + 1], Bs[RK][T + 1], Zs[T][T + 1];
  const int lt = blockIdx.x % lane_tiles;
  int ct = blockIdx.x / lane_tiles, g = 0, c_lo = 0, c_hi = p.cols, r_lo = 0, r_hi = p.red;
  if (p.rag == MM_RAG_COLS) {
    for (g = 0; g < p.groups; ++g) {  // the group that holds column tile ct
      const int2 r = mm_range(p.offsets, g, p.cols);
      const int n = (r.y - r.x + T - 1) / T;
      if (ct < n) {
        c_lo = r.x, c_hi = r.y;
        break;
      }
      ct -= n;
    }
    if (g == p.groups) return;
  } else if (p.rag == MM_RAG_RED) {
    g = blockIdx.z;
    const int2 r = mm_range(p.offsets, g, p.red);
    r_lo = r.x, r_hi = r.y;
  }
  const int l0 = lt * T, c0 = c_lo + ct * T;
  const int64_t a_base = p.rag == MM_RAG_COLS ? g * p.a.group_stride : 0;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int r0 = r_lo; r0 < r_hi; r0 += RK) {
    for (int i = threadIdx.x; i < T * RK; i += 256) {
      const int ar = p.a.red_major ? i % RK : i / T, al = p.a.red_major ? i / RK : i % T;
      const int br = p.b.red_major ? i % RK : i / T, bc = p.b.red_major ? i / RK : i % T;
      float a = 0.f, b = 0.f;
      if (r0 + ar < r_hi && l0 + al < p.lanes)
        a = ld16(p.a.p, a_base + (p.a.red_major ? (int64_t)(l0 + al) * p.a.ld + r0 + ar : (int64_t)(r0 + ar) * p.a.ld + l0 + al), p.f16);
      if (r0 + br < r_hi && c0 + bc < c_hi)
        b = ld16(p.b.p, p.b.red_major ? (int64_t)(c0 + bc) * p.b.ld + r0 + br : (int64_t)(r0 + br) * p.b.ld + c0 + bc, p.f16);
      As[ar][al] = a;
      Bs[br][bc] = b;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += Bs[r][ty + 16 * i] * As[r][tx + 16 * j];
    __syncthreads();
  }
  const MmEpiArgs& e = p.e;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + ty + 16 * i, l = l0 + tx + 16 * j;
      float v = acc[i][j];
      if (p.epi == MM_EPI_STATS) {
        Zs[ty + 16 * i][tx + 16 * j] = l < p.lanes ? v : -INFINITY;
        if (c < c_hi && l < p.lanes && l + e.lane0 == __ldg(e.labels + c)) e.zlab[c] = v;
        continue;
      }
      if (c >= c_hi || l >= p.lanes) continue;
      if (p.epi == MM_EPI_SOFTGRAD) {
        const int lab = __ldg(e.labels + c);
        const bool skip = lab == e.ignore || lab < 0 || lab >= e.vocab;
        v = skip ? 0.f : (expf(v - __ldg(e.lse + c)) - (l + e.lane0 == lab ? 1.f : 0.f)) * (__ldg(e.g + c) / __ldg(e.gscale) * kMmGradOne);
        st16(e.out, (int64_t)c * e.ld + l, v, p.f16);
        continue;
      }
      if (e.acc_in) v += e.acc_in[(int64_t)c * e.acc_ld + l];
      if (e.scale) v *= __ldg(e.scale);
      if (e.bias) v += ld16(e.bias, l, p.f16);
      if (e.z) st16(e.z, (int64_t)c * e.ldz + l, v, p.f16);
      v = mm_act(v, e.act);
      if (e.residual) v += ld16(e.residual, (int64_t)c * e.ldr + l, p.f16);
      const int64_t o = (p.rag == MM_RAG_RED ? g * e.group_stride : 0) + (int64_t)c * e.ld + l;
      if (e.out_f32) {
        float* out = static_cast<float*>(e.out);
        out[o] = e.accumulate ? out[o] + v : v;
      } else {
        st16(e.out, o, e.accumulate ? ld16(e.out, o, p.f16) + v : v, p.f16);
      }
    }
  if (p.epi == MM_EPI_STATS) {
    __syncthreads();
    const int c = c0 + threadIdx.x;
    if (threadIdx.x < T && c < c_hi) {
      float m = -INFINITY, sum = 0.f;
      for (int l = 0; l < T; ++l) m = fmaxf(m, Zs[threadIdx.x][l]);
      if (m != -INFINITY)  // (a tile of infinitely improbable words adds nothing)
        for (int l = 0; l < T && l0 + l < p.lanes; ++l) sum += expf(Zs[threadIdx.x][l] - m);
      e.part[(int64_t)lt * p.cols + c] = make_float2(m, sum);
    }
  }
}

}  // namespace

cudaError_t mm_prepare() { return cudaSuccess; }

cudaError_t mm_launch(const MmProblem& p, cudaStream_t s) {
  if (p.lanes <= 0 || p.cols <= 0) return cudaSuccess;
  const int lane_tiles = (p.lanes + T - 1) / T;
  const int64_t col_tiles = (p.cols + T - 1) / T + (p.rag == MM_RAG_COLS ? p.groups : 0);
  if (lane_tiles * col_tiles > 0x7fffffff) return cudaErrorInvalidValue;
  mm_simple_kernel<<<dim3((unsigned)(lane_tiles * col_tiles), 1, p.rag == MM_RAG_RED ? p.groups : 1), 256, 0, s>>>(p, lane_tiles);
  return cudaGetLastError();
}

}  // namespace ds4
