// C entry points of the operators on 16-bit matrices: argument checks, workspace layout and the
// sequence of launches. Host code, and the device word that the kernels raise flags in.
#include <algorithm>
#include <mutex>
#include <string>

#include "../../include/ds4moe.h"
#include "mm16.cuh"

namespace ds4 {
int set_error(int code, const char* msg);  // records the message returned by ds4moe_last_error
}

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxWidth = 1 << 24;
constexpr int kMaxGroups = 1024;
constexpr int kPieceMax = 16384, kPieceMin = 256;  // words of one piece of the vocabulary

static __device__ int g_mm_err;  // flags of ds4moe_ops_status
std::mutex g_mu;
int* g_err_ptr[kMaxDevices] = {};

// The checks of one call: the first failure is recorded under the entry point's name.
struct Check {
  const char* fn;
  int code = DS4MOE_OK, dev = -1;
  explicit Check(const char* f) : fn(f) {}
  bool ok() const { return code == DS4MOE_OK; }
  void fail(int c, const std::string& msg) {
    if (ok()) code = ds4::set_error(c, (std::string(fn) + ": " + msg).c_str());
  }
  void invalid(const std::string& msg) { fail(DS4MOE_ERR_INVALID_ARG, msg); }
  void rows(int64_t v) {
    if (v < 0 || v > kMaxWidth) invalid("rows=" + std::to_string(v) + " must be in 0..2^24");
  }
  void width(const char* name, int64_t v) {
    if (v < 1 || v > kMaxWidth) invalid(std::string(name) + "=" + std::to_string(v) + " must be in 1..2^24");
  }
  void dtype(int v) {
    if (v != DS4MOE_BF16 && v != DS4MOE_FP16) fail(DS4MOE_ERR_UNSUPPORTED_FORMAT, "dtype=" + std::to_string(v) + " is not DS4MOE_BF16 or DS4MOE_FP16");
  }
  void act(int v) {
    if (v < DS4MOE_ACT_NONE || v > DS4MOE_ACT_GELU) invalid("act=" + std::to_string(v) + " is not a ds4moe_act");
  }
  // A row distance: 0 stands for the width.
  int64_t ld(const char* name, int64_t v, int64_t width) {
    if (v == 0) return width;
    if (v < width || v > (int64_t)1 << 40) invalid(std::string(name) + "=" + std::to_string(v) + " is less than the row's width " + std::to_string(width) + " (or above 2^40)");
    return v;
  }
  void device() {
    if (!ok()) return;
    if (cudaGetDevice(&dev) != cudaSuccess) {
      cudaGetLastError();
      fail(DS4MOE_ERR_CUDA, "no current CUDA device");
    } else if (dev < 0 || dev >= kMaxDevices) {
      invalid("device ordinal above 63");
    }
  }
  // A required (or, with optional, possibly null) device pointer.
  void ptr(const char* name, const void* p, int align, bool optional = false) {
    if (!ok() || (optional && !p)) return;
    if (!p) return invalid(std::string(name) + " is NULL");
    if ((uintptr_t)p % align) return invalid(std::string(name) + " is not aligned to " + std::to_string(align) + " bytes");
    if (dev < 0) return;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return invalid(std::string(name) + " is not device memory");
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return invalid(std::string(name) + " is not device memory");
    if (at.device != dev && at.type == cudaMemoryTypeDevice) fail(DS4MOE_ERR_DEVICE_MISMATCH, std::string(name) + " lives on another device than the current one");
  }
  int cuda(cudaError_t e) {
    if (e != cudaSuccess) {
      cudaGetLastError();  // reported here, not at the caller's next check
      fail(DS4MOE_ERR_CUDA, cudaGetErrorString(e));
    }
    return code;
  }
  // The current device's error word.
  int* err_word() {
    if (!ok()) return nullptr;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_err_ptr[dev]) {
      void* p = nullptr;
      cudaError_t e = cudaGetSymbolAddress(&p, g_mm_err);
      if (e == cudaSuccess) e = ds4::mm_prepare();
      if (e != cudaSuccess) {
        cudaGetLastError();
        fail(DS4MOE_ERR_CUDA, std::string("setting the kernels up failed: ") + cudaGetErrorString(e));
        return nullptr;
      }
      g_err_ptr[dev] = static_cast<int*>(p);
    }
    return g_err_ptr[dev];
  }
};

// No exception may leave a C entry point.
template <class F>
int guarded(const char* fn, F&& f) {
  try {
    return f();
  } catch (...) {
    return ds4::set_error(DS4MOE_ERR_OOM, fn);
  }
}

ds4::MmProblem product(const void* a, int64_t lda, bool a_red, const void* b, int64_t ldb, bool b_red, int lanes,
                       int cols, int red, int dtype, void* out, int64_t ld, int* err) {
  ds4::MmProblem p = {};
  p.a = {a, lda, 0, a_red};
  p.b = {b, ldb, 0, b_red};
  p.lanes = lanes, p.cols = cols, p.red = red;
  p.groups = 1;
  p.f16 = dtype == DS4MOE_FP16;
  p.e.out = out;
  p.e.ld = ld;
  p.err = err;
  return p;
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

void groups(Check& c, int n) {
  if (n < 1 || n > kMaxGroups) c.invalid("n_groups=" + std::to_string(n) + " must be in 1..1024");
}
// The distance between the groups' [n x k] matrices.
int64_t stride(Check& c, const char* name, int64_t v, int64_t n, int64_t ld) {
  if (v == 0) return n * ld;
  if (v < n * ld) c.invalid(std::string(name) + "=" + std::to_string(v) + " is less than one matrix (n * its row distance)");
  return v;
}

// Workspace of the cross entropy: the forward's partials and label logits, or the gradient's scale
// words, fp32 sum of dx and one piece of dz.
int64_t ce_forward_bytes(int64_t rows, int64_t vocab) { return up(8 * rows * ((vocab + ds4::kMmStatTile - 1) / ds4::kMmStatTile), 16) + 4 * rows; }
int64_t ce_grad_bytes(int64_t rows, int64_t d, int64_t piece) { return 16 + up(4 * rows * d, 16) + 2 * up(rows, 8) * piece; }

// The piece of the vocabulary, up to `most` words, with the shortest schedule: a piece whose products leave the last
// round over the SMs nearly full beats a larger one that does not (2048 rows, 129280 words, d 4096: 14592 words make
// 456 and 912 tiles, whole rounds of 76 pairs).
int64_t best_piece(int64_t most, int rows, int vocab, int d, bool dx, bool dw) {
  const auto one = [&](int64_t words) -> int64_t {
    if (words <= 0) return 0;
    const int64_t launch = 3400;  // about 4 us, in mm_cost's units
    return ds4::mm_cost(rows, (int)words, d, true) + launch + (dx ? ds4::mm_cost(d, rows, (int)words, false) + launch : 0) +
           (dw ? ds4::mm_cost(d, (int)words, rows, true) + launch : 0);
  };
  int64_t best = most, best_cost = INT64_MAX;
  for (int64_t piece = most; 2 * piece > most && piece >= kPieceMin; piece -= kPieceMin) {
    const int64_t cost = vocab / piece * one(piece) + one(vocab % piece);
    if (cost < best_cost) best_cost = cost, best = piece;
  }
  return best;
}

}  // namespace

extern "C" int ds4moe_grouped_mm(const void* x, const void* w, const int32_t* offsets, void* y, int32_t rows,
                                 int32_t n, int32_t k, int32_t n_groups, int32_t dtype, int64_t ldx, int64_t ldw,
                                 int64_t w_stride, int64_t ldy, void* stream) {
  return guarded("ds4moe_grouped_mm", [&]() -> int {
    Check c("ds4moe_grouped_mm");
    c.rows(rows), c.width("n", n), c.width("k", k), c.dtype(dtype), groups(c, n_groups);
    ldx = c.ld("ldx", ldx, k), ldw = c.ld("ldw", ldw, k), ldy = c.ld("ldy", ldy, n);
    w_stride = stride(c, "w_stride", w_stride, n, ldw);
    if (!c.ok() || rows == 0) return c.code;
    c.device();
    c.ptr("x", x, 2), c.ptr("w", w, 2), c.ptr("offsets", offsets, 4), c.ptr("y", y, 2);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmProblem p = product(w, ldw, true, x, ldx, true, n, rows, k, dtype, y, ldy, err);
    p.a.group_stride = w_stride;
    p.groups = n_groups, p.offsets = offsets, p.rag = ds4::MM_RAG_COLS;
    return c.cuda(ds4::mm_launch(p, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int ds4moe_grouped_mm_dx(const void* dy, const void* w, const int32_t* offsets, void* dx, int32_t rows,
                                    int32_t n, int32_t k, int32_t n_groups, int32_t dtype, int64_t lddy, int64_t ldw,
                                    int64_t w_stride, int64_t lddx, void* stream) {
  return guarded("ds4moe_grouped_mm_dx", [&]() -> int {
    Check c("ds4moe_grouped_mm_dx");
    c.rows(rows), c.width("n", n), c.width("k", k), c.dtype(dtype), groups(c, n_groups);
    lddy = c.ld("lddy", lddy, n), ldw = c.ld("ldw", ldw, k), lddx = c.ld("lddx", lddx, k);
    w_stride = stride(c, "w_stride", w_stride, n, ldw);
    if (!c.ok() || rows == 0) return c.code;
    c.device();
    c.ptr("dy", dy, 2), c.ptr("w", w, 2), c.ptr("offsets", offsets, 4), c.ptr("dx", dx, 2);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmProblem p = product(w, ldw, false, dy, lddy, true, k, rows, n, dtype, dx, lddx, err);
    p.a.group_stride = w_stride;
    p.groups = n_groups, p.offsets = offsets, p.rag = ds4::MM_RAG_COLS;
    return c.cuda(ds4::mm_launch(p, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int ds4moe_grouped_mm_dw(const void* dy, const void* x, const int32_t* offsets, void* dw, int32_t rows,
                                    int32_t n, int32_t k, int32_t n_groups, int32_t dtype, int32_t dw_dtype,
                                    int32_t accumulate, int64_t lddy, int64_t ldx, int64_t lddw, int64_t dw_stride,
                                    void* stream) {
  return guarded("ds4moe_grouped_mm_dw", [&]() -> int {
    Check c("ds4moe_grouped_mm_dw");
    c.rows(rows), c.width("n", n), c.width("k", k), c.dtype(dtype), groups(c, n_groups);
    if (dw_dtype != dtype && dw_dtype != DS4MOE_FP32) c.fail(DS4MOE_ERR_UNSUPPORTED_FORMAT, "dw_dtype must be dtype or DS4MOE_FP32");
    lddy = c.ld("lddy", lddy, n), ldx = c.ld("ldx", ldx, k), lddw = c.ld("lddw", lddw, k);
    dw_stride = stride(c, "dw_stride", dw_stride, n, lddw);
    if (!c.ok()) return c.code;
    c.device();
    c.ptr("offsets", offsets, 4), c.ptr("dw", dw, dw_dtype == DS4MOE_FP32 ? 4 : 2);
    c.ptr("dy", dy, 2, rows == 0), c.ptr("x", x, 2, rows == 0);  // without rows nothing of them is read
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmProblem p = product(x, ldx, false, dy, lddy, false, k, n, rows, dtype, dw, lddw, err);
    p.groups = n_groups, p.offsets = offsets, p.rag = ds4::MM_RAG_RED;
    p.e.group_stride = dw_stride;
    p.e.out_f32 = dw_dtype == DS4MOE_FP32, p.e.accumulate = accumulate != 0;
    return c.cuda(ds4::mm_launch(p, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int ds4moe_linear(const void* x, const void* w, const void* bias, const void* residual, void* y, void* zout,
                             int32_t rows, int32_t n, int32_t k, int32_t act, int32_t dtype, int64_t ldx, int64_t ldw,
                             int64_t ldr, int64_t ldy, int64_t ldz, void* stream) {
  return guarded("ds4moe_linear", [&]() -> int {
    Check c("ds4moe_linear");
    c.rows(rows), c.width("n", n), c.width("k", k), c.act(act), c.dtype(dtype);
    ldx = c.ld("ldx", ldx, k), ldw = c.ld("ldw", ldw, k), ldr = c.ld("ldr", ldr, n), ldy = c.ld("ldy", ldy, n);
    ldz = c.ld("ldz", ldz, n);
    if (!c.ok() || rows == 0) return c.code;
    c.device();
    c.ptr("x", x, 2), c.ptr("w", w, 2), c.ptr("y", y, 2);
    c.ptr("bias", bias, 2, true), c.ptr("residual", residual, 2, true), c.ptr("zout", zout, 2, true);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmProblem p = product(w, ldw, true, x, ldx, true, n, rows, k, dtype, y, ldy, err);
    p.e.bias = bias, p.e.residual = residual, p.e.ldr = ldr, p.e.z = zout, p.e.ldz = ldz, p.e.act = act;
    return c.cuda(ds4::mm_launch(p, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int64_t ds4moe_linear_grad_workspace(int32_t rows, int32_t n, int32_t act) {
  if (rows <= 0 || n <= 0) return 16;  // (without rows nothing is kept: ds4moe_linear_grad writes the zeros directly)
  return 16 + (act == DS4MOE_ACT_NONE ? 0 : up(2 * (int64_t)rows * up(n, 8), 16)) + 4 * (int64_t)ds4::mm_colsum_chunks(rows) * n;
}

extern "C" int ds4moe_linear_grad(const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                                  void* db, int32_t rows, int32_t n, int32_t k, int32_t act, int32_t dtype,
                                  int64_t lddy, int64_t ldx, int64_t ldw, int64_t ldz, int64_t lddx, int64_t lddw,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded("ds4moe_linear_grad", [&]() -> int {
    Check c("ds4moe_linear_grad");
    c.rows(rows), c.width("n", n), c.width("k", k), c.act(act), c.dtype(dtype);
    lddy = c.ld("lddy", lddy, n), ldx = c.ld("ldx", ldx, k), ldw = c.ld("ldw", ldw, k), ldz = c.ld("ldz", ldz, n);
    lddx = c.ld("lddx", lddx, k), lddw = c.ld("lddw", lddw, k);
    if (!c.ok()) return c.code;
    if (workspace_bytes < ds4moe_linear_grad_workspace(rows, n, act)) {
      c.fail(DS4MOE_ERR_CAPACITY, "workspace_bytes is less than ds4moe_linear_grad_workspace");
      return c.code;
    }
    c.device();
    const bool none = rows == 0;
    c.ptr("dy", dy, 2, none), c.ptr("x", x, 2, none || !dw), c.ptr("w", w, 2, none || !dx);
    c.ptr("z", z, 2, none || act == DS4MOE_ACT_NONE);
    c.ptr("dx", dx, 2, true), c.ptr("dw", dw, 2, true), c.ptr("db", db, 2, true);
    c.ptr("workspace", workspace, 16);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (none) {  // empty sums, which need no scratch: dw is the product's own zeros, db (0 is +0 in either type) a fill
      cudaError_t e = db ? cudaMemsetAsync(db, 0, 2 * (size_t)n, s) : cudaSuccess;
      if (e == cudaSuccess && dw) e = ds4::mm_launch(product(x, ldx, false, dy, lddy, false, k, n, 0, dtype, dw, lddw, err), s);
      return c.cuda(e);
    }
    char* ws = static_cast<char*>(workspace);
    const void* dz = dy;
    int64_t lddz = lddy;
    cudaError_t e = cudaSuccess;
    if (act != DS4MOE_ACT_NONE && (dx || dw)) dz = ws, lddz = up(n, 8);
    float* part = db ? reinterpret_cast<float*>(ws + (act == DS4MOE_ACT_NONE ? 0 : up(2 * (int64_t)rows * up(n, 8), 16))) : nullptr;
    if (db || dz != dy) e = ds4::mm_act_grad(dy, lddy, z, ldz, dz == dy ? nullptr : ws, lddz, part, db, rows, n, act, dtype == DS4MOE_FP16, s);
    if (e == cudaSuccess && dx) e = ds4::mm_launch(product(w, ldw, false, dz, lddz, true, k, rows, n, dtype, dx, lddx, err), s);
    if (e == cudaSuccess && dw) e = ds4::mm_launch(product(x, ldx, false, dz, lddz, false, k, n, rows, dtype, dw, lddw, err), s);
    return c.cuda(e);
  });
}

extern "C" int64_t ds4moe_cross_entropy_workspace(int32_t rows, int32_t vocab, int32_t d) {
  if (rows <= 0 || vocab <= 0 || d <= 0) return 16;
  const int64_t f = ce_forward_bytes(rows, vocab), g = ce_grad_bytes(rows, d, std::min<int64_t>(kPieceMax, up(vocab, kPieceMin)));
  return f > g ? f : g;
}

extern "C" int ds4moe_cross_entropy(const void* x, const void* w, const int32_t* labels, float* loss, float* lse,
                                    int32_t rows, int32_t vocab, int32_t d, int32_t dtype, int32_t ignore_index,
                                    int64_t ldx, int64_t ldw, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded("ds4moe_cross_entropy", [&]() -> int {
    Check c("ds4moe_cross_entropy");
    c.rows(rows), c.width("vocab", vocab), c.width("d", d), c.dtype(dtype);
    ldx = c.ld("ldx", ldx, d), ldw = c.ld("ldw", ldw, d);
    if (!c.ok() || rows == 0) return c.code;
    if (workspace_bytes < ce_forward_bytes(rows, vocab)) {
      c.fail(DS4MOE_ERR_CAPACITY, "workspace_bytes is less than the " + std::to_string(ce_forward_bytes(rows, vocab)) + " that the softmax partials take");
      return c.code;
    }
    c.device();
    c.ptr("x", x, 2), c.ptr("w", w, 2), c.ptr("labels", labels, 4), c.ptr("loss", loss, 4), c.ptr("lse", lse, 4);
    c.ptr("workspace", workspace, 16);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ds4::MmProblem p = product(x, ldx, true, w, ldw, true, rows, vocab, d, dtype, nullptr, 0, err);
    p.epi = ds4::MM_EPI_STATS;
    const int tiles = (vocab + ds4::kMmStatTile - 1) / ds4::kMmStatTile;
    p.e.labels = labels, p.e.vocab = vocab, p.e.ignore = ignore_index;
    p.e.part = static_cast<float2*>(workspace);
    p.e.zlab = reinterpret_cast<float*>(static_cast<char*>(workspace) + up(8 * (int64_t)rows * tiles, 16));
    cudaError_t e = ds4::mm_launch(p, s);
    if (e == cudaSuccess) e = ds4::mm_softmax_join(p.e.part, tiles, p.e.zlab, labels, ignore_index, vocab, rows, loss, lse, err, s);
    return c.cuda(e);
  });
}

extern "C" int ds4moe_cross_entropy_grad(const void* x, const void* w, const int32_t* labels, const float* lse,
                                         const float* dloss, void* dx, void* dw, int32_t rows, int32_t vocab,
                                         int32_t d, int32_t dtype, int32_t ignore_index, int64_t ldx, int64_t ldw,
                                         int64_t lddx, int64_t lddw, void* workspace, int64_t workspace_bytes,
                                         void* stream) {
  return guarded("ds4moe_cross_entropy_grad", [&]() -> int {
    Check c("ds4moe_cross_entropy_grad");
    c.rows(rows), c.width("vocab", vocab), c.width("d", d), c.dtype(dtype);
    ldx = c.ld("ldx", ldx, d), ldw = c.ld("ldw", ldw, d), lddx = c.ld("lddx", lddx, d), lddw = c.ld("lddw", lddw, d);
    if (!c.ok() || (!dx && !dw)) return c.code;
    if (rows && workspace_bytes < ce_grad_bytes(rows, d, kPieceMin)) {  // (compared before it is reduced: it may be any number)
      c.fail(DS4MOE_ERR_CAPACITY, "workspace_bytes is less than the " + std::to_string(ce_grad_bytes(rows, d, kPieceMin)) + " of the smallest piece of the vocabulary");
      return c.code;
    }
    c.device();
    const bool none = rows == 0;
    c.ptr("x", x, 2, none), c.ptr("w", w, 2, none), c.ptr("labels", labels, 4, none), c.ptr("lse", lse, 4, none);
    c.ptr("dloss", dloss, 4, none), c.ptr("dx", dx, 2, true), c.ptr("dw", dw, 2, true), c.ptr("workspace", workspace, 16, none);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (none) {  // an empty sum
      if (dw) return c.cuda(ds4::mm_launch(product(x, ldx, false, x, ldx, false, d, vocab, 0, dtype, dw, lddw, err), s));
      return c.code;
    }
    char* ws = static_cast<char*>(workspace);
    float* gs = reinterpret_cast<float*>(ws);
    float* sum = reinterpret_cast<float*>(ws + 16);
    char* dz = ws + 16 + up(4 * (int64_t)rows * d, 16);
    const char* wb = static_cast<const char*>(w);
    const int64_t lddz = up(rows, 8);
    // the largest piece of the vocabulary that the workspace holds
    const int64_t fits = (workspace_bytes - ce_grad_bytes(rows, d, 0)) / (2 * lddz) / kPieceMin * kPieceMin;
    const int64_t piece = best_piece(std::min<int64_t>({fits, kPieceMax, up(vocab, kPieceMin)}), rows, vocab, d, dx, dw);
    cudaError_t e = ds4::mm_grad_scale(dloss, labels, ignore_index, vocab, rows, gs, s);
    for (int64_t v0 = 0; v0 < vocab && e == cudaSuccess; v0 += piece) {
      const int pv = (int)std::min<int64_t>(piece, vocab - v0);
      const bool last = v0 + pv == vocab;
      ds4::MmProblem p = product(x, ldx, true, wb + 2 * v0 * ldw, ldw, true, rows, pv, d, dtype, dz, lddz, err);
      p.epi = ds4::MM_EPI_SOFTGRAD;
      p.e.word0 = (int)v0, p.e.vocab = vocab, p.e.ignore = ignore_index;
      p.e.labels = labels, p.e.lse = lse, p.e.g = dloss, p.e.gscale = gs;
      e = ds4::mm_launch(p, s);
      if (e == cudaSuccess && dx) {  // the pieces add up in fp32; the last one rounds
        p = product(wb + 2 * v0 * ldw, ldw, false, dz, lddz, false, d, rows, pv, dtype, last ? dx : sum, last ? lddx : d, err);
        p.e.out_f32 = !last;
        p.e.acc_in = v0 ? sum : nullptr, p.e.acc_ld = d;
        p.e.scale = last ? gs + 1 : nullptr;
        e = ds4::mm_launch(p, s);
      }
      if (e == cudaSuccess && dw) {
        p = product(x, ldx, false, dz, lddz, true, d, pv, rows, dtype, static_cast<char*>(dw) + 2 * v0 * lddw, lddw, err);
        p.e.scale = gs + 1;
        e = ds4::mm_launch(p, s);
      }
    }
    return c.cuda(e);
  });
}

extern "C" int ds4moe_ops_status(int32_t* flags) {
  return guarded("ds4moe_ops_status", [&]() -> int {
    Check c("ds4moe_ops_status");
    if (!flags) c.invalid("flags is NULL");
    c.device();
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(flags, err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(err, 0, 4);
    return c.cuda(e);
  });
}
