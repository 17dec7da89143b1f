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
constexpr int kMaxListed = ds4::kMmListed, kMaxTop = ds4::kMmTop;
constexpr int kScoreRows = 128;                    // scores take blocks of so many rows at least, whatever the workspace

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
  void listed(const char* name, int v, int least, int most) {
    if (v < least || v > most) invalid(std::string(name) + "=" + std::to_string(v) + " must be in " + std::to_string(least) + ".." + std::to_string(most));
  }
  void temperature(float v) {
    if (!(v >= 1e-3f && v <= 1e3f)) invalid("temperature=" + std::to_string(v) + " must be in 0.001..1000");
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
  p.e.inv_t = 1.f;
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
  const int64_t step = up(most / 64, kPieceMin);  // (32 tries, a few microseconds)
  for (int64_t piece = most; 2 * piece > most && piece >= kPieceMin; piece -= step) {
    const int64_t cost = vocab / piece * one(piece) + one(vocab % piece);
    if (cost < best_cost) best_cost = cost, best = piece;
  }
  return best;
}

// The gradient of a softmax loss in pieces of the vocabulary: the logits again, dz of one piece in the workspace, its
// parts of dx and dw. labels: the cross entropy's; ids, places: the distillation's listed words.
struct SoftGrad {
  const void *x, *w;
  int64_t ldx, ldw;
  void *dx, *dw;
  int64_t lddx, lddw;
  int rows, vocab, d, dtype;
  int* err;
  float *gs, *sum;
  char* dz;
  int64_t dz_bytes;
  const float *lse, *g;
  float inv_t;
  const int* labels;
  int ignore;
  const int* ids;
  const float* places;
  int listed;
  int64_t piece_max;  // words of a piece
};
cudaError_t soft_grad(const SoftGrad& q, cudaStream_t s) {
  const char* wb = static_cast<const char*>(q.w);
  const int rows = q.rows, vocab = q.vocab, d = q.d, dtype = q.dtype;
  const int64_t lddz = up(rows, 8), ldx = q.ldx, ldw = q.ldw;
  // the largest piece of the vocabulary that the workspace holds
  const int64_t fits = q.dz_bytes / (2 * lddz) / kPieceMin * kPieceMin;
  const int64_t piece = best_piece(std::min<int64_t>({fits, q.piece_max, up(vocab, kPieceMin)}), rows, vocab, d, q.dx, q.dw);
  cudaError_t e = cudaSuccess;
  for (int64_t v0 = 0; v0 < vocab && e == cudaSuccess; v0 += piece) {
    const int pv = (int)std::min<int64_t>(piece, vocab - v0);
    const bool last = v0 + pv == vocab;
    ds4::MmProblem p = product(q.x, ldx, true, wb + 2 * v0 * ldw, ldw, true, rows, pv, d, dtype, q.dz, lddz, q.err);
    p.epi = ds4::MM_EPI_SOFTGRAD;
    p.e.word0 = (int)v0, p.e.vocab = vocab, p.e.ignore = q.ignore;
    p.e.labels = q.labels, p.e.lse = q.lse, p.e.g = q.g, p.e.gscale = q.gs, p.e.inv_t = q.inv_t;
    e = ds4::mm_launch(p, s);
    if (e == cudaSuccess && q.ids) e = ds4::mm_distill_scatter(q.ids, q.places, q.g, q.gs, q.listed, rows, (int)v0, pv, q.dz, lddz, p.f16, s);
    if (e == cudaSuccess && q.dx) {  // the pieces add up in fp32; the last one rounds
      p = product(wb + 2 * v0 * ldw, ldw, false, q.dz, lddz, false, d, rows, pv, dtype, last ? q.dx : q.sum, last ? q.lddx : d, q.err);
      p.e.out_f32 = !last;
      p.e.acc_in = v0 ? q.sum : nullptr, p.e.acc_ld = d;
      p.e.scale = last ? q.gs + 1 : nullptr;
      p.may_spread = q.ids != nullptr;
      e = ds4::mm_launch(p, s);
    }
    if (e == cudaSuccess && q.dw) {
      p = product(q.x, ldx, false, q.dz, lddz, true, d, pv, rows, dtype, static_cast<char*>(q.dw) + 2 * v0 * q.lddw, q.lddw, q.err);
      p.e.scale = q.gs + 1;
      e = ds4::mm_launch(p, s);
    }
  }
  return e;
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
    const int64_t held = ce_grad_bytes(rows, d, 0);
    cudaError_t e = ds4::mm_grad_scale(dloss, labels, ignore_index, vocab, rows, gs, s);
    if (e != cudaSuccess) return c.cuda(e);
    SoftGrad q = {x, w, ldx, ldw, dx, dw, lddx, lddw, rows, vocab, d, dtype, err};
    q.gs = gs, q.sum = sum, q.dz = ws + held, q.dz_bytes = workspace_bytes - held;
    q.lse = lse, q.g = dloss, q.inv_t = 1.f, q.labels = labels, q.ignore = ignore_index, q.piece_max = kPieceMax;
    return c.cuda(soft_grad(q, s));
  });
}

namespace {

// The gradient of rows whose dz is given: dx and dW of W [n x k], grouped or (offsets null) dense.
cudaError_t block_grad(const void* dz, int64_t lddz, const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t w_stride,
                       const int32_t* offsets, int n_groups, void* dx, int64_t lddx, void* dw, int64_t lddw, int64_t dw_stride,
                       int rows, int n, int k, int dtype, int* err, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (dx && rows) {
    ds4::MmProblem p = product(w, ldw, false, dz, lddz, true, k, rows, n, dtype, dx, lddx, err);
    p.a.group_stride = w_stride;
    if (offsets) p.groups = n_groups, p.offsets = offsets, p.rag = ds4::MM_RAG_COLS;
    p.may_spread = 1;
    e = ds4::mm_launch(p, s);
  }
  if (e == cudaSuccess && dw) {
    ds4::MmProblem p = product(x, ldx, false, dz, lddz, false, k, n, rows, dtype, dw, lddw, err);
    if (offsets) p.groups = n_groups, p.offsets = offsets, p.rag = ds4::MM_RAG_RED;
    p.e.group_stride = dw_stride;
    e = ds4::mm_launch(p, s);
  }
  return e;
}

// A block without offsets is one dense one.
void block_groups(Check& c, const void* offsets, int n_groups) {
  groups(c, n_groups);
  if (!offsets && n_groups > 1) c.invalid("offsets is NULL with n_groups=" + std::to_string(n_groups) + " (a dense block has one)");
}

// Workspace of the scores of `rows` rows: softmax partials, sorted lists with their logits; where the best words are asked
// for all logits, and the largest of each chunk.
struct ScoreSpace {
  int64_t part, ent, want, first, zwant, chunk_max, logits, total;
  ScoreSpace(int64_t rows, int64_t vocab, int64_t n, int top_k) {
    const int tile = ds4::mm_score_tile(1, rows <= ds4::kMmFewRows);  // (the smallest of any number of rows, up to kMmFewRows or beyond)
    const int64_t tiles = (vocab + tile - 1) / tile;
    const int64_t parts = rows <= ds4::kMmFewRows ? std::min<int64_t>(ds4::kMmFewParts, 4 * ((vocab + 127) / 128)) : tiles;
    part = 0;
    ent = up(8 * rows * parts, 16);
    want = ent + up(4 * rows * parts, 16);
    first = want + up(8 * rows * n, 16);
    zwant = first + (n ? up(2 * rows * tiles, 16) : 0);
    chunk_max = zwant + up(4 * rows * n, 16);
    logits = chunk_max + (top_k ? up(4 * rows * ((vocab + ds4::kMmStatChunk - 1) / ds4::kMmStatChunk), 16) : 0);
    total = logits + (top_k ? up(4 * rows * vocab, 16) : 0);
  }
  // What a query returns. Few rows have more partials and more entries of `first` each, so that 33 may take less than 32
  // (129280 words, one token: 467056 bytes, 652160): a workspace for more rows has to serve fewer.
  static int64_t bytes(int64_t rows, int64_t vocab, int64_t n, int top_k) {
    return std::max(ScoreSpace(rows, vocab, n, top_k).total, ScoreSpace(std::min<int64_t>(rows, ds4::kMmFewRows), vocab, n, top_k).total);
  }
};

// The scores of all rows, in blocks that the workspace holds: what `a` asks for, from its row 0 on.
struct ScoreCall {
  const void *x, *w;
  int64_t ldx, ldw;
  int vocab, d, dtype;
  int* err;
};
int score_rows(Check& c, int rows, int vocab, int n, int top_k, int64_t bytes) {
  const int64_t least = ScoreSpace(std::min(rows, kScoreRows), vocab, n, top_k).total;
  if (bytes < least) {
    c.fail(DS4MOE_ERR_CAPACITY, "workspace_bytes is less than the " + std::to_string(least) + " of a block of rows");
    return 0;
  }
  if (bytes >= ScoreSpace(rows, vocab, n, top_k).total) return rows;
  int64_t lo = 1, hi = (rows + kScoreRows - 1) / kScoreRows;  // blocks of kScoreRows that fit, and that do not
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    (bytes >= ScoreSpace(mid * kScoreRows, vocab, n, top_k).total ? lo : hi) = mid;
  }
  return (int)lo * kScoreRows;
}
cudaError_t scores(const ScoreCall& call, ds4::MmScores a, int rows, int block, char* ws, cudaStream_t s) {
  const int vocab = call.vocab;
  const bool few = block <= ds4::kMmFewRows;
  a.tile = ds4::mm_score_tile(rows, few);  // (of the call: its blocks take the same tiles)
  a.vocab = vocab, a.parts = few ? ds4::mm_few_parts(vocab) : (vocab + a.tile - 1) / a.tile, a.err = call.err;
  const ScoreSpace at(block, vocab, a.n, a.top_k);
  cudaError_t e = cudaSuccess;
  for (int64_t t0 = 0; t0 < rows && e == cudaSuccess; t0 += block) {
    const int nr = (int)std::min<int64_t>(block, rows - t0);
    ds4::MmScores b = a;
    b.rows = nr;
    const auto move = [&](auto*& p, int64_t per_row) { if (p) p += t0 * per_row; };
    move(b.words, a.n), move(b.lse, 1), move(b.logprob, a.n), move(b.entropy, 1), move(b.top_index, a.top_k);
    move(b.top_logprob, a.top_k), move(b.teacher, a.n), move(b.loss, 1);
    const char* x = static_cast<const char*>(call.x) + 2 * t0 * call.ldx;
    ds4::MmProblem p = few ? product(call.w, call.ldw, true, x, call.ldx, true, vocab, nr, call.d, call.dtype, nullptr, 0, call.err)
                           : product(x, call.ldx, true, call.w, call.ldw, true, nr, vocab, call.d, call.dtype, nullptr, 0, call.err);
    p.epi = few ? ds4::MM_EPI_SCORE_FEW : ds4::MM_EPI_SCORE;
    p.e.inv_t = a.inv_t;
    p.e.tile = a.tile;
    p.e.part = reinterpret_cast<float2*>(ws + at.part), p.e.ent = a.entropy ? reinterpret_cast<float*>(ws + at.ent) : nullptr;
    p.e.want = reinterpret_cast<int2*>(ws + at.want), p.e.n_want = a.n, p.e.zwant = reinterpret_cast<float*>(ws + at.zwant);
    p.e.first = reinterpret_cast<uint16_t*>(ws + at.first);
    p.e.logits = a.top_k ? reinterpret_cast<float*>(ws + at.logits) : nullptr;
    p.e.chunk_max = reinterpret_cast<float*>(ws + at.chunk_max);
    b.part = p.e.part, b.ent = p.e.ent, b.zwant = p.e.zwant, b.logits = p.e.logits, b.chunk_max = p.e.chunk_max;
    p.e.vocab = vocab;
    if (a.n <= (few ? ds4::kMmDirect : 1))
      p.e.words = b.words;
    else
      e = ds4::mm_sort_words(b.words, a.n, vocab, nr, a.tile, reinterpret_cast<int2*>(ws + at.want), reinterpret_cast<uint16_t*>(ws + at.first), s);
    if (e == cudaSuccess) e = ds4::mm_launch(p, s);
    if (e == cudaSuccess) e = ds4::mm_score_join(b, s);
  }
  return e;
}

// Workspace of the distillation's gradient: the scale words, fp32 sum of dx, each row's weight, the listed words' places,
// one piece of dz.
struct DistillSpace {
  int64_t sum, g, at, dz;
  DistillSpace(int64_t rows, int64_t d, int64_t n) {
    sum = 16;
    g = sum + up(4 * rows * d, 16);
    at = g + up(4 * rows, 16);
    dz = at + up(4 * rows * n, 16);
  }
  int64_t total(int64_t rows, int64_t piece) const { return dz + 2 * up(rows, 8) * piece; }
};
// Its pieces of the vocabulary: of up to 512 rows as many words as make 64 MB of dz, which still come from L2 (inputs in turns: 128 rows,
// 129280 words, d 2048 604 us in pieces of 16384, 383 in one; 512 rows, d 512 496, 335; 16 rows, 32000 words, d 1024 121, 91; but 256
// rows, 32000 words, d 4096 261, 292, and 512 rows, 129280 words, d 2048 940, 962). Beyond, the longer sums of dx, in several
// accumulators, cost more than fewer launches save (1024 rows, 64000 words, d 1024: 431 us, 505 in halves).
constexpr int64_t kDistillRows = 512, kDistillDz = (int64_t)1 << 26;
int64_t distill_piece(int64_t rows) {
  return rows > kDistillRows ? kPieceMax : std::max<int64_t>(kPieceMax, kDistillDz / 2 / up(rows, 8) / kPieceMin * kPieceMin);
}
// The bytes of dz for which a workspace is made: such a piece of these rows and of any smaller number.
int64_t distill_dz(int64_t rows, int64_t vocab) {
  const int64_t words = up(vocab, kPieceMin);
  return std::max(2 * up(rows, 8) * std::min<int64_t>(kPieceMax, words), std::min(kDistillDz, 2 * std::min(up(rows, 8), kDistillRows) * words));
}

}  // namespace

extern "C" int ds4moe_grouped_glu(const void* x, const void* w, const int32_t* offsets, void* h, void* zout, int32_t rows,
                                  int32_t n, int32_t k, int32_t n_groups, int32_t act, int32_t dtype, int64_t ldx,
                                  int64_t ldw, int64_t w_stride, int64_t ldh, int64_t ldz, void* stream) {
  return guarded("ds4moe_grouped_glu", [&]() -> int {
    Check c("ds4moe_grouped_glu");
    c.rows(rows), c.listed("n", n, 1, kMaxWidth / 2), c.width("k", k), c.act(act), c.dtype(dtype), groups(c, n_groups);
    ldx = c.ld("ldx", ldx, k), ldw = c.ld("ldw", ldw, k), ldh = c.ld("ldh", ldh, n), ldz = c.ld("ldz", ldz, 2 * (int64_t)n);
    w_stride = stride(c, "w_stride", w_stride, 2 * (int64_t)n, ldw);
    if (!c.ok() || rows == 0) return c.code;
    block_groups(c, offsets, n_groups);
    c.device();
    c.ptr("x", x, 2), c.ptr("w", w, 2), c.ptr("offsets", offsets, 4, true), c.ptr("h", h, 2), c.ptr("zout", zout, 2, true);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmProblem p = product(w, ldw, true, x, ldx, true, n, rows, k, dtype, h, ldh, err);
    p.epi = ds4::MM_EPI_GLU;
    p.a.group_stride = w_stride;
    if (offsets) p.groups = n_groups, p.offsets = offsets, p.rag = ds4::MM_RAG_COLS;
    p.e.z = zout, p.e.ldz = ldz, p.e.act = act;
    return c.cuda(ds4::mm_launch(p, static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int ds4moe_grouped_glu_grad(const void* dh, const void* x, const void* w, const int32_t* offsets, const void* z,
                                       void* dz, void* dx, void* dw, int32_t rows, int32_t n, int32_t k, int32_t n_groups,
                                       int32_t act, int32_t dtype, int64_t lddh, int64_t ldx, int64_t ldw, int64_t w_stride,
                                       int64_t ldz, int64_t lddz, int64_t lddx, int64_t lddw, int64_t dw_stride, void* stream) {
  return guarded("ds4moe_grouped_glu_grad", [&]() -> int {
    Check c("ds4moe_grouped_glu_grad");
    const int64_t n2 = 2 * (int64_t)n;
    c.rows(rows), c.listed("n", n, 1, kMaxWidth / 2), c.width("k", k), c.act(act), c.dtype(dtype), groups(c, n_groups);
    lddh = c.ld("lddh", lddh, n), ldx = c.ld("ldx", ldx, k), ldw = c.ld("ldw", ldw, k), ldz = c.ld("ldz", ldz, n2);
    lddz = c.ld("lddz", lddz, n2), lddx = c.ld("lddx", lddx, k), lddw = c.ld("lddw", lddw, k);
    w_stride = stride(c, "w_stride", w_stride, n2, ldw), dw_stride = stride(c, "dw_stride", dw_stride, n2, lddw);
    if (dz && dz == z && rows > 1 && lddz != ldz)  // (a row would be written while another one is read there)
      c.invalid("dz is z, but lddz=" + std::to_string(lddz) + " is not ldz=" + std::to_string(ldz));
    if (!c.ok()) return c.code;
    block_groups(c, offsets, n_groups);
    c.device();
    const bool none = rows == 0;  // (nothing of the operands is read, dw is zeros)
    c.ptr("dh", dh, 2, none), c.ptr("x", x, 2, none || !dw), c.ptr("w", w, 2, none || !dx), c.ptr("offsets", offsets, 4, true);
    c.ptr("z", z, 2, none), c.ptr("dz", dz, 2, none), c.ptr("dx", dx, 2, true), c.ptr("dw", dw, 2, true);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (!none) e = ds4::mm_glu_grad(dh, lddh, z, ldz, dz, lddz, offsets, n_groups, rows, n, act, dtype == DS4MOE_FP16, s);
    if (e == cudaSuccess)
      e = block_grad(dz, lddz, x, ldx, w, ldw, w_stride, offsets, n_groups, dx, lddx, dw, lddw, dw_stride, rows, (int)n2, k, dtype, err, s);
    return c.cuda(e);
  });
}

extern "C" int64_t ds4moe_logprobs_workspace(int32_t rows, int32_t vocab, int32_t n_tokens, int32_t top_k) {
  if (rows <= 0 || vocab <= 0 || n_tokens < 0) return 16;
  return std::max<int64_t>(16, ScoreSpace::bytes(rows, vocab, n_tokens, top_k));
}

extern "C" int ds4moe_logprobs(const void* x, const void* w, const int32_t* tokens, float* logprob, float* lse,
                               float* entropy, int32_t* top_index, float* top_logprob, int32_t rows, int32_t vocab,
                               int32_t d, int32_t n_tokens, int32_t top_k, int32_t dtype, float temperature, int64_t ldx,
                               int64_t ldw, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded("ds4moe_logprobs", [&]() -> int {
    Check c("ds4moe_logprobs");
    c.rows(rows), c.width("vocab", vocab), c.width("d", d), c.dtype(dtype), c.temperature(temperature);
    c.listed("n_tokens", n_tokens, 0, kMaxListed), c.listed("top_k", top_k, 0, std::min(kMaxTop, vocab));
    ldx = c.ld("ldx", ldx, d), ldw = c.ld("ldw", ldw, d);
    if (!c.ok() || rows == 0) return c.code;
    const int block = score_rows(c, rows, vocab, n_tokens, top_k, workspace_bytes);
    if (!c.ok()) return c.code;
    c.device();
    c.ptr("x", x, 2), c.ptr("w", w, 2), c.ptr("tokens", tokens, 4, n_tokens == 0), c.ptr("logprob", logprob, 4, n_tokens == 0);
    c.ptr("lse", lse, 4, true), c.ptr("entropy", entropy, 4, true);
    c.ptr("top_index", top_index, 4, top_k == 0), c.ptr("top_logprob", top_logprob, 4, top_k == 0);
    c.ptr("workspace", workspace, 16);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmScores a = {};
    a.inv_t = 1.f / temperature;
    a.words = tokens, a.n = n_tokens, a.logprob = logprob, a.lse = lse, a.entropy = entropy;
    a.top_k = top_k, a.top_index = top_index, a.top_logprob = top_logprob;
    return c.cuda(scores({x, w, ldx, ldw, vocab, d, dtype, err}, a, rows, block, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int64_t ds4moe_distill_workspace(int32_t rows, int32_t vocab, int32_t d, int32_t top_k) {
  if (rows <= 0 || vocab <= 0 || d <= 0 || top_k <= 0) return 16;
  return std::max<int64_t>(ScoreSpace::bytes(rows, vocab, top_k, 0),
                           DistillSpace(rows, d, top_k).dz + distill_dz(rows, vocab));
}

extern "C" int ds4moe_distill(const void* x, const void* w, const int32_t* ids, const float* teacher, float* loss,
                              float* lse, float* logq, int32_t rows, int32_t vocab, int32_t d, int32_t top_k, int32_t dtype,
                              float temperature, int64_t ldx, int64_t ldw, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  return guarded("ds4moe_distill", [&]() -> int {
    Check c("ds4moe_distill");
    c.rows(rows), c.width("vocab", vocab), c.width("d", d), c.dtype(dtype), c.temperature(temperature);
    c.listed("top_k", top_k, 1, kMaxListed);
    ldx = c.ld("ldx", ldx, d), ldw = c.ld("ldw", ldw, d);
    if (!c.ok() || rows == 0) return c.code;
    const int block = score_rows(c, rows, vocab, top_k, 0, workspace_bytes);
    if (!c.ok()) return c.code;
    c.device();
    c.ptr("x", x, 2), c.ptr("w", w, 2), c.ptr("ids", ids, 4), c.ptr("teacher", teacher, 4), c.ptr("loss", loss, 4);
    c.ptr("lse", lse, 4), c.ptr("logq", logq, 4), c.ptr("workspace", workspace, 16);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    ds4::MmScores a = {};
    a.inv_t = 1.f / temperature;
    a.words = ids, a.n = top_k, a.teacher = teacher, a.loss = loss, a.lse = lse, a.logprob = logq;
    return c.cuda(scores({x, w, ldx, ldw, vocab, d, dtype, err}, a, rows, block, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
  });
}

extern "C" int ds4moe_distill_grad(const void* x, const void* w, const int32_t* ids, const float* teacher, const float* lse,
                                   const float* logq, const float* dloss, void* dx, void* dw, int32_t rows, int32_t vocab,
                                   int32_t d, int32_t top_k, int32_t dtype, float temperature, int64_t ldx, int64_t ldw,
                                   int64_t lddx, int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded("ds4moe_distill_grad", [&]() -> int {
    Check c("ds4moe_distill_grad");
    c.rows(rows), c.width("vocab", vocab), c.width("d", d), c.dtype(dtype), c.temperature(temperature);
    c.listed("top_k", top_k, 1, kMaxListed);
    ldx = c.ld("ldx", ldx, d), ldw = c.ld("ldw", ldw, d), lddx = c.ld("lddx", lddx, d), lddw = c.ld("lddw", lddw, d);
    if (!c.ok() || (!dx && !dw)) return c.code;
    const DistillSpace at(rows, d, top_k);
    if (rows && workspace_bytes < at.total(rows, kPieceMin)) {
      c.fail(DS4MOE_ERR_CAPACITY, "workspace_bytes is less than the " + std::to_string(at.total(rows, kPieceMin)) + " of the smallest piece of the vocabulary");
      return c.code;
    }
    c.device();
    const bool none = rows == 0;
    c.ptr("x", x, 2, none), c.ptr("w", w, 2, none), c.ptr("ids", ids, 4, none), c.ptr("teacher", teacher, 4, none);
    c.ptr("lse", lse, 4, none), c.ptr("logq", logq, 4, none), c.ptr("dloss", dloss, 4, none);
    c.ptr("dx", dx, 2, true), c.ptr("dw", dw, 2, true), c.ptr("workspace", workspace, 16, none);
    int* err = c.err_word();
    if (!c.ok()) return c.code;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (none) {  // an empty sum
      if (dw) return c.cuda(ds4::mm_launch(product(x, ldx, false, x, ldx, false, d, vocab, 0, dtype, dw, lddw, err), s));
      return c.code;
    }
    char* ws = static_cast<char*>(workspace);
    float *gs = reinterpret_cast<float*>(ws), *g = reinterpret_cast<float*>(ws + at.g), *places = reinterpret_cast<float*>(ws + at.at);
    const float inv_t = 1.f / temperature;
    cudaError_t e = ds4::mm_distill_prepare(ids, teacher, logq, dloss, top_k, vocab, rows, inv_t, g, places, s);
    if (e == cudaSuccess) e = ds4::mm_grad_scale(g, nullptr, 0, vocab, rows, gs, s);
    if (e != cudaSuccess) return c.cuda(e);
    SoftGrad q = {x, w, ldx, ldw, dx, dw, lddx, lddw, rows, vocab, d, dtype, err};
    q.gs = gs, q.sum = reinterpret_cast<float*>(ws + at.sum), q.dz = ws + at.dz, q.dz_bytes = workspace_bytes - at.dz;
    q.lse = lse, q.g = g, q.inv_t = inv_t, q.ids = ids, q.places = places, q.listed = top_k, q.piece_max = distill_piece(rows);
    return c.cuda(soft_grad(q, s));
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
