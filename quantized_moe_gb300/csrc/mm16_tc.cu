// The 16-bit products on the 5th-generation tensor cores: out[c][l] = sum_r A(l, r) B(c, r).
//
// Persistent: one CTA (or pair of CTAs) per SM (or two SMs) loops over output tiles of 128 lanes per
// CTA x up to 256 columns. The lanes are the contiguous index of the output, so that a tensor-memory
// lane is a lane of the output; the columns are rows of tokens (or of dW), of which a tile takes
// exactly what its group has, rounded up to the MMA's granule, so that a group's weights cross HBM
// once however ragged the counts are.
//
// Operands are staged by TMA in 128-byte swizzled sub-tiles of 64 of the reduction, read by the MMA
// in either order: rows with the reduction contiguous (K-major) or with the lane or column index
// contiguous (MN-major: boxes of 64 lanes x 64 of the reduction). Pairs (cta_group::2): the leader's
// MMA spans both SMs' tiles, 256 lanes, and each CTA stages half of the columns, which halves
// the shared-memory and L2 traffic of the column operand.
//
// Warp roles: warps 0 and 3 issue the TMA loads of one operand each (their lanes issue the copies of a
// stage in parallel); one thread of warp 1 issues the MMAs (the leader's, in a pair); warp 2 clears what a
// ragged end of the reduction leaves in a stage; warps 4-11 run the epilogue of one tile while the next one's main loop
// fills the other accumulator. Where an operand's address or row distance is not a multiple of 16
// bytes, eight loader warps (12-19) read it with ordinary loads and write the same swizzled layout.
// Few tiles share their reduction out over a cluster of CTAs, which join their sums in shared memory.
//
// What bounds it (GB300, measured): the experts' products stream their weights (256 experts, 32768
// rows, n 2048, k 4096: 0.70-0.72 ms = 6.5-6.8 TB/s, 96-99 % of the copy bandwidth, for y and dx; the
// weight gradients, 4.3 GB of results, 0.85 ms = 5.5 TB/s: their way through shared memory beside the MMAs' operands);
// large dense products the tensor pipe and the SMs' L2 reads (2048 x 129280 x 4096: 1.12 ms = 1.94
// PFLOP/s, the rate of a large library product; 4096^3 with its epilogue 94 us = 1.46 PFLOP/s, of
// which a seventh is the last, partial round and the launch); single tokens the launch and one pass of
// loads (1 x 4096 x 4096: 9.8 us a launch in a graph, against 4.9 us of HBM time).
//
// Every wait is bounded (tc::mbar_wait). On a timeout the CTA raises error bit 2, waits for its copies
// and MMAs in flight, frees its tensor memory and returns.
#include <cudaTypedefs.h>

#include <algorithm>

#include "mm16.cuh"
#include "tc_ptx.cuh"

namespace ds4 {
namespace {

using namespace tc;

constexpr int BM = 128, BK = 64;          // lanes per CTA; reduction of one stage
constexpr int A_BYTES = BM * BK * 2;      // 16 KB
constexpr int kMaxStages = 12;
constexpr int kSegStats = 2048, kSegStore = 512;  // reduction of one accumulator where the result is fp32
constexpr int kSegFold = 16384;           // and where it has 16 bits
constexpr int kEpiPlain = 3;              // MM_EPI_STORE of 16-bit rows with nothing to add: a kernel of its own (mm_launch)
constexpr int kPanel = 8;                 // column tiles that a raster panel spans
constexpr int kEpiWarps = 8;              // epilogue warps: two per quadrant of tensor-memory lanes
constexpr int kFirstLoader = 4 + kEpiWarps;
constexpr int kLoaders = 8;               // loader warps of the unaligned form
constexpr int kThreads = 32 * kFirstLoader;
constexpr int kRowBytes = 2 * BM + 16;    // a staged row of 128 lanes: 16 bytes on, so that eight rows' chunks hit all banks
constexpr int kPartLd = BM + 4;           // floats from one column of a partial sum to the next (conflict-free as fragments)
constexpr int kOutBytes = 32 * kRowBytes;  // 32 columns of 128 lanes on their way out, one per half of the epilogue
constexpr int kSmemMax = 232448;

// n / d for 0 <= n < 2^31 by a multiplication: m = floor(2^32 (2^l - d) / d) + 1, l = ceil(log2 d) (T. Granlund and
// P. L. Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct Divider {
  uint32_t m, l;
  Divider() = default;
  explicit Divider(uint32_t d) : l(0) {
    while (l < 31 && (1u << l) < d) ++l;
    m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> l); }
};

struct TcArgs {
  MmProblem p;
  int bn, stages, b_box;      // column tile, pipeline depth, rows of a column-operand box
  int a_blocks, b_blocks;     // boxes of 64 x 64 that one copy of an MN-major operand brings
  int lane_tiles, col_tiles;  // of BM * CG lanes; of bn columns (without ragged columns)
  int rows_out;               // the 16-bit output (and residual, z) can be moved 8 lanes at a time
  int seg;                    // reduction that one accumulator takes before its sums are added up in fp32 (a multiple of BK)
  int accs;                   // accumulators of one tile that lie side by side in tensor memory (1: two take turns; 2: none is left to)
  int fold;                   // a tile with more reduction than seg is summed up in tensor memory (fold_acc), seg by seg
  int split;                  // CTAs (a cluster) that share a tile's reduction; 1: none
  int tail_from, tail_lg;     // tiles from here on are split into 2^tail_lg parts of their columns
  Divider by_lanes, by_panel, by_matrix;  // lane_tiles, lane_tiles * kPanel, lane_tiles * col_tiles
};

// Barriers, the tensor-memory address and the abort flag, then the group tables (tile_of).
__host__ __device__ constexpr int ctrl_bytes(int rag, int groups) {
  return 24 * kMaxStages + 32 + 16 + (rag == MM_DENSE ? 0 : 4 * (groups + 1) * (rag == MM_RAG_COLS ? 2 : 1));
}

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(addr) : "memory");
}

// Programmatic dependent launch: the next launch of the stream may set itself up while this one runs; nothing of
// global memory is read or written before the launches in front are complete.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int g, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(g), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(g), "r"(bar)
        : "memory");
}

// Shared-memory descriptor of a 128-byte swizzled operand. K-major: 8-row atoms of 1024 bytes along
// the rows (stride offset). MN-major: atoms of 64 lanes x 8 of the reduction; the next 8 of the
// reduction 1024 bytes on (stride offset), the next 64 lanes one 64 x 64 box on (leading offset).
__device__ __forceinline__ uint64_t op_desc(uint32_t addr, bool red_major) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(red_major ? 1 : 8192 >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}
// One MMA of 16 of the reduction, and the arrival on a barrier (in a pair: on both CTAs' barriers) once all
// MMAs issued before are complete. One thread of the CTA issues all of them.
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (CG == 2)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CG == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(su32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(su32(bar)) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_get(uint32_t* slot, uint32_t cols) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  } else {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(cols) : "memory");
  else
    tmem_dealloc(addr, cols);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_get16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// One output tile.
struct Tile {
  int g, l0, c0, n, r0, red;  // group, first lane of the CTA (pair), first column, columns, first of the reduction, its length
};

// Tables in shared memory: lo[g], g = 0..groups, the first row of each group, clamped to the matrix (a group
// ends where the next one begins, or is empty if that lies before it); for ragged columns pref[g], the running
// count of the groups' column tiles.
template <int CG>
__device__ __forceinline__ Tile tile_of(const TcArgs& a, const int* lo_of, const int* pref, int t, int share) {
  const MmProblem& p = a.p;
  Tile o;
  int col_tiles = a.col_tiles, c_lo = 0, c_n = p.cols, part = 0, width = a.bn;
  o.g = 0, o.r0 = 0, o.red = p.red;
  if (p.rag == MM_RAG_COLS) {
    const int ct = a.by_lanes.div(t);  // a group takes lane_tiles * its column tiles consecutive tiles
    int lo = 0, hi = p.groups;
    while (hi - lo > 1) {  // the last group whose running count is at most ct
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= ct) lo = mid; else hi = mid;
    }
    o.g = lo;
    col_tiles = pref[lo + 1] - pref[lo];
    t -= pref[lo] * a.lane_tiles;
    c_lo = lo_of[lo], c_n = max(lo_of[lo + 1] - c_lo, 0);
  } else if (p.rag == MM_RAG_RED) {
    o.g = a.by_matrix.div(t);
    t -= o.g * a.lane_tiles * col_tiles;
    o.r0 = lo_of[o.g], o.red = max(lo_of[o.g + 1] - o.r0, 0);
  } else if (t >= a.tail_from) {
    const int u = t - a.tail_from;
    part = u & ((1 << a.tail_lg) - 1);
    width = a.bn >> a.tail_lg;
    t = a.tail_from + (u >> a.tail_lg);
  }
  int panel = 0;
  if (col_tiles > kPanel) {
    panel = a.by_panel.div(t);
    t -= panel * a.lane_tiles * kPanel;
  }
  const int w = min(kPanel, col_tiles - panel * kPanel);
  const int lt = w == 1 ? t : w == kPanel ? t / kPanel : t / w, ct = panel * kPanel + t - lt * w;
  o.l0 = lt * BM * CG;
  o.c0 = c_lo + ct * a.bn + part * width;
  o.n = min(width, c_n - ct * a.bn - part * width);  // (a part past the last column has none)
  if (CG == 1 && a.split > 1) {  // this CTA's share of the reduction, whole stages
    const int blocks = (o.red + BK - 1) / BK;
    const int b0 = blocks * share / a.split * BK, b1 = blocks * (share + 1) / a.split * BK;
    o.red = min(o.red, b1) - b0;
    o.r0 += b0;
  }
  return o;
}

// The tiles of a warp in turn, every `step`-th one from `first`: tile_of takes a few hundred cycles of dependent
// arithmetic, so the lanes work out 32 tiles at once and hand them round (weight gradients of 256 experts, 128 rows
// each, where a tile has two or three stages: 910 -> 857 us with this and the cleaner's stores unrolled).
template <int CG>
struct Walk {
  Tile mine;
  int i = 31;
  __device__ __forceinline__ Tile next(const TcArgs& a, const int* lo_of, const int* pref, int t, int step, int tiles, int share, int lane) {
    if (++i == 32) {
      i = 0;
      mine = tile_of<CG>(a, lo_of, pref, min(t + lane * step, tiles - 1), share);
    }
    Tile o;
    o.g = __shfl_sync(0xffffffffu, mine.g, i);
    o.l0 = __shfl_sync(0xffffffffu, mine.l0, i);
    o.c0 = __shfl_sync(0xffffffffu, mine.c0, i);
    o.n = __shfl_sync(0xffffffffu, mine.n, i);
    o.r0 = __shfl_sync(0xffffffffu, mine.r0, i);
    o.red = __shfl_sync(0xffffffffu, mine.red, i);
    return o;
  }
};

// Columns of the tile's MMA: its columns rounded up to the granule (16, in a pair 32); whole 64-column
// boxes where the columns are the contiguous index.
template <int CG>
__device__ __forceinline__ int mma_n(const MmProblem& p, int n) {
  const int q = p.b.red_major ? 16 * CG : 64 * CG;
  return (n + q - 1) / q * q;
}

// One operand's stages by ordinary loads, in the layout that the TMA's 128-byte swizzle gives (16-byte chunk index XOR
// row mod 8). K-major: the rows of 64 elements are lanes or columns and their elements the reduction; MN-major the other
// way round, in boxes of 64 x 64. A thread owns one 16-byte chunk of every 32nd row, so that neither its chunk nor the
// parity of its addresses changes: it reads the aligned words that hold its eight elements and, where the row starts in
// the middle of a word, shifts them by an element. Elements outside the matrix are zeros; their words are not read.
struct Loader {
  const uint16_t* src;  // of the thread's chunk in its first row
  int64_t step;         // elements to the chunk 32 rows on
  int odd, red_major, row, ch;
  int mn_left, r_left;  // lanes or columns, and reduction, from the thread's first element to their ends
  __device__ __forceinline__ void start(const uint16_t* base, int64_t ld, int red, int mn0, int mn_end, int r0, int r_end, int tid) {
    red_major = red;
    row = tid >> 3, ch = tid & 7;
    const int mn = red ? mn0 + row : mn0 + ch * 8, r = red ? r0 + ch * 8 : r0 + row;
    src = base + (red ? (int64_t)mn * ld + r : (int64_t)r * ld + mn);
    step = 32 * ld;
    odd = (int)(reinterpret_cast<uintptr_t>(src) >> 1) & 1;
    mn_left = mn_end - mn, r_left = r_end - r;
  }
  __device__ __forceinline__ int valid(int u) const {
    if (red_major) return mn_left > 32 * u ? min(8, r_left) : 0;
    return r_left > 32 * (u & 1) ? min(8, mn_left - 64 * (u >> 1)) : 0;
  }
  // The words of the chunks in rows 32 u0 .. 32 u0 + 96 of the current stage, and their way into the stage: other work
  // goes in between, while they are in flight.
  __device__ __forceinline__ void load(int u0, int units, uint32_t (&w)[4][5]) const {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(src - odd);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + i, v = u < units ? valid(u) : 0;
      const uint32_t* qu = q + (red_major ? u * step : (u & 1) * step + 64 * (u >> 1)) / 2;
      if (v >= 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i][k] = qu[k];
        w[i][4] = odd ? qu[4] : 0u;
      } else {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[i][k] = v > 0 && 2 * k < v + odd ? qu[k] : 0u;  // (a word with a wanted element)
      }
    }
  }
  __device__ __forceinline__ void put(uint8_t* dst, int u0, int units, const uint32_t (&w)[4][5]) const {
    const uint32_t sh = odd * 16;
    uint8_t* to = dst + row * 128 + ((ch ^ (row & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + i;
      if (u >= units) break;
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = __funnelshift_r(w[i][k], w[i][k + 1], sh);
      const int v = valid(u);
      if (v < 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = v - 2 * k < 1 ? 0u : v - 2 * k < 2 ? r[k] & 0xffffu : r[k];
      }
      *reinterpret_cast<uint4*>(to + u * 4096) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
  __device__ __forceinline__ void next_stage(int64_t elements) {
    src += elements;
    r_left -= BK;
  }
};

// ------------------------------------------------------------------------------------ epilogues

// The running sum of a long reduction: adds (first: copies) an accumulator of n columns to the other one's place, from column
// c0 on every second 32 columns, the warp's own lanes. Only this warp reads what it wrote there.
__device__ __forceinline__ void fold_acc(uint32_t acc, uint32_t sum, bool first, int c0, int n) {
  for (int c = c0; c < n; c += 64) {
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      uint32_t v[16], w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
      tmem_get16(acc + c + h, v);
      if (!first) tmem_get16(sum + c + h, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
      tmem_put16(sum + c + h, v);
    }
  }
  tmem_st_wait();
}

// 32 elements of one lane, nv of them there, `ld` apart: the type is chosen once for all of them.
__device__ __forceinline__ void to16(const float (&v)[32], uint16_t (&h)[32], int f16) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    uint32_t u;
    if (f16) {
      const __half2 t = __floats2half2_rn(v[j], v[j + 1]);
      u = *reinterpret_cast<const uint32_t*>(&t);
    } else {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[j], v[j + 1]);
      u = *reinterpret_cast<const uint32_t*>(&t);
    }
    h[j] = (uint16_t)u, h[j + 1] = (uint16_t)(u >> 16);
  }
}
template <class T>
__device__ __forceinline__ void store_col(T* q, int64_t ld, int nv, const T (&h)[32]) {
  if (nv >= 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j, q += ld) *q = h[j];
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j, q += ld)
      if (j < nv) *q = h[j];
  }
}
template <class T>
__device__ __forceinline__ void load_col(const T* q, int64_t ld, int nv, T (&h)[32]) {
  if (nv >= 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j, q += ld) h[j] = *q;
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j, q += ld) h[j] = j < nv ? *q : T(0);
  }
}
__device__ __forceinline__ void add16(float (&v)[32], const void* base, int64_t at, int64_t ld, int nv, int f16) {
  uint16_t h[32];
  load_col(static_cast<const uint16_t*>(base) + at, ld, nv, h);
  if (f16) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += __half2float(__ushort_as_half(h[j]));
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += __uint_as_float((uint32_t)h[j] << 16);
  }
}
__device__ __forceinline__ void add32(float (&v)[32], const float* q, int64_t ld, int nv) {
  float h[32];
  load_col(q, ld, nv, h);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += h[j];
}

// Writes 32 columns (nv exist for this lane) of lane l.
__device__ __forceinline__ void put(const MmProblem& p, int g, int l, int c, int nv, const float (&v)[32]) {
  const MmEpiArgs& e = p.e;
  if (l >= p.lanes) return;
  const int64_t o = (p.rag == MM_RAG_RED ? g * e.group_stride : 0) + (int64_t)c * e.ld + l;
  if (e.out_f32) {
    store_col(static_cast<float*>(e.out) + o, e.ld, nv, v);
  } else {
    uint16_t h[32];
    to16(v, h, p.f16);
    store_col(static_cast<uint16_t*>(e.out) + o, e.ld, nv, h);
  }
}

// The arithmetic of a stored result: 32 columns (nv exist for this lane) of lane l.
__device__ __forceinline__ void epi_store(const MmProblem& p, int g, int l, int c, int nv, bool accumulate, float (&v)[32]) {
  const MmEpiArgs& e = p.e;
  if (l >= p.lanes) nv = 0;
  if (e.acc_in) add32(v, e.acc_in + (int64_t)c * e.acc_ld + l, e.acc_ld, nv);
  if (e.scale) {
    const float s = *e.scale;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= s;
  }
  if (e.bias) {
    const float b = nv ? ld16(e.bias, l, p.f16) : 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += b;
  }
  if (e.z) {
    uint16_t h[32];
    to16(v, h, p.f16);
    store_col(static_cast<uint16_t*>(e.z) + (int64_t)c * e.ldz + l, e.ldz, nv, h);
  }
  if (e.act == MM_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = mm_silu(v[j]);
  } else if (e.act == MM_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = mm_gelu(v[j]);
  } else if (e.act == MM_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = mm_relu(v[j]);
  }
  if (e.residual) add16(v, e.residual, (int64_t)c * e.ldr + l, e.ldr, nv, p.f16);
  if (accumulate) {
    const int64_t o = (p.rag == MM_RAG_RED ? g * e.group_stride : 0) + (int64_t)c * e.ld + l;
    if (e.out_f32)
      add32(v, static_cast<const float*>(e.out) + o, e.ld, nv);
    else
      add16(v, e.out, o, e.ld, nv, p.f16);
  }
}

// ---- 16-bit results by rows: the warps hold 32 lanes x 32 columns as fragments (a thread: lanes i/4 + 8 r, columns
// 8 j + 2 (i % 4) and the next), which stmatrix writes transposed into shared memory, from where whole rows of 128
// lanes leave as 16-byte stores.
struct Frag {
  float v[4][4][2];  // [block of 8 columns][block of 8 lanes][column parity]
};
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, Frag& f) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) f.v[(i >> 2) & 3][2 * (i >> 4) + ((i >> 1) & 1)][i & 1] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int f16) {
  if (f16) {
    const __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
  }
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
// The address that lane i gives for its row of an 8 x 8 block: block i / 8 of the warp's four, row i % 8.
__device__ __forceinline__ uint32_t frag_addr(uint32_t stage, int quad, int j, int lane) {
  return stage + (uint32_t)((8 * j + (lane & 7)) * kRowBytes + quad * 64 + (lane >> 3) * 16);
}
__device__ __forceinline__ void frag_out(uint32_t stage, int quad, int lane, const Frag& f, int f16) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(frag_addr(stage, quad, j, lane)),
                 "r"(pack16(f.v[j][0][0], f.v[j][0][1], f16)), "r"(pack16(f.v[j][1][0], f.v[j][1][1], f16)),
                 "r"(pack16(f.v[j][2][0], f.v[j][2][1], f16)), "r"(pack16(f.v[j][3][0], f.v[j][3][1], f16))
                 : "memory");
}
__device__ __forceinline__ void frag_add(uint32_t stage, int quad, int lane, Frag& f, int f16) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t r[4];
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(frag_addr(stage, quad, j, lane))
                 : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (f16) {
        f.v[j][i][0] += __half2float(__ushort_as_half((uint16_t)r[i]));
        f.v[j][i][1] += __half2float(__ushort_as_half((uint16_t)(r[i] >> 16)));
      } else {
        f.v[j][i][0] += __uint_as_float(r[i] << 16);
        f.v[j][i][1] += __uint_as_float(r[i] & 0xffff0000u);
      }
    }
  }
}
// Rows of 16-byte pieces between shared and global memory: thread i of 128 takes piece i % 16 of rows i / 16 + 8 k.
struct Rows {
  uint32_t smem;  // of the thread's first piece
  int row;
  bool live;  // the piece lies inside the matrix
  __device__ __forceinline__ void store(void* base, int64_t at, int64_t ld, int nv) const {
    uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (live && row + 8 * k < nv) q[k * ld] = lds128(smem + 8 * k * kRowBytes);  // (ld: 8 rows of ld elements, in pieces)
  }
  __device__ __forceinline__ void load(const void* base, int64_t at, int64_t ld, int nv, uint4 (&r)[4]) const {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = live && row + 8 * k < nv ? q[k * ld] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void stage(const uint4 (&r)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(smem + 8 * k * kRowBytes), "r"(r[k].x), "r"(r[k].y), "r"(r[k].z), "r"(r[k].w) : "memory");
  }
};

// Running maximum m and sum s of exp(z - m) of one token over 32 words (nv exist).
__device__ __forceinline__ void epi_stats(float (&v)[32], int nv, float& m, float& s) {
  float top = m;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < nv) top = fmaxf(top, v[j]);
  if (top == -INFINITY) {  // only words of probability zero so far (NaN logits still reach the sum)
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 32; ++j) bad |= j < nv && v[j] != v[j];
    if (bad) s = NAN;
    return;
  }
  s *= __expf(m - top);
  float t = 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < nv) t += __expf(v[j] - top);
  s += t;
  m = top;
}

template <int CG, int EPI, bool GEN>
__global__ void __launch_bounds__(GEN ? kThreads + 32 * kLoaders : kThreads, 1)
    mm_tc_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                 const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const MmProblem& p = a.p;
  // the stages start on a 1024-byte boundary (the swizzle's period); in a pair both CTAs have the same layout
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int stage_bytes = A_BYTES + a.bn / CG * BK * 2;
  uint8_t* out_stage = smem + a.stages * stage_bytes;  // [2][kOutBytes]
  float* parts = reinterpret_cast<float*>(out_stage + 2 * kOutBytes);  // [split - 1][bn][kPartLd], in the cluster's first CTA
  uint8_t* ctrl = out_stage + 2 * kOutBytes + (a.split - 1) * a.bn * kPartLd * 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* clean = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(clean + kMaxStages);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* lo_of = reinterpret_cast<int*>(tmem_slot + 4);
  int* pref = lo_of + p.groups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
  const int acc_stride = max(a.bn, 32);
  uint32_t tmem_cols = 32;
  while (tmem_cols < 2u * max(a.bn, 32)) tmem_cols *= 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full + i, GEN ? kLoaders : 1);
      mbar_init(empty + i, !GEN && p.rag == MM_RAG_RED ? 2 : 1);  // the MMAs' commit, and the cleaner
      mbar_init(clean + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, kEpiWarps * CG);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_get<CG>(tmem_slot, tmem_cols);
  if (warp == 0 && lane == 0 && !GEN) {
    tmap_prefetch(&ta);
    tmap_prefetch(&tb);
  }
  wait_for_previous();
  let_next_start();
  if (p.rag != MM_DENSE) {
    const int total = p.rag == MM_RAG_COLS ? p.cols : p.red;
    for (int g = threadIdx.x; g <= p.groups; g += blockDim.x) lo_of[g] = min(max(*(p.offsets + g), 0), total);
    __syncthreads();
    if (p.rag == MM_RAG_COLS && warp == 2) {
      int run = 0;
      for (int g0 = 0; g0 <= p.groups; g0 += 32) {
        const int g = g0 + lane;
        const int n = g < p.groups ? (max(lo_of[g + 1] - lo_of[g], 0) + a.bn - 1) / a.bn : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += u;
        }
        if (g <= p.groups) pref[g] = run + inc - n;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  tc_fence_before();
  if (CG == 2 || a.split > 1) cluster_sync();  // every CTA of the cluster runs and has set its barriers up
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int tiles = a.lane_tiles * (p.rag == MM_RAG_COLS ? pref[p.groups] : a.col_tiles) * (p.rag == MM_RAG_RED ? p.groups : 1);
  if (p.rag == MM_DENSE) tiles += (tiles - a.tail_from) * ((1 << a.tail_lg) - 1);
  const int share = CG == 2 ? 2 : a.split;  // CTAs that work on the same tile
  const int first = blockIdx.x / share, step = gridDim.x / share;
  const int part = CG == 1 && a.split > 1 ? (int)cluster_ctarank() : 0;
  if (CG == 1 && a.split > 1) tiles = min(tiles, first + 1);  // one tile a cluster, whatever the offsets say

  if ((warp == 0 || warp == 3) && !GEN) {
    // ------------------------------------------------------------------ TMA producers: warp 0 of A, warp 3 of B
    // One warp for both issues a stage's copies no faster than the MMAs use it up (y of 256 experts, 128 rows each: 726
    // us, 714 with two; gradients of 4096 x 2048 x 4096: 108, 105).
    const bool a_red = p.a.red_major, b_red = p.b.red_major, of_a = warp == 0;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int a_boxes = a_red ? 1 : 2 / a.a_blocks;
    Walk<CG> walk;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile o = walk.next(a, lo_of, pref, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const int nb = mma_n<CG>(p, o.n) / CG;  // columns that this CTA stages
      const int b_boxes = b_red ? (nb + a.b_box - 1) / a.b_box : (nb / 64 + a.b_blocks - 1) / a.b_blocks;
      const int b_box_bytes = b_red ? a.b_box * 128 : a.b_blocks * 8192;
      const uint32_t bytes = CG * (A_BYTES + b_boxes * b_box_bytes);
      const int la = o.l0 + BM * rank, cb = o.c0 + nb * rank;
      const int ga = p.rag == MM_RAG_COLS ? o.g : 0;
      for (int k = 0; k < o.red; k += BK) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + s, ph ^ 1, abort_flag, p.err, 1));
        if (!ok) break;
        const uint32_t st = su32(smem + s * stage_bytes), bar = CG == 2 ? mapa(su32(full + s), 0) : su32(full + s);
        const int r = o.r0 + k;
        if (of_a) {
          if (lane == 0 && rank == 0) mbar_expect_tx(full + s, bytes);  // (copies may report before it)
          if (lane < a_boxes) {
            if (a_red)
              tma_load<CG>(st, &ta, r, la, 0, ga, bar);
            else if (a.a_blocks > 1)
              tma_load<CG>(st, &ta, 0, r, la / 64, ga, bar);
            else
              tma_load<CG>(st + lane * 8192, &ta, la + 64 * lane, r, 0, ga, bar);
          }
        } else if (lane < b_boxes) {
          const uint32_t to = st + A_BYTES + lane * b_box_bytes;
          if (b_red)
            tma_load<CG>(to, &tb, r, cb + lane * a.b_box, 0, 0, bar);
          else if (a.b_blocks > 1)
            tma_load<CG>(to, &tb, 0, r, cb / 64 + lane * a.b_blocks, 0, bar);
          else
            tma_load<CG>(to, &tb, cb + 64 * lane, r, 0, 0, bar);
        }
        if (++s == a.stages) s = 0, ph ^= 1;
      }
    }
  } else if (GEN && warp >= kFirstLoader) {
    // ------------------------------------------------------------------ loaders (any alignment)
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int tid = threadIdx.x - kThreads;
    Walk<CG> walk;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile o = walk.next(a, lo_of, pref, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const uint16_t* pa = static_cast<const uint16_t*>(p.a.p) + (p.rag == MM_RAG_COLS ? o.g * p.a.group_stride : 0);
      const int nb = mma_n<CG>(p, o.n);
      Loader la, lb;
      la.start(pa, p.a.ld, p.a.red_major, o.l0, p.lanes, o.r0, o.r0 + o.red, tid);
      lb.start(static_cast<const uint16_t*>(p.b.p), p.b.ld, p.b.red_major, o.c0, o.c0 + o.n, o.r0, o.r0 + o.red, tid);
      const int b_units = (nb + 31) / 32;
      uint32_t wa[4][5], wb[4][5];
      if (o.red > 0) la.load(0, BM / 32, wa);
      for (int k = 0; k < o.red; k += BK) {
        lb.load(0, b_units, wb);
        ok = __all_sync(0xffffffffu, mbar_wait(empty + s, ph ^ 1, abort_flag, p.err, 1));
        if (!ok) break;
        uint8_t* st = smem + s * stage_bytes;
        la.put(st, 0, BM / 32, wa);
        la.next_stage(p.a.red_major ? BK : BK * p.a.ld);
        if (k + BK < o.red) la.load(0, BM / 32, wa);  // in flight over the next stage's wait
        lb.put(st + A_BYTES, 0, b_units, wb);
        if (b_units > 4) {
          lb.load(4, b_units, wb);
          lb.put(st + A_BYTES, 4, b_units, wb);
        }
        lb.next_stage(p.b.red_major ? BK : BK * p.b.ld);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full + s);
        if (++s == a.stages) s = 0, ph ^= 1;
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------------ MMA (one thread)
    if (elect_one()) {
      int s = 0, buf = 0;
      uint32_t ph = 0, cleaned = 0, used = 0;  // (used: the parity of each accumulator's uses)
      bool ok = true;
      const uint64_t a_step = (p.a.red_major ? 32 : 2048) >> 4, b_step = (p.b.red_major ? 32 : 2048) >> 4;
      const uint64_t a_desc = op_desc(su32(smem), p.a.red_major), b_desc = op_desc(su32(smem + A_BYTES), p.b.red_major);
      const uint32_t type = p.f16 ? 0u : 1u;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile o = tile_of<CG>(a, lo_of, pref, t, part);
        if (o.red <= 0 || o.n <= 0) continue;  // an empty sum: the epilogue writes zeros without an accumulator
        const int n = mma_n<CG>(p, o.n);
        const uint32_t idesc = (1u << 4) | type << 7 | type << 10 | (p.a.red_major ? 0u : 1u << 15) |
                               (p.b.red_major ? 0u : 1u << 16) | (uint32_t)(n >> 3) << 17 | (uint32_t)(BM * CG >> 4) << 24;
        // Accumulators take turns from tile to tile (or, of a result added up in memory, from seg to seg). A tile that is
        // summed up in tensor memory stays with its own one, seg after seg, and so does the tile after it: the other
        // one holds the sum, which the epilogue is done with when it hands the last seg's accumulator back.
        const bool folds = a.fold && o.red > a.seg;
        uint32_t d = 0;
        int in_seg = 0;  // reduction already in this accumulator
        for (int k = 0; k < o.red; k += BK) {
          if (in_seg == 0) {
            const int b = a.accs == 1 || k == 0 ? buf : 1;  // (1: the second accumulator of the same tile)
            if (!mbar_wait(acc_empty + b, (used >> b & 1) ^ 1, abort_flag, p.err, 6)) {
              ok = false;
              break;
            }
            tc_fence_after();
            d = tmem + (uint32_t)(b * acc_stride);
          }
          const int left = min(BK, o.red - k);
          if (!mbar_wait(full + s, ph, abort_flag, p.err, 7) ||
              (!GEN && p.rag == MM_RAG_RED && (left & 15) && !mbar_wait(clean + s, cleaned >> s & 1, abort_flag, p.err, 2))) {
            ok = false;
            break;
          }
          if (left & 15) cleaned ^= 1u << s;
          tc_fence_after();
          const uint64_t da = a_desc + (uint32_t)(s * stage_bytes >> 4), db = b_desc + (uint32_t)(s * stage_bytes >> 4);
          if (left > 48) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma<CG>(d, da + i * a_step, db + i * b_step, idesc, in_seg | i);
          } else {
            for (int i = 0; 16 * i < left; ++i) mma<CG>(d, da + i * a_step, db + i * b_step, idesc, in_seg | i);
          }
          commit<CG>(empty + s);
          if (++s == a.stages) s = 0, ph ^= 1;
          in_seg += BK;
          if (in_seg == a.seg || k + BK >= o.red) {
            if (a.accs == 1) {
              commit<CG>(acc_full + buf);
              used ^= 1u << buf;
              if (!folds) buf ^= 1;
            } else if (k + BK >= o.red) {
              commit<CG>(acc_full);
              used ^= 3u;
            }
            in_seg = 0;
          }
        }
      }
    }
  } else if (warp == 2 && !GEN && p.rag == MM_RAG_RED) {
    // ------------------------------------------------------------------ cleaner of ragged ends
    // Where a group ends inside a step of 16, the rows of the next group that the boxes also brought are
    // cleared in both operands before the MMA reads them (0 * NaN would not vanish). A row is 128 bytes of a box.
    // The warp passes every stage in turn and arrives on its empty barrier too, so that the ring cannot lap it.
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    Walk<CG> walk;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile o = walk.next(a, lo_of, pref, t, step, tiles, part, lane);
      for (int k = 0; k < o.red; k += BK) {
        ok = __all_sync(0xffffffffu, mbar_wait(full + s, ph, abort_flag, p.err, 2));
        if (!ok) break;
        const int left = min(BK, o.red - k);
        if (left & 15) {
          const int boxes = 2 + mma_n<CG>(p, o.n) / 64, from = left + (lane >> 3), end = (left + 15) & ~15;
          uint8_t* st = smem + s * stage_bytes + from * 128 + (lane & 7) * 16;
#pragma unroll
          for (int box = 0; box < 6; ++box) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (box < boxes && from + 4 * r < end) *reinterpret_cast<uint4*>(st + box * 8192 + r * 512) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        }
        __syncwarp();
        if (lane == 0) {
          if (left & 15) mbar_arrive(clean + s);
          mbar_arrive(empty + s);
        }
        if (++s == a.stages) s = 0, ph ^= 1;
      }
    }
  } else if (EPI == kEpiPlain && warp >= 4 && warp < kFirstLoader) {
    // ------------------------------------------------------------------ epilogue without anything to add
    const int quad = warp & 3, half = (warp - 4) >> 2, piece = threadIdx.x & 15, row = (threadIdx.x & 127) >> 4;
    const uint32_t stage = su32(out_stage) + half * kOutBytes, from = stage + (uint32_t)(row * kRowBytes + piece * 16);
    const int64_t ld = p.e.ld;
    int buf = 0;
    uint32_t used = 0;  // as the MMA counts them
    Walk<CG> walk;
    for (int t = first; t < tiles; t += step) {
      const Tile o = walk.next(a, lo_of, pref, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const bool sum = o.red > 0;
      const int l = o.l0 + BM * rank + 8 * piece;
      uint32_t taddr = tmem + (uint32_t)(buf * acc_stride) + ((uint32_t)(32 * quad) << 16);
      int left = l < p.lanes ? o.n - 32 * half - row : 0;  // rows from the thread's first to the tile's end
      uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.e.out) + (p.rag == MM_RAG_RED ? o.g * p.e.group_stride : 0) +
                                          (o.c0 + 32 * half + row) * ld + l);
      const bool folds = a.fold && o.red > a.seg;
      const uint32_t held = tmem + (uint32_t)((buf ^ 1) * acc_stride) + ((uint32_t)(32 * quad) << 16);
      bool ok = true;
      for (int k = 0; ok && k < o.red; k += a.seg) {  // (one round unless the tile folds)
        ok = mbar_wait(acc_full + buf, used >> buf & 1, abort_flag, p.err, 5);
        __syncwarp();
        tc_fence_after();
        used ^= 1u << buf;
        if (!folds || !ok) break;
        fold_acc(taddr, held, k == 0, 32 * half, o.n);
        if (k + a.seg >= o.red) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            mbar_arrive_cluster(mapa(su32(acc_empty + buf), 0));
          else
            mbar_arrive(acc_empty + buf);
        }
      }
      if (folds) taddr = held;
      if (!named_bar_all(2 + half, 128, ok)) break;  // (the warps that share barriers leave together)
      for (int c = 32 * half; c < o.n; c += 64) {
        Frag f;
        if (sum) {
          tmem_ld_frag(taddr + c, f);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) f.v[j][r][0] = f.v[j][r][1] = 0.f;
        }
        frag_out(stage, quad, lane, f, p.f16);
        named_bar(2 + half, 128);
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = lds128(from + 8 * k * kRowBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (8 * k < left) q[k * ld] = w[k];  // (8 rows of ld elements are ld pieces)
        left -= 64;
        q += 8 * ld;
        named_bar(2 + half, 128);
      }
      if (sum) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {  // the MMA may overwrite this buffer
          if (CG == 2)
            mbar_arrive_cluster(mapa(su32(acc_empty + buf), 0));
          else
            mbar_arrive(acc_empty + buf);
        }
        if (!folds) buf ^= 1;
      }
    }
  } else if (EPI != kEpiPlain && warp >= 4 && warp < kFirstLoader) {
    // ------------------------------------------------------------------ epilogue
    // Two warps per lane quadrant take the tile's 32-column chunks in turn; the four warps of a half work on the same
    // chunk.
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const MmEpiArgs& e = p.e;
    const uint32_t stage = su32(out_stage) + half * kOutBytes;
    Rows rows;
    {
      const int i = threadIdx.x & 127;
      rows.row = i >> 4;
      rows.smem = stage + (uint32_t)(rows.row * kRowBytes + (i & 15) * 16);
      rows.live = false;
    }
    const int c_first = 32 * half, c_step = 64;
    int buf = 0;
    uint32_t used = 0;  // as the MMA counts them
    Walk<CG> walk;
    for (int t = first; t < tiles; t += step) {
      const Tile o = walk.next(a, lo_of, pref, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const int l0 = o.l0 + BM * rank;
      const bool sum = o.red > 0;
      // what the tile needs besides its sums is fetched before they are waited for
      const bool by_rows = EPI != MM_EPI_STATS && a.rows_out;
      const int64_t group_out = p.rag == MM_RAG_RED ? o.g * e.group_stride : 0;
      const void* add = e.accumulate ? e.out : e.residual;
      const int64_t add_ld = e.accumulate ? e.ld : e.ldr;
      const int piece = l0 + (threadIdx.x & 15) * 8;
      const int64_t first_row = o.c0 + c_first + rows.row;
      int64_t add_at = (e.accumulate ? group_out : 0) + first_row * add_ld + piece;
      uint4 next[4];
      rows.live = piece < p.lanes;
      if (by_rows && add && part == 0) rows.load(add, add_at, add_ld, o.n - c_first, next);
      // lanes of the fragments (four per thread) or the thread's own lane
      float lse[4], gw[4], bias[4];
      int lab[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int l = l0 + 32 * quad + (by_rows ? (lane >> 2) + 8 * r : lane);
        lse[r] = 0.f, gw[r] = 0.f, bias[r] = 0.f, lab[r] = -1;
        if (l >= p.lanes || (!by_rows && r)) continue;
        if (EPI == MM_EPI_STORE) {
          if (e.bias) bias[r] = ld16(e.bias, l, p.f16);
        } else {
          lab[r] = max(*(e.labels + l), -1);
          if (EPI == MM_EPI_SOFTGRAD) {
            const bool skip = lab[r] == e.ignore || lab[r] < 0 || lab[r] >= e.vocab;
            lse[r] = *(e.lse + l);
            gw[r] = skip ? 0.f : *(e.g + l) / *e.gscale * kMmGradOne;
            lab[r] = skip ? -1 : lab[r] - e.word0;
          }
        }
      }
      float m = -INFINITY, total = 0.f;
      constexpr bool kHold = EPI == MM_EPI_STATS && CG == 2;  // sums over accumulators are held in registers
      float z[kHold ? 4 : 1][32];                             // the logits of the thread's four chunks
      const bool folds = a.fold && o.red > a.seg;
      bool ok = true;
      for (int k = 0; k == 0 || k < o.red; k += a.accs == 1 ? a.seg : o.red) {  // accumulators of the tile
        uint32_t taddr = tmem + (uint32_t)(buf * acc_stride) + ((uint32_t)(32 * quad) << 16);
        if (sum) {
          ok = mbar_wait(acc_full + buf, used >> buf & 1, abort_flag, p.err, 5);
          __syncwarp();
          tc_fence_after();
          used ^= 1u << buf;
        }
        if (folds && ok) {
          const uint32_t held = tmem + (uint32_t)((buf ^ 1) * acc_stride) + ((uint32_t)(32 * quad) << 16);
          fold_acc(taddr, held, k == 0, c_first, o.n);
          taddr = held;
          if (k + a.seg < o.red) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (CG == 2)
                mbar_arrive_cluster(mapa(su32(acc_empty + buf), 0));
              else
                mbar_arrive(acc_empty + buf);
            }
            continue;
          }
        }
        // (the warps that share barriers in what follows leave together)
        ok = EPI == MM_EPI_STATS ? named_bar_all(1, 32 * kEpiWarps, ok) : named_bar_all(2 + half, 128, ok);
        if (CG == 1 && a.split > 1) {
          // the CTAs of a cluster have each summed a share of the reduction: the others hand theirs to the first one's
          // shared memory, which adds them in order
          if (part > 0 && ok) {
            for (int c = c_first; c < o.n; c += c_step) {
              float v[32];
              if (sum) {
                tmem_ld32(taddr + c, v);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.f;
              }
              const uint32_t to = mapa(su32(parts + ((part - 1) * a.bn + c) * kPartLd + 32 * quad + lane), 0);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + j * kPartLd * 4), "f"(v[j]) : "memory");
            }
          }
          cluster_sync();
          if (part > 0) ok = false;
        }
        if (!ok) break;
        const bool two = EPI == MM_EPI_STATS && !kHold && a.accs > 1;
        if (two) {  // fold the first accumulator into the second and hand it back: the next tile's first half needs it soon
          for (int c = c_first; o.red > a.seg && c < o.n && l0 + 32 * quad < p.lanes; c += c_step) {
            float v[32], more[32];
            tmem_ld32(taddr + c, v);
            tmem_ld32(taddr + acc_stride + c, more);
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j] + more[j]);
            tmem_st32(taddr + acc_stride + c, w);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty);
        }
        if (EPI == MM_EPI_STATS) {
          const uint32_t sums = two && o.red > a.seg ? taddr + acc_stride : taddr;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c_first + i * c_step;
            if (c >= o.n || l0 + 32 * quad >= p.lanes) break;  // (no words, or no tokens)
            float v[32];
            float(&y)[32] = kHold ? z[kHold ? i : 0] : v;
            tmem_ld32(sums + c, v);
            if (kHold) {
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = k ? y[j] + v[j] : v[j];
              if (k + a.seg < o.red) continue;
            }
            const int nv = min(32, o.n - c), at = lab[0] - (o.c0 + c);
            epi_stats(y, nv, m, total);
            if (at >= 0 && at < nv) {  // (the label of a lane that exists)
              float own = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == at) own = y[j];
              e.zlab[l0 + 32 * quad + lane] = own;
            }
          }
        } else if (by_rows) {
          for (int c = c_first; c < o.n; c += c_step) {
            Frag f;
            if (sum) {
              tmem_ld_frag(taddr + c, f);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) f.v[j][r][0] = f.v[j][r][1] = 0.f;
            }
            if (CG == 1) {
              for (int k = 1; k < a.split; ++k) {
                const float* q = parts + ((k - 1) * a.bn + c + 2 * (lane & 3)) * kPartLd + 32 * quad + (lane >> 2);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    f.v[j][r][0] += q[8 * j * kPartLd + 8 * r];
                    f.v[j][r][1] += q[(8 * j + 1) * kPartLd + 8 * r];
                  }
              }
            }
            const int64_t row_at = first_row + (c - c_first);
            if (EPI == MM_EPI_SOFTGRAD) {
              const int word = o.c0 + c + 2 * (lane & 3);
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    // (a row without gradient stays zero even where its logits are not finite)
                    const float d = (__expf(f.v[j][r][q] - lse[r]) - (word + 8 * j + q == lab[r] ? 1.f : 0.f)) * gw[r];
                    f.v[j][r][q] = gw[r] == 0.f ? 0.f : d;
                  }
            } else {
              if (e.scale) {
                const float sc = *e.scale;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) f.v[j][r][0] *= sc, f.v[j][r][1] *= sc;
              }
              if (e.bias) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) f.v[j][r][0] += bias[r], f.v[j][r][1] += bias[r];
              }
              if (e.z) {
                frag_out(stage, quad, lane, f, p.f16);
                named_bar(2 + half, 128);
                rows.store(e.z, row_at * e.ldz + piece, e.ldz, o.n - c);
                named_bar(2 + half, 128);
              }
              if (e.act == MM_ACT_SILU) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) f.v[j][r][0] = mm_silu(f.v[j][r][0]), f.v[j][r][1] = mm_silu(f.v[j][r][1]);
              } else if (e.act == MM_ACT_GELU) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) f.v[j][r][0] = mm_gelu(f.v[j][r][0]), f.v[j][r][1] = mm_gelu(f.v[j][r][1]);
              } else if (e.act == MM_ACT_RELU) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) f.v[j][r][0] = mm_relu(f.v[j][r][0]), f.v[j][r][1] = mm_relu(f.v[j][r][1]);
              }
              if (add) {
                rows.stage(next);
                named_bar(2 + half, 128);
                add_at += c_step * add_ld;
                if (c + c_step < o.n) rows.load(add, add_at, add_ld, o.n - c - c_step, next);
                frag_add(stage, quad, lane, f, p.f16);  // (each warp rereads and overwrites its own quarter only)
                __syncwarp();
              }
            }
            frag_out(stage, quad, lane, f, p.f16);
            named_bar(2 + half, 128);
            rows.store(e.out, group_out + row_at * e.ld + piece, e.ld, o.n - c);
            named_bar(2 + half, 128);
          }
        } else {
          const int l = l0 + 32 * quad + lane;
          for (int c = c_first; c < o.n; c += c_step) {
            float v[32];
            if (sum) {
              tmem_ld32(taddr + c, v);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
            if (CG == 1) {
              for (int k = 1; k < a.split; ++k) {
                const float* q = parts + ((k - 1) * a.bn + c) * kPartLd + 32 * quad + lane;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += q[j * kPartLd];
              }
            }
            const int nv = min(32, o.n - c);
            if (EPI == MM_EPI_STORE) {
              epi_store(p, o.g, l, o.c0 + c, nv, e.accumulate || (k && !folds), v);
              put(p, o.g, l, o.c0 + c, nv, v);
            } else {
              const int at = lab[0] - (o.c0 + c);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = gw[0] == 0.f ? 0.f : (__expf(v[j] - lse[0]) - (j == at ? 1.f : 0.f)) * gw[0];
              put(p, 0, l, o.c0 + c, nv, v);
            }
          }
        }
        if (sum) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {  // the MMA may overwrite this buffer
            if (CG == 2)
              mbar_arrive_cluster(mapa(su32(acc_empty + buf), 0));
            else
              mbar_arrive(acc_empty + (two ? 1 : buf));
          }
          if (a.accs == 1 && !folds) buf ^= 1;
        }
      }
      if (!ok) break;
      if (EPI == MM_EPI_STATS) {  // the two halves' partials are joined
        float2* x = reinterpret_cast<float2*>(out_stage) + 32 * quad + lane;
        const int l = l0 + 32 * quad + lane;
        if (half) *x = make_float2(m, total);
        named_bar(2, 32 * kEpiWarps);
        if (!half && l < p.lanes) {
          const float2 q = *x;
          const float top = fmaxf(m, q.x);
          // (a half without likely words has m = -inf and adds its sum, 0 or NaN)
          const float s0 = m == top ? total : total * __expf(m - top), s1 = q.x == top ? q.y : q.y * __expf(q.x - top);
          e.part[(int64_t)(o.c0 / a.bn) * p.lanes + l] = make_float2(top, s0 + s1);
        }
      }
    }
  }
  __syncwarp();
  if (CG == 1 && a.split > 1 && first < tiles && (warp < 4 || warp >= kFirstLoader)) cluster_sync();
  if (*abort_flag) {  // after a timeout: let the copies and MMAs in flight finish (about a millisecond)
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000ll) {
    }
  }
  tc_fence_before();
  if (CG == 2)
    cluster_sync();  // no copy, MMA or commit still targets the other CTA
  else
    __syncthreads();
  if (warp == 1) tmem_free<CG>(tmem, tmem_cols);
}

// ------------------------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
int g_sms[64] = {}, g_pairs[64] = {};  // per device: SMs, and pairs that can be resident at once

// 4D map with boxes of 64 contiguous elements, 128-byte swizzle: (contiguous index, row, -, group) with box_rows rows;
// or, for an MN-major operand whose width is a multiple of 64, (index in a block of 64, row, block, group) with
// `blocks` blocks of BK rows, which one copy lays one after the other.
bool make_map(CUtensorMap* m, const MmOperand& o, int f16, uint64_t inner, uint64_t rows, uint64_t groups, uint32_t box_rows, int blocks) {
  const cuuint64_t row = (cuuint64_t)o.ld * 2;
  const cuuint64_t dims[4] = {blocks > 1 ? 64 : inner, rows, blocks > 1 ? inner / 64 : 1, groups};
  const cuuint64_t strides[3] = {row, blocks > 1 ? 128 : row, groups > 1 ? (cuuint64_t)o.group_stride * 2 : row};
  const cuuint32_t box[4] = {BK, box_rows, (cuuint32_t)blocks, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return g_encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(o.p),
                  dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int smem_bytes(int cg, int bn, int stages, int split, const MmProblem& p) {
  return 1024 + stages * (A_BYTES + bn / cg * BK * 2) + 2 * kOutBytes + (split - 1) * bn * kPartLd * 4 + ctrl_bytes(p.rag, p.groups);
}

template <int CG, int EPI, bool GEN>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const TcArgs& a, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(GEN ? kThreads + 32 * kLoaders : kThreads);
  cfg.dynamicSmemBytes = smem_bytes(CG, a.bn, a.stages, a.split, a.p);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG == 2 ? 2 : a.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 || a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, mm_tc_kernel<CG, EPI, GEN>, ta, tb, a);
}

template <int CG, bool GEN>
cudaError_t launch_epi(const CUtensorMap& ta, const CUtensorMap& tb, const TcArgs& a, int grid, cudaStream_t s) {
  switch (a.p.epi) {
    case MM_EPI_STATS: return launch<CG, MM_EPI_STATS, GEN>(ta, tb, a, grid, s);
    case MM_EPI_SOFTGRAD: return launch<CG, MM_EPI_SOFTGRAD, GEN>(ta, tb, a, grid, s);
    default: break;
  }
  const MmEpiArgs& e = a.p.e;
  const bool plain = a.rows_out && a.split == 1 && !e.scale && !e.bias && !e.z && !e.residual && !e.accumulate && e.act == MM_ACT_NONE;
  if (!GEN && plain) return launch<CG, kEpiPlain, false>(ta, tb, a, grid, s);
  return launch<CG, MM_EPI_STORE, GEN>(ta, tb, a, grid, s);
}

template <int CG, int EPI, bool GEN>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(mm_tc_kernel<CG, EPI, GEN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
}
template <int CG, bool GEN>
cudaError_t prepare_epi() {
  cudaError_t e = prepare_one<CG, MM_EPI_STORE, GEN>();
  if (e == cudaSuccess) e = prepare_one<CG, MM_EPI_STATS, GEN>();
  if (e == cudaSuccess) e = prepare_one<CG, MM_EPI_SOFTGRAD, GEN>();
  return e;
}

// The column tile with the shortest schedule: rounds over the SMs times a tile's columns (and what a tile costs
// whatever its width, about 24 columns' time). Widths that are no multiple of 64 run at the next larger one's rate
// (4096^3, main loop alone: 256 74 us, 192 74 us, 224 100 us). Groups of a ragged reduction (0: a dense product, the only
// one whose last round is split) run on single CTAs, where a tile costs 200 columns more, the loads of its 128 lanes
// (one group, 8192 rows, 4096 x 4096: 256 columns 189 us in 4 rounds, 192 194 us in 5, 128 238 us in 7).
struct Schedule {
  int64_t cost;  // columns' time
  int bn, tail_lg, tail_from;
};
Schedule schedule(int64_t lane_tiles, int cols, bool b_red, int groups, int cg, int units) {
  Schedule best = {INT64_MAX, 256, 0, 0};
  const int grain = b_red ? 64 : 64 * cg, fixed = groups ? 200 : 24;
  for (int bn = 256; bn >= grain; bn -= grain) {
    const int64_t tiles = lane_tiles * ((cols + bn - 1) / bn) * std::max(1, groups);
    const int64_t tail = tiles % units;
    // the last, partial round of a dense product: its tiles are split while all parts still fit one round
    int lg = 0;
    while (groups == 0 && tail && lg < 2 && (tail << (lg + 1)) <= units && (bn >> (lg + 1)) % grain == 0) ++lg;
    const int64_t cost = tiles / units * (bn + fixed) + (tail ? (bn >> lg) + fixed : 0);
    if (cost < best.cost) best = {cost, bn, lg, (int)std::min<int64_t>(tiles - tail, INT32_MAX)};
  }
  return best;
}

}  // namespace

int64_t mm_cost(int lanes, int cols, int red, bool b_red) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int cg = lanes > BM && g_pairs[dev & 63] > 0 ? 2 : 1, units = std::max(1, cg == 2 ? g_pairs[dev & 63] : g_sms[dev & 63]);
  return schedule((lanes + BM * cg - 1) / (BM * cg), cols, b_red, 0, cg, units).cost * ((red + BK - 1) / BK + 4);
}

cudaError_t mm_prepare() {
  if (!g_encode) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&g_sms[dev & 63], cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = prepare_epi<1, false>();
  if (e == cudaSuccess) e = prepare_epi<2, false>();
  if (e == cudaSuccess) e = prepare_epi<1, true>();
  if (e == cudaSuccess) e = prepare_one<1, kEpiPlain, false>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiPlain, false>();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&g_pairs[dev & 63], mm_tc_kernel<2, MM_EPI_STORE, false>, &cfg);
  }
  return e;
}

cudaError_t mm_launch(const MmProblem& p, cudaStream_t s) {
  if (p.lanes <= 0 || p.cols <= 0) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = g_sms[dev & 63], pairs = g_pairs[dev & 63];
  TcArgs a = {};
  a.p = p;
  const bool gen = p.red <= 0 || !mm_aligned(p.a) || !mm_aligned(p.b);
  // Few tiles (at most one for every two SMs): the reduction of a tile is split over a cluster of CTAs, as many as keep
  // every SM busy once, with six stages each at least (1 x 4096 x 4096, 64 stages: 18.9 us alone, 10.0 in four shares;
  // 16 x 2048 x 1024, 16 stages: 7.4 alone, 6.6 in two; but 64 x 1024 x 512, 8 stages: 5.6 alone, 6.4 in two, and
  // 300 x 1000 x 576, 9 stages: 6.0 alone, 7.0 in two).
  a.split = 1;
  const int64_t lanes128 = (p.lanes + BM - 1) / BM;
  const int blocks = (p.red + BK - 1) / BK;
  const int split_bn = p.cols <= 32 && p.b.red_major ? 32 : 64;
  // tiles of that width (ragged columns: where they all fit one, each group with rows has one)
  const int64_t few = lanes128 * (p.rag == MM_RAG_COLS ? std::min(p.groups, p.cols) : (p.cols + split_bn - 1) / split_bn);
  if (p.rag != MM_RAG_RED && p.epi == MM_EPI_STORE && (p.rag == MM_DENSE || p.cols <= 64) && 2 * few <= sms)
    a.split = (int)std::max<int64_t>(1, std::min<int64_t>({sms / few, blocks / 6, split_bn == 32 ? 8 : 4}));
  // Pairs where there are at least two 128-lane tiles (a half-empty pair would double the work of a
  // narrow product) and the reduction is not ragged (a group's end has to be cleared in both CTAs).
  const int cg = !gen && p.rag != MM_RAG_RED && p.lanes > BM && pairs > 0 && a.split == 1 ? 2 : 1;
  const int units = cg == 2 ? pairs : sms;
  a.lane_tiles = (p.lanes + BM * cg - 1) / (BM * cg);
  a.bn = 256;
  if (a.split > 1) {
    a.bn = split_bn;
  } else if (p.rag == MM_RAG_COLS) {
    // the groups' sizes are only known on the device: a tile that holds twice the average (a smaller tile
    // leaves room for more stages in flight; a group beyond it takes several tiles, which share its weights in L2)
    const int64_t typical = std::min<int64_t>(2 * (((int64_t)p.cols + p.groups - 1) / p.groups), p.cols);
    while (a.bn > 64 && a.bn / 2 >= typical) a.bn /= 2;
  } else if (p.epi != MM_EPI_STATS) {
    const Schedule w = schedule(a.lane_tiles, p.cols, p.b.red_major, p.rag == MM_RAG_RED ? p.groups : 0, cg, units);
    a.bn = w.bn, a.tail_lg = w.tail_lg, a.tail_from = w.tail_from;
  }
  a.stages = 1;
  while (a.stages < kMaxStages && smem_bytes(cg, a.bn, a.stages + 1, a.split, p) <= kSmemMax) ++a.stages;
  // the rows of a copy divide what a CTA stages; large copies where the columns are not ragged (4096^3 with copies of
  // 128 rows 81.7 us, of 64 rows 83.8)
  const int staged = a.bn / cg;
  a.b_box = p.rag == MM_RAG_COLS || staged % 64 ? 32 : staged % 128 ? 64 : 128;
  a.a_blocks = !p.a.red_major && p.lanes % 64 == 0 ? 2 : 1;
  a.b_blocks = !p.b.red_major && p.cols % 64 == 0 && (staged == 256 || staged == 128) ? staged / 64 : 1;
  a.col_tiles = (p.cols + a.bn - 1) / a.bn;
  const int64_t tiles = a.lane_tiles * (int64_t)(p.rag == MM_RAG_COLS ? a.col_tiles + p.groups : a.col_tiles) * (p.rag == MM_RAG_RED ? p.groups : 1);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  if (a.tail_lg == 0) a.tail_from = (int)tiles;
  a.by_lanes = Divider(a.lane_tiles), a.by_panel = Divider(a.lane_tiles * kPanel), a.by_matrix = Divider(a.lane_tiles * a.col_tiles);
  const MmEpiArgs& ep = p.e;
  const auto by_rows = [](const void* base, int64_t ld) { return !base || ((uintptr_t)base % 16 == 0 && ld % 8 == 0); };
  a.rows_out = !ep.out_f32 && !ep.acc_in && p.lanes % 8 == 0 && ep.group_stride % 8 == 0 && by_rows(ep.out, ep.ld) &&
               by_rows(ep.residual, ep.ldr) && by_rows(ep.z, ep.ldz);
  CUtensorMap ta = {}, tb = {};
  if (!gen) {
    const uint64_t groups = p.rag == MM_RAG_COLS ? p.groups : 1;
    const uint64_t red = p.red;
    const bool ok = make_map(&ta, p.a, p.f16, p.a.red_major ? red : p.lanes, p.a.red_major ? p.lanes : red, groups, p.a.red_major ? BM : BK, a.a_blocks) &&
                    make_map(&tb, p.b, p.f16, p.b.red_major ? red : p.cols, p.b.red_major ? p.cols : red, 1, p.b.red_major ? a.b_box : BK, a.b_blocks);
    if (!ok) return cudaErrorInvalidValue;
  }
  // The tensor cores' fp32 accumulation cuts instead of rounding: a sum of positive terms loses 2^-24 of its size for every
  // step of 16 (measured: 9.7e-4 over 2^18 terms), so that no accumulator may take all of a long reduction.
  //  * Results in 16 bits: one accumulator for every 16384 terms, 6e-5 at most, an eighth of fp16's rounding; the epilogue
  //    adds them up in the other accumulator's place, which costs a long tile the overlap of the two.
  //  * Weight gradients in fp32: one for every 512 rows, added to what the tile has stored.
  //  * Losses: one for every 2048 of d (their relative error at d 4096: 9.3e-7 with one accumulator, 4.6e-7 with two; four,
  //    1.6e-7, cost the 2048-row forward 7 % for their hand-overs, two 1 %). Pairs hold the sums in registers; single
  //    CTAs, where that many registers keep the next launch from starting early (16 rows: 195 us, 174 without), use all
  //    of tensor memory for the two of a tile, and the epilogue folds the first into the second at once and hands it
  //    back. A longer d is added up as for 16 bits.
  a.seg = kSegFold;
  a.accs = 1;
  if (p.epi == MM_EPI_STATS && (cg == 2 || p.red > 2 * kSegStats))
    a.seg = kSegStats, a.fold = cg == 1;
  else if (p.epi == MM_EPI_STATS && p.red > kSegStats)
    a.seg = (p.red + 2 * BK - 1) / (2 * BK) * BK, a.accs = 2;
  else if (ep.out_f32 && !ep.acc_in && p.rag == MM_RAG_RED)
    a.seg = kSegStore;
  else
    a.fold = 1;
  if (a.split > 1) {
    const int64_t most = a.lane_tiles * (p.rag == MM_RAG_COLS ? (int64_t)std::min(p.groups, p.cols) : a.col_tiles);
    return gen ? launch_epi<1, true>(ta, tb, a, (int)most * a.split, s) : launch_epi<1, false>(ta, tb, a, (int)most * a.split, s);
  }
  const int grid = cg * (int)std::max<int64_t>(1, std::min<int64_t>(units, tiles + (tiles - (p.rag == MM_DENSE ? a.tail_from : tiles)) * ((1 << a.tail_lg) - 1)));
  if (gen) return launch_epi<1, true>(ta, tb, a, grid, s);
  return cg == 2 ? launch_epi<2, false>(ta, tb, a, grid, s) : launch_epi<1, false>(ta, tb, a, grid, s);
}

}  // namespace ds4
