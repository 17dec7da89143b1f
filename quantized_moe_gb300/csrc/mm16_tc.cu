// The 16-bit products on the 5th-generation tensor cores: out[c][l] = sum_r A(l, r) B(c, r).
//
// Persistent: one CTA (or pair of CTAs) per SM (or two SMs) loops over output tiles of 128 lanes per
// CTA x up to 256 columns (of groups around that size 512, in both accumulators). The lanes are the contiguous index of the output, so that a tensor-memory
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
// bytes, 16 loader warps (12-27) read it with ordinary loads and write the same swizzled layout.
// Few tiles share their reduction out over a cluster of CTAs, which join their sums in shared memory.
//
// The gated block is a product whose lanes are 16 gate features, the same 16 up features, and so on, so that a thread of the
// epilogue holds both factors of its results. Scores have tokens as lanes, a thread each, or, few of them, as columns.
//
// What bounds it (GB300, measured): the experts' products stream their weights (256 experts, 32768
// rows, n 2048, k 4096: 0.70-0.72 ms = 6.5-6.8 TB/s, 96-99 % of the copy bandwidth, for y and dx; the
// weight gradients, 4.3 GB of results, 0.79 ms = 5.9 TB/s: their busiest unit is shared memory, for operands and results, 72 %);
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
constexpr int kEpiPlain = 6;              // MM_EPI_STORE of 16-bit rows with nothing to add: a kernel of its own (mm_launch)
constexpr int kEpiScoreOne = 7;           // MM_EPI_SCORE where one accumulator takes a logit's whole sum
// Pairs with more to do, in kernels of their own (their branches in the common ones cost 4096^3 3 %, its gradients 5 %):
constexpr int kEpiPlainWide = 8, kEpiGluWide = 9;  // kEpiPlain, MM_EPI_GLU with tiles wider than an accumulator
constexpr int kEpiPlainRag = 10;          // kEpiPlain of a ragged reduction
constexpr int kEpiSpread = 11;            // MM_EPI_STORE of tiles whose sums are joined a share of the columns in each CTA
__host__ __device__ constexpr bool is_store(int epi) { return epi == MM_EPI_STORE || epi == kEpiSpread; }
constexpr int kEpiPlainScaled = 12;       // kEpiPlain times a number (a softmax loss's weight gradients of 256 rows, 32000 words, d 1024: 80 -> 72 us)
constexpr int kEpiPlainSoft = 13;         // MM_EPI_SOFTGRAD without labels, by rows, with no branch or label in a logit's arithmetic (726 tokens,
                                          // 114183 words, d 96, all of the gradient: 449 us by lanes, 382 by rows, 320 so)
__host__ __device__ constexpr bool is_plain(int epi) { return epi == kEpiPlain || epi == kEpiPlainScaled || epi == kEpiPlainSoft || epi == kEpiPlainWide || epi == kEpiPlainRag; }
__host__ __device__ constexpr bool is_glu(int epi) { return epi == MM_EPI_GLU || epi == kEpiGluWide; }
__host__ __device__ constexpr bool is_wide(int epi) { return epi == kEpiPlainWide || epi == kEpiGluWide; }
constexpr int kAccCols = 256;             // columns of one accumulator, the widest MMA
constexpr int kMaxSpread = 8;             // CTAs of a cluster that share out a tile's reduction and its columns
constexpr int kRagBox = 32;               // rows of a box where the columns are ragged
constexpr int kPanel = 8;                 // column tiles that a raster panel spans
constexpr int kEpiWarps = 8;              // epilogue warps: two per quadrant of tensor-memory lanes
constexpr int kFirstLoader = 4 + kEpiWarps;
// Loader warps of the unaligned form: with 16 a thread's share of a stage is small enough to be held a whole stage ahead (with 8 a
// stage's second half of B waited for its first: 1231 x 7770 x 3498 276 us, 211; 42 groups, 16356 rows, n 1696, k 3315 1880, 1378).
constexpr int kLoaders = 16;
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
  int bn, stages, b_box;      // column tile (above kAccCols: tiles that need it take both accumulators), pipeline depth, rows of a column-operand box
  int a_blocks, b_blocks;     // boxes of 64 x 64 that one copy of an MN-major operand brings
  int glu_whole;              // one copy brings a gated block's 64 gate and 64 up rows (else 16 rows each)
  int ring;                   // bytes of all stages
  int lane_tiles, col_tiles;  // of BM * CG lanes; of bn columns (without ragged columns)
  int rows_out;               // the 16-bit output (and residual, z) can be moved 8 lanes at a time
  int plain;                  // and nothing is to be added (a dense one may be scaled)
  int seg;                    // reduction that one accumulator takes before its sums are added up in fp32 (a multiple of BK)
  int accs;                   // accumulators of one tile that lie side by side in tensor memory (1: two take turns; 2: none is left to)
  int fold;                   // a tile with more reduction than seg is summed up in tensor memory (fold_acc), seg by seg
  int split;                  // CTAs (a cluster) that share a tile's reduction; 1: none
  int spread;                 // they join their sums a share of the columns each (0: all in the first one); columns of a share
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
// An arrival at a pair's leader that hands tensor memory back: no memory is passed on with it (tcgen05.wait::ld and the fence
// before it order the reads), and a release at cluster scope would wait for the warp's stores to global memory.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(addr) : "memory");
}

// One that passes on what the warp has written, or seen arrive, in its own CTA's shared memory, and the other side of it, of a phase
// that is known to be complete: ordered at cluster scope, since MMAs that the leader issues read that memory, but for shared memory
// alone (a release of everything waits for the epilogue's stores: 64 groups around 256 rows, 4096 x 4096 480 us so, 531).
__device__ __forceinline__ void mbar_arrive_leader(uint32_t addr) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mbar_acquire_pair(uint64_t* b, uint32_t parity) {
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%0], %1;\n}\n"
      "fence.acquire.sync_restrict::shared::cluster.cluster;\n" ::"r"(su32(b)), "r"(parity)
      : "memory");
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

template <int CG>
__device__ __forceinline__ void tma_load5(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int u, int g, uint32_t bar) {
  if (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5, %6}], [%7];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(g), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(g), "r"(bar)
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
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, v); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  tmem_get16(taddr, r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// The columns of the widest tile where tiles may take both accumulators, from the sizes that the groups have: a multiple of 64
// above kAccCols, up to a.bn, if one tile for each group of so many rows takes less time than tiles of kAccCols, else
// kAccCols. A wide tile passes over its group's weights once, but nothing overlaps the storing of its results. Time is estimated
// as the rounds of an average tile and what the largest takes longer, in cycles fitted to 465 shapes of 16 to 128 groups of 171 to
// 448 rows on average: a step of 64 loads 256 lanes and n columns in 1.1 cycles each, or multiplies them in 2 n (tiles of kAccCols
// first: 64 groups of 264, 2048 x 4096 346 us, 223; 64 of 0 to 600, 2048 x 768 63, 76). The choice costs 0.2 % on average, wide
// tiles throughout 2 % for products and 4 % for blocks, none 6 % and 5 %. Both CTAs of a pair come to the same.
template <bool GLU>
__device__ __forceinline__ int widest_tile(const TcArgs& a, const int* lo_of, int units, int lane) {
  int most = 0;
#pragma unroll 1
  for (int g = lane; g < a.p.groups; g += 32) {
    const int n = lo_of[g + 1] - lo_of[g];
    if (n <= a.bn) most = max(most, n);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (most <= kAccCols) return kAccCols;
  const float blocks = (float)((a.p.red + BK - 1) / BK), store = GLU ? 18.f : 6.f;  // (cycles of a column's results)
  const auto main_loop = [&](float n) { return blocks * fmaxf(1.1f * (2 * BM + n), 2.f * n); };
  const auto cost = [&](int n) -> unsigned { return n ? (unsigned)(fmaxf(main_loop((float)n), store * (float)n) + 3000.f) : 0u; };
  const unsigned of_full = cost(kAccCols);
  unsigned sum[2] = {}, largest[2] = {}, tiles[2] = {};
#pragma unroll 1
  for (int g = lane; g < a.p.groups; g += 32) {
    const unsigned n = (unsigned)max(lo_of[g + 1] - lo_of[g], 0), full = n / kAccCols, rest = n % kAccCols;
    const unsigned of_rest = cost((int)rest), narrow = full * of_full + of_rest, top = full ? of_full : of_rest, count = full + (rest > 0);
    const bool one = n > kAccCols && n <= a.bn;
    const unsigned wide = (unsigned)(main_loop((float)n) + store * (float)n + (GLU ? 3000.f : 4500.f));
    sum[0] += narrow, tiles[0] += count, largest[0] = max(largest[0], top);
    sum[1] += one ? wide : narrow, tiles[1] += one ? 1 : count, largest[1] = max(largest[1], one ? wide : top);
  }
  float time[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float count = (float)__reduce_add_sync(0xffffffffu, tiles[i]), mean = __fdividef((float)__reduce_add_sync(0xffffffffu, sum[i]), count);
    const float rounds = ceilf(__fdividef((float)a.lane_tiles * count, (float)units) - 1e-3f);
    time[i] = (rounds - 1.f) * mean + (float)__reduce_max_sync(0xffffffffu, largest[i]);
  }
  return (GLU ? 1.03f : 1.06f) * time[1] < time[0] ? (most + 63) / 64 * 64 : kAccCols;
}

// One output tile.
struct Tile {
  int g, l0, c0, n, r0, red;  // group, first lane of the CTA (pair), first column, columns, first of the reduction, its length
};

// Tables in shared memory: lo[g], g = 0..groups, the first row of each group, clamped to the matrix (a group
// ends where the next one begins, or is empty if that lies before it); for ragged columns pref[g], the running
// count of the groups' column tiles.
// WIDE: a group of at most `widest` rows has one tile, which beyond kAccCols takes both accumulators; a larger one has tiles of
// kAccCols, whose accumulators take turns (64 groups of 20 and 400 rows in turn, 2048 x 4096: 231 us, in tiles of 320 and 80
// columns 300).
template <int CG, bool WIDE>
__device__ __forceinline__ Tile tile_of(const TcArgs& a, const int* lo_of, const int* pref, int widest, int t, int share) {
  const MmProblem& p = a.p;
  Tile o;
  int col_tiles = a.col_tiles, c_lo = 0, c_n = p.cols, part = 0, pitch = a.bn, width = a.bn;
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
    if (WIDE && c_n > widest) pitch = width = kAccCols;
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
  o.c0 = c_lo + ct * pitch + part * width;
  o.n = min(width, c_n - ct * pitch - part * width);  // (a part past the last column has none)
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
// each, where a tile has two or three stages: 910 -> 857 us with this and the cleaner's stores unrolled). The unaligned form
// does without: its threads have 72 registers, and the seven that a Walk holds spilled (2048 x 4096 x 513: 48 us, 46).
template <int CG, bool WIDE>
struct Walk {
  Tile mine;
  int i = 31;
  __device__ __forceinline__ Tile next(const TcArgs& a, const int* lo_of, const int* pref, int widest, int t, int step, int tiles, int share, int lane) {
    if (++i == 32) {
      i = 0;
      mine = tile_of<CG, WIDE>(a, lo_of, pref, widest, min(t + lane * step, tiles - 1), share);
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
// way round, in boxes of 64 x 64. A thread owns one 16-byte chunk of every 64th row, so that neither its chunk nor the
// parity of its addresses changes: it reads the aligned words that hold its eight elements and, where the row starts in
// the middle of a word, shifts them by an element. Elements outside the matrix are zeros; their words are not read.
struct Loader {
  const uint16_t* src;  // of the thread's chunk in its first row
  int64_t step;         // elements to the chunk 64 rows on
  int odd, red_major, row, ch;
  int mn_left, r_left;  // lanes or columns, and reduction, from the thread's first element to their ends
  int pitch;            // lanes or columns from one of the thread's rows to the next (K-major)
  __device__ __forceinline__ void start(const uint16_t* base, int64_t ld, int red, int mn0, int mn_end, int r0, int r_end, int tid) {
    red_major = red;
    row = tid >> 3, ch = tid & 7, pitch = 64;
    const int mn = red ? mn0 + row : mn0 + ch * 8, r = red ? r0 + ch * 8 : r0 + row;
    src = base + (red ? (int64_t)mn * ld + r : (int64_t)r * ld + mn);
    step = red ? 64 * ld : 64;
    odd = (int)(reinterpret_cast<uintptr_t>(src) >> 1) & 1;
    mn_left = mn_end - mn, r_left = r_end - r;
  }
  // The gated block's weights, `up` elements from a gate row to its up row: 16 gate rows, then the same 16 up rows.
  __device__ __forceinline__ void start_glu(const uint16_t* base, int64_t ld, int64_t up, int f0, int f_end, int r0, int r_end, int tid) {
    start(base, ld, 1, f0 + ((tid >> 4 & 16) | (tid >> 3 & 15)), f_end, r0, r_end, tid & 7);
    row = tid >> 3, pitch = 32;
    if (row & 16) src += up;
    step = 32 * ld;
    odd = (int)(reinterpret_cast<uintptr_t>(src) >> 1) & 1;
  }
  __device__ __forceinline__ int valid(int u) const {
    if (red_major) return mn_left > pitch * u ? min(8, r_left) : 0;
    return r_left > 0 ? min(8, mn_left - 64 * u) : 0;
  }
  // The words of the thread's chunks of the current stage, up to the operand's row `rows`, and their way into the stage: other
  // work goes in between, while they are in flight.
  template <int N>
  __device__ __forceinline__ void load(int rows, uint32_t (&w)[N][5]) const {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(src - odd);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int v = 64 * u < rows ? valid(u) : 0;
      const uint32_t* qu = q + u * step / 2;
      if (v >= 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[u][k] = qu[k];
        w[u][4] = odd ? qu[4] : 0u;
      } else {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[u][k] = v > 0 && 2 * k < v + odd ? qu[k] : 0u;  // (a word with a wanted element)
      }
    }
  }
  template <int N>
  __device__ __forceinline__ void put(uint8_t* dst, int rows, const uint32_t (&w)[N][5]) const {
    const uint32_t sh = odd * 16;
    uint8_t* to = dst + row * 128 + ((ch ^ (row & 7)) << 4);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (64 * u + (red_major ? row : 0) >= rows) break;
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = __funnelshift_r(w[u][k], w[u][k + 1], sh);
      const int v = valid(u);
      if (v < 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = v - 2 * k < 1 ? 0u : v - 2 * k < 2 ? r[k] & 0xffffu : r[k];
      }
      *reinterpret_cast<uint4*>(to + u * 8192) = make_uint4(r[0], r[1], r[2], r[3]);
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

// N elements of one lane, nv of them there, `ld` apart: the type is chosen once for all of them.
template <int N>
__device__ __forceinline__ void to16(const float (&v)[N], uint16_t (&h)[N], int f16) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
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
template <class T, int N>
__device__ __forceinline__ void store_col(T* q, int64_t ld, int nv, const T (&h)[N]) {
  if (nv >= N) {
#pragma unroll
    for (int j = 0; j < N; ++j, q += ld) *q = h[j];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j, q += ld)
      if (j < nv) *q = h[j];
  }
}
template <class T, int N>
__device__ __forceinline__ void load_col(const T* q, int64_t ld, int nv, T (&h)[N]) {
  if (nv >= N) {
#pragma unroll
    for (int j = 0; j < N; ++j, q += ld) h[j] = *q;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j, q += ld) h[j] = j < nv ? *q : T(0);
  }
}
template <int N>
__device__ __forceinline__ void add16(float (&v)[N], const void* base, int64_t at, int64_t ld, int nv, int f16) {
  uint16_t h[N];
  load_col(static_cast<const uint16_t*>(base) + at, ld, nv, h);
  if (f16) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += __half2float(__ushort_as_half(h[j]));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += __uint_as_float((uint32_t)h[j] << 16);
  }
}
template <int N>
__device__ __forceinline__ void add32(float (&v)[N], const float* q, int64_t ld, int nv) {
  float h[N];
  load_col(q, ld, nv, h);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] += h[j];
}

// Writes N columns (nv exist for this lane) of lane l.
template <int N>
__device__ __forceinline__ void put(const MmProblem& p, int g, int l, int c, int nv, const float (&v)[N]) {
  const MmEpiArgs& e = p.e;
  if (l >= p.lanes) return;
  const int64_t o = (p.rag == MM_RAG_RED ? g * e.group_stride : 0) + (int64_t)c * e.ld + l;
  if (e.out_f32) {
    store_col(static_cast<float*>(e.out) + o, e.ld, nv, v);
  } else {
    uint16_t h[N];
    to16(v, h, p.f16);
    store_col(static_cast<uint16_t*>(e.out) + o, e.ld, nv, h);
  }
}

// What `out` holds of N columns (nv exist) of lane l.
template <int N>
__device__ __forceinline__ void epi_fetch(const MmProblem& p, int g, int l, int c, int nv, uint32_t (&w)[N]) {
  const MmEpiArgs& e = p.e;
  if (l >= p.lanes) nv = 0;
  const int64_t at = (p.rag == MM_RAG_RED ? g * e.group_stride : 0) + (int64_t)c * e.ld + l;
  if (e.out_f32) {
    load_col(static_cast<const uint32_t*>(e.out) + at, e.ld, nv, w);
  } else {
    uint16_t h[N];
    load_col(static_cast<const uint16_t*>(e.out) + at, e.ld, nv, h);
#pragma unroll
    for (int j = 0; j < N; ++j) w[j] = h[j];
  }
}

// The arithmetic of a stored result: N columns (nv exist for this lane) of lane l.
template <int N>
__device__ __forceinline__ void epi_store(const MmProblem& p, int g, int l, int c, int nv, bool accumulate, float (&v)[N]) {
  const MmEpiArgs& e = p.e;
  if (l >= p.lanes) nv = 0;
  if (e.acc_in) add32(v, e.acc_in + (int64_t)c * e.acc_ld + l, e.acc_ld, nv);
  if (e.scale) {
    const float s = *e.scale;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= s;
  }
  if (e.bias) {
    const float b = nv ? ld16(e.bias, l, p.f16) : 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += b;
  }
  if (e.z) {
    uint16_t h[N];
    to16(v, h, p.f16);
    store_col(static_cast<uint16_t*>(e.z) + (int64_t)c * e.ldz + l, e.ldz, nv, h);
  }
  if (e.act == MM_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = mm_silu(v[j]);
  } else if (e.act == MM_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = mm_gelu(v[j]);
  } else if (e.act == MM_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = mm_relu(v[j]);
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

// The gated block: lanes l of a group of 32 hold 16 features' gates, then their ups; 32 columns, nv exist.
__device__ __forceinline__ void glu_out(const MmProblem& p, int l, int c, int nv, float (&v)[32]) {
  const MmEpiArgs& e = p.e;
  const int f = (l >> 5) * 16 + (l & 15), is_up = (l >> 4) & 1;
  if (f >= p.lanes) nv = 0;
  uint16_t h[32];
  if (e.z) {
    to16(v, h, p.f16);
    store_col(static_cast<uint16_t*>(e.z) + (int64_t)c * e.ldz + (is_up ? p.lanes : 0) + f, e.ldz, nv, h);
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = mm_act(v[j], e.act) * __shfl_xor_sync(0xffffffffu, v[j], 16);
  to16(v, h, p.f16);
  store_col(static_cast<uint16_t*>(e.out) + (int64_t)c * e.ld + f, e.ld, is_up ? 0 : nv, h);
}

// ---- 16-bit results by rows: the warps hold 32 lanes x 32 columns as fragments (a thread: lanes i/4 + 8 r, columns
// 8 j + 2 (i % 4) and the next), which stmatrix writes transposed into shared memory, from where whole rows of 128
// lanes leave as 16-byte stores.
template <int J>
struct FragOf {
  float v[J][4][2];  // [block of 8 columns][block of 8 lanes][column parity]
};
using Frag = FragOf<4>;
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, FragOf<2>& f) {  // (16 columns)
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) f.v[(i >> 2) & 1][2 * (i >> 3) + ((i >> 1) & 1)][i & 1] = __uint_as_float(r[i]);
}
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
template <int J>
__device__ __forceinline__ void frag_out(uint32_t stage, int quad, int lane, const FragOf<J>& f, int f16, int j0 = 0) {
#pragma unroll
  for (int j = 0; j < J; ++j)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(frag_addr(stage, quad, j0 + j, lane)),
                 "r"(pack16(f.v[j][0][0], f.v[j][0][1], f16)), "r"(pack16(f.v[j][1][0], f.v[j][1][1], f16)),
                 "r"(pack16(f.v[j][2][0], f.v[j][2][1], f16)), "r"(pack16(f.v[j][3][0], f.v[j][3][1], f16))
                 : "memory");
}
// The gated block's fragments: the warp's lanes are 16 features' gates and their ups, so that a thread holds both factors of
// its results. z: a staged row is the tile's 64 gates and then their 64 ups; h: its 64 features.
__device__ __forceinline__ void glu_frag_out(uint32_t stage, int quad, int lane, const Frag& f, int f16) {
  const uint32_t at = stage + (uint32_t)((lane & 7) * kRowBytes + (lane >> 4) * 128 + quad * 32 + ((lane >> 3) & 1) * 16);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(at + 8 * j * kRowBytes),
                 "r"(pack16(f.v[j][0][0], f.v[j][0][1], f16)), "r"(pack16(f.v[j][1][0], f.v[j][1][1], f16)),
                 "r"(pack16(f.v[j][2][0], f.v[j][2][1], f16)), "r"(pack16(f.v[j][3][0], f.v[j][3][1], f16))
                 : "memory");
}
__device__ __forceinline__ void glu_frag_act(Frag& f, int act) {
  const auto each = [&](auto fn) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 2; ++q) f.v[j][r][q] = fn(f.v[j][r][q]) * f.v[j][r + 2][q];
  };
  if (act == MM_ACT_SILU)
    each([](float v) { return mm_silu(v); });
  else if (act == MM_ACT_GELU)
    each([](float v) { return mm_gelu(v); });
  else if (act == MM_ACT_RELU)
    each([](float v) { return mm_relu(v); });
  else
    each([](float v) { return v; });
}
__device__ __forceinline__ void glu_frag_out_h(uint32_t stage, int quad, int lane, const Frag& f, int f16) {
  const uint32_t at = stage + (uint32_t)((8 * (lane >> 4) + (lane & 7)) * kRowBytes + quad * 32 + ((lane >> 3) & 1) * 16);
#pragma unroll
  for (int j = 0; j < 4; j += 2)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(at + 8 * j * kRowBytes),
                 "r"(pack16(f.v[j][0][0], f.v[j][0][1], f16)), "r"(pack16(f.v[j][1][0], f.v[j][1][1], f16)),
                 "r"(pack16(f.v[j + 1][0][0], f.v[j + 1][0][1], f16)), "r"(pack16(f.v[j + 1][1][0], f.v[j + 1][1][1], f16))
                 : "memory");
}
template <int J>
__device__ __forceinline__ void frag_add(uint32_t stage, int quad, int lane, FragOf<J>& f, int f16, int j0) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    uint32_t r[4];
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(frag_addr(stage, quad, j0 + j, lane))
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

// The same for scores: c = log2(e) / T, u the running sum of (z - m) exp((z - m) / T), from which the entropy comes
// without the cancellation that a sum of p z would have.
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(v));
  return r;
}
// Words from nv on are made -inf: they add nothing, and no word's arithmetic hangs on a branch (written with a condition for
// each word the chunk ran one word after the other, 4.5 thousand cycles where this takes one). Returns the chunk's largest.
// It and the running maximum m, which starts as NaN, are NaN as long as there is no number: the search for the best words
// may not take such tiles and chunks for closed words (-inf), which are listed after the open ones.
template <bool ENT>
__device__ __forceinline__ float epi_score(float (&v)[32], int nv, float c, float& m, float& s, float& u) {
  if (nv < 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = j < nv ? v[j] : -INFINITY;
  }
  float q[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int j = 4; j < 32; ++j) q[j & 3] = fmaxf(q[j & 3], v[j]);
  const float chunk = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3])), top = fmaxf(m, chunk);
  if (!(top > -INFINITY)) {  // only words of probability zero so far, or that are NaN (which still reach the sum)
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 32; ++j) bad |= v[j] != v[j];
    if (bad) s = NAN;
    m = top;
    return chunk;
  }
  const float d = fmaxf(m - top, -1e30f), r = exp2_fast(d * c);  // (m = -inf or NaN: s and u are 0, or NaN)
  float t[4] = {s * r, 0.f, 0.f, 0.f}, w[4] = {(u + d * s) * r, 0.f, 0.f, 0.f};
  m = top;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float dj = v[j] - top, e = exp2_fast(dj * c);
    t[j & 3] += e;
    if (ENT) w[j & 3] += fmaxf(dj, -1e30f) * e;  // (words of probability zero add nothing)
  }
  s = (t[0] + t[1]) + (t[2] + t[3]);
  if (ENT) u = (w[0] + w[1]) + (w[2] + w[3]);
  return chunk;
}

// The listed words of one of few tokens in ascending order, from a sorted list or, of up to kMmDirect words, straight from
// the caller's (the next one is looked for among them).
struct Wanted {
  int next = INT32_MAX, at = 0;  // the word, its place (in the sorted or in the caller's list)
  __device__ __forceinline__ void look(const MmEpiArgs& e, const int* words, int word, int place) {  // the first behind (word, place)
    next = INT32_MAX;
    for (int i = 0; i < e.n_want; ++i) {
      const int w = words[i];
      if (w < e.vocab && (w > word || (w == word && i > place)) && w < next) next = w, at = i;
    }
  }
  __device__ __forceinline__ void start(const MmEpiArgs& e, int64_t t, int tile, int tiles, int w0) {
    if (e.words) return look(e, e.words + t * e.n_want, w0 - 1, INT32_MAX);
    at = *(e.first + t * tiles + tile);
    if (at < e.n_want) next = e.want[t * e.n_want + at].x;
  }
  // Stores the logits of those among the nv words from w0 on and passes over earlier ones.
  __device__ __forceinline__ void take(const MmEpiArgs& e, const float (&v)[32], int w0, int nv, int64_t t) {
    while (next < w0 + nv) {
      if (next >= w0) {
        float own = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == next - w0) own = v[j];
        e.zwant[t * e.n_want + (e.words ? at : e.want[t * e.n_want + at].y)] = own;
      }
      if (e.words)
        look(e, e.words + t * e.n_want, next, at);
      else
        next = ++at < e.n_want ? e.want[t * e.n_want + at].x : INT32_MAX;
    }
  }
};

// One chunk of few tokens' scores: thread's token t of `tokens`, 32 words from w0 (nv exist).
__device__ __forceinline__ void score_few(const MmEpiArgs& e, float (&v)[32], int w0, int nv, int t, int tokens, int tiles, float& m,
                                          float& s, float& u) {
  const int64_t tile = w0 / kMmStatChunk;
  Wanted wanted;
  if (e.n_want > 0) wanted.start(e, t, (int)tile, tiles, w0);
  const float most = epi_score<true>(v, nv, e.inv_t * 1.4426950408889634f, m, s, u);
  if (e.logits) {
    store_col(e.logits + (int64_t)w0 * tokens + t, tokens, nv, v);
    e.chunk_max[tile * tokens + t] = most;
  }
  wanted.take(e, v, w0, nv, t);
}

template <int CG, int EPI, bool GEN>
__global__ void __launch_bounds__(GEN ? kThreads + 32 * kLoaders : kThreads, 1)
    mm_tc_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                 const __grid_constant__ TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const MmProblem& p = a.p;
  // the stages start on a 1024-byte boundary (the swizzle's period); in a pair both CTAs have the same layout
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  int stages = a.stages, stage_bytes = A_BYTES + a.bn / CG * BK * 2;
  uint8_t* out_stage = smem + a.ring;  // [2][kOutBytes]
  float* parts = reinterpret_cast<float*>(out_stage + 2 * kOutBytes);  // [split - 1][bn][kPartLd], in the cluster's first CTA
  uint8_t* ctrl = out_stage + 2 * kOutBytes + (a.spread ? 0 : (a.split - 1) * a.bn * kPartLd * 4);
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* clean = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(clean + kMaxStages);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* widest_slot = reinterpret_cast<int*>(tmem_slot + 2);
  int* lo_of = reinterpret_cast<int*>(tmem_slot + 4);
  int* pref = lo_of + p.groups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
  const int acc_stride = min(max(a.bn, 32), kAccCols);
  // Tiles wider than an accumulator: their columns run on into the other one, so that one pass over A serves up to 512.
  constexpr bool kWide = is_wide(EPI);
  uint32_t tmem_cols = 32;
  while (tmem_cols < 2u * acc_stride) tmem_cols *= 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < (kWide ? kMaxStages : a.stages); ++i) {
      mbar_init(full + i, GEN ? kLoaders : 1);
      mbar_init(empty + i, !GEN && p.rag == MM_RAG_RED && rank == 0 ? 2 : 1);  // the MMAs' commit, and the cleaner
      mbar_init(clean + i, CG);
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
  // (The scores' join has a block or a warp for each row: started early, its blocks would all settle on the SMs that the
  // product leaves first and wait there. 2048 rows, a block for eight rows: 1340 us instead of 345.)
  if (EPI != MM_EPI_SCORE && EPI != kEpiScoreOne && EPI != MM_EPI_SCORE_FEW) let_next_start();
  if (p.rag != MM_DENSE) {
    const int total = p.rag == MM_RAG_COLS ? p.cols : p.red;
    for (int g = threadIdx.x; g <= p.groups; g += blockDim.x) lo_of[g] = min(max(*(p.offsets + g), 0), total);
    __syncthreads();
    if (p.rag == MM_RAG_COLS && warp == 2) {
      int run = 0, most = a.bn;
      if (kWide) {
        most = widest_tile<is_glu(EPI)>(a, lo_of, gridDim.x / CG, lane);
        if (lane == 0) *widest_slot = most;
      }
      for (int g0 = 0; g0 <= p.groups; g0 += 32) {
        const int g = g0 + lane;
        const int rows = g < p.groups ? max(lo_of[g + 1] - lo_of[g], 0) : 0;
        const int n = kWide ? rows > most ? (rows + kAccCols - 1) / kAccCols : rows > 0 : (rows + a.bn - 1) / a.bn;
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
  const int widest = kWide ? *widest_slot : a.bn;
  if (kWide) {  // the ring has as many stages as these tiles leave room for
    stage_bytes = A_BYTES + widest / CG * BK * 2;
    stages = min(kMaxStages, a.ring / stage_bytes);
  }
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
    const int a_boxes = is_glu(EPI) ? (a.glu_whole ? 1 : BM / 16) : a_red ? 1 : 2 / a.a_blocks;
    Walk<CG, kWide> walk;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile o = walk.next(a, lo_of, pref, widest, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const bool wide = kWide && o.n > kAccCols;
      const int nb = mma_n<CG>(p, wide ? o.n - kAccCols : o.n) / CG;  // columns that this CTA stages (of the second part)
      const int b_boxes = kWide ? (wide ? kAccCols / CG / kRagBox : 0) + (nb + kRagBox - 1) / kRagBox :
                          b_red ? (nb + a.b_box - 1) / a.b_box : (nb / 64 + a.b_blocks - 1) / a.b_blocks;
      const int b_box_bytes = kWide ? kRagBox * 128 : b_red ? a.b_box * 128 : a.b_blocks * 8192;
      const uint32_t bytes = A_BYTES + b_boxes * b_box_bytes;
      const int la = o.l0 + BM * rank, cb = o.c0 + nb * rank;
      // The lane's box: of a wide tile the first part's columns, split between the CTAs, and then the second's. (Worked out for
      // every stage it slowed narrow tiles too: 16 groups of 200 rows, 2048 x 768 15.4 us, 14.1.)
      int y_wide = cb + lane * kRagBox;
      if (kWide && wide) y_wide += lane < kAccCols / CG / kRagBox ? (kAccCols / CG - nb) * (int)rank : kAccCols - kAccCols / CG;
      const int ga = p.rag == MM_RAG_COLS ? o.g : 0;
      for (int k = 0; k < o.red; k += BK) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + s, ph ^ 1, abort_flag, p.err, 1));
        if (!ok) break;
        const bool own = EPI == kEpiPlainRag && o.red - k < BK && ((o.red - k) & 15);
        const auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z, int g, uint32_t bar) {
          if (own)  // the copies of a pair's ragged end report to their own CTA's barrier, for its cleaner
            tma_load<1>(dst, map, x, y, z, g, bar);
          else
            tma_load<CG>(dst, map, x, y, z, g, bar);
        };
        const uint32_t st = su32(smem + s * stage_bytes), bar = CG == 2 && !own ? mapa(su32(full + s), 0) : su32(full + s);
        const int r = o.r0 + k;
        if (of_a) {
          if (lane == 0 && (rank == 0 || own)) mbar_expect_tx(full + s, CG == 2 && !own ? 2 * bytes : bytes);  // (copies may report before it)
          if (lane < a_boxes) {
            if (is_glu(EPI) && a.glu_whole)  // 16 rows of the gate, the same 16 of up, and so on
              tma_load5<CG>(st, &ta, r, 0, 0, la / 32, ga, bar);
            else if (is_glu(EPI))
              tma_load<CG>(st + lane * 2048, &ta, r, la / 2 + 16 * (lane >> 1) + (lane & 1 ? p.lanes : 0), 0, ga, bar);
            else if (a_red)
              tma_load<CG>(st, &ta, r, la, 0, ga, bar);
            else if (a.a_blocks > 1)
              load(st, &ta, 0, r, la / 64, ga, bar);
            else
              load(st + lane * 8192, &ta, la + 64 * lane, r, 0, ga, bar);
          }
        } else if (lane < b_boxes) {
          const uint32_t to = st + A_BYTES + lane * b_box_bytes;
          if (kWide)
            tma_load<CG>(to, &tb, r, y_wide, 0, 0, bar);
          else if (b_red)
            tma_load<CG>(to, &tb, r, cb + lane * a.b_box, 0, 0, bar);
          else if (a.b_blocks > 1)
            load(to, &tb, 0, r, cb / 64 + lane * a.b_blocks, 0, bar);
          else
            load(to, &tb, cb + 64 * lane, r, 0, 0, bar);
        }
        if (++s == stages) s = 0, ph ^= 1;
      }
    }
  } else if (GEN && warp >= kFirstLoader) {
    // ------------------------------------------------------------------ loaders (any alignment)
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int tid = threadIdx.x - kThreads;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile o = tile_of<CG, kWide>(a, lo_of, pref, widest, t, part);
      if (o.n <= 0) continue;
      const uint16_t* pa = static_cast<const uint16_t*>(p.a.p) + (p.rag == MM_RAG_COLS ? o.g * p.a.group_stride : 0);
      const int nb = mma_n<CG>(p, o.n);
      Loader la, lb;
      if (is_glu(EPI))
        la.start_glu(pa, p.a.ld, p.lanes * p.a.ld, o.l0 / 2, p.lanes, o.r0, o.r0 + o.red, tid);
      else
        la.start(pa, p.a.ld, p.a.red_major, o.l0, p.lanes, o.r0, o.r0 + o.red, tid);
      lb.start(static_cast<const uint16_t*>(p.b.p), p.b.ld, p.b.red_major, o.c0, o.c0 + o.n, o.r0, o.r0 + o.red, tid);
      const int b_rows = (nb + 31) / 32 * 32;  // (a stage has room for whole 32s)
      uint32_t wa[BM / 64][5], wb[kAccCols / 64][5];  // a stage ahead
      if (o.red > 0) {
        la.load(BM, wa);
        lb.load(b_rows, wb);
      }
      for (int k = 0; k < o.red; k += BK) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + s, ph ^ 1, abort_flag, p.err, 1));
        if (!ok) break;
        uint8_t* st = smem + s * stage_bytes;
        la.put(st, BM, wa);
        la.next_stage(p.a.red_major ? BK : BK * p.a.ld);
        if (k + BK < o.red) la.load(BM, wa);
        lb.put(st + A_BYTES, b_rows, wb);
        lb.next_stage(p.b.red_major ? BK : BK * p.b.ld);
        if (k + BK < o.red) lb.load(b_rows, wb);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full + s);
        if (++s == stages) s = 0, ph ^= 1;
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
        const Tile o = tile_of<CG, kWide>(a, lo_of, pref, widest, t, part);
        if (o.red <= 0 || o.n <= 0) continue;  // an empty sum: the epilogue writes zeros without an accumulator
        const bool wide = kWide && o.n > kAccCols;
        const int n = wide ? kAccCols : mma_n<CG>(p, o.n);
        const uint32_t idesc = (1u << 4) | type << 7 | type << 10 | (p.a.red_major ? 0u : 1u << 15) |
                               (p.b.red_major ? 0u : 1u << 16) | (uint32_t)(n >> 3) << 17 | (uint32_t)(BM * CG >> 4) << 24;
        // Accumulators take turns from tile to tile (or, of a result added up in memory, from seg to seg). A tile that is
        // summed up in tensor memory stays with its own one, seg after seg, and so does the tile after it: the other
        // one holds the sum, which the epilogue is done with when it hands the last seg's accumulator back.
        const bool folds = a.fold && o.red > a.seg;
        const uint32_t idesc_rest = wide ? (idesc & ~(0x3fu << 17)) | (uint32_t)(mma_n<CG>(p, o.n - kAccCols) >> 3) << 17 : 0u;
        uint32_t d = 0;
        int in_seg = 0;  // reduction already in this accumulator
        for (int k = 0; k < o.red; k += BK) {
          if (in_seg == 0) {
            const int b = wide ? 0 : a.accs == 1 || k == 0 ? buf : 1;  // (1: the second accumulator of the same tile)
            if (!mbar_wait(acc_empty + b, (used >> b & 1) ^ 1, abort_flag, p.err, 6) ||
                (kWide && wide && !mbar_wait(acc_empty + 1, (used >> 1 & 1) ^ 1, abort_flag, p.err, 6))) {
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
          if (CG == 2 && p.rag == MM_RAG_RED && (left & 15)) mbar_acquire_pair(clean + s, cleaned >> s & 1);
          if (left & 15) cleaned ^= 1u << s;
          tc_fence_after();
          const uint64_t da = a_desc + (uint32_t)(s * stage_bytes >> 4), db = b_desc + (uint32_t)(s * stage_bytes >> 4);
          if (kWide && wide) {
            const uint64_t rest = db + (kAccCols / CG * BK * 2 >> 4);
            for (int i = 0; 16 * i < left; ++i) {
              mma<CG>(d, da + i * a_step, db + i * b_step, idesc, in_seg | i);
              mma<CG>(d + kAccCols, da + i * a_step, rest + i * b_step, idesc_rest, in_seg | i);
            }
          } else if (left > 48) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma<CG>(d, da + i * a_step, db + i * b_step, idesc, in_seg | i);
          } else {
            for (int i = 0; 16 * i < left; ++i) mma<CG>(d, da + i * a_step, db + i * b_step, idesc, in_seg | i);
          }
          commit<CG>(empty + s);
          if (++s == stages) s = 0, ph ^= 1;
          in_seg += BK;
          if (in_seg == a.seg || k + BK >= o.red) {
            if (kWide && wide) {  // (its reduction fits one accumulator: mm_launch)
              commit<CG>(acc_full);
              commit<CG>(acc_full + 1);
              used ^= 3u;
            } else if (a.accs == 1) {
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
    // The warp passes every stage in turn and arrives on its empty barrier too, so that the ring cannot lap it. In a pair
    // the other CTA's full barriers see ragged ends alone, and its cleaner waits for nothing else: neither can lap the other.
    // The MMA waits for both cleaners (64 groups around 256 rows, 4096 x 4096: 564 us on single CTAs, 480 on pairs).
    int s = 0;
    uint32_t ph = 0, cleaned = 0;
    bool ok = true;
    Walk<CG, kWide> walk;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile o = walk.next(a, lo_of, pref, widest, t, step, tiles, part, lane);
      for (int k = 0; k < o.red; k += BK) {
        const int left = min(BK, o.red - k);
        if (CG == 2 && rank && !(left & 15)) {
          if (++s == stages) s = 0;
          continue;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(full + s, CG == 2 && rank ? cleaned >> s & 1 : ph, abort_flag, p.err, 2));
        if (!ok) break;
        cleaned ^= 1u << s;
        if (left & 15) {
          const int boxes = 2 + mma_n<CG>(p, o.n) / CG / 64, from = left + (lane >> 3), end = (left + 15) & ~15;
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
          if (CG == 2 && rank) {
            mbar_arrive_leader(mapa(su32(clean + s), 0));
          } else {
            if (left & 15) mbar_arrive(clean + s);
            mbar_arrive(empty + s);
          }
        }
        if (++s == stages) s = 0, ph ^= 1;
      }
    }
  } else if (is_plain(EPI) && warp >= 4 && warp < kFirstLoader) {
    // ------------------------------------------------------------------ epilogue without anything to add
    const int quad = warp & 3, half = (warp - 4) >> 2, piece = threadIdx.x & 15, row = (threadIdx.x & 127) >> 4;
    const uint32_t stage = su32(out_stage) + half * kOutBytes, from = stage + (uint32_t)(row * kRowBytes + piece * 16);
    const int64_t ld = p.e.ld;
    int buf = 0;
    uint32_t used = 0;  // as the MMA counts them
    Walk<CG, kWide> walk;
    for (int t = first; t < tiles; t += step) {
      const Tile o = GEN ? tile_of<CG, kWide>(a, lo_of, pref, widest, t, part) : walk.next(a, lo_of, pref, widest, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const bool sum = o.red > 0;
      const int l = o.l0 + BM * rank + 8 * piece;
      const bool wide = kWide && o.n > kAccCols;
      uint32_t taddr = tmem + (uint32_t)(wide ? 0 : buf * acc_stride) + ((uint32_t)(32 * quad) << 16);
      int left = l < p.lanes ? o.n - 32 * half - row : 0;  // rows from the thread's first to the tile's end
      uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.e.out) + (p.rag == MM_RAG_RED ? o.g * p.e.group_stride : 0) +
                                          (o.c0 + 32 * half + row) * ld + l);
      const bool folds = a.fold && o.red > a.seg;
      const uint32_t held = tmem + (uint32_t)((buf ^ 1) * acc_stride) + ((uint32_t)(32 * quad) << 16);
      float lse[4], gw[4];  // of the fragments' lanes
      if (EPI == kEpiPlainSoft) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int token = o.l0 + BM * rank + 32 * quad + (lane >> 2) + 8 * r;
          const bool there = token < p.lanes;
          lse[r] = there ? *(p.e.lse + token) : 0.f;
          gw[r] = there ? *(p.e.g + token) / *p.e.gscale * kMmGradOne : 0.f;
        }
      }
      bool ok = true;
      if (kWide && wide && sum) {
        ok = mbar_wait(acc_full, used & 1, abort_flag, p.err, 5) && mbar_wait(acc_full + 1, used >> 1 & 1, abort_flag, p.err, 5);
        __syncwarp();
        tc_fence_after();
        used ^= 3u;
      }
      for (int k = 0; !wide && ok && k < o.red; k += a.seg) {  // (one round unless the tile folds)
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
      const float scale = EPI == kEpiPlainScaled ? *p.e.scale : 1.f, inv_t = p.e.inv_t;
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
        if (EPI == kEpiPlainScaled) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) f.v[j][r][0] *= scale, f.v[j][r][1] *= scale;
        }
        if (EPI == kEpiPlainSoft) {  // (probabilities below 2^-126 are 0, far below what the sums over dz resolve)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float d = exp2_fast((f.v[j][r][h] * inv_t - lse[r]) * 1.4426950408889634f) * gw[r];
                f.v[j][r][h] = gw[r] == 0.f ? 0.f : d;  // (a row without gradient stays zero even where its logits are not finite)
              }
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
          if (kWide && wide) {
            mbar_arrive_cluster(mapa(su32(acc_empty), 0));
            mbar_arrive_cluster(mapa(su32(acc_empty + 1), 0));
          } else if (CG == 2)
            mbar_arrive_cluster(mapa(su32(acc_empty + buf), 0));
          else
            mbar_arrive(acc_empty + buf);
        }
        if (!folds && !wide) buf ^= 1;
      }
    }
  } else if (!is_plain(EPI) && warp >= 4 && warp < kFirstLoader) {
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
    constexpr bool kSpread = EPI == kEpiSpread;
    // Columns that a thread holds of a stored result. In the unaligned form it has 72 registers: with 32 columns, what is added
    // and the bias fetched ahead and a Walk it spilled 648 bytes (2048 x 4096 x 101 with bias, gelu and kept z 48 us, now 36; dW of
    // 24 groups, 8 rows, n 2000, k 711, added to an older one in fp32 137, now 90).
    constexpr int kPieces = GEN && is_store(EPI) ? 16 : 32;
    const auto part_of = [&](int k, int c) -> const float* {  // the k-th other CTA's sums of columns c to c + 31
      if (kSpread) return reinterpret_cast<const float*>(smem) + ((k - 1) * a.spread + (c >> 5) / a.split * 32) * kPartLd;
      return parts + ((k - 1) * a.bn + c) * kPartLd;
    };
    constexpr bool kScore = EPI == MM_EPI_SCORE || EPI == kEpiScoreOne, kStats = EPI == MM_EPI_STATS || kScore;
    int buf = 0;
    uint32_t used = 0;  // as the MMA counts them
    float few_m = NAN, few_s = 0.f, few_u = 0.f;  // few tokens: of all the warp's words
    Walk<CG, kWide> walk;
    for (int t = first; t < tiles; t += step) {
      const Tile o = GEN ? tile_of<CG, kWide>(a, lo_of, pref, widest, t, part) : walk.next(a, lo_of, pref, widest, t, step, tiles, part, lane);
      if (o.n <= 0) continue;
      const int l0 = o.l0 + BM * rank;
      const bool sum = o.red > 0;
      // what the tile needs besides its sums is fetched before they are waited for
      const bool by_rows = EPI == MM_EPI_SOFTGRAD || (!kStats && EPI != MM_EPI_SCORE_FEW && a.rows_out);
      const int64_t group_out = p.rag == MM_RAG_RED ? o.g * e.group_stride : 0;
      const void* add = e.accumulate ? e.out : e.residual;
      const int64_t add_ld = e.accumulate ? e.ld : e.ldr;
      const int piece = l0 + (threadIdx.x & 15) * 8;
      const int64_t first_row = o.c0 + c_first + rows.row;
      int64_t add_at = (e.accumulate ? group_out : 0) + first_row * add_ld + piece;
      uint4 next[4];
      rows.live = piece < p.lanes;
      if (!GEN && by_rows && add && part == 0) rows.load(add, add_at, add_ld, o.n - c_first, next);
      // lanes of the fragments (four per thread) or the thread's own lane
      float lse[4], gw[4], bias[4];
      int lab[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int l = l0 + 32 * quad + (by_rows ? (lane >> 2) + 8 * r : lane);
        lse[r] = 0.f, gw[r] = 0.f, bias[r] = 0.f, lab[r] = -1;
        if (l >= p.lanes || (!by_rows && r)) continue;
        if (is_store(EPI)) {
          if (e.bias) bias[r] = ld16(e.bias, l, p.f16);
        } else if (EPI == MM_EPI_STATS || EPI == MM_EPI_SOFTGRAD) {
          if (EPI == MM_EPI_STATS || e.labels) lab[r] = max(*(e.labels + l), -1);
          if (EPI == MM_EPI_SOFTGRAD) {
            const bool skip = e.labels && (lab[r] == e.ignore || lab[r] < 0 || lab[r] >= e.vocab);
            lse[r] = *(e.lse + l);
            gw[r] = skip ? 0.f : *(e.g + l) / *e.gscale * kMmGradOne;
            lab[r] = skip ? -1 : lab[r] - e.word0;
          }
        }
      }
      float m = kScore ? NAN : -INFINITY, total = 0.f, spread = 0.f;
      // the listed words of the thread's token: the first one from the tile's start on
      const int2* want = nullptr;
      int want_left = 0, want_next = INT32_MAX;
      if (kScore && e.n_want > 0 && l0 + 32 * quad + lane < p.lanes) {
        const int64_t token = l0 + 32 * quad + lane;
        if (e.words) {
          want_left = 1, want_next = *(e.words + token);
          if (want_next < o.c0 || want_next >= e.vocab) want_next = INT32_MAX;
        } else {
          const int at = *(e.first + token * a.col_tiles + o.c0 / a.bn);
          want = e.want + token * e.n_want + at;
          want_left = e.n_want - at;
          if (want_left > 0) want_next = want->x;
        }
      }
      constexpr bool kHold = kStats && CG == 2 && EPI != kEpiScoreOne;  // sums over accumulators are held in registers
      float z[kHold ? 4 : 1][32];                             // the logits of the thread's four chunks
      const bool folds = a.fold && o.red > a.seg, wide = kWide && o.n > kAccCols;
      bool ok = true;
      for (int k = 0; k == 0 || k < o.red; k += a.accs == 1 ? a.seg : o.red) {  // accumulators of the tile
        uint32_t taddr = tmem + (uint32_t)(wide ? 0 : buf * acc_stride) + ((uint32_t)(32 * quad) << 16);
        if (kWide && wide && sum) {
          ok = mbar_wait(acc_full, used & 1, abort_flag, p.err, 5) && mbar_wait(acc_full + 1, used >> 1 & 1, abort_flag, p.err, 5);
          __syncwarp();
          tc_fence_after();
          used ^= 3u;
        } else if (sum) {
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
        ok = kStats ? named_bar_all(1, 32 * kEpiWarps, ok) : named_bar_all(2 + half, 128, ok);
        if (kSpread) {
          // The CTAs of a cluster have each summed a share of the reduction, and each adds up the sums of every split-th chunk
          // of 32 columns, its own and then the others' in order: these go where its stages were, once all are done with theirs.
          cluster_sync();
          for (int c = c_first; ok && c < o.n; c += c_step) {
            const int owner = (c >> 5) % a.split;
            if (owner == part) continue;
            float v[32];
            tmem_ld32(taddr + c, v);
            const uint32_t to = mapa(su32(reinterpret_cast<float*>(smem) +
                                          ((part < owner ? part : part - 1) * a.spread + (c >> 5) / a.split * 32) * kPartLd + 32 * quad + lane), owner);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(to + j * kPartLd * 4), "f"(v[j]) : "memory");
          }
          cluster_sync();
        } else if (CG == 1 && a.split > 1) {
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
        const bool two = kStats && !kHold && EPI != kEpiScoreOne && a.accs > 1;
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
        if (kStats) {
          const uint32_t sums = two && o.red > a.seg ? taddr + acc_stride : taddr;
#pragma unroll(EPI == kEpiScoreOne || GEN ? 1 : 4)  // (GEN has fewer registers: 1350 x 48737 x 70 129 us unrolled, 106)
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
            if (kScore) {
              const float scale = e.inv_t * 1.4426950408889634f;
              const float most = e.ent ? epi_score<true>(y, nv, scale, m, total, spread) : epi_score<false>(y, nv, scale, m, total, spread);
              if (e.logits && l0 + 32 * quad + lane < p.lanes) {
                store_col(e.logits + (int64_t)(o.c0 + c) * p.lanes + l0 + 32 * quad + lane, p.lanes, nv, y);
                e.chunk_max[(int64_t)((o.c0 + c) / kMmStatChunk) * p.lanes + l0 + 32 * quad + lane] = most;
              }
              while (want_next < o.c0 + c + nv) {
                const int j_at = want_next - (o.c0 + c);
                if (j_at >= 0) {  // (the other half's words are passed over)
                  float own = 0.f;
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (j == j_at) own = y[j];
                  e.zwant[(int64_t)(l0 + 32 * quad + lane) * e.n_want + (e.words ? 0 : want->y)] = own;
                }
                ++want;
                want_next = --want_left > 0 ? want->x : INT32_MAX;
              }
              continue;
            }
            epi_stats(y, nv, m, total);
            if (at >= 0 && at < nv) {  // (the label of a lane that exists)
              float own = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == at) own = y[j];
              e.zlab[l0 + 32 * quad + lane] = own;
            }
          }
        } else if (EPI == MM_EPI_SCORE_FEW) {
          const int w0 = l0 + 32 * quad;  // the warp's words; a thread has one of them for every token, and takes one token's
          if (half == 0 && w0 < p.lanes) {
            float v[32];
            float* x = reinterpret_cast<float*>(out_stage) + quad * (32 * 33);
            tmem_ld32(taddr, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j * 33 + lane] = v[j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = x[lane * 33 + j];
            __syncwarp();
            if (lane < o.n) score_few(e, v, w0, min(32, p.lanes - w0), lane, p.cols, (p.lanes + kMmStatChunk - 1) / kMmStatChunk, few_m, few_s, few_u);
          }
        } else if (by_rows && is_glu(EPI)) {
          for (int c = c_first; c < o.n; c += c_step) {
            Frag f;
            tmem_ld_frag(taddr + c, f);
            if (CG == 1) {
              for (int k = 1; k < a.split; ++k) {
                const float* q = part_of(k, c) + 2 * (lane & 3) * kPartLd + 32 * quad + (lane >> 2);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    f.v[j][r][0] += q[8 * j * kPartLd + 8 * r];
                    f.v[j][r][1] += q[(8 * j + 1) * kPartLd + 8 * r];
                  }
              }
            }
            const int i = threadIdx.x & 127;
            const int64_t row0 = o.c0 + c;
            if (e.z) {
              glu_frag_out(stage, quad, lane, f, p.f16);
              named_bar(2 + half, 128);
              const int feature = l0 / 2 + (i & 7) * 8;
              rows.live = feature < p.lanes;
              rows.store(e.z, (row0 + rows.row) * e.ldz + ((i & 8) ? p.lanes : 0) + feature, e.ldz, o.n - c);
              named_bar(2 + half, 128);
            }
            glu_frag_act(f, e.act);
            glu_frag_out_h(stage, quad, lane, f, p.f16);
            named_bar(2 + half, 128);
            const int feature = l0 / 2 + (i & 7) * 8;
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // a row's 64 features are eight pieces of 16 bytes
              const int row = (i >> 3) + 16 * k;
              if (feature < p.lanes && c + row < o.n)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.out) + (row0 + row) * e.ld + feature) =
                    lds128(stage + (uint32_t)(row * kRowBytes + (i & 7) * 16));
            }
            named_bar(2 + half, 128);
          }
        } else if (by_rows) {
          constexpr int kJ = kPieces / 8;
          for (int c = c_first; c < o.n; c += c_step) {
            if (kSpread && (c >> 5) % a.split != part) continue;
            FragOf<kJ> f;
            const auto each = [&](auto fn) {
#pragma unroll
              for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) f.v[j][r][0] = fn(f.v[j][r][0], r), f.v[j][r][1] = fn(f.v[j][r][1], r);
            };
            const auto sums = [&](int j0) {  // of 8 kJ columns from 8 j0 on
              if (sum)
                tmem_ld_frag(taddr + c + 8 * j0, f);
              else
                each([](float, int) { return 0.f; });
              if (CG == 1) {
                for (int k = 1; k < a.split; ++k) {
                  const float* q = part_of(k, c) + (8 * j0 + 2 * (lane & 3)) * kPartLd + 32 * quad + (lane >> 2);
#pragma unroll
                  for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                      f.v[j][r][0] += q[8 * j * kPartLd + 8 * r];
                      f.v[j][r][1] += q[(8 * j + 1) * kPartLd + 8 * r];
                    }
                }
              }
              if (is_store(EPI)) {
                if (e.scale) {
                  const float sc = *e.scale;
                  each([&](float v, int) { return v * sc; });
                }
                if (e.bias) each([&](float v, int r) { return v + bias[r]; });
              }
            };
            const auto act = [&] {
              if (e.act == MM_ACT_SILU)
                each([](float v, int) { return mm_silu(v); });
              else if (e.act == MM_ACT_GELU)
                each([](float v, int) { return mm_gelu(v); });
              else if (e.act == MM_ACT_RELU)
                each([](float v, int) { return mm_relu(v); });
            };
            const int64_t row_at = first_row + (c - c_first);
            if (kJ == 4) sums(0);
            if (EPI == MM_EPI_SOFTGRAD) {
              const int word = o.c0 + c + 2 * (lane & 3);
#pragma unroll
              for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    // (a row without gradient stays zero even where its logits are not finite)
                    const float d = (__expf(f.v[j][r][q] * e.inv_t - lse[r]) - (word + 8 * j + q == lab[r] ? 1.f : 0.f)) * gw[r];
                    f.v[j][r][q] = gw[r] == 0.f ? 0.f : d;
                  }
              frag_out(stage, quad, lane, f, p.f16);
            } else {
              if (e.z) {
#pragma unroll 1
                for (int j0 = 0; j0 < 4; j0 += kJ) {
                  if (kJ < 4) sums(j0);
                  frag_out(stage, quad, lane, f, p.f16, j0);
                }
                named_bar(2 + half, 128);
                rows.store(e.z, row_at * e.ldz + piece, e.ldz, o.n - c);
                named_bar(2 + half, 128);
              }
              if (kJ == 4) act();
              if (add) {
                if (GEN) rows.load(add, add_at, add_ld, o.n - c, next);
                rows.stage(next);
                named_bar(2 + half, 128);
                add_at += c_step * add_ld;
                if (!GEN && c + c_step < o.n) rows.load(add, add_at, add_ld, o.n - c - c_step, next);
              }
#pragma unroll 1
              for (int j0 = 0; j0 < 4; j0 += kJ) {
                if (kJ < 4) sums(j0), act();
                if (add) {
                  frag_add(stage, quad, lane, f, p.f16, j0);  // (each warp rereads and overwrites its own quarter only)
                  __syncwarp();
                }
                frag_out(stage, quad, lane, f, p.f16, j0);
              }
            }
            named_bar(2 + half, 128);
            rows.store(e.out, group_out + row_at * e.ld + piece, e.ld, o.n - c);
            named_bar(2 + half, 128);
          }
        } else {
          const int l = l0 + 32 * quad + lane;
          for (int c = c_first; c < o.n; c += c_step) {
            if (kSpread && (c >> 5) % a.split != part) continue;
            const bool accumulate = e.accumulate || (k && !folds);
            if constexpr (GEN && is_store(EPI)) {
              // What a weight gradient (to which nothing else is done) is added to comes 32 columns at a time, as in the aligned
              // form: with 16 loads in flight 64 groups of 128 rows, n 2000, k 711 took 296 us, so 228.
              if (accumulate) {
                uint32_t old[32];
                epi_fetch(p, o.g, l, o.c0 + c, min(32, o.n - c), old);
#pragma unroll
                for (int h = 0; h < 32; h += kPieces) {
                  float v[kPieces];
                  if (sum) {
                    tmem_ld(taddr + c + h, v);
                  } else {
#pragma unroll
                    for (int j = 0; j < kPieces; ++j) v[j] = 0.f;
                  }
#pragma unroll
                  for (int j = 0; j < kPieces; ++j) {
                    const uint32_t w = old[h + j];
                    v[j] += e.out_f32 ? __uint_as_float(w) : p.f16 ? __half2float(__ushort_as_half((uint16_t)w)) : __uint_as_float(w << 16);
                  }
                  put(p, o.g, l, o.c0 + c + h, min(kPieces, o.n - c - h), v);
                }
                continue;
              }
            }
#pragma unroll 1
            for (int h = 0; h < 32; h += kPieces) {
              const int nv = min(kPieces, o.n - c - h);
              if (nv <= 0) break;
              float v[kPieces];
              if (sum) {
                tmem_ld(taddr + c + h, v);
              } else {
#pragma unroll
                for (int j = 0; j < kPieces; ++j) v[j] = 0.f;
              }
              if (CG == 1) {
                for (int k = 1; k < a.split; ++k) {
                  const float* q = part_of(k, c) + h * kPartLd + 32 * quad + lane;
#pragma unroll
                  for (int j = 0; j < kPieces; ++j) v[j] += q[j * kPartLd];
                }
              }
              if constexpr (is_glu(EPI)) {
                glu_out(p, l, o.c0 + c, nv, v);
              } else {
                epi_store(p, o.g, l, o.c0 + c + h, nv, !GEN && accumulate, v);
                put(p, o.g, l, o.c0 + c + h, nv, v);
              }
            }
          }
        }
        if (sum) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {  // the MMA may overwrite this buffer
            if (kWide && wide) {
              mbar_arrive_cluster(mapa(su32(acc_empty), 0));
              mbar_arrive_cluster(mapa(su32(acc_empty + 1), 0));
            } else if (CG == 2)
              mbar_arrive_cluster(mapa(su32(acc_empty + buf), 0));
            else
              mbar_arrive(acc_empty + (two ? 1 : buf));
          }
          if (a.accs == 1 && !folds && !wide) buf ^= 1;
        }
      }
      if (!ok) break;
      if (kScore) {
        float4* x = reinterpret_cast<float4*>(out_stage) + 32 * quad + lane;
        const int l = l0 + 32 * quad + lane;
        if (half) *x = make_float4(m, total, spread, 0.f);
        named_bar(2, 32 * kEpiWarps);
        if (!half && l < p.lanes) {
          const float4 q = *x;
          const float top = fmaxf(m, q.x), c = e.inv_t * 1.4426950408889634f;
          const float d0 = m == top ? 0.f : fmaxf(m - top, -1e30f), d1 = q.x == top ? 0.f : fmaxf(q.x - top, -1e30f);
          const float r0 = exp2_fast(d0 * c), r1 = exp2_fast(d1 * c);
          const int64_t at = (int64_t)(o.c0 / a.bn) * p.lanes + l;
          e.part[at] = make_float2(top, total * r0 + q.y * r1);
          if (e.ent) e.ent[at] = (spread + d0 * total) * r0 + (q.z + d1 * q.y) * r1;
        }
      }
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
    if (EPI == MM_EPI_SCORE_FEW && half == 0 && lane < p.cols) {
      const int64_t at = (int64_t)(blockIdx.x * 4 + quad) * p.cols + lane;
      e.part[at] = make_float2(few_m, few_s);
      if (e.ent) e.ent[at] = few_u;
    }
  }
  __syncwarp();
  if (CG == 1 && a.split > 1 && first < tiles && (warp < 4 || warp >= kFirstLoader)) {
    cluster_sync();
    if (EPI == kEpiSpread) cluster_sync();
  }
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
int g_clusters[64][kMaxSpread + 1] = {};  // and clusters of so many CTAs

// A gated block's weights, n a multiple of 16: (reduction, row of 16, gate or up, 16 rows, group); one copy brings four times 16
// gate rows and the same 16 up rows.
bool make_glu_map(CUtensorMap* m, const MmOperand& o, int f16, uint64_t red, uint64_t n, uint64_t groups) {
  const cuuint64_t row = (cuuint64_t)o.ld * 2;
  const cuuint64_t dims[5] = {red, 16, 2, n / 16, groups};
  const cuuint64_t strides[4] = {row, row * n, row * 16, groups > 1 ? (cuuint64_t)o.group_stride * 2 : row};
  const cuuint32_t box[5] = {BK, 16, 2, BM / 32, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return g_encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(o.p),
                  dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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

int smem_bytes(int cg, int bn, int stages, int split, const MmProblem& p) {  // (split 1: also where it is spread)
  return 1024 + stages * (A_BYTES + bn / cg * BK * 2) + 2 * kOutBytes + (split - 1) * bn * kPartLd * 4 + ctrl_bytes(p.rag, p.groups);
}

template <int CG, int EPI, bool GEN>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const TcArgs& a, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(GEN ? kThreads + 32 * kLoaders : kThreads);
  cfg.dynamicSmemBytes = smem_bytes(CG, a.bn, 0, a.spread ? 1 : a.split, a.p) + a.ring;
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
    case MM_EPI_SOFTGRAD:
      if (!GEN && !a.p.e.labels) return launch<CG, kEpiPlainSoft, false>(ta, tb, a, grid, s);
      return launch<CG, MM_EPI_SOFTGRAD, GEN>(ta, tb, a, grid, s);
    case MM_EPI_GLU:
      if (a.bn > kAccCols) return CG == 2 && !GEN ? launch<2, kEpiGluWide, false>(ta, tb, a, grid, s) : cudaErrorInvalidValue;
      return launch<CG, MM_EPI_GLU, GEN>(ta, tb, a, grid, s);
    case MM_EPI_SCORE:
      if (!GEN && a.p.red <= kSegStats) return launch<CG, kEpiScoreOne, false>(ta, tb, a, grid, s);
      return launch<CG, MM_EPI_SCORE, GEN>(ta, tb, a, grid, s);
    case MM_EPI_SCORE_FEW: return CG == 1 ? launch<1, MM_EPI_SCORE_FEW, GEN>(ta, tb, a, grid, s) : cudaErrorInvalidValue;
    default: break;
  }
  if (CG == 2 && a.bn > kAccCols) return launch<2, kEpiPlainWide, false>(ta, tb, a, grid, s);
  if (CG == 2 && a.p.rag == MM_RAG_RED) return launch<2, kEpiPlainRag, false>(ta, tb, a, grid, s);
  if (CG == 1 && a.spread) return launch<1, kEpiSpread, false>(ta, tb, a, grid, s);
  if (GEN && a.plain && a.split == 1 && !a.p.e.scale) return launch<1, kEpiPlain, true>(ta, tb, a, grid, s);
  if (!GEN && a.plain && a.split == 1)
    return a.p.e.scale ? launch<CG, kEpiPlainScaled, false>(ta, tb, a, grid, s) : launch<CG, kEpiPlain, false>(ta, tb, a, grid, s);
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
  if (e == cudaSuccess) e = prepare_one<CG, MM_EPI_GLU, GEN>();
  if (e == cudaSuccess) e = prepare_one<CG, MM_EPI_SCORE, GEN>();
  return e;
}

// The column tile with the shortest schedule: rounds over the SMs times a tile's columns (and what a tile costs
// whatever its width, about 24 columns' time). Widths that are no multiple of 64 run at the next larger one's rate
// (4096^3, main loop alone: 256 74 us, 192 74 us, 224 100 us). Groups of a ragged reduction (0: a dense product, the only
// one whose last round is split) have tiles that cost 200 columns more, the loads of their lanes (measured on single CTAs;
// one group, 8192 rows, 4096 x 4096: 256 columns 189 us in 4 rounds, 192 194 us in 5, 128 238 us in 7).
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

// Whether a ragged reduction runs on pairs. They halve the operands' way into the SMs, but start 0.8 us later, waste half a
// pair where the tiles of 128 lanes are odd, and leave half as many units to share few tiles out to. Measured over 759 shapes of 1
// to 256 groups of 7 to 16384 rows (single CTAs first): 64 groups of 256 rows, 4096 x 4096 510 us, 459, but 256 x 512 8.8, 9.5;
// 64 of 128 rows, 1000 x 1024 33.8, 31.8, but 512 x 4096 58.0, 61.5; 24 of 64 rows, 2048 x 1024 22.9, 23.8; 64 of 256 rows,
// 2048 x 264 (three tiles of lanes) 33.4, 35.4; one of 16384 rows, 2048 x 2048 90, 79, 512 x 512 (four tiles) 62.8, 70.3, and
// 4096 x 1152 (nine) 95, 147. Of the 113 with an even number of tiles that this takes none is slower on pairs.
bool rag_pairs(const MmProblem& p, int pairs) {
  const int64_t lanes128 = (p.lanes + BM - 1) / BM, average = p.red / p.groups;
  const int64_t tiles = (lanes128 + 1) / 2 * ((p.cols + 255) / 256) * p.groups;
  if (lanes128 % 2 && lanes128 <= 16) return false;
  if (average >= 192 ? p.lanes <= 256 || p.cols <= 256 : average < 128 || p.lanes <= 512 || p.cols <= 512) return false;
  return 5 * tiles >= 4 * pairs && tiles * (average + 4 * BK) >= (int64_t)33 * BK * pairs;  // (33 steps of 64 for each pair, with what a tile costs)
}

}  // namespace

int mm_few_parts(int vocab) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return 4 * std::min({g_sms[dev & 63], kMmFewParts / 4, (vocab + BM - 1) / BM});
}

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
  if (e == cudaSuccess) e = prepare_one<1, kEpiPlain, true>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiPlainWide, false>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiGluWide, false>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiPlainRag, false>();
  if (e == cudaSuccess) e = prepare_one<1, kEpiPlainSoft, false>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiPlainSoft, false>();
  if (e == cudaSuccess) e = prepare_one<1, kEpiPlainScaled, false>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiPlainScaled, false>();
  if (e == cudaSuccess) e = prepare_one<1, kEpiSpread, false>();
  if (e == cudaSuccess) e = prepare_one<1, kEpiScoreOne, false>();
  if (e == cudaSuccess) e = prepare_one<2, kEpiScoreOne, false>();
  if (e == cudaSuccess) e = prepare_one<1, MM_EPI_SCORE_FEW, false>();
  if (e == cudaSuccess) e = prepare_one<1, MM_EPI_SCORE_FEW, true>();
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
    for (int n = 2; e == cudaSuccess && n <= kMaxSpread; ++n) {
      cfg.gridDim = dim3(n);
      attr[0].val.clusterDim.x = n;
      e = cudaOccupancyMaxActiveClusters(&g_clusters[dev & 63][n], mm_tc_kernel<1, kEpiSpread, false>, &cfg);
    }
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
  const bool stats = p.epi == MM_EPI_STATS || p.epi == MM_EPI_SCORE;
  const int lanes = p.epi == MM_EPI_GLU ? 2 * p.lanes : p.lanes;  // (a gated block's features take two each)
  const int64_t lanes128 = (lanes + BM - 1) / BM;
  const int blocks = (p.red + BK - 1) / BK;
  const int split_bn = p.cols <= 32 && p.b.red_major ? 32 : 64;
  // tiles of that width (ragged columns: where they all fit one, each group with rows has one)
  const int64_t few = lanes128 * (p.rag == MM_RAG_COLS ? std::min(p.groups, p.cols) : (p.cols + split_bn - 1) / split_bn);
  if (p.rag != MM_RAG_RED && (p.epi == MM_EPI_STORE || p.epi == MM_EPI_GLU) && (p.rag == MM_DENSE || p.cols <= 64) && 2 * few <= sms)
    a.split = (int)std::max<int64_t>(1, std::min<int64_t>({sms / few, blocks / 6, split_bn == 32 ? 8 : 4}));
  // Clusters that do not all run at once take two rounds (1 token, a gated block of 1024 features, k 3664, 16 tiles: 16.4 us
  // in eight shares, 9.3 in six). Not all that the device is said to hold always find room, but of two and of four (said 28 of
  // five: 25 took 14.3 us, 24 10.5; 46 of three: 44 took 34 us, in two shares 26): an eighth is left. Products whose bits
  // earlier callers rely on keep their shares.
  const auto held_at_once = [&](int n) { return n == 2 || n == 4 ? g_clusters[dev & 63][n] : g_clusters[dev & 63][n] * 7 / 8; };
  if (p.epi == MM_EPI_GLU || p.may_spread)
    while (a.split > 1 && held_at_once(a.split) < few) --a.split;
  // Where that leaves a long reduction of more columns to few CTAs, tiles of 64 to 256 columns over clusters that also share out
  // the joining of their sums, if they are estimated to take less time (cycles: a CTA's stage brings its operands at 64
  // bytes a cycle, and so does the exchange at 32; dx of 512 rows, 16128 words, d 1024: 41 us, 31 so).
  int spread_bn = 0;
  if (p.may_spread && !gen && p.rag == MM_DENSE && p.epi == MM_EPI_STORE && !p.e.residual && !p.e.accumulate && p.cols > 32 && p.red <= kSegFold) {
    const auto stage = [](int bn) { return 256 + 2 * bn; };
    int64_t best = a.split > 1 ? (int64_t)(blocks + a.split - 1) / a.split * stage(64) : INT64_MAX;
    if (a.split == 1) {
      const int units = p.lanes > BM ? pairs : sms, cgs = p.lanes > BM ? 2 : 1;
      best = schedule((p.lanes + BM * cgs - 1) / (BM * cgs), p.cols, p.b.red_major, 0, cgs, std::max(1, units)).cost * 2 * blocks;
    }
    for (int bn = 64; bn <= 256; bn *= 2) {
      const int64_t tiles = lanes128 * ((p.cols + bn - 1) / bn);
      int n = (int)std::min<int64_t>({sms / tiles, kMaxSpread, blocks / 6});
      // (what a CTA receives has to fit where its stages were)
      const int stage_bytes = A_BYTES + bn * BK * 2, held = (kSmemMax - smem_bytes(1, bn, 0, 1, p)) / stage_bytes * stage_bytes;
      while (n > 1 && (n - 1) * ((bn / 32 + n - 1) / n * 32) * kPartLd * 4 > held) --n;
      if (n < 2 || held_at_once(n) < tiles) continue;
      const int64_t cost = (blocks + n - 1) / n * stage(bn) + bn * 16 + 3000;
      if (cost < best) best = cost, spread_bn = bn, a.split = n;
    }
  }
  const MmEpiArgs& ep = p.e;
  const auto by_rows = [](const void* base, int64_t ld) { return !base || ((uintptr_t)base % 16 == 0 && ld % 8 == 0); };
  // (dz of a softmax loss always leaves by rows, see MM_EPI_SOFTGRAD)
  a.rows_out = !ep.out_f32 && !ep.acc_in && p.lanes % 8 == 0 && ep.group_stride % 8 == 0 && by_rows(ep.out, ep.ld) &&
               by_rows(ep.residual, ep.ldr) && by_rows(ep.z, ep.ldz);
  a.plain = a.rows_out && p.epi == MM_EPI_STORE && (!ep.scale || p.rag == MM_DENSE) && !ep.bias && !ep.z && !ep.residual && !ep.accumulate && ep.act == MM_ACT_NONE;
  // Pairs where there are at least two 128-lane tiles (a half-empty pair would double the work of a
  // narrow product); of ragged reductions those whose results leave by rows and that rag_pairs takes.
  const bool few_tokens = p.epi == MM_EPI_SCORE_FEW;
  const int cg = !gen && !few_tokens && (p.rag != MM_RAG_RED || (a.plain && rag_pairs(p, pairs))) && lanes > BM && pairs > 0 && a.split == 1 ? 2 : 1;
  const int units = cg == 2 ? pairs : few_tokens ? std::min(sms, kMmFewParts / 4) : sms;
  a.lane_tiles = (lanes + BM * cg - 1) / (BM * cg);
  a.bn = 256;
  if (spread_bn) {
    a.bn = spread_bn;
    a.spread = (spread_bn / 32 + a.split - 1) / a.split * 32;
  } else if (a.split > 1) {
    a.bn = split_bn;
  } else if (few_tokens) {
    if (p.cols > kMmFewRows) return cudaErrorInvalidValue;
    a.bn = kMmFewRows;
  } else if (p.rag == MM_RAG_COLS) {
    // the groups' sizes are only known on the device: a tile that holds twice the average (a smaller tile
    // leaves room for more stages in flight; a group beyond it takes several tiles, which share its weights in L2)
    const int64_t average = ((int64_t)p.cols + p.groups - 1) / p.groups, typical = std::min<int64_t>(2 * average, p.cols);
    while (a.bn > 64 && a.bn / 2 >= typical) a.bn /= 2;
    // Groups around 256 rows: those above would pass over their weights once more for a few rows (64 groups of 264, 4096 x
    // 4096: 677 us, 462 in one pass). Where there are tiles for every pair of SMs, the tile may hold half as much again as the average (widest_tile).
    if (cg == 2 && p.red <= kSegFold && p.b.red_major && (a.plain || p.epi == MM_EPI_GLU) && 3 * average > 2 * kAccCols &&
        average <= 448 && a.lane_tiles * (int64_t)std::min(p.groups, p.cols) >= units)
      a.bn = (int)std::min<int64_t>(2 * kAccCols, (3 * average / 2 + 63) / 64 * 64);
  } else if (p.epi == MM_EPI_SCORE) {
    a.bn = p.e.tile;
  } else if (!stats) {
    const Schedule w = schedule(a.lane_tiles, p.cols, p.b.red_major, p.rag == MM_RAG_RED ? p.groups : 0, cg, units);
    a.bn = w.bn, a.tail_lg = w.tail_lg, a.tail_from = w.tail_from;
  }
  a.stages = 1;
  while (a.stages < kMaxStages && smem_bytes(cg, a.bn, a.stages + 1, a.spread ? 1 : a.split, p) <= kSmemMax) ++a.stages;
  const int room = kSmemMax - smem_bytes(cg, a.bn, 0, a.spread ? 1 : a.split, p);
  a.ring = a.bn > kAccCols ? room / 1024 * 1024 : a.stages * (A_BYTES + a.bn / cg * BK * 2);
  // the rows of a copy divide what a CTA stages; large copies where the columns are not ragged (4096^3 with copies of
  // 128 rows 81.7 us, of 64 rows 83.8)
  const int staged = a.bn / cg;
  a.b_box = p.rag == MM_RAG_COLS || staged % 64 ? kRagBox : staged % 128 ? 64 : 128;
  a.a_blocks = !p.a.red_major && p.lanes % 64 == 0 ? 2 : 1;
  a.b_blocks = !p.b.red_major && p.cols % 64 == 0 && (staged == 256 || staged == 128) ? staged / 64 : 1;
  a.col_tiles = (p.cols + std::min(a.bn, kAccCols) - 1) / std::min(a.bn, kAccCols);
  const int64_t tiles = a.lane_tiles * (int64_t)(p.rag == MM_RAG_COLS ? a.col_tiles + p.groups : a.col_tiles) * (p.rag == MM_RAG_RED ? p.groups : 1);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  if (a.tail_lg == 0) a.tail_from = (int)tiles;
  a.by_lanes = Divider(a.lane_tiles), a.by_panel = Divider(a.lane_tiles * kPanel), a.by_matrix = Divider(a.lane_tiles * a.col_tiles);
  a.glu_whole = p.epi == MM_EPI_GLU && p.lanes % 16 == 0 && p.a.ld < ((int64_t)1 << 38) / p.lanes;  // (a map's strides end at 2^40 bytes)
  CUtensorMap ta = {}, tb = {};
  if (!gen) {
    const uint64_t groups = p.rag == MM_RAG_COLS ? p.groups : 1;
    const uint64_t red = p.red;
    const bool ok = (a.glu_whole ? make_glu_map(&ta, p.a, p.f16, red, p.lanes, groups) :
                     make_map(&ta, p.a, p.f16, p.a.red_major ? red : p.lanes, p.a.red_major ? lanes : red, groups, p.epi == MM_EPI_GLU ? 16 : p.a.red_major ? BM : BK, a.a_blocks)) &&
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
  if (few_tokens)  // (the sums of 32 tokens are added up while the ring fills: accumulators side by side were no faster)
    a.seg = kSegStats, a.fold = 1;
  else if (stats && (cg == 2 || p.red > 2 * kSegStats))
    a.seg = kSegStats, a.fold = cg == 1;
  else if (stats && p.red > kSegStats)
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
