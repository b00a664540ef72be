// linear_mma.cuh -- the linear operator's products on the tensor cores
// (tcgen05, sm_103a), for 16-bit types.
//
// C[m, n] = sum_k A[m, k] B[n, k], 128 rows of C per CTA and BN columns per
// tile.  Six warps, or ten:
//
//   warp 0   copies a 64-deep slice of both operands per stage into a ring of
//            shared-memory stages (TMA, 128-byte swizzle), a full / empty
//            mbarrier pair per stage;
//   warp 1   one thread issues the matrix instructions of a stage and commits
//            them to its empty barrier; the binary32 sums stay in tensor memory;
//   the rest read a finished tile's sums (each warp its quarter of the 128
//            lanes), apply the epilogue and store.
//
// The tile's sums are double-buffered in tensor memory, so that the epilogue of
// a tile runs under the products of the next; the grid is persistent.
//
// CG = 2: a pair of CTAs makes a 256-row tile; each holds its 128 rows of A and
// half of B's columns, and one thread of the pair issues for both, so each SM
// reads half of B from the other's shared memory instead of from L2.
//
// SWAP: C is stored transposed (row = column of C): with few rows of x, the
// weight's rows fill the 128 lanes and the tokens are the columns.
//
// GATED: the weight's rows are those of a gate, then as many of what it gates; a tile
// holds the same columns of both (half of its B operand each: of a pair, one CTA's
// half; with SWAP, half of the lanes), and the epilogue stores act(gate) * up.
//
// splits > 1: the CTAs of a cluster each take a part of K, and add their sums
// through distributed shared memory in rank order (no atomics: equal calls give
// equal bits).
//
// Operands may be stored with k contiguous (KC) or with m / n contiguous (the
// gradients' operands): the copy brings 64 x 64 squares then, and the matrix
// instruction's descriptors say so; nothing is transposed in memory.
//
// TO float with bfloat16 operands: float32 products.  An operand's row holds three pieces
// of its values side by side (each the rounding of what the ones before leave: 24 bits in
// all).  The three pieces of a slice of K arrive one after another, and the six pairs of them
// whose products reach 2^-24 of the whole are multiplied while they are in shared memory (K
// walked once for each pair took twice the copies: 4096 x 4096 x 8192 1,124 us, 939 so).  The
// tensor cores cut a sum's last place at each addition of 16 products (4.4e-6 in the norm over
// 4096 of k), so each slice has a sum of its own, the pair of the first pieces last, and the
// slices' sums are added with rounding by the epilogue's warps, in their registers (1.5e-7 over
// 10,330 of k; the library's float32 product 1.8e-6).  An infinity, or a product past binary32,
// meets zeros and terms of the other sign there that the values' own product has not: a sum that
// is not finite is made again from the values, in binary32 (pieces_again).
//
// Every wait is bounded: the first that gives up records its site in `status`;
// one that gives up ends its role, the others then run out as well, and all meet
// at the end to free the tensor memory.  A warp that waits as a whole decides as
// a whole.
#pragma once

#include <cuda.h>

#include "bulk.cuh"
#include "linear.cuh"

namespace b200norm {

constexpr int kMmaK = 64;              // elements of k per stage: 128 bytes
constexpr int kMmaRows = 128;          // rows of C per CTA
constexpr int kMmaABytes = kMmaRows * kMmaK * 2;
constexpr int kMmaWithheld = 20;       // how much sooner a test's site gives up
constexpr int kMmaGroup = 8;           // row tiles a column of tiles is walked down by (16
                                       // does as well; 4 and 32 lose 4 and 6 percent)

struct MmaArgs {
  int64_t M, N;        // of the product as the tensor cores see it
  int kblocks;         // 64-deep slices of K
  int tiles_m, tiles_n;
  int splits;
  int64_t gate;        // GATED: columns of the result (the weight has twice as many rows)
  int piece_a, piece_b;  // pieces: elements from one of an operand's to the next
  Epilogue e;
  bool vec;            // rows of the result, bias and residual are whole 16-byte vectors
  unsigned* status;
  unsigned long long limit_ns;
  bool late;           // pdl_wait() at the end
  bool stall;          // a test: nothing is copied, and the waits give up
  unsigned withhold;   // a test: the site whose event is left out (0: none)
};

// The operands in pieces as they lie in memory, for sums that are not finite.  They take the
// place of a tensor map that results in pieces do not need: 48 bytes more of arguments cost a
// launch 0.4 us.
struct MmaPieces {
  const __nv_bfloat16 *a, *b;
  int64_t lda, ldb, K;
  int piece_a, piece_b;
};
template <bool PIECES>
using MmaLastMap = typename std::conditional<PIECES, MmaPieces, CUtensorMap>::type;

// Shared memory of a CTA: the ring, then room for each epilogue warp's results (unless
// SWAP): two of 4 KB, or with pieces one of 32 by 33 floats.  Two small CTAs share an SM.
constexpr int kMmaStageRows = 32 * 128;  // 32 rows of 64 results, 128 bytes each
template <int CG, int BN, bool SWAP, bool GATED = false, bool PIECES = false>
struct MmaShape {
  static constexpr int kBRows = BN / CG;                 // of B, per CTA
  static constexpr int kBBytes = kBRows * kMmaK * 2;
  static constexpr int kStageBytes = kMmaABytes + kBBytes;
  // warps of the epilogue: a quarter of the lanes each, and of the wide tiles
  // half of the columns (with four, 16384 x 512 x 512 bf16 took 15.4 us, 12.6
  // with eight)
  // (GATED: 64 columns of the result each)
  static constexpr int kWarps = BN >= (GATED ? 256 : 128) ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kCols = BN / (kWarps / 4);
  static constexpr int kStageOut = PIECES ? 32 * 33 * 4 : 2 * kMmaStageRows;
  static constexpr int kOut = SWAP ? 0 : kWarps * kStageOut;
  // (with pieces two slices of K, six stages, and for that the SM to itself)
  static constexpr int kCtas = BN <= 64 && (SWAP || !PIECES) ? 2 : 1;  // on an SM
  static constexpr int kBudget =
      (kCtas == 2 ? 112 * 1024 : PIECES ? 226 * 1024 : 225 * 1024) - kOut;
  static constexpr int kStages = kBudget / kStageBytes > 8 ? 8 : kBudget / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  // buffers of columns for sums, and what is allocated: a power of two
  static constexpr int kBuffers = 2;
  static constexpr int kColumns = kBuffers * BN;
  static constexpr int kTmem = kColumns <= 32    ? 32
                               : kColumns <= 64  ? 64
                               : kColumns <= 128 ? 128
                               : kColumns <= 256 ? 256
                                                 : 512;
  static constexpr size_t kSmem = 1024 + kRing + kOut;
};

// -- instructions ---------------------------------------------------------------

// One warp (of each CTA of a pair) takes the columns, and gives up the right to
// take more at once: the SM's other CTAs wait for that right.
template <int CG>
__device__ __forceinline__ void tmem_alloc(unsigned* dst, unsigned cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}

template <int CG>
__device__ __forceinline__ void tmem_free(unsigned addr, unsigned cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D (+)= A B^T over 16 of k, both operands from shared memory.
template <int CG>
__device__ __forceinline__ void mma_f16(unsigned d, unsigned long long a, unsigned long long b,
                                        unsigned idesc, bool accumulate) {
  const unsigned acc = accumulate ? 1u : 0u;
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// The barrier (of both CTAs of a pair) completes once this thread's earlier
// matrix instructions have.
template <int CG>
__device__ __forceinline__ void mma_commit(unsigned long long* bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_addr(bar)) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;"
        :: "r"(smem_addr(bar)), "h"(static_cast<unsigned short>(3)) : "memory");
}

// 32 columns of this warp's 32 lanes; complete after tmem_wait().
__device__ __forceinline__ void tmem_load32(unsigned addr, float (&v)[32]) {
  unsigned r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_load16(unsigned addr, float (&v)[16]) {
  unsigned r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_store16(unsigned addr, const float (&v)[16]) {
  unsigned r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
         "r"(r[15]), "r"(addr) : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One column of this warp's 32 lanes.
__device__ __forceinline__ float tmem_load1(unsigned addr) {
  unsigned r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_store1(unsigned addr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};"
               :: "r"(__float_as_uint(v)), "r"(addr) : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A box of the tensor map at (x, y) into this CTA's shared memory, completing
// on `bar` (a shared::cluster address: of the pair's first CTA when CG is 2).
template <int CG>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y,
                                         unsigned bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];"
        :: "r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier"
        "::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// 32 rows of 64 results from shared memory (written by this warp's lanes, then
// stage_ready() and a warp barrier) to (x, y) of the tensor; what lies past its
// edges is not stored.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
               :: "l"(map), "r"(x), "r"(y), "r"(smem_addr(src)) : "memory");
}
__device__ __forceinline__ void stage_ready() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores, all but the latest N groups, have read their source.
template <int N>
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(N) : "memory");
}
__device__ __forceinline__ void stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A shared-memory operand's descriptor: 128-byte swizzle.  KC: rows of 128
// bytes, eight of them (1024 bytes) a group; `lead` is not used.  Otherwise
// the same groups hold 64 of m / n by eight of k, `lead` bytes lie between
// neighbouring squares of 64 x 64.
__device__ __forceinline__ unsigned long long smem_desc(unsigned addr, unsigned lead) {
  return static_cast<unsigned long long>((addr >> 4) & 0x3fff) |
         (static_cast<unsigned long long>((lead >> 4) & 0x3fff) << 16) |
         (static_cast<unsigned long long>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// binary32 sums; operand type (0 float16, 1 bfloat16), which index is
// contiguous (1: m / n), and the instruction's shape.
__host__ __device__ constexpr unsigned mma_idesc(bool bf16, bool a_kc, bool b_kc, int m, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((a_kc ? 0u : 1u) << 15) | ((b_kc ? 0u : 1u) << 16) |
         (static_cast<unsigned>(n >> 3) << 17) | (static_cast<unsigned>(m >> 4) << 24);
}

// -- waits ----------------------------------------------------------------------

// The sites recorded when a wait gives up.
enum MmaSite : unsigned {
  kSiteEmpty = 1, kSiteFull = 2, kSiteSums = 3, kSiteDrained = 4, kSiteResidual = 5
};

// A test's site gives up long before the others do.
__device__ __forceinline__ unsigned long long wait_limit(const MmaArgs& g, unsigned site) {
  return site == g.withhold ? g.limit_ns / kMmaWithheld : g.limit_ns;
}

// The whole warp's wait: each lane sees the barrier's phase, and one that gave up
// stops them all, so that they go on together.
__device__ __forceinline__ bool warp_wait(unsigned long long* bar, unsigned parity,
                                          unsigned long long limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns));
}

// -- epilogue -------------------------------------------------------------------

// z and y of N results (bias and residual already widened, or absent).
template <typename T, int NC>
__device__ __forceinline__ void add_to(float (&v)[NC], const T* p) {
  float f[NC];
  unpack(ld_reuse<T, NC>(p), f);
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i] += f[i];
}

// A warp's 32 rows m0.. of a tile, COLS columns n0.., whole 16-byte vectors: 64
// columns at a time to shared memory (a lane per row; the 16-byte chunks of a row
// permuted by the row, as the tensor copy's 128-byte swizzle has them, so that
// eight lanes never meet in a bank) and from there by tensor copies.  Stored
// straight from the registers, a lane per row, each instruction touches 32 lines.
// The residual comes the other way through the same buffer.
// `drained` is called once the sums have been read.  False: the wait for a residual
// gave up.
template <typename T, int COLS, bool FULL, int ACT, class Drained>
__device__ __forceinline__ bool epilogue_tile(const MmaArgs& g, const CUtensorMap* map_y,
                                              const CUtensorMap* map_z, const CUtensorMap* map_r,
                                              unsigned d, int64_t m0, int64_t n0, int lane,
                                              unsigned char* stage, unsigned long long* bar,
                                              unsigned& phase, unsigned& turn,
                                              Drained&& drained) {
  const T* bias = FULL ? static_cast<const T*>(g.e.bias) : nullptr;
  const bool res = FULL && g.e.residual, keep = FULL && g.e.z;
  const bool rows = m0 < g.M;
#pragma unroll 1
  for (int c = 0; c < COLS / 64; ++c) {
    const int64_t n = n0 + c * 64;
    const bool some = rows && n < g.N;
    // the two buffers take turns, from tile to tile as well: the one that the
    // latest store still reads is not this one
    unsigned char* at_y = stage + (keep ? 0 : turn * kMmaStageRows);
    unsigned char* at_z = stage + kMmaStageRows;
    if (lane == 0 && some) {
      if (keep) stores_read<0>();
      else stores_read<1>();
      if (res) {
        mbar_arrive_expect_tx(bar, kMmaStageRows);
        if (g.withhold != kSiteResidual)
          tma_load<1>(at_y, map_r, static_cast<int>(n), static_cast<int>(m0), smem_addr(bar));
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      tmem_load32(d + c * 64 + h * 32, v);
      if (c == COLS / 64 - 1 && h == 1) drained();
      if (!some) continue;
      const int64_t col = n + h * 32;
      // the row's chunk j of these 32 columns
      auto chunk = [&](int j) { return ((h * 4 + j) ^ (lane & 7)) * 16 + lane * 128; };
      if (bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (col + j * 8 >= g.N) continue;
          float b[8];
          unpack(ld_reuse<T, 8>(bias + col + j * 8), b);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j * 8 + i] += b[i];
        }
      }
      auto put = [&](unsigned char* at) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = v[j * 8 + i];
          *reinterpret_cast<Pack<T, 8>*>(at + chunk(j)) = pack_from<T, 8>(f);
        }
      };
      if (keep) put(at_z);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = act_value<ACT>(v[i]);
      if (res) {
        if (h == 0) {
          if (!warp_wait(bar, phase, wait_limit(g, kSiteResidual))) {
            // the copy may still be on its way to this CTA's shared memory
            if (lane == 0) mbar_wait(bar, phase, wait_limit(g, kSiteResidual));
            return false;
          }
          phase ^= 1;
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float r[8];
          unpack(*reinterpret_cast<const Pack<T, 8>*>(at_y + chunk(j)), r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j * 8 + i] += r[i];
        }
      }
      put(at_y);
    }
    if (!some) continue;
    turn ^= 1;
    stage_ready();
    __syncwarp();
    if (lane == 0) {
      tma_store(map_y, at_y, static_cast<int>(n), static_cast<int>(m0));
      if (keep) tma_store(map_z, at_z, static_cast<int>(n), static_cast<int>(m0));
      store_commit();
    }
  }
  return true;
}

// The same where rows are not whole vectors: 32 columns at a time are turned
// around in shared memory, so that a warp's lanes hold neighbouring columns.
template <typename T, int COLS, bool FULL, class Drained>
__device__ __forceinline__ void epilogue_tile_scalar(const MmaArgs& g, unsigned d, int64_t m0,
                                                     int64_t n0, int lane, float* stage,
                                                     Drained&& drained) {
  const T* bias = FULL ? static_cast<const T*>(g.e.bias) : nullptr;
  const T* res = FULL ? static_cast<const T*>(g.e.residual) : nullptr;
  T* y = static_cast<T*>(g.e.y);
  T* z = FULL ? static_cast<T*>(g.e.z) : nullptr;
  const int rows = g.M - m0 < 32 ? (g.M > m0 ? static_cast<int>(g.M - m0) : 0) : 32;
#pragma unroll 1
  for (int c = 0; c < COLS; c += 32) {
    float v[32];
    tmem_load32(d + c, v);
    if (c + 32 == COLS) drained();
#pragma unroll
    for (int i = 0; i < 32; ++i) stage[lane * 33 + i] = v[i];
    __syncwarp();
    const int64_t n = n0 + c + lane;
    if (n < g.N) {
      const float b = bias ? to_f32(bias[n]) : 0.0f;
      const int64_t at = m0 * g.N + n;
      auto run = [&](auto act) {
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
          float f = stage[r * 33 + lane];
          if (bias) f += b;
          if (z) z[at + r * g.N] = from_f32<T>(f);
          f = act_value<decltype(act)::value>(f);
          if (res) f += to_f32(res[at + r * g.N]);
          y[at + r * g.N] = from_f32<T>(f);
        }
      };
      if constexpr (FULL) with_act(g.e.act, run);
      else run(Const<kActNone>());
    }
    __syncwarp();
  }
}

// NC consecutive columns n.. of row m of the result, straight from registers.
template <typename T, int NC>
__device__ __forceinline__ void epilogue_row(const Epilogue& e, bool vec, int64_t m, int64_t n,
                                             int64_t N, float (&v)[NC]) {
  const T* bias = static_cast<const T*>(e.bias);
  const T* res = static_cast<const T*>(e.residual);
  T* y = static_cast<T*>(e.y);
  T* z = static_cast<T*>(e.z);
  const int64_t at = m * N + n;
  with_act(e.act, [&](auto act) {
    if (vec && n + NC <= N) {
      if (bias) add_to<T, NC>(v, bias + n);
      if (z) *reinterpret_cast<Pack<T, NC>*>(z + at) = pack_from<T, NC>(v);
#pragma unroll
      for (int i = 0; i < NC; ++i) v[i] = act_value<decltype(act)::value>(v[i]);
      if (res) add_to<T, NC>(v, res + at);
      *reinterpret_cast<Pack<T, NC>*>(y + at) = pack_from<T, NC>(v);
      return;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (n + i >= N) continue;
      float f = v[i];
      if (bias) f += to_f32(bias[n + i]);
      if (z) z[at + i] = from_f32<T>(f);
      f = act_value<decltype(act)::value>(f);
      if (res) f += to_f32(res[at + i]);
      y[at + i] = from_f32<T>(f);
    }
  });
}

// NC consecutive rows (tokens) m.. of column n of the result: lanes hold
// neighbouring columns.
template <typename T, int NC>
__device__ __forceinline__ void epilogue_col(const Epilogue& e, int64_t m, int64_t M, int64_t n,
                                             int64_t N, float (&v)[NC]) {
  const T* bias = static_cast<const T*>(e.bias);
  const T* res = static_cast<const T*>(e.residual);
  T* y = static_cast<T*>(e.y);
  T* z = static_cast<T*>(e.z);
  const float b = bias ? to_f32(bias[n]) : 0.0f;
  float r[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i)  // on their way together
    r[i] = res && m + i < M ? to_f32(res[(m + i) * N + n]) : 0.0f;
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (m + i >= M) continue;
      const int64_t at = (m + i) * N + n;
      float f = v[i];
      if (bias) f += b;
      if (z) z[at] = from_f32<T>(f);
      f = act_value<decltype(act)::value>(f);
      if (res) f += r[i];
      y[at] = from_f32<T>(f);
    }
  });
}

// -- epilogue of a gate and what it gates -----------------------------------------

// z from the sums of columns n.., and then act(gate) * up, into `gate`.
template <typename T, int NC>
__device__ __forceinline__ void gated_bias(const Epilogue& e, int64_t n, int64_t N,
                                           float (&gate)[NC], float (&up)[NC]) {
  const T* bias = static_cast<const T*>(e.bias);
  if (!bias) return;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (n + i >= N) continue;
    gate[i] += to_f32(bias[n + i]);
    up[i] += to_f32(bias[N + n + i]);
  }
}
template <int NC>
__device__ __forceinline__ void gated_values(const Epilogue& e, float (&gate)[NC],
                                             const float (&up)[NC]) {
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < NC; ++i) gate[i] = act_value<decltype(act)::value>(gate[i]) * up[i];
  });
}

// A warp's 32 rows m0.. of a tile, 64 columns n0.. of the result, whole 16-byte vectors,
// through shared memory as in epilogue_tile; `gate` and `up` are their sums' places.  With z
// its two parts leave first, from both buffers, and the sums are read once more.
template <typename T, int ACT, class Drained>
__device__ __forceinline__ void epilogue_gated(const MmaArgs& g, const CUtensorMap* map_y,
                                               const CUtensorMap* map_gate,
                                               const CUtensorMap* map_up, unsigned gate,
                                               unsigned up, int64_t m0, int64_t n0, int lane,
                                               unsigned char* stage, unsigned& turn,
                                               Drained&& drained) {
  const T* bias = static_cast<const T*>(g.e.bias);
  const bool some = m0 < g.M && n0 < g.N, keep = g.e.z;
  unsigned char* at_y = stage + (keep ? 0 : turn * kMmaStageRows);
  unsigned char* at_up = stage + kMmaStageRows;
  if (lane == 0 && some) {
    if (keep) stores_read<0>();
    else stores_read<1>();
  }
  __syncwarp();
  // f(place of 8 columns in the row's 128 bytes, gate, up) over the 64 columns
  auto columns = [&](bool last, auto&& f) {
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      float a[16], b[16];
      tmem_load16(gate + h * 16, a);
      tmem_load16(up + h * 16, b);
      if (last && h == 3) drained();
      if (!some) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t col = n0 + h * 16 + j * 8;
        float v[8], w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = a[j * 8 + i];
          w[i] = b[j * 8 + i];
        }
        if (bias && col < g.N) {
          add_to<T, 8>(v, bias + col);
          add_to<T, 8>(w, bias + g.N + col);
        }
        f(((h * 2 + j) ^ (lane & 7)) * 16 + lane * 128, v, w);
      }
    }
  };
  if (keep) {
    columns(false, [&](int at, float(&v)[8], float(&w)[8]) {
      *reinterpret_cast<Pack<T, 8>*>(stage + at) = pack_from<T, 8>(v);
      *reinterpret_cast<Pack<T, 8>*>(at_up + at) = pack_from<T, 8>(w);
    });
    if (some) {
      stage_ready();
      __syncwarp();
      if (lane == 0) {
        tma_store(map_gate, stage, static_cast<int>(n0), static_cast<int>(m0));
        store_commit();
        tma_store(map_up, at_up, static_cast<int>(n0), static_cast<int>(m0));
        store_commit();
        stores_read<1>();
      }
      __syncwarp();
    }
  }
  columns(true, [&](int at, float(&v)[8], float(&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value<ACT>(v[i]) * w[i];
    *reinterpret_cast<Pack<T, 8>*>(at_y + at) = pack_from<T, 8>(v);
  });
  if (!some) return;
  turn ^= 1;
  stage_ready();
  __syncwarp();
  if (lane == 0) {
    tma_store(map_y, at_y, static_cast<int>(n0), static_cast<int>(m0));
    store_commit();
  }
}

// The same where rows are not whole vectors: 32 columns of z and of the result at a time are
// turned around in shared memory, so that a warp's lanes hold neighbouring columns.
template <typename T, class Drained>
__device__ __forceinline__ void epilogue_gated_scalar(const MmaArgs& g, unsigned gate, unsigned up,
                                                      int64_t m0, int64_t n0, int lane,
                                                      float* stage, Drained&& drained) {
  const int rows = g.M - m0 < 32 ? (g.M > m0 ? static_cast<int>(g.M - m0) : 0) : 32;
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    float v[32], w[32];
    tmem_load32(gate + c, v);
    tmem_load32(up + c, w);
    if (c == 32) drained();
    gated_bias<T, 32>(g.e, n0 + c, g.N, v, w);
    const int64_t n = n0 + c + lane;
    auto put = [&](float (&f)[32], T* p, int64_t ld) {  // element (m, n) at p[m * ld + n]
#pragma unroll
      for (int i = 0; i < 32; ++i) stage[lane * 33 + i] = f[i];
      __syncwarp();
      if (n < g.N) {
#pragma unroll 4
        for (int r = 0; r < rows; ++r) p[(m0 + r) * ld + n] = from_f32<T>(stage[r * 33 + lane]);
      }
      __syncwarp();
    };
    if (g.e.z) {
      put(v, static_cast<T*>(g.e.z), 2 * g.N);
      put(w, static_cast<T*>(g.e.z) + g.N, 2 * g.N);
    }
    gated_values<32>(g.e, v, w);
    put(v, static_cast<T*>(g.e.y), g.N);
  }
}

// NC consecutive columns n.. of row m of the result, straight from registers.
template <typename T, int NC>
__device__ __forceinline__ void gated_row(const Epilogue& e, bool vec, int64_t m, int64_t n,
                                          int64_t N, float (&gate)[NC], float (&up)[NC]) {
  gated_bias<T, NC>(e, n, N, gate, up);
  T* y = static_cast<T*>(e.y) + m * N + n;
  T* z = e.z ? static_cast<T*>(e.z) + m * 2 * N + n : nullptr;
  if (vec && n + NC <= N) {
    if (z) {
      *reinterpret_cast<Pack<T, NC>*>(z) = pack_from<T, NC>(gate);
      *reinterpret_cast<Pack<T, NC>*>(z + N) = pack_from<T, NC>(up);
    }
    gated_values<NC>(e, gate, up);
    *reinterpret_cast<Pack<T, NC>*>(y) = pack_from<T, NC>(gate);
    return;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (n + i >= N || !z) continue;
    z[i] = from_f32<T>(gate[i]);
    z[N + i] = from_f32<T>(up[i]);
  }
  gated_values<NC>(e, gate, up);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (n + i < N) y[i] = from_f32<T>(gate[i]);
}

// NC consecutive rows (tokens) m.. of column n of the result: lanes hold neighbouring columns.
template <typename T, int NC>
__device__ __forceinline__ void gated_col(const Epilogue& e, int64_t m, int64_t M, int64_t n,
                                          int64_t N, float (&gate)[NC], float (&up)[NC]) {
  const T* bias = static_cast<const T*>(e.bias);
  T* y = static_cast<T*>(e.y);
  T* z = static_cast<T*>(e.z);
  const float bg = bias ? to_f32(bias[n]) : 0.0f, bu = bias ? to_f32(bias[N + n]) : 0.0f;
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (m + i >= M) continue;
      const float a = bias ? gate[i] + bg : gate[i], b = bias ? up[i] + bu : up[i];
      if (z) {
        z[(m + i) * 2 * N + n] = from_f32<T>(a);
        z[((m + i) * 2 + 1) * N + n] = from_f32<T>(b);
      }
      y[(m + i) * N + n] = from_f32<T>(act_value<decltype(act)::value>(a) * b);
    }
  });
}

// -- sums in pieces that are not finite --------------------------------------------

// N values of an operand in pieces: of row i, from k on (a multiple of N; zeros past K).
// Through L2, as the tensor copies: a late launch has not waited when it gets here.
template <bool KC, int N>
__device__ __forceinline__ void piece_values(const __nv_bfloat16* p, int64_t ld, int piece,
                                             int64_t i, int64_t k, int64_t K, float (&f)[N]) {
  const unsigned short* at =
      reinterpret_cast<const unsigned short*>(p) + (KC ? i * ld + k : k * ld + i);
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = 0.0f;
  // each sum exact (eight values at a time where registers matter less)
#pragma unroll(N == 8 ? 3 : 1)
  for (int j = 2; j >= 0; --j) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (KC) {
        if (e % 4) continue;
        const uint2 q = __ldcg(reinterpret_cast<const uint2*>(at + j * piece + e));
        f[e] += __uint_as_float(q.x << 16);
        f[e + 1] += __uint_as_float(q.x & 0xffff0000u);
        f[e + 2] += __uint_as_float(q.y << 16);
        f[e + 3] += __uint_as_float(q.y & 0xffff0000u);
      } else if (k + e < K) {
        f[e] += __uint_as_float(static_cast<unsigned>(__ldcg(at + e * ld + j * piece)) << 16);
      }
    }
  }
}

// t and N more products of row m of A and row n of B.
template <bool A_KC, bool B_KC, int N>
__device__ __forceinline__ float pieces_add(const MmaPieces& o, int64_t m, int64_t n, int64_t k,
                                            float t) {
  float a[N], b[N];
  piece_values<A_KC, N>(o.a, o.lda, o.piece_a, m, k, o.K, a);
  piece_values<B_KC, N>(o.b, o.ldb, o.piece_b, n, k, o.K, b);
#pragma unroll
  for (int e = 0; e < N; ++e) t = fmaf(a[e], b[e], t);
  return t;
}

// A warp's sums of a tile, made again in binary32 where they are not finite: each lane's row m of
// A (-1: none) and `cols` columns, over k in [k0, k1) (multiples of 64, or K).
struct MmaAgain {
  unsigned at;       // tensor memory, the tile's column 0
  int first, far;    // column c of the warp's is first + c % 64 + c / 64 * far
  int cols, half;    // columns from `half` on are of what is gated
  int64_t m, n0;     // of column 0
  int64_t N, gate;   // columns of the result; rows of B from a gate's to its other
  int64_t k0, k1;
};

// A NaN stays one, and is soon known where all of x is NaN.  A few sums of a column are made by
// the whole warp, one after another, many by a lane each.  4096 x 4096 x 4096, forward and
// gradients: one infinity in x and dh 4 and 54 ms, all of them NaN 2.2 and 4 ms, all the same
// infinity 0.7 and 4.7 s (otherwise 0.94 and 2.0 ms).  What this costs the other calls matters
// more: it is a call, of few registers (inlined, or with twice as many loads on their way, the
// gradients' CTAs found no room beside the launch before, 512 x 256 x 512 20.6 us; 19.4 so, 18.7
// without).
template <bool A_KC, bool B_KC>
__device__ __noinline__ void pieces_again(const MmaPieces o, const MmaAgain p) {
  constexpr int N = A_KC && B_KC ? 8 : 4;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < p.cols; ++c) {
    const int col = p.first + c % 64 + c / 64 * p.far;
    const int64_t j = p.n0 + (col < p.half ? col : col - p.half);
    const int64_t n = col < p.half ? j : p.gate + j;
    float v = tmem_load1(p.at + col);
    const bool off = p.m >= 0 && j < p.N && !isfinite(v);
    float t = 0.0f;
    if (off) t = pieces_add<A_KC, B_KC, N>(o, p.m, n, p.k0, t);
    unsigned todo = __ballot_sync(0xffffffffu, off && t == t);
    if (__popc(todo) > 4) {
      if (off)
#pragma unroll 1
        for (int64_t k = p.k0 + N; k < p.k1 && t == t; k += N)
          t = pieces_add<A_KC, B_KC, N>(o, p.m, n, k, t);
      todo = 0;
    }
    if (off) v = t;
#pragma unroll 1
    for (; todo; todo &= todo - 1) {
      const int source = __ffs(todo) - 1;
      const int64_t row = __shfl_sync(0xffffffffu, p.m, source);
      t = 0.0f;
#pragma unroll 1
      for (int64_t k = p.k0; k < p.k1 && !__any_sync(0xffffffffu, t != t); k += 32 * N)
        if (k + lane * N < p.k1) t = pieces_add<A_KC, B_KC, N>(o, row, n, k + lane * N, t);
      t = warp_sum(t);
      if (lane == source) v = t;
    }
    __syncwarp();
    tmem_store1(p.at + col, v);
  }
}

// -- kernel ---------------------------------------------------------------------

// (GATED: map_z is of z's gate columns, map_r of the others; in pieces map_r is the operands.)
template <typename T, int CG, int BN, bool A_KC, bool B_KC, bool SWAP, bool GATED = false,
          typename TO = T>
__global__ void __launch_bounds__(MmaShape<CG, BN, SWAP, GATED, sizeof(TO) == 4>::kThreads,
                                  GATED ? 1 : 0)
linear_mma_kernel(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_y,
                  const __grid_constant__ CUtensorMap map_z,
                  const __grid_constant__ MmaLastMap<!std::is_same<T, TO>::value> map_r,
                  const MmaArgs g) {
  constexpr bool kPieces = !std::is_same<T, TO>::value;
  using S = MmaShape<CG, BN, SWAP, GATED, kPieces>;
  constexpr bool kFull = A_KC && B_KC;  // the gradients' products are stored as they are
  static_assert(!GATED || kFull, "a gate is of the forward product");
  static_assert(!kPieces || !SWAP || GATED, "pieces with few rows are of a gated product");
  // a gate and what it gates lie in different lanes: they meet in shared memory
  constexpr bool kMeet = GATED && SWAP;
  constexpr int kTileM = kMeet ? kMmaRows / 2 : kMmaRows;  // rows and columns of the result
  constexpr int kTileN = GATED && !SWAP ? BN / 2 : BN;
  constexpr int kStages = S::kStages;
  constexpr bool kBf16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
  extern __shared__ unsigned char raw[];
  // the swizzle counts from 1024-byte boundaries
  unsigned char* ring = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  __shared__ alignas(8) unsigned long long full[kStages], empty[kStages], sums[2], drained[2],
      fetched[S::kWarps];
  __shared__ unsigned tmem_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned rank = cluster_rank();
  const bool leader = CG == 1 || rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sums[i], 1);
      mbar_init(&drained[i], S::kWarps * CG);
    }
    for (int i = 0; i < S::kWarps; ++i) mbar_init(&fetched[i], 1);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<CG>(&tmem_slot, S::kTmem);
  tc_fence_before();
  __syncthreads();
  if (CG == 2 || g.splits > 1) cluster_sync();  // the peers' barriers are ready
  tc_fence_after();
  const unsigned tmem = tmem_slot;
  if (!g.late) pdl_wait();
  pdl_trigger();  // after the allocation: a later grid cannot take the columns first

  // this CTA's (pair's) tiles and its part of K (with pieces there may be more parts than slices,
  // which the plan counts three times: the sums of a part without one are zeros)
  const int unit = CG == 2 || g.splits > 1 ? blockIdx.x / cluster_size() : blockIdx.x;
  const int units = CG == 2 || g.splits > 1 ? gridDim.x / cluster_size() : gridDim.x;
  const int tiles = g.tiles_m * g.tiles_n;
  const int part = g.splits > 1 ? rank : 0;
  const int k_lo = static_cast<int>(static_cast<int64_t>(g.kblocks) * part / g.splits);
  const int k_hi = static_cast<int>(static_cast<int64_t>(g.kblocks) * (part + 1) / g.splits);

  // tile t: groups of kMmaGroup row tiles, walked column by column, so that
  // tiles made at the same time share rows and columns of the operands in L2
  auto tile_at = [&](int t, int& tm, int& tn) {
    const int per = kMmaGroup * g.tiles_n;
    const int first = t / per * kMmaGroup;
    const int size = g.tiles_m - first < kMmaGroup ? g.tiles_m - first : kMmaGroup;
    tm = first + t % per % size;
    tn = t % per / size;
  };
  auto give_up = [&](unsigned site) {
    if (atomicCAS(g.status, 0u, kStatusDeviceTimeout) == 0u) atomicExch(g.status + 1, site);
  };

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool alive = true;
      const unsigned full0 = CG == 2 ? peer_addr(&full[0], 0) : smem_addr(&full[0]);
      for (int t = unit; t < tiles && alive && !g.stall; t += units) {
        int tm, tn;
        tile_at(t, tm, tn);
        const int m0 = (tm * CG + (CG == 2 ? static_cast<int>(rank) : 0)) * kTileM;
        const int gate = static_cast<int>(g.gate);  // rows of the weight from a gate's to its other
        const int n0 = GATED && !SWAP
                           ? tn * kTileN + (CG == 2 ? static_cast<int>(rank) * gate : 0)
                           : tn * BN + (CG == 2 ? static_cast<int>(rank) * S::kBRows : 0);
        constexpr int kParts = kPieces ? 3 : 1;
        for (int q = k_lo * kParts; q < k_hi * kParts; ++q, ++it) {
          const int kb = q / kParts;
          const int s = it % kStages;
          if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, wait_limit(g, kSiteEmpty))) {
            give_up(kSiteEmpty);
            alive = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[s], CG * S::kStageBytes);
          unsigned char* a = ring + s * S::kStageBytes;
          unsigned char* b = a + kMmaABytes;
          const unsigned bar = full0 + s * 8;
          const int k = kb * kMmaK;
          int xa = 0, xb = 0;  // along the operands' rows
          if constexpr (kPieces) {  // the second, the first, the third
            const int r = q - kb * kParts, piece = r == 0 ? 1 : r == 1 ? 0 : 2;
            xa = piece * g.piece_a;
            xb = piece * g.piece_b;
          }
          if constexpr (kMeet) {
            tma_load<CG>(a, &map_a, xa + k, m0, bar);
            tma_load<CG>(a + kMmaABytes / 2, &map_a, xa + k, gate + m0, bar);
          } else if constexpr (A_KC) {
            tma_load<CG>(a, &map_a, xa + k, m0, bar);
          } else {
#pragma unroll
            for (int i = 0; i < kMmaRows / 64; ++i)
              tma_load<CG>(a + i * 8192, &map_a, xa + m0 + i * 64, k, bar);
          }
          if constexpr (GATED && !SWAP && CG == 1) {
            tma_load<CG>(b, &map_b, xb + k, n0, bar);
            tma_load<CG>(b + S::kBBytes / 2, &map_b, xb + k, gate + n0, bar);
          } else if constexpr (B_KC) {
            tma_load<CG>(b, &map_b, xb + k, n0, bar);
          } else {
#pragma unroll
            for (int i = 0; i < S::kBRows / 64; ++i)
              tma_load<CG>(b + i * 8192, &map_b, xb + n0 + i * 64, k, bar);
          }
        }
      }
      // Nothing may still be on its way to this CTA's shared memory when it
      // ends: not the last commits' arrivals, and after a timeout no copy.
      const int from = it > kStages ? it - kStages : 0;
      for (int i = from; i < it; ++i) {
        if (alive) mbar_wait(&empty[i % kStages], (i / kStages) & 1, g.limit_ns);
        else if (leader) mbar_wait(&full[i % kStages], (i / kStages) & 1, g.limit_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      constexpr unsigned idesc = mma_idesc(kBf16, A_KC, B_KC, kMmaRows * CG, BN);
      // 16 of k further: 32 bytes along a row, or two groups of eight rows
      constexpr unsigned step_a = (A_KC ? 32 : 2048) >> 4, step_b = (B_KC ? 32 : 2048) >> 4;
      int it = 0, n = 0;
      bool alive = true;
      for (int t = unit; t < tiles && alive; t += units) {
        // a sum over all of this CTA's K, or with pieces over a slice
        for (int kb = k_lo; kb < k_hi && alive; ++n) {
          const int buf = n % S::kBuffers;
          if (!mbar_wait(&drained[buf], ((n / S::kBuffers) & 1) ^ 1, wait_limit(g, kSiteDrained))) {
            give_up(kSiteDrained);
            alive = false;
            break;
          }
          tc_fence_after();
          const unsigned d = tmem + buf * BN;
          unsigned at[3];  // stages
          auto arrived = [&](int i) {
            const int s = (it + i) % kStages;
            at[i] = smem_addr(ring + s * S::kStageBytes);
            alive = mbar_wait(&full[s], ((it + i) / kStages) & 1, g.limit_ns);
            if (!alive) give_up(kSiteFull);
            tc_fence_after();
            return alive;
          };
          auto multiply = [&](unsigned a, unsigned b, bool add) {  // A of one stage, B of another
            const unsigned long long da = smem_desc(a, 8192);
            const unsigned long long db = smem_desc(b + kMmaABytes, 8192);
#pragma unroll
            for (int k = 0; k < kMmaK / 16; ++k)
              mma_f16<CG>(d, da + k * step_a, db + k * step_b, idesc, add || k > 0);
          };
          auto used = [&](int i) {
            if (g.withhold != kSiteEmpty) mma_commit<CG>(&empty[(it + i) % kStages]);
          };
          if constexpr (kPieces) {
            // stages: the second pieces, the first, the third
            if (!arrived(0)) break;
            multiply(at[0], at[0], false);
            if (!arrived(1)) break;
            multiply(at[0], at[1], true);
            multiply(at[1], at[0], true);
            used(0);
            if (!arrived(2)) break;
            multiply(at[1], at[2], true);
            multiply(at[2], at[1], true);
            used(2);
            multiply(at[1], at[1], true);
            used(1);
            it += 3;
            ++kb;
          } else {
            const int first = kb;
            for (; kb < k_hi && arrived(0); ++kb, ++it) {
              multiply(at[0], at[0], kb > first);
              used(0);
            }
          }
          mma_commit<CG>(&sums[buf]);
        }
      }
    }
  } else {
    const int quarter = warp & 3;  // the lanes of tensor memory this warp may read
    const int row = quarter * 32 + lane;
    const int c0 = (warp - 2) / 4 * S::kCols;  // this warp's columns of a tile: c0, kCols of them
    unsigned char* stage = ring + S::kRing + (warp - 2) * S::kStageOut;  // not SWAP
    unsigned phase = 0, turn = 0;
    int n = 0;
    bool alive = true;
    for (int t = unit; t < tiles && alive; t += units, ++n) {
      auto await = [&] {  // a buffer's sums
        alive = warp_wait(&sums[n % S::kBuffers], (n / S::kBuffers) & 1, g.limit_ns);
        if (!alive && lane == 0) give_up(kSiteSums);
        tc_fence_after();
        return alive;
      };
      auto release = [&] {  // they have been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && g.withhold != kSiteDrained) {
          if constexpr (CG == 1) {
            mbar_arrive(&drained[n % S::kBuffers]);
          } else {
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                         :: "r"(peer_addr(&drained[n % S::kBuffers], 0)) : "memory");
          }
        }
      };
      unsigned at = tmem + n % S::kBuffers * BN + (static_cast<unsigned>(quarter * 32) << 16);
      if constexpr (kPieces) {
        // the slices' sums added up, the columns that this warp stores; then back to the last
        // one's place
        constexpr bool kApart = GATED && !SWAP && BN == 256;  // 64 of each half
        auto column = [&](int c) {
          return kApart ? (warp - 2) / 4 * 64 + c % 64 + c / 64 * 128 : c0 + c;
        };
        float total[S::kCols / 16][16] = {};
        for (int kb = k_lo; kb < k_hi; ++kb) {
          if (kb > k_lo) {
            release();
            ++n;
          }
          if (!await()) break;
          at = tmem + n % S::kBuffers * BN + (static_cast<unsigned>(quarter * 32) << 16);
#pragma unroll
          for (int c = 0; c < S::kCols / 16; ++c) {
            float v[16];
            tmem_load16(at + column(16 * c), v);
#pragma unroll
            for (int i = 0; i < 16; ++i) total[c][i] += v[i];
          }
        }
        if (!alive) break;
        float zero[4] = {};  // NaN if a sum is not finite
#pragma unroll
        for (int c = 0; c < S::kCols / 16; ++c) {
#pragma unroll
          for (int i = 0; i < 16; ++i) zero[i % 4] = fmaf(total[c][i], 0.0f, zero[i % 4]);
          tmem_store16(at + column(16 * c), total[c]);
        }
        if (__any_sync(0xffffffffu, (zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.0f)) {
          int tm, tn;
          tile_at(t, tm, tn);
          const int64_t i = static_cast<int64_t>(tm * CG + (CG == 2 ? static_cast<int>(rank) : 0)) *
                                kTileM + (kMeet ? row % kTileM : row);
          const int64_t k1 = static_cast<int64_t>(k_hi) * kMmaK;
          pieces_again<A_KC, B_KC>(
              map_r, {at, column(0), kApart ? 128 : 64, S::kCols, GATED && !SWAP ? kTileN : BN,
                      i >= g.M ? -1 : kMeet && row >= kTileM ? g.gate + i : i,
                      static_cast<int64_t>(tn) * kTileN, g.N, g.gate,
                      static_cast<int64_t>(k_lo) * kMmaK, k1 < map_r.K ? k1 : map_r.K});
        }
      } else if (!await()) {
        break;
      }
      auto drain = [&] { release(); };
      int tm, tn;
      tile_at(t, tm, tn);
      const int64_t m0 =
          static_cast<int64_t>(tm * CG + (CG == 2 ? static_cast<int>(rank) : 0)) * kTileM;
      const int64_t n0 = static_cast<int64_t>(tn) * kTileN;
      const unsigned d = at + c0;
      if (kMeet || g.splits > 1) {
        // to shared memory (every copy and matrix instruction on it is done),
        // a column of 128 rows after another
        float* mine = reinterpret_cast<float*>(ring);
        if constexpr (BN >= 32) {
#pragma unroll
          for (int c = 0; c < S::kCols; c += 32) {
            float v[32];
            tmem_load32(d + c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) mine[(c0 + c + i) * kMmaRows + row] = v[i];
          }
        } else {
          float v[16];
          tmem_load16(d, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[i * kMmaRows + row] = v[i];
        }
        break;  // one tile per cluster
      }
      if constexpr (GATED) {
        if constexpr (!SWAP) {
          const int64_t n = n0 + (warp - 2) / 4 * 64;
          const unsigned first = d - c0 + (warp - 2) / 4 * 64;
          bool stored = false;
          if constexpr (!kPieces) if (g.vec) {
            stored = true;
            with_act(g.e.act, [&](auto act) {
              epilogue_gated<T, decltype(act)::value>(g, &map_y, &map_z, &map_r, first,
                                                      first + BN / 2, m0 + quarter * 32, n, lane,
                                                      stage, turn, drain);
            });
          }
          if (!stored) {
            epilogue_gated_scalar<TO>(g, first, first + BN / 2, m0 + quarter * 32, n, lane,
                                     reinterpret_cast<float*>(stage), drain);
          }
        }
      } else if constexpr (SWAP) {
        const int64_t m = m0 + row;
        if constexpr (BN >= 32) {
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            float v[32];
            tmem_load32(d + c, v);
            if (m < g.M) epilogue_col<TO, 32>(g.e, n0 + c, g.N, m, g.M, v);
            __syncwarp();
          }
        } else {
          float v[16];
          tmem_load16(d, v);
          if (m < g.M) epilogue_col<TO, 16>(g.e, n0, g.N, m, g.M, v);
        }
        drain();
      } else {
        bool stored = false;
        if constexpr (!kPieces) {
          if (g.vec) {
            stored = true;
            bool fetched_all = true;
            auto run = [&](auto act) {
              fetched_all = epilogue_tile<T, S::kCols, kFull, decltype(act)::value>(
                  g, &map_y, &map_z, &map_r, d, m0 + quarter * 32, n0 + c0, lane, stage,
                  &fetched[warp - 2], phase, turn, drain);
            };
            if constexpr (kFull) with_act(g.e.act, run);
            else run(Const<kActNone>());
            if (!fetched_all) {
              if (lane == 0) give_up(kSiteResidual);
              break;
            }
          }
        }
        if (!stored)
          epilogue_tile_scalar<TO, S::kCols, kFull>(g, d, m0 + quarter * 32, n0 + c0, lane,
                                                    reinterpret_cast<float*>(stage), drain);
      }
    }
    if constexpr (!SWAP)
      if (lane == 0) stores_done();
  }
  __syncwarp();

  if (CG == 1 && (kMeet || g.splits > 1)) {
    cluster_sync();
    if constexpr (GATED) {
      if (warp >= 2 && unit < tiles) {
        // this rank's columns of the result, summed over the ranks in order: with SWAP a
        // thread takes one of the tile's 64 features and half of the tokens, otherwise a row
        const int row = (warp & 3) * 32 + lane;
        const int cols = kTileN / g.splits / (SWAP ? 2 : 1);
        const int c0 = static_cast<int>(rank) * (kTileN / g.splits) + (SWAP ? row / 64 * cols : 0);
        const int lead = SWAP ? row % 64 : row;                // the gate's place, and
        const int other = SWAP ? 64 : BN / 2 * kMmaRows;       // the other's from it on
        int tm, tn;
        tile_at(unit, tm, tn);
        const int64_t m = static_cast<int64_t>(tm) * kTileM + lead;
        const int64_t n0 = static_cast<int64_t>(tn) * kTileN;
        unsigned peer[kMaxSplits];
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r)
          peer[r] = peer_addr(reinterpret_cast<const float*>(ring) + lead, r < g.splits ? r : 0);
        auto columns = [&](auto nc) {
          constexpr int NC = decltype(nc)::value;
          for (int c = c0; c < c0 + cols; c += NC) {
            float part[2][kMaxSplits][NC];
#pragma unroll
            for (int r = 0; r < kMaxSplits; ++r) {
              if (r >= g.splits) continue;
#pragma unroll
              for (int i = 0; i < NC; ++i) {
                part[0][r][i] = peer_load(peer[r] + (c + i) * kMmaRows * 4);
                part[1][r][i] = peer_load(peer[r] + ((c + i) * kMmaRows + other) * 4);
              }
            }
            float v[NC] = {}, w[NC] = {};
#pragma unroll
            for (int r = 0; r < kMaxSplits; ++r) {
              if (r >= g.splits) continue;
#pragma unroll
              for (int i = 0; i < NC; ++i) {
                v[i] += part[0][r][i];
                w[i] += part[1][r][i];
              }
            }
            if (m < g.M) {
              if constexpr (SWAP) gated_col<TO, NC>(g.e, n0 + c, g.N, m, g.M, v, w);
              else gated_row<TO, NC>(g.e, g.vec, m, n0 + c, g.N, v, w);
            }
          }
        };
        if (cols % 4 == 0) columns(Const<4>());
        else if (cols % 2 == 0) columns(Const<2>());
        else columns(Const<1>());
      }
    } else if (warp >= 2 && unit < tiles) {
      // this rank's columns (this warp's share of them), summed over the ranks in
      // order
      const int row = (warp & 3) * 32 + lane;
      const int cols = BN / g.splits / (S::kWarps / 4);
      const int c0 = static_cast<int>(rank) * (BN / g.splits) + (warp - 2) / 4 * cols;
      int tm, tn;
      tile_at(unit, tm, tn);
      const int64_t m = static_cast<int64_t>(tm) * kMmaRows + row;
      const int64_t n0 = static_cast<int64_t>(tn) * BN;
      unsigned peer[kMaxSplits];
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        peer[r] = peer_addr(reinterpret_cast<const float*>(ring) + row, r < g.splits ? r : 0);
      auto columns = [&](auto nc) {
        constexpr int NC = decltype(nc)::value;
        for (int c = c0; c < c0 + cols; c += NC) {
          float part[kMaxSplits][NC];
#pragma unroll
          for (int r = 0; r < kMaxSplits; ++r) {
            if (r >= g.splits) continue;
#pragma unroll
            for (int i = 0; i < NC; ++i) part[r][i] = peer_load(peer[r] + (c + i) * kMmaRows * 4);
          }
          float v[NC] = {};
#pragma unroll
          for (int r = 0; r < kMaxSplits; ++r) {
            if (r >= g.splits) continue;
#pragma unroll
            for (int i = 0; i < NC; ++i) v[i] += part[r][i];
          }
          if (m < g.M) {
            if constexpr (SWAP) epilogue_col<TO, NC>(g.e, n0 + c, g.N, m, g.M, v);
            else epilogue_row<TO, NC>(g.e, g.vec, m, n0 + c, g.N, v);
          }
        }
      };
      if constexpr (SWAP) {
        if (cols % 8 == 0) columns(Const<8>());
        else if (cols % 4 == 0) columns(Const<4>());
        else columns(Const<2>());
      } else {
        columns(Const<16 / sizeof(TO)>());
      }
    }
    cluster_sync();  // the peers may still read this CTA's sums
  }
  tc_fence_before();
  if (CG == 2) cluster_sync();  // the pair frees its columns together
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CG>(tmem, S::kTmem);
  }
  if (g.late) pdl_wait();
}

}  // namespace b200norm
