// heads.cuh -- query and key heads on the way to attention: rotation of pairs of
// elements by the token's position, with or without an RMS norm of the head before
// it, and the gradients (sm_103a).
//
// With the pair (a, b) of a head, its frequency f and the token's position p:
//   (a, b) -> (a c - b s, b c + a s),  c = scale cos(p f), s = scale sin(p f);
// the norm before it is u = x r, r = 1 / sqrt(mean(x^2) + eps), a = u gamma.
//
// Bound by HBM: a head is read once and written once.  A row (one head of one token)
// is held by a group of lanes in registers; a lane holds both elements of its pairs, so
// the rotation needs no exchange.  A warp takes an equal share of all tokens' heads, as
// many at a time as it has groups (a step), and makes a token's cosines and sines once
// for all of them.
//
// 16384 tokens of 32 + 8 heads of 128 bf16: rotation 60 us, with the norm 59 (5.7 TB/s, 86% of
// the copy rate; a bare copy by as many resident warps, reads and writes mixed, takes 56 to
// 58), gradient 91, interleaved 87 (5.5 and 5.8 TB/s); one token 2.1, 2.5 and 4.5.
//
// Angles: a frequency is kept as turns per position in units of 2^-64, so that the
// low 64 bits of position * frequency are the angle without its whole turns, exactly:
// positions cost no digits, and no binary64 operation is made per token.
#pragma once

#include "bulk.cuh"
#include "common.cuh"
#include "heads.h"
#include "pair.cuh"

namespace b200norm {

constexpr int kHeadWarps = 8;

struct HeadsArgs {
  HeadsCall c;
  unsigned tokens, seq;
  int units, lanes;
  int pitch;       // angles a warp keeps: whole units
  int steps[2];    // per token: the heads in groups of 32 / lanes
  int parts[2];    // gradient: CTAs of queries and of keys
  bool whole;      // half a unit's pairs are all rotated, or none
  bool full;       // every pair of a head is rotated
};

// Rows on their way to a warp: each lane copies its own accesses to shared memory
// asynchronously and reads them back itself, so that a step waits for copies issued
// stages ago and nothing is exchanged.  (With the next row in registers instead, 16 KB an SM
// were on their way, and 16384 x 40 x 128 bf16 took 117 us; three stages 58.6 and 56 without
// the norm but 61.6 for heads of 256, six 61.)
template <typename T, int VE, int K>
struct HeadRow {
  static constexpr int kStages = 64 * VE * K * sizeof(T) <= 1024 ? 4
                                 : VE * K * sizeof(T) <= 32      ? 3
                                                                 : 2;
  Pack<T, VE> lo[K][32], hi[K][32];  // [lane]
};
constexpr int kHeadStages = 4;  // at most

// Dynamic shared memory: turns per position (8 bytes a pair), gamma widened (queries',
// keys'), each warp's cosines and sines, positions that are on their way with a token's
// first row, and rows.
__host__ __device__ inline int head_table_floats(const HeadsArgs& g) {
  return g.pitch * (2 * (1 + kHeadWarps) + (g.c.norm ? 4 : 0)) + kHeadWarps * kHeadStages * 2;
}
template <typename T, int VE, int K>
size_t head_smem(const HeadsArgs& g, bool gradient) {
  return static_cast<size_t>(head_table_floats(g)) * 4 +
         sizeof(HeadRow<T, VE, K>) * HeadRow<T, VE, K>::kStages * kHeadWarps * (gradient ? 2 : 1);
}

// -- angles -----------------------------------------------------------------------

// Radians per position to turns per position, mod 1, in units of 2^-64.  A frequency that is
// not finite has no angle, at any position: a number that no half turn and more can be (there
// binary64 has steps of 2^-53 turns).
constexpr unsigned long long kNoAngle = (1ull << 63) + 1;
__device__ __forceinline__ unsigned long long phase_step(double radians) {
  constexpr double kInv2Pi = 0.15915494309189535;
  if (!isfinite(radians)) return kNoAngle;
  double t = radians * kInv2Pi;
  t -= floor(t);
  return __double2ull_rz(t * 18446744073709551616.0);
}

// Cosine and sine of `phase` 2^-32 turns: the nearest quarter turn is taken off
// exactly, and on the eighth of a turn that is left to either side (|a| <= pi / 4) the
// Taylor series end below 2.5e-8.
__device__ __forceinline__ void phase_cos_sin(unsigned phase, float& c, float& s) {
  constexpr float kTurn = 1.4629180792671596e-9f;  // 2 pi / 2^32
  const unsigned quarter = (phase + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int>(phase - (quarter << 30))) * kTurn;
  const float q = a * a;
  float sn = fmaf(q, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, 1/7!, 1/5!, 1/3!
  sn = fmaf(sn, q, 8.3333333e-3f);
  sn = fmaf(sn, q, -1.6666667e-1f);
  sn = fmaf(sn * q, a, a);
  float cs = fmaf(q, -2.7557319e-7f, 2.4801587e-5f);  // 1/10!, 1/8!, 1/6!, 1/4!
  cs = fmaf(cs, q, -1.3888889e-3f);
  cs = fmaf(cs, q, 4.1666667e-2f);
  cs = fmaf(cs, q, -0.5f);
  cs = fmaf(cs, q, 1.0f);
  const bool swap = quarter & 1;
  const float x = swap ? sn : cs, y = swap ? cs : sn;
  c = (quarter + 1) & 2 ? -x : x;  // quarters 1 and 2
  s = quarter & 2 ? -y : y;        // quarters 2 and 3
}

// -- rows -------------------------------------------------------------------------

// A row's elements in registers: two at a time, for one instruction on both, where an
// access holds two or more.
template <int VE>
struct HeadVec {
  using V = typename std::conditional<VE == 1, float, float2>::type;
  static constexpr int N = VE == 1 ? 1 : VE / 2;
};

// The first (a) and second (b) elements of a unit's VE pairs, widened, from its accesses lo
// and hi: these themselves, or, interleaved, the even and odd elements of both.
template <typename T, int VE>
__device__ __forceinline__ void unit_widen(const Pack<T, VE>& lo, const Pack<T, VE>& hi,
                                           bool interleaved,
                                           typename HeadVec<VE>::V (&a)[HeadVec<VE>::N],
                                           typename HeadVec<VE>::V (&b)[HeadVec<VE>::N]) {
  if constexpr (VE == 1) {
    a[0] = to_f32(lo.v[0]);
    b[0] = to_f32(hi.v[0]);
  } else if (!interleaved) {
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      a[i] = get2(lo, i);
      b[i] = get2(hi, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      const int j = 2 * i, k = 2 * i + 1, n = VE / 2;  // pairs j and k
      const float2 x = j < n ? get2(lo, j) : get2(hi, j - n);
      const float2 y = k < n ? get2(lo, k) : get2(hi, k - n);
      a[i] = make_float2(x.x, y.x);
      b[i] = make_float2(x.y, y.y);
    }
  }
}

template <typename T, int VE>
__device__ __forceinline__ void unit_narrow(const typename HeadVec<VE>::V (&a)[HeadVec<VE>::N],
                                            const typename HeadVec<VE>::V (&b)[HeadVec<VE>::N],
                                            bool interleaved, Pack<T, VE>& lo, Pack<T, VE>& hi) {
  if constexpr (VE == 1) {
    lo.v[0] = from_f32<T>(a[0]);
    hi.v[0] = from_f32<T>(b[0]);
  } else if (!interleaved) {
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      set2(lo, i, a[i].x, a[i].y);
      set2(hi, i, b[i].x, b[i].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      const int j = 2 * i, k = 2 * i + 1, n = VE / 2;
      if (j < n) set2(lo, j, a[i].x, b[i].x);
      else set2(hi, j - n, a[i].x, b[i].x);
      if (k < n) set2(lo, k, a[i].y, b[i].y);
      else set2(hi, k - n, a[i].y, b[i].y);
    }
  }
}

// VE floats of shared memory, 16 bytes at a time where they are whole.
template <int VE>
__device__ __forceinline__ Pack<float, VE> read_floats(const float* p) {
  Pack<float, VE> v;
  if constexpr (VE <= 2) {
    v = *reinterpret_cast<const Pack<float, VE>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) {
      const float4 f = reinterpret_cast<const float4*>(p)[i];
      v.v[4 * i] = f.x;
      v.v[4 * i + 1] = f.y;
      v.v[4 * i + 2] = f.z;
      v.v[4 * i + 3] = f.w;
    }
  }
  return v;
}

// Where a lane's units lie: accesses lo and hi of the row, VE elements each, such that
// neighbouring lanes' accesses are neighbours in memory.  A unit's VE pairs are, in the half
// layout, elements i of lo and i of hi; interleaved, neighbours inside lo (the first VE / 2
// pairs) and inside hi.
template <int VE, int K>
struct HeadUnits {
  int lo[K], hi[K];    // element of the row, -1: none
  int pa[K], pb[K];    // pair of the first and of the second half of the unit's pairs
};

template <int VE, int K>
__device__ __forceinline__ HeadUnits<VE, K> head_units(const HeadsArgs& g, int sub) {
  HeadUnits<VE, K> u;
  const int half = g.c.interleaved ? 0 : g.c.rot / 2;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int i = sub + k * g.lanes;
    const bool in = i < g.units;
    int lo = i * VE, hi = lo + half;
    u.pa[k] = lo;
    u.pb[k] = lo + VE / 2;
    if (lo >= half) {  // past the half layout's pairs: the row's last part, in two halves
      if (VE == 1 && g.c.interleaved) {
        lo = 2 * i;
        hi = lo + 1;
      } else {
        lo += half;
        hi = lo + (g.units - half / VE) * VE;
        u.pa[k] = lo / 2;
        u.pb[k] = hi / 2;
      }
    }
    u.lo[k] = in ? lo : -1;
    u.hi[k] = in && hi < g.c.size ? hi : -1;
    if (!in) u.pa[k] = u.pb[k] = 0;
  }
  return u;
}

// This lane's accesses of a row to its place of a stage (zeros where it has none).  Two
// bytes alone cannot be copied asynchronously: they are loaded.
template <typename T, int VE>
__device__ __forceinline__ void head_copy(Pack<T, VE>* dst, const T* src, bool in) {
  constexpr int kBytes = sizeof(T) * VE;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(smem_addr(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
  else if constexpr (kBytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                 :: "r"(smem_addr(dst)), "l"(src), "r"(in ? 8 : 0) : "memory");
  else if constexpr (kBytes == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(smem_addr(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
  else
    *dst = in ? ld_stream<T, VE>(src) : Pack<T, VE>{};
}

// A copy of no bytes names an aligned address all the same: `none`, the start of a tensor
// (in lanes without a row p may lie anywhere).
template <typename T, int VE, int K>
__device__ __forceinline__ void head_fetch(HeadRow<T, VE, K>& r, const T* p, const T* none,
                                           bool in, const HeadUnits<VE, K>& u) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const bool l = in && u.lo[k] >= 0, h = in && u.hi[k] >= 0;
    head_copy<T, VE>(&r.lo[k][lane], l ? p + u.lo[k] : none, l);
    head_copy<T, VE>(&r.hi[k][lane], h ? p + u.hi[k] : none, h);
  }
}

__device__ __forceinline__ void fetch_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the latest N groups of this thread have arrived.
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

template <int VE, int K>
struct HeadValues {
  typename HeadVec<VE>::V a[K][HeadVec<VE>::N], b[K][HeadVec<VE>::N];
};

template <typename T, int VE, int K>
__device__ __forceinline__ void head_widen(const HeadRow<T, VE, K>& r, bool interleaved,
                                           HeadValues<VE, K>& v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < K; ++k)
    unit_widen<T, VE>(r.lo[k][lane], r.hi[k][lane], interleaved, v.a[k], v.b[k]);
}

template <typename T, int VE, int K>
__device__ __forceinline__ void head_store(T* p, bool in, bool interleaved,
                                           const HeadUnits<VE, K>& u, const HeadValues<VE, K>& v) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Pack<T, VE> lo, hi;
    unit_narrow<T, VE>(v.a[k], v.b[k], interleaved, lo, hi);
    if (in && u.lo[k] >= 0) st_stream<T, VE>(p + u.lo[k], lo);
    if (in && u.hi[k] >= 0) st_stream<T, VE>(p + u.hi[k], hi);
  }
}

// Sum over the row's lanes (a power of two); fixed steps where LANES says how many.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, int lanes) {
  if constexpr (LANES == 0) {
    return seg_sum(v, lanes);
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
}

// -- what a CTA's rows share --------------------------------------------------------

struct HeadShared {
  unsigned long long* steps;  // [pitch]
  float* gamma;               // [2][2 * pitch]
  float* cosines;             // this warp's [pitch], and its sines behind them
  long long* position;        // this warp's [stage]
};

__device__ __forceinline__ HeadShared head_shared(const HeadsArgs& g, unsigned char* raw) {
  HeadShared sh;
  sh.steps = reinterpret_cast<unsigned long long*>(raw);
  sh.gamma = reinterpret_cast<float*>(sh.steps + g.pitch);
  float* tables = sh.gamma + (g.c.norm ? 4 * g.pitch : 0);
  sh.cosines = tables + (threadIdx.x >> 5) * 2 * g.pitch;
  sh.position = reinterpret_cast<long long*>(tables + kHeadWarps * 2 * g.pitch) +
                (threadIdx.x >> 5) * kHeadStages;
  return sh;
}

__device__ __forceinline__ float head_gamma_at(const HeadsArgs& g, int n, int j) {
  const void* p = g.c.set[n].gamma;
  if (!p || j >= g.c.size || g.c.set[n].heads == 0) return 1.0f;
  return g.c.m == DType::F32   ? static_cast<const float*>(p)[j]
         : g.c.m == DType::F16 ? to_f32(static_cast<const __half*>(p)[j])
                               : to_f32(static_cast<const __nv_bfloat16*>(p)[j]);
}

__device__ __forceinline__ void head_fill(const HeadsArgs& g, const HeadShared& sh) {
  for (int i = threadIdx.x; i < g.c.rot / 2; i += blockDim.x)
    sh.steps[i] = phase_step(__ldg(g.c.inv_freq + i));
  if (g.c.norm)
    for (int i = threadIdx.x; i < 4 * g.pitch; i += blockDim.x) {
      const int n = i >= 2 * g.pitch;
      sh.gamma[i] = head_gamma_at(g, n, i - n * 2 * g.pitch);
    }
  __syncthreads();
}

// A token's position on its way to a stage (lane 0 copies it, the warp reads it).
__device__ __forceinline__ void head_fetch_position(const HeadsArgs& g, const HeadShared& sh,
                                                    int stage, unsigned b, unsigned t) {
  if (g.c.rot == 0 || (threadIdx.x & 31) != 0) return;
  const int64_t at = b * g.c.pos_batch + t * g.c.pos_token;
  const unsigned dst = smem_addr(sh.position + stage);
  if (g.c.pos64)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                 :: "r"(dst), "l"(static_cast<const long long*>(g.c.positions) + at) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                 :: "r"(dst), "l"(static_cast<const int*>(g.c.positions) + at) : "memory");
}

// This warp's token: scaled cosines, and sines of the sign wanted; 1 and 0 past the pairs.
__device__ __forceinline__ void head_angles(const HeadsArgs& g, const HeadShared& sh, int stage,
                                            float sine) {
  __syncwarp();  // the position is there for all lanes; the angles before are no longer read
  const long long p =
      g.c.pos64 ? sh.position[stage] : *reinterpret_cast<const int*>(sh.position + stage);
  for (int n = threadIdx.x & 31; n < g.pitch; n += 32) {
    float c = 1.0f, s = 0.0f;
    if (n < g.c.rot / 2) {
      const unsigned long long step = sh.steps[n];
      const unsigned long long phase = static_cast<unsigned long long>(p) * step;
      phase_cos_sin(static_cast<unsigned>(phase >> 32), c, s);
      if (step == kNoAngle) c = s = __int_as_float(0x7fffffff);
      c *= g.c.scale;
      s *= sine;
    }
    sh.cosines[n] = c;
    sh.cosines[g.pitch + n] = s;
  }
  __syncwarp();
}

// A warp's share: `left` steps on end of all tokens' steps, the same for every warp but for
// one; the first is step i of token t of sequence b.
struct HeadShare {
  unsigned b, t;
  int i, left;
};

__device__ __forceinline__ HeadShare head_share(const HeadsArgs& g, int steps, int64_t warp,
                                                int64_t warps) {
  const unsigned long long all = static_cast<unsigned long long>(g.tokens) * steps;
  const unsigned long long lo = all * warp / warps, hi = all * (warp + 1) / warps;
  HeadShare s;
  const unsigned token = steps ? static_cast<unsigned>(lo / steps) : 0;
  s.i = static_cast<int>(lo - static_cast<unsigned long long>(token) * steps);
  s.left = static_cast<int>(hi - lo);
  s.b = token / g.seq;
  s.t = token - s.b * g.seq;
  return s;
}

// To the next token, `done` steps on.
__device__ __forceinline__ void head_next(const HeadsArgs& g, HeadShare& s, int done) {
  s.left -= done;
  s.i = 0;
  if (++s.t == g.seq) {
    s.t = 0;
    ++s.b;
  }
}

__device__ __forceinline__ int head_end(const HeadShare& s, int steps) {
  return s.left < steps - s.i ? s.i + s.left : steps;
}

// FORM 1 and 2: all of a head is rotated, in the half layout or interleaved; 0: known at run
// time (branches on it inside the gradient's step cost a tenth: they keep its instructions
// in order).
template <int FORM>
__device__ __forceinline__ bool is_interleaved(const HeadsArgs& g) {
  return FORM == 0 ? g.c.interleaved : FORM == 2;
}

// gamma of a unit's pairs.
template <int VE, int K>
__device__ __forceinline__ void unit_gamma(const float* gamma, const HeadUnits<VE, K>& u, int k,
                                           bool interleaved,
                                           typename HeadVec<VE>::V (&a)[HeadVec<VE>::N],
                                           typename HeadVec<VE>::V (&b)[HeadVec<VE>::N]) {
  // (a unit that is not there has values of 0 and is not stored: gamma's first element will do,
  // which if not finite makes the row's sums so anyway)
  unit_widen<float, VE>(read_floats<VE>(gamma + (u.lo[k] >= 0 ? u.lo[k] : 0)),
                        read_floats<VE>(gamma + (u.hi[k] >= 0 ? u.hi[k] : 0)), interleaved, a, b);
}

// Cosines and sines of a unit's pairs.
template <int VE, int K>
__device__ __forceinline__ void unit_angles(const float* p, const HeadUnits<VE, K>& u, int k,
                                            typename HeadVec<VE>::V (&v)[HeadVec<VE>::N]) {
  if constexpr (VE == 1) {
    v[0] = p[u.pa[k]];
  } else {
    const Pack<float, VE / 2> a = read_floats<VE / 2>(p + u.pa[k]);
    const Pack<float, VE / 2> b = read_floats<VE / 2>(p + u.pb[k]);
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
      const int j = 2 * i, k2 = 2 * i + 1, n = VE / 2;
      v[i] = make_float2(j < n ? a.v[j] : b.v[j - n], k2 < n ? a.v[k2] : b.v[k2 - n]);
    }
  }
}

// (a, b) -> (a ca + b sa, b cb + a sb), what a pair of the rotation becomes; one past the
// pairs (a ca, b cb): an infinity must not reach the neighbour through a factor of zero.
template <int FORM, int VE, int K, typename V, int N>
__device__ __forceinline__ void unit_turn(const HeadsArgs& g, const HeadUnits<VE, K>& u, int k,
                                          V (&a)[N], V (&b)[N], const V (&ca)[N],
                                          const V (&sa)[N], const V (&cb)[N], const V (&sb)[N]) {
  const int left_a = g.c.rot / 2 - u.pa[k], left_b = g.c.rot / 2 - u.pb[k];
  V x[N], y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = a[i];
    y[i] = b[i];
    a[i] = mul2(a[i], ca[i]);
    b[i] = mul2(b[i], cb[i]);
  }
  if (FORM != 0 || g.full) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = fma2(y[i], sa[i], a[i]);
      b[i] = fma2(x[i], sb[i], b[i]);
    }
    return;
  }
  if (VE != 2 && g.whole) {
    if (left_a > 0) {
#pragma unroll
      for (int i = 0; i < (N + 1) / 2; ++i) {
        a[i] = fma2(y[i], sa[i], a[i]);
        b[i] = fma2(x[i], sb[i], b[i]);
      }
    }
    if (left_b > 0) {
#pragma unroll
      for (int i = (N + 1) / 2; i < N; ++i) {
        a[i] = fma2(y[i], sa[i], a[i]);
        b[i] = fma2(x[i], sb[i], b[i]);
      }
    }
    return;
  }
  if constexpr (VE > 1) {
    auto turns = [&](int i) { return i < VE / 2 ? i < left_a : i - VE / 2 < left_b; };
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (turns(2 * i)) {
        a[i].x = fmaf(y[i].x, sa[i].x, a[i].x);
        b[i].x = fmaf(x[i].x, sb[i].x, b[i].x);
      }
      if (turns(2 * i + 1)) {
        a[i].y = fmaf(y[i].y, sa[i].y, a[i].y);
        b[i].y = fmaf(x[i].y, sb[i].y, b[i].y);
      }
    }
  }
}

// -- forward ----------------------------------------------------------------------

// What multiplies a lane's pairs: gamma and the angles in one.
template <int VE, int K>
struct HeadFactors {
  using V = typename HeadVec<VE>::V;
  static constexpr int N = HeadVec<VE>::N;
  V ca[K][N], sa[K][N], cb[K][N], sb[K][N];
};

template <int FORM, int VE, int K, bool NORM>
__device__ __forceinline__ void head_factors(const HeadsArgs& g, const HeadShared& sh,
                                             const float* gamma, const HeadUnits<VE, K>& u,
                                             HeadFactors<VE, K>& f) {
  using V = typename HeadVec<VE>::V;
  constexpr int N = HeadVec<VE>::N;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    V c[N], s[N], ga[N], gb[N];
    unit_angles<VE, K>(sh.cosines, u, k, c);
    unit_angles<VE, K>(sh.cosines + g.pitch, u, k, s);
    if constexpr (NORM) unit_gamma<VE, K>(gamma, u, k, is_interleaved<FORM>(g), ga, gb);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (!NORM) ga[i] = gb[i] = every<V>(1.0f);
      f.ca[k][i] = mul2(ga[i], c[i]);
      f.sa[k][i] = mul2(mul2(gb[i], s[i]), every<V>(-1.0f));
      f.cb[k][i] = mul2(gb[i], c[i]);
      f.sb[k][i] = mul2(ga[i], s[i]);
    }
  }
}

// What a warp fetches next: step i of its share, a row of one tensor for each group of
// lanes.  `p` is this lane's row.
template <typename T>
struct HeadCursor {
  HeadShare at;
  int end;         // of the token's steps
  const T* p;
  int64_t step;    // elements from a step's row to the next
  int left;        // this lane's rows from here on, of the tensor
  bool fresh;      // a token's first row: its position comes with it
};

template <typename T, int VE, int K, int LANES, int FORM, bool NORM>
__global__ void __launch_bounds__(32 * kHeadWarps) heads_kernel(const HeadsArgs g) {
  using V = typename HeadVec<VE>::V;
  constexpr int N = HeadVec<VE>::N, S = HeadRow<T, VE, K>::kStages;
  extern __shared__ __align__(16) unsigned char raw[];
  const HeadShared sh = head_shared(g, raw);
  HeadRow<T, VE, K>* ring = reinterpret_cast<HeadRow<T, VE, K>*>(raw + head_table_floats(g) * 4) +
                            (threadIdx.x >> 5) * S;
  const int lanes = LANES ? LANES : g.lanes;
  const int lane = threadIdx.x & 31;
  const int sub = lane & (lanes - 1), row = lane / lanes, rows = 32 / lanes;
  const HeadUnits<VE, K> u = head_units<VE, K>(g, sub);
  const int steps = g.steps[0] + g.steps[1];
  const bool inter = is_interleaved<FORM>(g);
  const float inv_size = 1.0f / static_cast<float>(g.c.size);
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kHeadWarps + (threadIdx.x >> 5);
  HeadShare at = head_share(g, steps, me, static_cast<int64_t>(gridDim.x) * kHeadWarps);
  pdl_wait();
  pdl_trigger();

  // what is fetched, some steps ahead of what is worked on
  const T* none = static_cast<const T*>(g.c.set[g.c.set[0].heads ? 0 : 1].x);
  HeadCursor<T> c;
  c.at = at;
  auto seek = [&] {  // to step i of the token: queries first, then keys
    const int n = c.at.i >= g.steps[0];
    const HeadSet& set = g.c.set[n];
    const int64_t h = static_cast<int64_t>(c.at.i - (n ? g.steps[0] : 0)) * rows + row;
    c.p = static_cast<const T*>(set.x) + c.at.b * set.xs.batch + c.at.t * set.xs.token +
          h * set.xs.head;
    c.step = rows * set.xs.head;
    c.left = static_cast<int>(set.heads - h);
  };
  auto open = [&] {
    c.end = head_end(c.at, steps);
    c.fresh = true;
    if (c.at.left > 0) seek();
  };
  auto fetch = [&](int stage) {
    if (c.at.left > 0) {
      head_fetch<T, VE, K>(ring[stage], c.p, none, c.left > 0, u);
      if (c.fresh) head_fetch_position(g, sh, stage, c.at.b, c.at.t);
      c.fresh = false;
      --c.at.left;
      if (++c.at.i == c.end) {
        head_next(g, c.at, 0);
        open();
      } else if (c.at.i == g.steps[0]) {
        seek();
      } else {
        c.p += c.step;
        c.left -= rows;
      }
    }
    fetch_commit();
  };
  open();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i);
  head_fill(g, sh);
  int stage = 0;
  while (at.left > 0) {
    fetch_wait<S - 2>();
    head_angles(g, sh, stage, g.c.inverse ? -g.c.scale : g.c.scale);
    const int begin = at.i, end = head_end(at, steps);
#pragma unroll 1
    for (int n = 0; n < 2; ++n) {
      const HeadSet& set = g.c.set[n];
      const int off = n ? g.steps[0] : 0;
      const int first = begin > off ? begin - off : 0;
      const int last = end - off < g.steps[n] ? end - off : g.steps[n];
      if (first >= last) continue;
      HeadFactors<VE, K> f;
      head_factors<FORM, VE, K, NORM>(g, sh, sh.gamma + (n ? 2 * g.pitch : 0), u, f);
      const int64_t h = static_cast<int64_t>(first) * rows + row;
      T* y = static_cast<T*>(set.y) + at.b * set.ys.batch + at.t * set.ys.token + h * set.ys.head;
      const int64_t step = rows * set.ys.head;
      int left = static_cast<int>(set.heads - h);
#pragma unroll 1
      for (int i = first; i < last; ++i, y += step, left -= rows) {
        fetch_wait<S - 2>();
        HeadValues<VE, K> x;
        head_widen<T, VE, K>(ring[stage], inter, x);
        float r = 1.0f;
        if constexpr (NORM) {
          V sa = every<V>(0.0f), sb = every<V>(0.0f);
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
              sa = fma2(x.a[k][e], x.a[k][e], sa);
              sb = fma2(x.b[k][e], x.b[k][e], sb);
            }
          r = rsqrtf(row_sum<LANES>(total(add2(sa, sb)), lanes) * inv_size + g.c.eps);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
          unit_turn<FORM, VE, K>(g, u, k, x.a[k], x.b[k], f.ca[k], f.sa[k], f.cb[k], f.sb[k]);
        if constexpr (NORM) {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) {
              x.a[k][e] = mul2(x.a[k][e], every<V>(r));
              x.b[k][e] = mul2(x.b[k][e], every<V>(r));
            }
        }
        head_store<T, VE, K>(y, left > 0, inter, u, x);
        // into the stage before this one, whose values have all been used
        fetch(stage == 0 ? S - 1 : stage - 1);
        stage = stage + 1 == S ? 0 : stage + 1;
      }
    }
    head_next(g, at, end - begin);
  }
  fetch_wait<0>();
}

// -- gradient ---------------------------------------------------------------------

// With da = the rotation transposed of dy and g = da gamma:
//   dx = r (g - u mean(g u)) = r g - x r^3 mean(g x),  dgamma = sum over rows of da u.
// The first parts[0] CTAs take the queries, the others the keys; each keeps its
// columns' sums in registers over all its rows and stores them as one part.  What bounds it
// next to HBM is the latency of a step's arithmetic: two CTAs of 128 registers fit on an SM.
template <typename T, int VE, int K, int LANES, int FORM>
__global__ void __launch_bounds__(32 * kHeadWarps, 2 * VE * K <= 16 ? 2 : 1)
heads_grad_kernel(const HeadsArgs g) {
  using V = typename HeadVec<VE>::V;
  constexpr int N = HeadVec<VE>::N, S = HeadRow<T, VE, K>::kStages;
  extern __shared__ __align__(16) unsigned char raw[];
  const HeadShared sh = head_shared(g, raw);
  HeadRow<T, VE, K>* ring = reinterpret_cast<HeadRow<T, VE, K>*>(raw + head_table_floats(g) * 4) +
                            (threadIdx.x >> 5) * 2 * S;
  const int lanes = LANES ? LANES : g.lanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (lanes - 1), row = lane / lanes, rows = 32 / lanes;
  const int n = blockIdx.x >= static_cast<unsigned>(g.parts[0]);
  const HeadSet& set = g.c.set[n];
  const unsigned part = blockIdx.x - (n ? g.parts[0] : 0);
  const HeadUnits<VE, K> u = head_units<VE, K>(g, sub);
  const float inv_size = 1.0f / static_cast<float>(g.c.size);
  const int steps = g.steps[n];
  const bool inter = is_interleaved<FORM>(g);
  HeadShare at = head_share(g, steps, static_cast<int64_t>(part) * kHeadWarps + warp,
                            static_cast<int64_t>(g.parts[n]) * kHeadWarps);
  pdl_wait();
  pdl_trigger();

  // what is fetched, some steps ahead of what is worked on
  const T* none = static_cast<const T*>(set.x);
  HeadCursor<T> c;
  const T* pd = nullptr;
  const int64_t step_d = rows * set.dys.head, step_y = rows * set.ys.head;
  c.step = rows * set.xs.head;
  c.at = at;
  auto open = [&] {
    c.end = head_end(c.at, steps);
    c.fresh = true;
    if (c.at.left <= 0) return;
    const int64_t h = static_cast<int64_t>(c.at.i) * rows + row;
    c.p = static_cast<const T*>(set.x) + c.at.b * set.xs.batch + c.at.t * set.xs.token +
          h * set.xs.head;
    pd = static_cast<const T*>(set.dy) + c.at.b * set.dys.batch + c.at.t * set.dys.token +
         h * set.dys.head;
    c.left = static_cast<int>(set.heads - h);
  };
  auto fetch = [&](int stage) {
    if (c.at.left > 0) {
      head_fetch<T, VE, K>(ring[2 * stage], c.p, none, c.left > 0, u);
      head_fetch<T, VE, K>(ring[2 * stage + 1], pd, none, c.left > 0, u);
      if (c.fresh) head_fetch_position(g, sh, stage, c.at.b, c.at.t);
      c.fresh = false;
      --c.at.left;
      if (++c.at.i == c.end) {
        head_next(g, c.at, 0);
        open();
      } else {
        c.p += c.step;
        pd += step_d;
        c.left -= rows;
      }
    }
    fetch_commit();
  };
  open();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i);
  head_fill(g, sh);
  int stage = 0;
  V da[K][N], db[K][N];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < N; ++e) da[k][e] = db[k][e] = every<V>(0.0f);
  while (at.left > 0) {
    fetch_wait<S - 2>();
    head_angles(g, sh, stage, g.c.scale);
    const int first = at.i, last = head_end(at, steps);
    const int64_t h = static_cast<int64_t>(first) * rows + row;
    T* y = static_cast<T*>(set.y) + at.b * set.ys.batch + at.t * set.ys.token + h * set.ys.head;
    int left = static_cast<int>(set.heads - h);
#pragma unroll 1
    for (int i = first; i < last; ++i, y += step_y, left -= rows) {
      fetch_wait<S - 2>();
      HeadValues<VE, K> x, d;
      head_widen<T, VE, K>(ring[2 * stage], inter, x);
      head_widen<T, VE, K>(ring[2 * stage + 1], inter, d);
      V sa = every<V>(0.0f), sb = every<V>(0.0f), ta = every<V>(0.0f), tb = every<V>(0.0f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        // turned back; angles and gamma come from shared memory every time: kept in
        // registers they took 40 of them, and spilled
        V c[N], s[N], t[N], ga[N], gb[N];
        unit_angles<VE, K>(sh.cosines, u, k, c);
        unit_angles<VE, K>(sh.cosines + g.pitch, u, k, s);
#pragma unroll
        for (int e = 0; e < N; ++e) t[e] = mul2(s[e], every<V>(-1.0f));
        unit_turn<FORM, VE, K>(g, u, k, d.a[k], d.b[k], c, s, c, t);
        unit_gamma<VE, K>(sh.gamma + n * 2 * g.pitch, u, k, inter, ga, gb);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          sa = fma2(x.a[k][e], x.a[k][e], sa);
          sb = fma2(x.b[k][e], x.b[k][e], sb);
          ta = fma2(mul2(d.a[k][e], ga[e]), x.a[k][e], ta);
          tb = fma2(mul2(d.b[k][e], gb[e]), x.b[k][e], tb);
        }
      }
      // (lanes without a row here hold zeros, and r would be infinite for eps 0)
      const bool in = left > 0;
      const float length = row_sum<LANES>(total(add2(sa, sb)), lanes) * inv_size + g.c.eps;
      const float r = in ? rsqrtf(length) : 0.0f;
      const float m = row_sum<LANES>(total(add2(ta, tb)), lanes) * inv_size * r * r;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        V ga[N], gb[N];
        unit_gamma<VE, K>(sh.gamma + n * 2 * g.pitch, u, k, inter, ga, gb);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const V ua = mul2(x.a[k][e], every<V>(r)), ub = mul2(x.b[k][e], every<V>(r));
          da[k][e] = fma2(d.a[k][e], ua, da[k][e]);
          db[k][e] = fma2(d.b[k][e], ub, db[k][e]);
          d.a[k][e] = mul2(mul2(d.a[k][e], ga[e]), every<V>(r));
          d.b[k][e] = mul2(mul2(d.b[k][e], gb[e]), every<V>(r));
          d.a[k][e] = fma2(ua, every<V>(-m), d.a[k][e]);
          d.b[k][e] = fma2(ub, every<V>(-m), d.b[k][e]);
        }
      }
      if (set.y) head_store<T, VE, K>(y, in, inter, u, d);
      // into the stage before this one, whose values have all been used
      fetch(stage == 0 ? S - 1 : stage - 1);
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    head_next(g, at, last - first);
  }
  fetch_wait<0>();
  if (!set.dgamma) return;
  // the groups of a warp, then the warps in order, through the shared memory that held
  // the angles and gammas
  float* red = reinterpret_cast<float*>(raw);  // [kHeadWarps][2 * pitch]
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Pack<float, VE> lo, hi;
    unit_narrow<float, VE>(da[k], db[k], inter, lo, hi);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      for (int o = lanes; o < 32; o <<= 1) {
        lo.v[e] += __shfl_xor_sync(0xffffffffu, lo.v[e], o);
        hi.v[e] += __shfl_xor_sync(0xffffffffu, hi.v[e], o);
      }
      if (row == 0) {
        if (u.lo[k] >= 0) red[warp * 2 * g.pitch + u.lo[k] + e] = lo.v[e];
        if (u.hi[k] >= 0) red[warp * 2 * g.pitch + u.hi[k] + e] = hi.v[e];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.c.size; i += blockDim.x) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kHeadWarps; ++w) t += red[w * 2 * g.pitch + i];
    g.c.part[static_cast<int64_t>(blockIdx.x) * g.c.size + i] = t;
  }
}

// The parts added in a fixed order: a CTA takes 32 columns of a tensor's, its 32 warps
// every 32nd part each, then the warps' sums are added.
template <typename M>
__global__ void __launch_bounds__(1024) heads_dgamma_kernel(const float* part, M* dq, M* dk,
                                                            int size, int parts_q, int parts_k) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool keys = blockIdx.y != 0;
  M* out = keys ? dk : dq;
  if (!out) return;
  const int parts = keys ? parts_k : parts_q;
  const float* p = part + (keys ? static_cast<int64_t>(parts_q) * size : 0);
  float t = 0.0f;
  if (col < size) {
#pragma unroll 4
    for (int i = warp; i < parts; i += 32) t += p[static_cast<int64_t>(i) * size + col];
  }
  red[warp][lane] = t;
  __syncthreads();
  if (warp != 0 || col >= size) return;
  t = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) t += red[w][lane];
  out[col] = from_f32<M>(t);
}

}  // namespace b200norm
