// linear.h -- host-side interface between the C ABI and the kernels of the
// linear operator (y = act(x W^T + b) + residual) and its gradients.
#pragma once

#include "launch.h"

namespace b200norm {

// Activation codes of the ABI.
enum Activation { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4 };
constexpr int kActivations = 5;

// One matrix product C[m, n] = sum_k A[m, k] * B[n, k].  An operand is stored
// with k contiguous (element (i, k) at p[i * ld + k]) or with i contiguous
// (p[k * ld + i]).
struct Operand {
  const void* p;
  int64_t ld;
  bool k_contiguous;
};

// What happens to C before it is stored (dense, row-major, N columns):
// z = C + bias[n]; y = act(z) + residual[m, n].
struct Epilogue {
  const void* bias;      // null: none
  const void* residual;  // null: none
  void* y;
  void* z;               // null: not stored
  int act;
};

// How a product is tiled: CTAs per tile (cg), columns per tile (bn), parts of K
// (a cluster each), and whether the result's columns fill the lanes (swap).
struct MmaPlan {
  int cg, bn, splits;
  bool swap;
};

struct Product {
  Operand a, b;
  int64_t M, N, K;
  Epilogue epi;
  DType t;
  MmaPlan forced;  // by a test (cg 0: automatic)
  // B has 2 N rows, a gate's and what it gates; C[m, n] = act(z[m, n]) * z[m, N + n] with
  // z = A B^T + bias (M x 2 N); no residual
  bool gated = false;
  // Both operands are three bfloat16 pieces of float32 values, this many elements apart in a
  // row (a multiple of 64; where k is contiguous, the rest of a piece is zeros); t is F32.
  // (0: operands of type t.)
  int64_t piece_a = 0, piece_b = 0;
  // The launch before this one is a product of the same call, of whose result nothing here is
  // needed: the tensor-core kernels run beside it.
  bool late = false;
  int* ctas = nullptr;  // receives how many CTAs a tensor-core product was launched with
};

cudaError_t launch_product(const Product& p, cudaStream_t stream);
cudaError_t launch_plain_f32(const Product& p, cudaStream_t stream);

// The tensor-core kernels (16-bit types) -----------------------------------------

// What they need of an operand: 16-byte aligned rows at a 16-byte aligned place.
inline bool mma_operand_ok(const Operand& o, DType t) {
  return t != DType::F32 && o.ld % 8 == 0 && reinterpret_cast<uintptr_t>(o.p) % 16 == 0;
}

MmaPlan plan_mma(int64_t M, int64_t N, int64_t K, bool b_kc, bool gated, bool pieces, int sms);
cudaError_t launch_mma(const Product& p, cudaStream_t stream);
template <typename T>
cudaError_t launch_mma_t(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                         cudaStream_t stream);

cudaError_t launch_mma_f32(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                           cudaStream_t stream);

// Whether a forced plan has a kernel for the product.
bool mma_plan_ok(const MmaPlan& plan, int64_t M, int64_t K, bool a_kc, bool b_kc, bool gated);

// Two words per device: a b200norm_status recorded by a wait that gave up, and
// its site (nullptr if they cannot be resolved).
unsigned* linear_status_words();
// A test's limit for the waits of launches that copy nothing (0: normal ones).
unsigned long long linear_stall_limit_ns();
void set_linear_stall(unsigned long long limit_ns);
// A test's site whose event is left out, and how long its wait lasts (site 0: none;
// false: not a site that can be).
struct LinearWithhold {
  unsigned site, limit_ns;
};
LinearWithhold linear_withhold();
bool set_linear_withhold(unsigned site, unsigned limit_ns);

// dz = round_T(dy * act'(z)) with rows `ldz` apart (null: not stored), and the
// column sums of dy * act'(z) (null: not wanted) through `part`.
struct LinearDzCall {
  const void* dy;
  const void* z;       // null when act is kActNone
  void* dz;
  int64_t ldz;
  void* db;
  float* part;         // [linear_db_parts(rows, out)][out]
  int64_t rows, out;
  int act;
  DType t;
  int64_t piece = 0;   // gated float32: dz as three bfloat16 pieces, this many elements apart
};
// Parts of the column sums: enough CTAs to fill the GPU (a CTA has 256 columns of
// a 16-bit type), at least 32 rows in each.
inline int linear_db_parts(int64_t rows, int64_t out) {
  int64_t p = (152 * 8 * 256 + out - 1) / out;
  const int64_t most = (rows + 31) / 32;
  if (p > most) p = most;
  if (p > 1024) p = 1024;
  return static_cast<int>(p < 1 ? 1 : p);
}
// The same of a gated call: about four CTAs of 256 threads (a thread has 16 bytes of a row)
// for each SM, four rows or more in each part.
constexpr int kGatedDzThreads = 256;
inline int gated_db_parts(int64_t rows, int64_t out, DType t) {
  const int64_t cols = kGatedDzThreads * (t == DType::F32 ? 4 : 8);
  int64_t p = 152 * 4 / ((out + cols - 1) / cols);
  const int64_t most = (rows + 3) / 4;
  if (p > most) p = most;
  if (p > 1024) p = 1024;
  return static_cast<int>(p < 1 ? 1 : p);
}
// Gated gradients of so few rows read the weight and write its gradient in one launch; dx comes
// in parts of the features, enough for two CTAs (of 256 columns, or 128) on each SM and 16
// features or more in each.
// (Four rows, float32 up to eight; of a 16-bit type up to eight with 2^25 products of a half:
// 8 x 768 x 768 (rows, in, out) bf16 7.8 us, 15.0 on the tensor cores, 8 x 4096 x 4096 48.5 and
// 45.4, 4 x 4096 x 4096 29.8 and 49.6.)
inline bool gated_few(int64_t rows, int64_t in, int64_t out, DType t) {
  return rows > 0 && (rows <= 4 || (rows <= 8 && (t == DType::F32 ||
                                                  rows * in * out <= int64_t{1} << 25)));
}
inline int gated_few_parts(int64_t rows, int64_t in, int64_t out, DType t) {
  const int64_t cols = t == DType::F32 || rows > 4 ? 128 : 256;
  int64_t p = 152 * 2 / ((in + cols - 1) / cols);
  const int64_t most = (out + 15) / 16;
  if (p > most) p = most;
  return static_cast<int>(p < 1 ? 1 : p);
}
// gated: `out` columns of the result, z and dz with twice as many.
cudaError_t launch_linear_dz(const LinearDzCall& c, bool gated, cudaStream_t stream);
// Then the parts of the column sums into db (nothing without it); late: the launch before is a
// product behind the former.
cudaError_t launch_linear_db(const LinearDzCall& c, bool gated, bool late, cudaStream_t stream);

// gated: y = act(gate) * up of out columns each; weight, bias, z (and db, dw) of both.
struct LinearCall {
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  void* y;
  void* z;
  int64_t rows, in, out;
  DType t;
  int act;
  void* workspace;
  MmaPlan forced;
  bool gated = false;
};

struct LinearGradCall {
  const void* dy;
  const void* x;
  const void* w;
  const void* z;
  void* dx;
  void* dw;
  void* db;
  int64_t rows, in, out;
  DType t;
  int act;
  void* workspace;
  MmaPlan forced;
  bool gated = false;
};

// What a call keeps in its workspace: offsets, and the bytes in all.  Operands
// of 16-bit types whose rows do not start on 16-byte boundaries are copied to
// rows that do (`pitch` elements apart), except for few rows of x, where the
// weight is read once and not worth a copy.
// Whether the row kernel takes a product.  float32: up to four rows (4 x 4096 x 4096
// 35 us, 60 as a tiled product).  Unaligned 16-bit operands: one row (1 x 4097 x 4099
// 14 us), or up to 2 M products (2 x 4097 x 4099 takes 21 us by way of aligned
// copies).  Aligned ones: up to four rows and 4 M products (1 x 768 x 768 2.1 us
// against 4.7 on the tensor cores, 4 x 768 x 768 4.1 against 4.7, 1 x 1024 x 4096 2.8
// against 5.7, but 1 x 4096 x 4096 11.2 against 10.1, 4 x 4096 x 4096 35 against 10).
inline bool few_rows(int64_t M, int64_t N, int64_t K, DType t, bool aligned) {
  if (M > 4) return false;
  if (t == DType::F32) return true;
  const int64_t products = M * N * K;
  return aligned ? products <= int64_t{1} << 22 : M == 1 || products <= int64_t{1} << 21;
}
// The same of a gated product (N columns of the result): one row always goes to it
// (1 x 4096 x 8192 bf16 22.8 us, 24.9 on the tensor cores; 1 x 1024 x 4096 4.9 and 7.3), and
// float32 up to eight where 4 divides K (8 x 4096 x 4096 54 us, 124 on the binary32 tiles and 100
// in pieces; 8 x 256 x 256 2.7 and 8.0; but 8 x 1027 x 1283 33 and 17).  Off 16-byte boundaries
// as well, where its loads are of 4 bytes: 5 x 256 x 256 5.4 and 8.5, 6 x 2048 x 2048 32 and 43,
// 8 x 1024 x 1024 16.8 and 16.3 (8 x 4096 x 1024 60 and 49), 8 x 4096 x 4096 131, in pieces 152.
inline bool gated_few_rows(int64_t M, int64_t N, int64_t K, DType t, bool aligned) {
  return M == 1 || (t == DType::F32 && M <= 8 && K % 4 == 0) || few_rows(M, 2 * N, K, t, aligned);
}
inline int64_t pitch16(int64_t n) { return (n + 7) / 8 * 8; }
struct LinearPlan {
  bool pack;              // x and weight are copied
  bool pieces;            // in three pieces (float32)
  size_t x, w, bytes;
};
struct LinearGradPlan {
  bool make_dz;           // dz is stored: with an activation, or to realign dy
  bool pack;              // x and weight are copied
  bool pieces;            // dz, x and weight are stored in three pieces (float32)
  bool few;               // gated, few rows: dx in parts, nothing else
  int64_t ldz;
  size_t dz, part, x, w, bytes;
};
// aligned16: x and weight (and dy) start on 16-byte boundaries.  `out` counts the weight's
// rows, a gate's and what it gates alike; a gated gradient has an activation (any).
LinearPlan linear_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16);
LinearGradPlan linear_grad_plan(int64_t rows, int64_t in, int64_t out, DType t, int act,
                                bool aligned16);
// The plans of a gated call (`out` counts the result's columns).  float32 products are made
// on the tensor cores where the copies in pieces pay (gated_pieces).
bool gated_pieces(int64_t rows, int64_t in, int64_t out, bool grad);
inline int64_t piece_of(int64_t n) { return (n + 63) / 64 * 64; }
LinearPlan gated_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16);
LinearGradPlan gated_grad_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16);
cudaError_t launch_linear(const LinearCall& c, const LinearPlan& plan, cudaStream_t stream);
cudaError_t launch_linear_grad(const LinearGradCall& c, const LinearGradPlan& plan,
                               cudaStream_t stream);

}  // namespace b200norm
