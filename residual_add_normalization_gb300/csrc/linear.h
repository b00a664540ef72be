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
};

cudaError_t launch_product(const Product& p, cudaStream_t stream);
cudaError_t launch_plain_f32(const Product& p, cudaStream_t stream);

// The tensor-core kernels (16-bit types) -----------------------------------------

// What they need of an operand: 16-byte aligned rows at a 16-byte aligned place.
inline bool mma_operand_ok(const Operand& o, DType t) {
  return t != DType::F32 && o.ld % 8 == 0 && reinterpret_cast<uintptr_t>(o.p) % 16 == 0;
}

MmaPlan plan_mma(int64_t M, int64_t N, int64_t K, bool b_kc, int sms);
cudaError_t launch_mma(const Product& p, cudaStream_t stream);
template <typename T>
cudaError_t launch_mma_t(const Product& p, const MmaPlan& plan, int sms, unsigned* status,
                         cudaStream_t stream);

// Whether a forced plan has a kernel for the product.
bool mma_plan_ok(const MmaPlan& plan, int64_t M, int64_t K, bool a_kc, bool b_kc);

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
cudaError_t launch_linear_dz(const LinearDzCall& c, cudaStream_t stream);

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
inline int64_t pitch16(int64_t n) { return (n + 7) / 8 * 8; }
struct LinearPlan {
  bool pack;              // x and weight are copied
  size_t x, w, bytes;
};
struct LinearGradPlan {
  bool make_dz;           // dz is stored: with an activation, or to realign dy
  bool pack;              // x and weight are copied
  int64_t ldz;
  size_t dz, part, x, w, bytes;
};
// aligned16: x and weight (and dy) start on 16-byte boundaries.
LinearPlan linear_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16);
LinearGradPlan linear_grad_plan(int64_t rows, int64_t in, int64_t out, DType t, int act,
                                bool aligned16);
cudaError_t launch_linear(const LinearCall& c, const LinearPlan& plan, cudaStream_t stream);
cudaError_t launch_linear_grad(const LinearGradCall& c, const LinearGradPlan& plan,
                               cudaStream_t stream);

}  // namespace b200norm
