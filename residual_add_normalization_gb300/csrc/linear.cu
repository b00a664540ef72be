// The linear operator's host side: which kernel a product takes, and its launch.
#include "layer_launch.cuh"
#include "linear.cuh"

namespace b200norm {

namespace {

template <typename T>
cudaError_t launch_plain(const Product& p, cudaStream_t stream) {
  const PlainProduct a{p.a.p, p.b.p, p.a.ld, p.b.ld, p.a.k_contiguous, p.b.k_contiguous,
                       p.M, p.N, p.K, p.epi};
  const dim3 grid(static_cast<unsigned>((p.M + kPlainTile - 1) / kPlainTile),
                  static_cast<unsigned>((p.N + kPlainTile - 1) / kPlainTile));
  return launch_pdl(linear_plain_kernel<T>, grid, 256, stream, a);
}

template <typename T>
cudaError_t launch_dz(const LinearDzCall& c, cudaStream_t stream) {
  const unsigned stripes = static_cast<unsigned>((c.out + 255) / 256);
  const int parts = c.rows > 0 ? linear_db_parts(c.rows) : 0;
  cudaError_t e = cudaSuccess;
  if (parts > 0) e = launch_pdl(linear_dz_kernel<T>, dim3(stripes, parts), 256, stream, c, parts);
  if (e == cudaSuccess && c.db)
    e = launch_pdl(linear_db_kernel<T>, dim3(stripes), 256, stream,
                   static_cast<const float*>(c.part), static_cast<T*>(c.db), c.out, parts);
  return e;
}

}  // namespace

cudaError_t launch_product(const Product& p, cudaStream_t stream) {
  if (mma_operand_ok(p.a, p.t) && mma_operand_ok(p.b, p.t) && p.K > 0)
    return launch_mma(p, stream);
  switch (p.t) {
    case DType::F32: return launch_plain<float>(p, stream);
    case DType::F16: return launch_plain<__half>(p, stream);
    default: return launch_plain<__nv_bfloat16>(p, stream);
  }
}

cudaError_t launch_linear_dz(const LinearDzCall& c, cudaStream_t stream) {
  switch (c.t) {
    case DType::F32: return launch_dz<float>(c, stream);
    case DType::F16: return launch_dz<__half>(c, stream);
    default: return launch_dz<__nv_bfloat16>(c, stream);
  }
}

namespace {
size_t round_256(size_t n) { return (n + 255) / 256 * 256; }
}  // namespace

LinearPlan linear_plan(int64_t, int64_t, int64_t, DType, bool) { return {0}; }

LinearGradPlan linear_grad_plan(int64_t rows, int64_t, int64_t out, DType t, int act, bool) {
  LinearGradPlan p;
  p.dz = 0;
  p.part = act != kActNone ? round_256(static_cast<size_t>(rows) * out * dtype_size(t)) : 0;
  p.bytes = p.part + round_256(static_cast<size_t>(linear_db_parts(rows)) * out * 4);
  return p;
}

cudaError_t launch_linear(const LinearCall& c, const LinearPlan&, cudaStream_t stream) {
  const Product p{{c.x, c.in, true}, {c.w, c.in, true}, c.rows, c.out, c.in,
                  {c.bias, c.residual, c.y, c.z, c.act}, c.t, c.forced};
  return launch_product(p, stream);
}

cudaError_t launch_linear_grad(const LinearGradCall& c, const LinearGradPlan& plan,
                               cudaStream_t stream) {
  char* ws = static_cast<char*>(c.workspace);
  const bool act = c.act != kActNone;
  void* dz = act && (c.dx || c.dw) ? ws + plan.dz : nullptr;
  cudaError_t e = cudaSuccess;
  if (dz || c.db) {
    const LinearDzCall d{c.dy, c.z, dz, c.out, c.db, reinterpret_cast<float*>(ws + plan.part),
                         c.rows, c.out, c.act, c.t};
    e = launch_linear_dz(d, stream);
    if (e != cudaSuccess) return e;
  }
  const void* g = act ? dz : c.dy;
  if (c.dx && c.rows > 0) {
    const Product p{{g, c.out, true}, {c.w, c.in, false}, c.rows, c.in, c.out,
                    {nullptr, nullptr, c.dx, nullptr, kActNone}, c.t, c.forced};
    e = launch_product(p, stream);
    if (e != cudaSuccess) return e;
  }
  if (c.dw) {
    const Product p{{g, c.out, false}, {c.x, c.in, false}, c.out, c.in, c.rows,
                    {nullptr, nullptr, c.dw, nullptr, kActNone}, c.t, c.forced};
    e = launch_product(p, stream);
  }
  return e;
}

}  // namespace b200norm
