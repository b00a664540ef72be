// The linear operator's host side: which kernel a product takes.
#include "linear_launch.cuh"

namespace b200norm {

extern template cudaError_t launch_rows<float>(const Product&, cudaStream_t);
extern template cudaError_t launch_dz<float>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_rows<__half>(const Product&, cudaStream_t);
extern template cudaError_t launch_dz<__half>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_pack<__half>(const void*, void*, int64_t, const void*,
                                      void*, int64_t, int64_t, cudaStream_t);
extern template cudaError_t launch_rows<__nv_bfloat16>(const Product&, cudaStream_t);
extern template cudaError_t launch_dz<__nv_bfloat16>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_pack<__nv_bfloat16>(const void*, void*, int64_t, const void*,
                                             void*, int64_t, int64_t, cudaStream_t);

namespace {

size_t round_256(size_t n) { return (n + 255) / 256 * 256; }

cudaError_t pack_rows(DType t, const void* src0, void* dst0, int64_t rows0, const void* src1,
                      void* dst1, int64_t rows1, int64_t n, cudaStream_t stream) {
  return t == DType::F16
             ? launch_pack<__half>(src0, dst0, rows0, src1, dst1, rows1, n, stream)
             : launch_pack<__nv_bfloat16>(src0, dst0, rows0, src1, dst1, rows1, n, stream);
}

}  // namespace

cudaError_t launch_product(const Product& p, cudaStream_t stream) {
  const bool mma = mma_operand_ok(p.a, p.t) && mma_operand_ok(p.b, p.t) && p.K > 0;
  if (p.a.k_contiguous && p.b.k_contiguous && !(mma && p.forced.cg) &&
      few_rows(p.M, p.N, p.K, p.t, mma)) {
    switch (p.t) {
      case DType::F32: return launch_rows<float>(p, stream);
      case DType::F16: return launch_rows<__half>(p, stream);
      default: return launch_rows<__nv_bfloat16>(p, stream);
    }
  }
  if (mma) return launch_mma(p, stream);
  // the plans see to it that 16-bit operands of more than a few rows are aligned
  return p.t == DType::F32 ? launch_plain_f32(p, stream) : cudaErrorMisalignedAddress;
}

cudaError_t launch_linear_dz(const LinearDzCall& c, cudaStream_t stream) {
  switch (c.t) {
    case DType::F32: return launch_dz<float>(c, stream);
    case DType::F16: return launch_dz<__half>(c, stream);
    default: return launch_dz<__nv_bfloat16>(c, stream);
  }
}

LinearPlan linear_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16) {
  LinearPlan p = {};
  p.pack = t != DType::F32 && (in % 8 != 0 || !aligned16) && !few_rows(rows, out, in, t, false);
  if (p.pack) {
    p.w = round_256(static_cast<size_t>(rows) * pitch16(in) * 2);
    p.bytes = p.w + round_256(static_cast<size_t>(out) * pitch16(in) * 2);
  }
  return p;
}

LinearGradPlan linear_grad_plan(int64_t rows, int64_t in, int64_t out, DType t, int act,
                                bool aligned16) {
  LinearGradPlan p = {};
  const bool half = t != DType::F32;
  p.make_dz = act != kActNone || (half && (out % 8 != 0 || !aligned16));
  p.pack = half && (in % 8 != 0 || !aligned16);
  p.ldz = half ? pitch16(out) : out;
  const size_t dz = p.make_dz ? static_cast<size_t>(rows) * p.ldz * dtype_size(t) : 0;
  p.part = round_256(dz);
  p.x = p.part + round_256(static_cast<size_t>(linear_db_parts(rows, out)) * out * 4);
  p.w = p.x + (p.pack ? round_256(static_cast<size_t>(rows) * pitch16(in) * 2) : 0);
  p.bytes = p.w + (p.pack ? round_256(static_cast<size_t>(out) * pitch16(in) * 2) : 0);
  return p;
}

cudaError_t launch_linear(const LinearCall& c, const LinearPlan& plan, cudaStream_t stream) {
  Operand x{c.x, c.in, true}, w{c.w, c.in, true};
  if (plan.pack) {
    char* ws = static_cast<char*>(c.workspace);
    const cudaError_t e = pack_rows(c.t, c.x, ws + plan.x, c.rows, c.w, ws + plan.w, c.out, c.in,
                                    stream);
    if (e != cudaSuccess) return e;
    x = {ws + plan.x, pitch16(c.in), true};
    w = {ws + plan.w, pitch16(c.in), true};
  }
  const Product p{x, w, c.rows, c.out, c.in, {c.bias, c.residual, c.y, c.z, c.act}, c.t, c.forced};
  return launch_product(p, stream);
}

cudaError_t launch_linear_grad(const LinearGradCall& c, const LinearGradPlan& plan,
                               cudaStream_t stream) {
  char* ws = static_cast<char*>(c.workspace);
  void* made = plan.make_dz && (c.dx || c.dw) ? ws + plan.dz : nullptr;
  cudaError_t e = cudaSuccess;
  if (made || c.db) {
    const LinearDzCall d{c.dy, c.z, made, plan.ldz, c.db, reinterpret_cast<float*>(ws + plan.part),
                         c.rows, c.out, c.act, c.t};
    e = launch_linear_dz(d, stream);
    if (e != cudaSuccess) return e;
  }
  if (plan.pack && c.rows > 0 && (c.dx || c.dw)) {
    e = pack_rows(c.t, c.x, ws + plan.x, c.dw ? c.rows : 0, c.w, ws + plan.w, c.dx ? c.out : 0,
                  c.in, stream);
    if (e != cudaSuccess) return e;
  }
  const void* dz = plan.make_dz ? made : c.dy;
  const int64_t ldz = plan.make_dz ? plan.ldz : c.out;
  if (c.dx && c.rows > 0) {
    Operand w{c.w, c.in, false};
    if (plan.pack) w = {ws + plan.w, pitch16(c.in), false};
    const Product p{{dz, ldz, true}, w, c.rows, c.in, c.out,
                    {nullptr, nullptr, c.dx, nullptr, kActNone}, c.t, c.forced};
    e = launch_product(p, stream);
    if (e != cudaSuccess) return e;
  }
  if (c.dw && c.rows == 0)  // empty sums: the zero of every type is zero bits
    return cudaMemsetAsync(c.dw, 0, static_cast<size_t>(c.out) * c.in * dtype_size(c.t), stream);
  if (c.dw) {
    Operand x{c.x, c.in, false};
    if (plan.pack) x = {ws + plan.x, pitch16(c.in), false};
    const Product p{{dz, ldz, false}, x, c.out, c.in, c.rows,
                    {nullptr, nullptr, c.dw, nullptr, kActNone}, c.t, c.forced};
    e = launch_product(p, stream);
  }
  return e;
}

}  // namespace b200norm
