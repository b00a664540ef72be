// The linear operator's host side: which kernel a product takes.
#include "gated_few.cuh"
#include "linear_launch.cuh"

namespace b200norm {

extern template cudaError_t launch_rows<float>(const Product&, cudaStream_t);
extern template cudaError_t launch_dz<float>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_gated_dz<float>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_db<float>(const LinearDzCall&, bool, bool, cudaStream_t);
extern template cudaError_t launch_gated_few<float>(const GatedFewArgs&, void*, cudaStream_t);
extern template cudaError_t launch_rows<__half>(const Product&, cudaStream_t);
extern template cudaError_t launch_dz<__half>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_gated_dz<__half>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_db<__half>(const LinearDzCall&, bool, bool, cudaStream_t);
extern template cudaError_t launch_gated_few<__half>(const GatedFewArgs&, void*, cudaStream_t);
extern template cudaError_t launch_pack<__half>(const void*, void*, int64_t, const void*,
                                      void*, int64_t, int64_t, cudaStream_t);
extern template cudaError_t launch_rows<__nv_bfloat16>(const Product&, cudaStream_t);
extern template cudaError_t launch_dz<__nv_bfloat16>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_gated_dz<__nv_bfloat16>(const LinearDzCall&, cudaStream_t);
extern template cudaError_t launch_db<__nv_bfloat16>(const LinearDzCall&, bool, bool, cudaStream_t);
extern template cudaError_t launch_gated_few<__nv_bfloat16>(
    const GatedFewArgs&, void*, cudaStream_t);
extern template cudaError_t launch_pack<__nv_bfloat16>(const void*, void*, int64_t, const void*,
                                             void*, int64_t, int64_t, cudaStream_t);

cudaError_t launch_pieces(const void* src0, void* dst0, int64_t rows0, const void* src1,
                          void* dst1, int64_t rows1, int64_t n, bool late, cudaStream_t stream);

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
  if (p.piece_a) return launch_mma(p, stream);
  const bool mma = mma_operand_ok(p.a, p.t) && mma_operand_ok(p.b, p.t) && p.K > 0;
  if (p.a.k_contiguous && p.b.k_contiguous && !(mma && p.forced.cg) &&
      (p.gated ? gated_few_rows(p.M, p.N, p.K, p.t, mma) : few_rows(p.M, p.N, p.K, p.t, mma))) {
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

cudaError_t launch_linear_dz(const LinearDzCall& c, bool gated, cudaStream_t stream) {
  switch (c.t) {
    case DType::F32: return gated ? launch_gated_dz<float>(c, stream) : launch_dz<float>(c, stream);
    case DType::F16:
      return gated ? launch_gated_dz<__half>(c, stream) : launch_dz<__half>(c, stream);
    default:
      return gated ? launch_gated_dz<__nv_bfloat16>(c, stream)
                   : launch_dz<__nv_bfloat16>(c, stream);
  }
}

cudaError_t launch_linear_db(const LinearDzCall& c, bool gated, bool late, cudaStream_t stream) {
  if (!c.db) return cudaSuccess;
  switch (c.t) {
    case DType::F32: return launch_db<float>(c, gated, late, stream);
    case DType::F16: return launch_db<__half>(c, gated, late, stream);
    default: return launch_db<__nv_bfloat16>(c, gated, late, stream);
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

// Where the copies in pieces pay, us on the binary32 units and in pieces.  Forward, 2^26 products
// of a half: 256 x 512 x 512 (rows, in, out) 16.1 and 12.0, 2048 x 1024 x 2048 387 and 74, but
// 512 x 256 x 256 9.5 and 11.0.  Gradients sooner: 512 x 256 x 256 30.5 and 16.4, 256 x 256 x 256
// 19.9 and 15.5, 512 x 768 x 768 71 and 38.  Few rows are bound by the weight and its copy:
// 12 x 4096 x 4096 124 and 100, gradients 165 and 147, but of 16 x 2048 x 2048 50 and 58; those
// that the row kernel takes are not copied.
bool gated_pieces(int64_t rows, int64_t in, int64_t out, bool grad) {
  const int64_t products = rows * in * out;
  if (!grad) return rows > (in % 4 == 0 ? 8 : 4) && products >= int64_t{1} << 26;
  return products >= int64_t{1} << (rows >= 64 ? 24 : 27);
}

LinearPlan gated_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16) {
  if (t != DType::F32 || !gated_pieces(rows, in, out, false))
    return linear_plan(rows, in, 2 * out, t, aligned16);
  LinearPlan p = {};
  p.pieces = true;
  p.w = round_256(static_cast<size_t>(rows) * 3 * piece_of(in) * 2);
  p.bytes = p.w + round_256(static_cast<size_t>(2 * out) * 3 * piece_of(in) * 2);
  return p;
}

LinearGradPlan gated_grad_plan(int64_t rows, int64_t in, int64_t out, DType t, bool aligned16) {
  LinearGradPlan p = {};
  if (gated_few(rows, in, out, t)) {
    p.few = true;
    p.bytes = round_256(static_cast<size_t>(gated_few_parts(rows, in, out, t)) * rows * in * 4);
    return p;
  }
  const bool half = t != DType::F32;
  p.make_dz = true;
  p.pieces = !half && gated_pieces(rows, in, out, true);
  p.pack = half && (in % 8 != 0 || !aligned16);
  p.ldz = p.pieces ? 3 * piece_of(2 * out) : half ? pitch16(2 * out) : 2 * out;
  const int64_t pitch = p.pieces ? 3 * piece_of(in) : p.pack ? pitch16(in) : 0;
  p.part = round_256(static_cast<size_t>(rows) * p.ldz * (p.pieces ? 2 : dtype_size(t)));
  p.x = p.part + round_256(static_cast<size_t>(gated_db_parts(rows, out, t)) * 2 * out * 4);
  p.w = p.x + round_256(static_cast<size_t>(rows) * pitch * 2);
  p.bytes = p.w + round_256(static_cast<size_t>(2 * out) * pitch * 2);
  return p;
}

cudaError_t launch_linear(const LinearCall& c, const LinearPlan& plan, cudaStream_t stream) {
  Operand x{c.x, c.in, true}, w{c.w, c.in, true};
  if (plan.pack) {
    char* ws = static_cast<char*>(c.workspace);
    const cudaError_t e = pack_rows(c.t, c.x, ws + plan.x, c.rows, c.w, ws + plan.w,
                                    c.gated ? 2 * c.out : c.out, c.in, stream);
    if (e != cudaSuccess) return e;
    x = {ws + plan.x, pitch16(c.in), true};
    w = {ws + plan.w, pitch16(c.in), true};
  }
  Product p{x, w, c.rows, c.out, c.in, {c.bias, c.residual, c.y, c.z, c.act}, c.t, c.forced,
            c.gated};
  if (plan.pieces) {
    char* ws = static_cast<char*>(c.workspace);
    const cudaError_t e =
        launch_pieces(c.x, ws + plan.x, c.rows, c.w, ws + plan.w, 2 * c.out, c.in, false, stream);
    if (e != cudaSuccess) return e;
    p.piece_a = p.piece_b = piece_of(c.in);
    p.a = {ws + plan.x, 3 * p.piece_a, true};
    p.b = {ws + plan.w, 3 * p.piece_b, true};
  }
  return launch_product(p, stream);
}

// Launches that need nothing of one another run side by side: the pieces beside dz, dW beside
// dx, and behind these the last step of db (one after another: gated bf16 512 x 1024 x 1024
// 26 us, 22 so; 16384 x 768 x 768 117 and 97, with dz's four CTAs an SM).
cudaError_t launch_linear_grad(const LinearGradCall& c, const LinearGradPlan& plan,
                               cudaStream_t stream) {
  char* ws = static_cast<char*>(c.workspace);
  if (plan.few) {
    const GatedFewArgs a{c.dy, c.x, c.w, c.z, c.dw, c.db,
                         c.dx ? reinterpret_cast<float*>(ws) : nullptr, c.rows, c.in, c.out, c.act};
    switch (c.t) {
      case DType::F32: return launch_gated_few<float>(a, c.dx, stream);
      case DType::F16: return launch_gated_few<__half>(a, c.dx, stream);
      default: return launch_gated_few<__nv_bfloat16>(a, c.dx, stream);
    }
  }
  const int64_t out = c.gated ? 2 * c.out : c.out;  // rows of the weight
  void* made = plan.make_dz && (c.dx || c.dw) ? ws + plan.dz : nullptr;
  cudaError_t e = cudaSuccess;
  const LinearDzCall d{c.dy, c.z, made, plan.ldz, c.db, reinterpret_cast<float*>(ws + plan.part),
                       c.rows, c.out, c.act, c.t, plan.pieces ? piece_of(out) : 0};
  if (made || c.db) {
    e = launch_linear_dz(d, c.gated, stream);
    if (e != cudaSuccess) return e;
  }
  if (c.rows == 0) {  // empty sums: the zero of every type is zero bits
    e = launch_linear_db(d, c.gated, false, stream);
    if (e != cudaSuccess || !c.dw) return e;
    return cudaMemsetAsync(c.dw, 0, static_cast<size_t>(out) * c.in * dtype_size(c.t), stream);
  }
  if (plan.pieces && (c.dx || c.dw)) {
    e = launch_pieces(c.x, ws + plan.x, c.dw ? c.rows : 0, c.w, ws + plan.w, c.dx ? out : 0, c.in,
                      true, stream);
    if (e != cudaSuccess) return e;
  }
  if (plan.pack && (c.dx || c.dw)) {
    e = pack_rows(c.t, c.x, ws + plan.x, c.dw ? c.rows : 0, c.w, ws + plan.w, c.dx ? out : 0,
                  c.in, stream);
    if (e != cudaSuccess) return e;
  }
  int ctas = 0;  // of dx
  const void* dz = plan.make_dz ? made : c.dy;
  const int64_t ldz = plan.make_dz ? plan.ldz : out;
  if (c.dx) {
    Operand w{c.w, c.in, false};
    if (plan.pack) w = {ws + plan.w, pitch16(c.in), false};
    Product p{{dz, ldz, true}, w, c.rows, c.in, out,
              {nullptr, nullptr, c.dx, nullptr, kActNone}, c.t, c.forced};
    if (plan.pieces) {
      p.piece_a = piece_of(out);
      p.piece_b = piece_of(c.in);
      p.b = {ws + plan.w, 3 * p.piece_b, false};
    }
    p.ctas = &ctas;
    e = launch_product(p, stream);
    if (e != cudaSuccess) return e;
  }
  if (c.dw) {
    Operand x{c.x, c.in, false};
    if (plan.pack) x = {ws + plan.x, pitch16(c.in), false};
    Product p{{dz, ldz, false}, x, out, c.in, c.rows,
              {nullptr, nullptr, c.dw, nullptr, kActNone}, c.t, c.forced};
    if (plan.pieces) {
      p.piece_a = piece_of(out);
      p.piece_b = piece_of(c.in);
      p.b = {ws + plan.x, 3 * p.piece_b, false};
    }
    // beside a dx that leaves many SMs, or none but at its end; the first CTAs on a few idle SMs
    // cost dx more than they gain (128 CTAs, 512 x 2048 x 2048 bf16: 40.3 us, 36.3)
    p.late = c.dx && (ctas <= 152 * 2 / 3 || ctas >= 152);
    e = launch_product(p, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_linear_db(d, c.gated, c.dx || c.dw, stream);
}

}  // namespace b200norm
