// api.cu -- the C ABI: argument validation, schedule selection and launch.
//
// Every entry point validates its arguments completely before enqueueing
// anything, picks a schedule from the shape, element type and pointer
// alignment (the GB300 counterpart of the pages' per-call choice among
// implementation variants), and launches on the caller's stream.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "b200norm.h"
#include "b200norm_testing.h"
#include "heads.h"
#include "launch.h"
#include "layer.h"
#include "linear.h"

using namespace b200norm;

namespace {

thread_local std::string g_error;
thread_local int g_force_row_mode = 0;
thread_local int g_force_group_route = 0;
thread_local int g_force_csize = 0;  // forced CTA / cluster row split (0: automatic)
thread_local int g_force_nv = 0;
thread_local MmaPlan g_force_linear = {0, 0, 0, false};

b200norm_status fail(b200norm_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_error = buf;
  return st;
}

b200norm_status ok() {
  g_error.clear();
  return B200NORM_OK;
}

b200norm_status cuda_fail(cudaError_t e, const char* what) {
  return fail(B200NORM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool dtype_ok(b200norm_dtype t) {
  return t == B200NORM_F32 || t == B200NORM_F16 || t == B200NORM_BF16;
}

DType to_dtype(b200norm_dtype t) {
  return t == B200NORM_F32 ? DType::F32 : t == B200NORM_F16 ? DType::F16 : DType::BF16;
}

// SkipGroupNorm (T, M) pairs with kernels: M = float32 or T, and float16
// gamma/beta under float32 X.
bool group_types_ok(b200norm_dtype t, b200norm_dtype m) {
  return dtype_ok(t) && (m == B200NORM_F32 || m == t || (t == B200NORM_F32 && m == B200NORM_F16));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};

bool overlaps(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Outputs may not overlap inputs or each other.
b200norm_status check_overlaps(const Range* in, int nin, const Range* out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i], in[j]))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps input %s", out[i].name,
                    in[j].name);
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i], out[j]))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "outputs %s and %s overlap", out[i].name,
                    out[j].name);
  }
  return B200NORM_OK;
}

b200norm_status check_eps(float eps) {
  if (std::isnan(eps) || eps < 0.0f)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "epsilon must be >= 0 and not NaN (got %g)",
                static_cast<double>(eps));
  return B200NORM_OK;
}

constexpr int64_t kMaxGrid = 0x7fffffffLL;

// The forced CTA / cluster split of b200norm_testing_force_split.
b200norm_status forced_split(int64_t rows, int64_t n, RowPlan* p) {
  const int64_t nvec = n / p->ve;
  const int64_t per = static_cast<int64_t>(g_force_nv) * g_force_csize;
  const int64_t block = ((nvec + per - 1) / per + 31) / 32 * 32;
  if (block > 512)
    return fail(B200NORM_ERR_UNSUPPORTED, "forced split needs %lld threads per CTA (max 512)",
                static_cast<long long>(block));
  p->mode = 1;
  p->nv = g_force_nv;
  p->rpg = 1;
  p->csize = g_force_csize;
  p->block = static_cast<int>(block);
  p->tpr = p->block * p->csize;
  p->grid = rows * p->csize;
  return B200NORM_OK;
}

RowPlan forced_walk(int64_t rows, RowPlan p) {
  p.mode = 2;
  p.block = p.tpr = 512;
  p.csize = 1;
  p.nv = p.rpg = 1;
  p.grid = rows;
  return p;
}

b200norm_status skip_rms_impl(const void* input, const void* skip, const void* gamma,
                              const void* bias, void* output, void* sum, float* mean,
                              float* inv_std, int64_t rows, int64_t hidden, b200norm_dtype T,
                              float epsilon, b200norm_stream_t stream) {
  if (!dtype_ok(T)) return fail(B200NORM_ERR_UNSUPPORTED, "element type %d not supported", T);
  if (rows < 0) return fail(B200NORM_ERR_INVALID_ARGUMENT, "rows must be >= 0");
  if (hidden <= 0) return fail(B200NORM_ERR_INVALID_ARGUMENT, "hidden must be > 0");
  if (hidden > 0x7fffffffLL) return fail(B200NORM_ERR_UNSUPPORTED, "hidden exceeds 2^31-1");
  if (b200norm_status st = check_eps(epsilon)) return st;
  if (rows == 0) return ok();
  if (!input || !skip || !gamma || !output)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "input, skip, gamma and output are required");
  const size_t es = dtype_size(to_dtype(T));
  const void* ptrs[] = {input, skip, gamma, bias, output, sum};
  for (const void* p : ptrs)
    if (p && !aligned(p, es))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "tensor pointer not aligned to its element size");
  if ((mean && !aligned(mean, 4)) || (inv_std && !aligned(inv_std, 4)))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "statistics pointers must be 4-byte aligned");
  const size_t tb = static_cast<size_t>(rows) * hidden * es, vb = hidden * es;
  const Range in[] = {{input, tb, "input"}, {skip, tb, "skip"}, {gamma, vb, "gamma"},
                      {bias, vb, "bias"}};
  const Range out[] = {{output, tb, "output"}, {sum, tb, "input_skip_bias_sum"},
                       {mean, static_cast<size_t>(rows) * 4, "mean"},
                       {inv_std, static_cast<size_t>(rows) * 4, "inv_std_var"}};
  if (b200norm_status st = check_overlaps(in, 4, out, 4)) return st;

  const int ve = static_cast<int>(16 / es);
  bool vec = hidden % ve == 0;
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) vec = false;
  RowPlan plan = plan_rows(rows, hidden, to_dtype(T), vec, RowOp::SkipRms);
  if (g_force_csize)
    if (b200norm_status st = forced_split(rows, hidden, &plan)) return st;
  if (g_force_row_mode == 0 && !g_force_csize)
    prefer_pipe_skip_rms(rows, hidden, to_dtype(T), vec, &plan);
  if (g_force_row_mode == 2) plan = forced_walk(rows, plan);
  if (g_force_row_mode == 3 && !pipe_plan(rows, hidden, to_dtype(T), vec, &plan))
    return fail(B200NORM_ERR_UNSUPPORTED, "forced pipelined schedule cannot take this call");
  if (plan.grid > kMaxGrid) return fail(B200NORM_ERR_UNSUPPORTED, "too many rows for one launch");
  SkipRmsCall c{input, skip, gamma, bias, output, sum, mean, inv_std, rows, hidden, to_dtype(T),
                epsilon};
  cudaError_t e = launch_skip_rms(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "skip_rms launch");
  return ok();
}

// A tensor argument of the layer and linear entry points (null: absent).
struct Tensor {
  const void* p;
  size_t bytes, elem;
  const char* name;
  bool output;
};

// Element alignment, and no output over an input or another output.
b200norm_status check_tensors(const Tensor* t, int n) {
  for (int i = 0; i < n; ++i)
    if (t[i].p && !aligned(t[i].p, t[i].elem))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s is not aligned to its element size",
                  t[i].name);
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (i != j && t[i].output && (!t[j].output || j > i) &&
          overlaps({t[i].p, t[i].bytes, t[i].name}, {t[j].p, t[j].bytes, t[j].name}))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps %s", t[i].name, t[j].name);
  return B200NORM_OK;
}

bool all_aligned16(const Tensor* t, int n) {
  for (int i = 0; i < n; ++i)
    if (t[i].p && !aligned(t[i].p, 16)) return false;
  return true;
}

b200norm_status check_workspace(const void* ws, size_t bytes, size_t need, const Tensor* t,
                                int n) {
  if (need == 0) return B200NORM_OK;
  if (!ws || bytes < need)
    return fail(B200NORM_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu at %p)", need, bytes,
                ws);
  if (!aligned(ws, 256)) return fail(B200NORM_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  for (int i = 0; i < n; ++i)
    if (overlaps({ws, need, "workspace"}, {t[i].p, t[i].bytes, t[i].name}))
      return fail(B200NORM_ERR_WORKSPACE, "workspace overlaps %s", t[i].name);
  return B200NORM_OK;
}

b200norm_status check_layer_shape(int64_t rows, int64_t hidden, b200norm_dtype T,
                                  b200norm_dtype M) {
  if (!dtype_ok(T) || (M != T && M != B200NORM_F32))
    return fail(B200NORM_ERR_UNSUPPORTED, "element types T=%d M=%d not supported", T, M);
  if (rows < 0) return fail(B200NORM_ERR_INVALID_ARGUMENT, "rows must be >= 0");
  if (hidden <= 0) return fail(B200NORM_ERR_INVALID_ARGUMENT, "hidden must be > 0");
  if (hidden > 0x7fffffffLL || rows > kMaxGrid)
    return fail(B200NORM_ERR_UNSUPPORTED, "hidden or rows exceeds 2^31-1");
  return B200NORM_OK;
}

constexpr int64_t kMaxFeatures = int64_t{1} << 20;
constexpr int64_t kMaxGated = kMaxFeatures / 2;
constexpr int64_t kMaxLinearRows = int64_t{1} << 30;  // tensor copies take int coordinates

b200norm_status check_linear_shape(int64_t rows, int64_t in, int64_t out, b200norm_dtype T,
                                   int activation) {
  if (!dtype_ok(T)) return fail(B200NORM_ERR_UNSUPPORTED, "element type %d not supported", T);
  if (rows < 0 || in <= 0 || out <= 0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "need rows >= 0, in_features > 0, out_features > 0");
  if (rows > kMaxLinearRows || in > kMaxFeatures || out > kMaxFeatures)
    return fail(B200NORM_ERR_UNSUPPORTED, "rows exceeds 2^30, or features 2^20");
  if (activation < 0 || activation >= kActivations)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "activation must be 0 (none), 1 (SiLU), 2 (GELU), 3 (GELU, tanh) or 4 (ReLU)");
  return B200NORM_OK;
}

b200norm_status check_gated_shape(int64_t rows, int64_t in, int64_t out, b200norm_dtype T,
                                  int activation) {
  if (b200norm_status st = check_linear_shape(rows, in, out, T, activation)) return st;
  if (out > kMaxGated)
    return fail(B200NORM_ERR_UNSUPPORTED, "out_features of a gated call exceeds 2^19");
  return B200NORM_OK;
}

// ---- query and key heads ----

// A strided tensor of heads, as an argument.
struct HeadsArg {
  const void* p;
  int64_t heads;
  const int64_t* strides;
  const char* name;
};

using Wide = unsigned __int128;

// Elements from the first to one past the last.
Wide heads_extent(const HeadsArg& a, int64_t batch, int64_t seq, int64_t size) {
  return static_cast<Wide>(batch - 1) * a.strides[0] + static_cast<Wide>(seq - 1) * a.strides[1] +
         static_cast<Wide>(a.heads - 1) * a.strides[2] + size;
}

b200norm_status check_heads(const HeadsArg& a, int64_t batch, int64_t seq, int64_t size,
                            size_t es) {
  if (!a.p) return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s is required", a.name);
  if (!aligned(a.p, es))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s is not aligned to its element size", a.name);
  for (int i = 0; i < 3; ++i)
    if (a.strides[i] < 0)
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "strides of %s must be >= 0", a.name);
  if (heads_extent(a, batch, seq, size) > static_cast<Wide>(INT64_MAX) / 8)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "strides of %s reach past the address space",
                a.name);
  return B200NORM_OK;
}

// Whether no element of an output has two places: each axis steps past all that the
// axes of smaller steps reach.
bool heads_distinct(const HeadsArg& a, int64_t batch, int64_t seq, int64_t size) {
  const int64_t n[3] = {batch, seq, a.heads};
  bool used[3] = {false, false, false};
  Wide extent = static_cast<Wide>(size);
  for (int round = 0; round < 3; ++round) {
    int least = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && n[i] > 1 && (least < 0 || a.strides[i] < a.strides[least])) least = i;
    if (least < 0) break;
    used[least] = true;
    if (static_cast<Wide>(a.strides[least]) < extent) return false;
    extent += static_cast<Wide>(n[least] - 1) * a.strides[least];
  }
  return true;
}

// Whether two tensors of heads share no element, as far as it can be told: they lie apart, or
// side by side in every stretch of one of their steps (in a sequence, a product's row, or a
// head's place of queries, keys and values).
bool heads_apart(const HeadsArg& a, const HeadsArg& b, int64_t batch, int64_t seq, int64_t size,
                 size_t es) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  if (a0 > b0) return heads_apart(b, a, batch, seq, size, es);
  const uintptr_t gap = (b0 - a0) / es;
  if (heads_extent(a, batch, seq, size) <= gap) return true;
  // elements from the first to one past the last, whole stretches left out
  auto within = [&](const HeadsArg& t, int64_t step) {
    const int64_t n[3] = {batch, seq, t.heads};
    Wide extent = static_cast<Wide>(size);
    for (int i = 0; i < 3; ++i)
      if (t.strides[i] % step) extent += static_cast<Wide>(n[i] - 1) * t.strides[i];
    return extent;
  };
  for (const HeadsArg* t : {&a, &b}) {
    const int64_t n[3] = {batch, seq, t->heads};
    for (int i = 0; i < 3; ++i) {
      const int64_t step = t->strides[i];
      if (n[i] < 2 || step < 1) continue;
      const Wide at = gap % static_cast<uintptr_t>(step);
      if (within(a, step) <= at && at + within(b, step) <= static_cast<Wide>(step)) return true;
    }
  }
  return false;
}

bool heads_same(const HeadsArg& a, const HeadsArg& b, int64_t batch, int64_t seq) {
  return a.p == b.p && a.heads == b.heads && (batch == 1 || a.strides[0] == b.strides[0]) &&
         (seq == 1 || a.strides[1] == b.strides[1]) &&
         (a.heads == 1 || a.strides[2] == b.strides[2]);
}

// What the rotation reads and gamma, as ranges of memory.
Range heads_range(const HeadsArg& a, int64_t batch, int64_t seq, int64_t size, size_t es) {
  return {a.p, static_cast<size_t>(heads_extent(a, batch, seq, size)) * es, a.name};
}

b200norm_status check_rotation(const b200norm_rotation* r, int64_t batch, int64_t seq,
                               int64_t head_size) {
  if (!r) return fail(B200NORM_ERR_INVALID_ARGUMENT, "rotation is required");
  if (r->rotary_size < 0 || r->rotary_size > head_size || r->rotary_size % 2)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "rotary_size must be even, in [0, head_size]");
  if (r->interleaved != 0 && r->interleaved != 1)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "interleaved must be 0 or 1");
  if (r->rotary_size == 0) return B200NORM_OK;
  if (!std::isfinite(r->scale))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (r->position_bytes != 4 && r->position_bytes != 8)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "position_bytes must be 4 or 8");
  if (batch == 0 || seq == 0) return B200NORM_OK;
  if (!r->positions || !r->inv_freq)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "positions and inv_freq are required");
  if (!aligned(r->positions, r->position_bytes) || !aligned(r->inv_freq, 8))
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "positions or inv_freq is not aligned to its element size");
  if (r->batch_stride < 0 || r->token_stride < 0 ||
      static_cast<Wide>(batch - 1) * r->batch_stride +
              static_cast<Wide>(seq - 1) * r->token_stride >
          static_cast<Wide>(INT64_MAX) / 16)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "strides of positions out of range");
  return B200NORM_OK;
}

b200norm_status check_heads_shape(int64_t batch, int64_t seq, int64_t q, int64_t k, int64_t size,
                                  b200norm_dtype T, b200norm_dtype M) {
  if (!dtype_ok(T) || (M != T && M != B200NORM_F32))
    return fail(B200NORM_ERR_UNSUPPORTED, "element types T=%d M=%d not supported", T, M);
  if (batch < 0 || seq < 0 || q < 0 || k < 0 || size <= 0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "need batch >= 0, seq >= 0, heads >= 0, head_size > 0");
  if (size > kMaxHeadSize || q > kMaxHeads || k > kMaxHeads)
    return fail(B200NORM_ERR_UNSUPPORTED, "head_size exceeds 1024, or heads 2^16");
  if (batch > kMaxGrid || seq > kMaxGrid || batch * seq > kMaxGrid)
    return fail(B200NORM_ERR_UNSUPPORTED, "batch * seq exceeds 2^31-1");
  if (batch * seq * (q + k) > int64_t{1} << 40)
    return fail(B200NORM_ERR_UNSUPPORTED, "batch * seq * heads exceeds 2^40");
  return B200NORM_OK;
}

// The steps that are taken: none along an axis of one, whatever is given for it.
HeadStrides to_strides(const int64_t* s, int64_t batch, int64_t seq, int64_t heads) {
  return {batch > 1 ? s[0] : 0, seq > 1 ? s[1] : 0, heads > 1 ? s[2] : 0};
}

HeadsCall heads_call(const b200norm_rotation* r, int64_t batch, int64_t seq, int64_t size,
                     b200norm_dtype T, b200norm_dtype M) {
  HeadsCall c = {};
  c.positions = r->positions;
  c.pos64 = r->position_bytes == 8;
  c.pos_batch = r->batch_stride;
  c.pos_token = r->token_stride;
  c.inv_freq = r->inv_freq;
  c.batch = batch;
  c.seq = seq;
  c.size = static_cast<int>(size);
  c.rot = static_cast<int>(r->rotary_size);
  c.interleaved = r->interleaved != 0;
  c.scale = r->scale;
  c.t = to_dtype(T);
  c.m = to_dtype(M);
  return c;
}

// The rotation's inputs.
int rotation_ranges(const HeadsCall& c, Range* out) {
  if (c.rot == 0) return 0;
  const size_t n = static_cast<size_t>((c.batch - 1) * c.pos_batch + (c.seq - 1) * c.pos_token + 1);
  out[0] = {c.positions, n * (c.pos64 ? 8 : 4), "positions"};
  out[1] = {c.inv_freq, static_cast<size_t>(c.rot / 2) * 8, "inv_freq"};
  return 2;
}

// The forward call of both entries.
b200norm_status heads_forward(const b200norm_heads* queries, const b200norm_heads* keys,
                              const b200norm_rotation* rotation, int64_t batch, int64_t seq,
                              int64_t head_size, b200norm_dtype T, b200norm_dtype M, bool norm,
                              int inverse, float epsilon, b200norm_stream_t stream) {
  const b200norm_heads* given[2] = {queries, keys};
  if (b200norm_status st = check_heads_shape(batch, seq, queries ? queries->heads : 0,
                                             keys ? keys->heads : 0, head_size, T, M))
    return st;
  if (b200norm_status st = check_rotation(rotation, batch, seq, head_size)) return st;
  if (inverse != 0 && inverse != 1)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "inverse must be 0 or 1");
  if (norm)
    if (b200norm_status st = check_eps(epsilon)) return st;
  if (batch * seq == 0) return ok();
  HeadsCall c = heads_call(rotation, batch, seq, head_size, T, M);
  c.inverse = inverse != 0;
  c.norm = norm;
  c.eps = epsilon;
  const size_t es = dtype_size(c.t), ms = dtype_size(c.m);
  static const char* names[2][3] = {{"queries x", "queries y", "queries gamma"},
                                    {"keys x", "keys y", "keys gamma"}};
  HeadsArg xs[2], ys[2];
  Range reads[4];
  int n = 0, nreads = rotation_ranges(c, reads);
  for (int i = 0; i < 2; ++i) {
    const b200norm_heads* h = given[i];
    if (!h || h->heads == 0) continue;
    xs[n] = {h->x, h->heads, h->x_strides, names[i][0]};
    ys[n] = {h->y, h->heads, h->y_strides, names[i][1]};
    for (const HeadsArg* a : {&xs[n], &ys[n]})
      if (b200norm_status st = check_heads(*a, batch, seq, head_size, es)) return st;
    if (h->gamma) {
      if (!norm) return fail(B200NORM_ERR_INVALID_ARGUMENT, "b200norm_rotary takes no gamma");
      if (!aligned(h->gamma, ms))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s is not aligned to its element size",
                    names[i][2]);
      reads[nreads++] = {h->gamma, static_cast<size_t>(head_size) * ms, names[i][2]};
    }
    auto steps = [&](const int64_t* s) { return to_strides(s, batch, seq, h->heads); };
    c.set[i] = {h->x, nullptr, h->gamma, h->y, nullptr, h->heads, steps(h->x_strides), {},
                steps(h->y_strides)};
    ++n;
  }
  if (n == 0) return ok();
  for (int i = 0; i < n; ++i) {
    if (!heads_distinct(ys[i], batch, seq, head_size))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s overlaps itself", ys[i].name);
    for (int j = 0; j < n; ++j)
      if (!(i == j && heads_same(ys[i], xs[j], batch, seq)) &&
          !heads_apart(ys[i], xs[j], batch, seq, head_size, es))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps %s", ys[i].name, xs[j].name);
    for (int j = 0; j < nreads; ++j)
      if (overlaps(heads_range(ys[i], batch, seq, head_size, es), reads[j]))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps %s", ys[i].name,
                    reads[j].name);
  }
  if (n == 2 && !heads_apart(ys[0], ys[1], batch, seq, head_size, es))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "outputs overlap");
  cudaError_t e = launch_heads(c, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, norm ? "head_rms_rotary launch" : "rotary launch");
  return ok();
}

// Skip shape classification (SkipGroupNorm README, Inputs, skip):
// returns 0 full, 1 broadcast per (n, c), -1 unrecognised.
int classify_skip(int rank, const int64_t* d, int64_t N, int64_t C, int64_t H, int64_t W,
                  bool cl) {
  if (rank == 4 && d) {
    const int64_t full_cl[4] = {N, H, W, C}, full_cf[4] = {N, C, H, W};
    const int64_t* f = cl ? full_cl : full_cf;
    if (d[0] == f[0] && d[1] == f[1] && d[2] == f[2] && d[3] == f[3]) return 0;
    if (d[0] == N && d[1] == 1 && d[2] == 1 && d[3] == C) return (H == 1 && W == 1) ? 0 : 1;
    return -1;
  }
  if (rank == 2 && d && d[0] == N && d[1] == C) return 1;
  return -1;
}

}  // namespace

namespace b200norm {

namespace {
std::atomic<bool> g_pdl{true};
}

bool pdl_enabled() { return g_pdl.load(std::memory_order_relaxed); }

void set_pdl_enabled(bool on) { g_pdl.store(on, std::memory_order_relaxed); }

}  // namespace b200norm

void b200norm::set_error_message(const char* msg) { g_error = msg; }

b200norm_status b200norm::skip_group_check(const void* x, const void* skip, int skip_rank,
                                           const int64_t* skip_dims, const void* bias,
                                           const void* gamma, const void* beta, const void* y,
                                           const void* s, int64_t N, int64_t C, int64_t H,
                                           int64_t W, b200norm_dtype T, b200norm_dtype M,
                                           int groups, float epsilon, int activation,
                                           int channels_last, bool* nothing_to_do) {
  *nothing_to_do = false;
  if (!group_types_ok(T, M))
    return fail(B200NORM_ERR_UNSUPPORTED, "element types T=%d M=%d not supported", T, M);
  if (N < 0 || C <= 0 || H < 0 || W < 0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "need N >= 0, C > 0, H >= 0, W >= 0");
  if (groups <= 0 || C % groups != 0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "groups (%d) must be > 0 and divide C (%lld)",
                groups, static_cast<long long>(C));
  if (activation != 0 && activation != 1)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "activation must be 0 (none) or 1 (SiLU)");
  if (b200norm_status st = check_eps(epsilon)) return st;
  const bool cl = channels_last != 0;
  const int bc = classify_skip(skip_rank, skip_dims, N, C, H, W, cl);
  if (bc < 0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "skip must have X's shape, (N, C) or (N, 1, 1, C)");
  if (N == 0 || H == 0 || W == 0) {
    *nothing_to_do = true;
    return B200NORM_OK;
  }
  if (C > 0x7fffffffLL || H * W > 0x7fffffffLL || N > 0x7fffffffLL)
    return fail(B200NORM_ERR_UNSUPPORTED, "C, H*W or N exceeds 2^31-1");
  if (!x || !skip || !gamma || !beta || !y)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "x, skip, gamma, beta and y are required");
  const size_t es = dtype_size(to_dtype(T)), ms = dtype_size(to_dtype(M));
  const void* tptrs[] = {x, skip, bias, y, s};
  for (const void* p : tptrs)
    if (p && !aligned(p, es))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "tensor pointer not aligned to its element size");
  if (!aligned(gamma, ms) || !aligned(beta, ms))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "gamma/beta not aligned to their element size");
  const size_t tb = static_cast<size_t>(N * C * H * W) * es;
  const size_t sb = bc ? static_cast<size_t>(N * C) * es : tb;
  const Range in[] = {{x, tb, "X"}, {skip, sb, "skip"}, {bias, C * es, "bias"},
                      {gamma, C * ms, "gamma"}, {beta, C * ms, "beta"}};
  const Range out[] = {{y, tb, "Y"}, {s, tb, "S"}};
  return check_overlaps(in, 5, out, 2);
}

extern "C" {

int b200norm_version(void) { return 1; }

const char* b200norm_status_string(b200norm_status s) {
  switch (s) {
    case B200NORM_OK: return "B200NORM_OK";
    case B200NORM_ERR_INVALID_ARGUMENT: return "B200NORM_ERR_INVALID_ARGUMENT";
    case B200NORM_ERR_UNSUPPORTED: return "B200NORM_ERR_UNSUPPORTED";
    case B200NORM_ERR_CUDA: return "B200NORM_ERR_CUDA";
    case B200NORM_ERR_WORKSPACE: return "B200NORM_ERR_WORKSPACE";
    case B200NORM_ERR_DEVICE_TIMEOUT: return "B200NORM_ERR_DEVICE_TIMEOUT";
  }
  return "B200NORM_UNKNOWN_STATUS";
}

const char* b200norm_last_error(void) { return g_error.c_str(); }

b200norm_status b200norm_skip_rms(const void* input, const void* skip, const void* gamma,
                                  const void* bias, void* output, void* input_skip_bias_sum,
                                  int64_t rows, int64_t hidden, b200norm_dtype T, float epsilon,
                                  b200norm_stream_t stream) {
  return skip_rms_impl(input, skip, gamma, bias, output, input_skip_bias_sum, nullptr, nullptr,
                       rows, hidden, T, epsilon, stream);
}

b200norm_status b200norm_skip_rms_stats(const void* input, const void* skip, const void* gamma,
                                        const void* bias, void* output,
                                        void* input_skip_bias_sum, float* mean,
                                        float* inv_std_var, int64_t rows, int64_t hidden,
                                        b200norm_dtype T, float epsilon,
                                        b200norm_stream_t stream) {
  return skip_rms_impl(input, skip, gamma, bias, output, input_skip_bias_sum, mean, inv_std_var,
                       rows, hidden, T, epsilon, stream);
}

b200norm_status b200norm_gated_rms(const void* x, const void* gate, const void* scale, void* y,
                                   int64_t numel, int64_t C, b200norm_dtype T, float epsilon,
                                   b200norm_stream_t stream) {
  if (!dtype_ok(T)) return fail(B200NORM_ERR_UNSUPPORTED, "element type %d not supported", T);
  if (C <= 0) return fail(B200NORM_ERR_INVALID_ARGUMENT, "C (numel of scale) must be > 0");
  if (numel < 0) return fail(B200NORM_ERR_INVALID_ARGUMENT, "numel must be >= 0");
  if (numel % C != 0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "numel (%lld) is not a multiple of C (%lld)",
                static_cast<long long>(numel), static_cast<long long>(C));
  if (C > 0x7fffffffLL) return fail(B200NORM_ERR_UNSUPPORTED, "C exceeds 2^31-1");
  if (b200norm_status st = check_eps(epsilon)) return st;
  if (numel == 0) return ok();
  if (!x || !gate || !scale || !y)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "x, gate, scale and y are required");
  const size_t es = dtype_size(to_dtype(T));
  const void* ptrs[] = {x, gate, scale, y};
  for (const void* p : ptrs)
    if (!aligned(p, es))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "tensor pointer not aligned to its element size");
  const size_t tb = static_cast<size_t>(numel) * es;
  const Range in[] = {{x, tb, "x"}, {gate, tb, "gate"}, {scale, C * es, "scale"}};
  const Range out[] = {{y, tb, "y"}};
  if (b200norm_status st = check_overlaps(in, 3, out, 1)) return st;
  const int64_t rows = numel / C;
  const int ve = static_cast<int>(16 / es);
  bool vec = C % ve == 0;
  for (const void* p : ptrs)
    if (!aligned(p, 16)) vec = false;
  RowPlan plan = plan_rows(rows, C, to_dtype(T), vec, RowOp::Gated);
  if (g_force_csize)
    if (b200norm_status st = forced_split(rows, C, &plan)) return st;
  if (g_force_row_mode == 2) plan = forced_walk(rows, plan);
  if (g_force_row_mode == 3 && !pipe_plan(rows, C, to_dtype(T), vec, &plan))
    return fail(B200NORM_ERR_UNSUPPORTED, "forced pipelined schedule cannot take this call");
  if (plan.grid > kMaxGrid) return fail(B200NORM_ERR_UNSUPPORTED, "too many rows for one launch");
  GatedCall c{x, gate, scale, y, rows, C, to_dtype(T), epsilon};
  cudaError_t e = launch_gated(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gated_rms launch");
  return ok();
}

size_t b200norm_skip_group_workspace_size(int64_t N, int64_t C, int64_t H, int64_t W, int groups,
                                          b200norm_dtype T, int channels_last) {
  if (!dtype_ok(T)) return kControlBytes;
  return group_workspace_bytes(N, C, H, W, groups, to_dtype(T), channels_last != 0);
}

b200norm_status b200norm_skip_group(const void* x, const void* skip, int skip_rank,
                                    const int64_t* skip_dims, const void* bias,
                                    const void* gamma, const void* beta, void* y, void* s,
                                    int64_t N, int64_t C, int64_t H, int64_t W,
                                    b200norm_dtype T, b200norm_dtype M, int groups,
                                    float epsilon, int activation, int channels_last,
                                    void* workspace, size_t workspace_bytes,
                                    b200norm_stream_t stream) {
  bool nothing_to_do = false;
  if (b200norm_status st = skip_group_check(x, skip, skip_rank, skip_dims, bias, gamma, beta, y,
                                            s, N, C, H, W, T, M, groups, epsilon, activation,
                                            channels_last, &nothing_to_do))
    return st;
  if (nothing_to_do) return ok();
  const bool cl = channels_last != 0;
  const size_t need = group_workspace_bytes(N, C, H, W, groups, to_dtype(T), cl);
  if (!workspace || workspace_bytes < need)
    return fail(B200NORM_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu at %p)", need,
                workspace_bytes, workspace);
  if (!aligned(workspace, 256))
    return fail(B200NORM_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t es = dtype_size(to_dtype(T)), ms = dtype_size(to_dtype(M));
  const int bc = classify_skip(skip_rank, skip_dims, N, C, H, W, cl);
  const size_t tb = static_cast<size_t>(N * C * H * W) * es;
  const size_t sb = bc ? static_cast<size_t>(N * C) * es : tb;
  const Range ws = {workspace, workspace_bytes, "workspace"};
  const Range others[] = {{x, tb, "X"}, {skip, sb, "skip"}, {bias, C * es, "bias"},
                          {gamma, C * ms, "gamma"}, {beta, C * ms, "beta"}, {y, tb, "Y"},
                          {s, tb, "S"}};
  for (const Range& r : others)
    if (overlaps(ws, r))
      return fail(B200NORM_ERR_WORKSPACE, "workspace overlaps %s", r.name);

  SkipGroupCall c{x, skip, bias, gamma, beta, y, s, N, C, H, W, groups, to_dtype(T), to_dtype(M),
                  bc == 1, activation, cl, epsilon, workspace, workspace_bytes};
  bool vec = true;
  const void* tptrs[] = {x, skip, bias, y, s};
  for (const void* p : tptrs)
    if (p && !aligned(p, 16)) vec = false;
  GroupPlan plan;
  cudaError_t e = plan_group(c, vec, g_force_group_route, &plan);
  if (e == cudaErrorNotSupported && g_force_group_route)
    return fail(B200NORM_ERR_UNSUPPORTED, "forced route %d cannot take this call",
                g_force_group_route);
  if (e != cudaSuccess) return cuda_fail(e, "skip_group planning");
  if (plan.grid > kMaxGrid) return fail(B200NORM_ERR_UNSUPPORTED, "problem too large for one launch");
  e = launch_group(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return fail(B200NORM_ERR_CUDA,
                "skip_group launch (route %d, grid %lld, block %d, cluster %d, smem %zu): %s",
                plan.route, static_cast<long long>(plan.grid), plan.block, plan.csize, plan.smem,
                cudaGetErrorString(e));
  return ok();
}

b200norm_status b200norm_workspace_init(void* workspace, size_t workspace_bytes,
                                        b200norm_stream_t stream) {
  if (!workspace || workspace_bytes < kControlBytes)
    return fail(B200NORM_ERR_WORKSPACE, "workspace missing or smaller than %zu bytes",
                kControlBytes);
  cudaError_t e = cudaMemsetAsync(workspace, 0, workspace_bytes,
                                  reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "workspace init");
  return ok();
}

b200norm_status b200norm_workspace_status(const void* workspace, b200norm_stream_t stream) {
  if (!workspace) return fail(B200NORM_ERR_WORKSPACE, "workspace is NULL");
  unsigned int ctl[4] = {0, 0, 0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(ctl, workspace, sizeof(ctl), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "workspace status read");
  if (ctl[2] != 0)
    return fail(static_cast<b200norm_status>(ctl[2]), "device wait %u gave up", ctl[3]);
  return ok();
}

b200norm_status b200norm_rows_status(b200norm_stream_t stream) {
  unsigned* word = pipe_status_word();
  if (!word) return fail(B200NORM_ERR_CUDA, "row status word not available on this device");
  unsigned v = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && v != 0) e = cudaMemsetAsync(word, 0, sizeof(v), st);
  if (e == cudaSuccess && v != 0) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "row status read");
  if (v != 0) return fail(static_cast<b200norm_status>(v), "a pipelined row wait gave up");
  return ok();
}

// ---- layer normalization and the linear operator -----------------------------

b200norm_status b200norm_skip_layer(const void* input, const void* skip, const void* gamma,
                                    const void* beta, const void* bias, void* output,
                                    void* input_skip_bias_sum, float* mean, float* inv_std_var,
                                    int64_t rows, int64_t hidden, b200norm_dtype T,
                                    b200norm_dtype M, float epsilon, b200norm_stream_t stream) {
  if (b200norm_status st = check_layer_shape(rows, hidden, T, M)) return st;
  if (b200norm_status st = check_eps(epsilon)) return st;
  if (!skip && (bias || input_skip_bias_sum))
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "bias and input_skip_bias_sum need a skip (S is the input without one)");
  if (rows == 0) return ok();
  if (!input || !gamma || !output)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "input, gamma and output are required");
  const size_t es = dtype_size(to_dtype(T)), ms = dtype_size(to_dtype(M));
  const size_t tb = static_cast<size_t>(rows) * hidden * es, sb = static_cast<size_t>(rows) * 4;
  const Tensor ts[] = {{input, tb, es, "input", false}, {skip, tb, es, "skip", false},
                       {gamma, hidden * ms, ms, "gamma", false},
                       {beta, hidden * ms, ms, "beta", false},
                       {bias, hidden * es, es, "bias", false},
                       {output, tb, es, "output", true},
                       {input_skip_bias_sum, tb, es, "input_skip_bias_sum", true},
                       {mean, sb, 4, "mean", true}, {inv_std_var, sb, 4, "inv_std_var", true}};
  if (b200norm_status st = check_tensors(ts, 9)) return st;
  LayerCall c{input, skip, gamma, beta, bias, output, input_skip_bias_sum, mean, inv_std_var,
              rows, hidden, to_dtype(T), to_dtype(M), epsilon,
              hidden % static_cast<int64_t>(16 / es) == 0 && all_aligned16(ts, 7)};
  cudaError_t e = launch_layer(c, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "skip_layer launch");
  return ok();
}

size_t b200norm_skip_layer_grad_workspace_size(int64_t rows, int64_t hidden) {
  if (rows < 0 || hidden <= 0) return 0;
  return layer_grad_workspace_bytes(rows, hidden);
}

b200norm_status b200norm_skip_layer_grad(const void* dy, const void* s, const float* mean,
                                         const float* inv_std_var, const void* gamma,
                                         const void* ds, void* dx, void* dgamma, void* dbeta,
                                         void* dbias, int64_t rows, int64_t hidden,
                                         b200norm_dtype T, b200norm_dtype M, void* workspace,
                                         size_t workspace_bytes, b200norm_stream_t stream) {
  if (b200norm_status st = check_layer_shape(rows, hidden, T, M)) return st;
  if (!dx && !dgamma && !dbeta && !dbias) return ok();
  if (rows > 0 && (!dy || !s || !mean || !inv_std_var || !gamma))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "dy, s, mean, inv_std_var and gamma are required");
  const size_t es = dtype_size(to_dtype(T)), ms = dtype_size(to_dtype(M));
  const size_t tb = static_cast<size_t>(rows) * hidden * es, sb = static_cast<size_t>(rows) * 4;
  const Tensor ts[] = {{dy, tb, es, "dy", false}, {s, tb, es, "s", false},
                       {gamma, hidden * ms, ms, "gamma", false}, {ds, tb, es, "ds", false},
                       {dx, tb, es, "dx", true}, {dgamma, hidden * ms, ms, "dgamma", true},
                       {dbeta, hidden * ms, ms, "dbeta", true},
                       {dbias, hidden * es, es, "dbias", true},
                       {mean, sb, 4, "mean", false}, {inv_std_var, sb, 4, "inv_std_var", false}};
  if (b200norm_status st = check_tensors(ts, 10)) return st;
  const size_t need = rows > 0 ? layer_grad_workspace_bytes(rows, hidden) : 0;
  if (b200norm_status st = check_workspace(workspace, workspace_bytes, need, ts, 10)) return st;
  LayerGradCall c{dy, s, mean, inv_std_var, gamma, ds, dx, dgamma, dbeta, dbias, rows, hidden,
                  to_dtype(T), to_dtype(M), workspace,
                  hidden % static_cast<int64_t>(16 / es) == 0 && all_aligned16(ts, 5)};
  cudaError_t e = launch_layer_grad(c, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "skip_layer_grad launch");
  return ok();
}

size_t b200norm_linear_workspace_size(int64_t rows, int64_t in_features, int64_t out_features,
                                      b200norm_dtype T, int aligned16) {
  if (check_linear_shape(rows, in_features, out_features, T, 0) != B200NORM_OK) return 0;
  return linear_plan(rows, in_features, out_features, to_dtype(T), aligned16 != 0).bytes;
}

b200norm_status b200norm_linear(const void* x, const void* weight, const void* bias,
                                const void* residual, void* y, void* z, int64_t rows,
                                int64_t in_features, int64_t out_features, b200norm_dtype T,
                                int activation, void* workspace, size_t workspace_bytes,
                                b200norm_stream_t stream) {
  if (b200norm_status st = check_linear_shape(rows, in_features, out_features, T, activation))
    return st;
  if (rows == 0) return ok();
  if (!x || !weight || !y)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "x, weight and y are required");
  const size_t es = dtype_size(to_dtype(T));
  const size_t xb = static_cast<size_t>(rows) * in_features * es;
  const size_t yb = static_cast<size_t>(rows) * out_features * es;
  const Tensor ts[] = {{x, xb, es, "x", false},
                       {weight, static_cast<size_t>(out_features) * in_features * es, es,
                        "weight", false},
                       {bias, out_features * es, es, "bias", false},
                       {residual, yb, es, "residual", false}, {y, yb, es, "y", true},
                       {z, yb, es, "z", true}};
  if (b200norm_status st = check_tensors(ts, 6)) return st;
  const LinearPlan plan =
      linear_plan(rows, in_features, out_features, to_dtype(T), all_aligned16(ts, 2));
  if (b200norm_status st = check_workspace(workspace, workspace_bytes, plan.bytes, ts, 6))
    return st;
  LinearCall c{x, weight, bias, residual, y, z, rows, in_features, out_features, to_dtype(T),
               activation, workspace, g_force_linear};
  cudaError_t e = launch_linear(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported && g_force_linear.cg)
    return fail(B200NORM_ERR_UNSUPPORTED, "forced tiling cannot take this call");
  if (e != cudaSuccess) return cuda_fail(e, "linear launch");
  return ok();
}

size_t b200norm_linear_grad_workspace_size(int64_t rows, int64_t in_features,
                                           int64_t out_features, b200norm_dtype T, int activation,
                                           int aligned16) {
  if (check_linear_shape(rows, in_features, out_features, T, activation) != B200NORM_OK) return 0;
  return linear_grad_plan(rows, in_features, out_features, to_dtype(T), activation,
                          aligned16 != 0).bytes;
}

b200norm_status b200norm_linear_grad(const void* dy, const void* x, const void* weight,
                                     const void* z, void* dx, void* dw, void* db, int64_t rows,
                                     int64_t in_features, int64_t out_features, b200norm_dtype T,
                                     int activation, void* workspace, size_t workspace_bytes,
                                     b200norm_stream_t stream) {
  if (b200norm_status st = check_linear_shape(rows, in_features, out_features, T, activation))
    return st;
  if (!dx && !dw && !db) return ok();
  if (activation == kActNone) z = nullptr;
  if (rows > 0 && (!dy || (dw && !x) || (dx && !weight) || (activation != kActNone && !z)))
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "dy, x (for dw), weight (for dx) and z (with an activation) are required");
  const size_t es = dtype_size(to_dtype(T));
  const size_t xb = static_cast<size_t>(rows) * in_features * es;
  const size_t yb = static_cast<size_t>(rows) * out_features * es;
  const size_t wb = static_cast<size_t>(out_features) * in_features * es;
  const Tensor ts[] = {{dy, yb, es, "dy", false}, {dw ? x : nullptr, xb, es, "x", false},
                       {dx ? weight : nullptr, wb, es, "weight", false}, {z, yb, es, "z", false},
                       {dx, xb, es, "dx", true}, {dw, wb, es, "dw", true},
                       {db, out_features * es, es, "db", true}};
  if (b200norm_status st = check_tensors(ts, 7)) return st;
  const LinearGradPlan plan = linear_grad_plan(rows, in_features, out_features, to_dtype(T),
                                               activation, all_aligned16(ts, 3));
  const size_t need = rows > 0 ? plan.bytes : 0;
  if (b200norm_status st = check_workspace(workspace, workspace_bytes, need, ts, 7)) return st;
  LinearGradCall c{dy, x, weight, z, dx, dw, db, rows, in_features, out_features, to_dtype(T),
                   activation, workspace, g_force_linear};
  cudaError_t e = launch_linear_grad(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported && g_force_linear.cg)
    return fail(B200NORM_ERR_UNSUPPORTED, "forced tiling cannot take this call");
  if (e != cudaSuccess) return cuda_fail(e, "linear_grad launch");
  return ok();
}

size_t b200norm_gated_linear_workspace_size(int64_t rows, int64_t in_features,
                                            int64_t out_features, b200norm_dtype T,
                                            int aligned16) {
  if (check_gated_shape(rows, in_features, out_features, T, 0) != B200NORM_OK) return 0;
  return gated_plan(rows, in_features, out_features, to_dtype(T), aligned16 != 0).bytes;
}

b200norm_status b200norm_gated_linear(const void* x, const void* weight, const void* bias, void* h,
                                      void* z, int64_t rows, int64_t in_features,
                                      int64_t out_features, b200norm_dtype T, int activation,
                                      void* workspace, size_t workspace_bytes,
                                      b200norm_stream_t stream) {
  if (b200norm_status st = check_gated_shape(rows, in_features, out_features, T, activation))
    return st;
  if (rows == 0) return ok();
  if (!x || !weight || !h)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "x, weight and h are required");
  const size_t es = dtype_size(to_dtype(T));
  const size_t xb = static_cast<size_t>(rows) * in_features * es;
  const size_t hb = static_cast<size_t>(rows) * out_features * es;
  const Tensor ts[] = {{x, xb, es, "x", false},
                       {weight, static_cast<size_t>(2 * out_features) * in_features * es, es,
                        "weight", false},
                       {bias, 2 * out_features * es, es, "bias", false}, {h, hb, es, "h", true},
                       {z, 2 * hb, es, "z", true}};
  if (b200norm_status st = check_tensors(ts, 5)) return st;
  const LinearPlan plan =
      gated_plan(rows, in_features, out_features, to_dtype(T), all_aligned16(ts, 2));
  if (b200norm_status st = check_workspace(workspace, workspace_bytes, plan.bytes, ts, 5))
    return st;
  LinearCall c{x, weight, bias, nullptr, h, z, rows, in_features, out_features, to_dtype(T),
               activation, workspace, g_force_linear, true};
  cudaError_t e = launch_linear(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported && g_force_linear.cg)
    return fail(B200NORM_ERR_UNSUPPORTED, "forced tiling cannot take this call");
  if (e != cudaSuccess) return cuda_fail(e, "gated_linear launch");
  return ok();
}

size_t b200norm_gated_linear_grad_workspace_size(int64_t rows, int64_t in_features,
                                                 int64_t out_features, b200norm_dtype T,
                                                 int aligned16) {
  if (check_gated_shape(rows, in_features, out_features, T, 0) != B200NORM_OK) return 0;
  return gated_grad_plan(rows, in_features, out_features, to_dtype(T), aligned16 != 0).bytes;
}

b200norm_status b200norm_gated_linear_grad(const void* dh, const void* x, const void* weight,
                                           const void* z, void* dx, void* dw, void* db,
                                           int64_t rows, int64_t in_features,
                                           int64_t out_features, b200norm_dtype T, int activation,
                                           void* workspace, size_t workspace_bytes,
                                           b200norm_stream_t stream) {
  if (b200norm_status st = check_gated_shape(rows, in_features, out_features, T, activation))
    return st;
  if (!dx && !dw && !db) return ok();
  if (rows > 0 && (!dh || !z || (dw && !x) || (dx && !weight)))
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "dh, z, x (for dw) and weight (for dx) are required");
  const size_t es = dtype_size(to_dtype(T));
  const size_t xb = static_cast<size_t>(rows) * in_features * es;
  const size_t hb = static_cast<size_t>(rows) * out_features * es;
  const size_t wb = static_cast<size_t>(2 * out_features) * in_features * es;
  const Tensor ts[] = {{dh, hb, es, "dh", false}, {dw ? x : nullptr, xb, es, "x", false},
                       {dx ? weight : nullptr, wb, es, "weight", false},
                       {z, 2 * hb, es, "z", false}, {dx, xb, es, "dx", true},
                       {dw, wb, es, "dw", true}, {db, 2 * out_features * es, es, "db", true}};
  if (b200norm_status st = check_tensors(ts, 7)) return st;
  const LinearGradPlan plan = gated_grad_plan(rows, in_features, out_features, to_dtype(T),
                                              all_aligned16(ts + 1, 2));
  const size_t need = rows > 0 ? plan.bytes : 0;
  if (b200norm_status st = check_workspace(workspace, workspace_bytes, need, ts, 7)) return st;
  LinearGradCall c{dh, x, weight, z, dx, dw, db, rows, in_features, out_features, to_dtype(T),
                   activation, workspace, g_force_linear, true};
  cudaError_t e = launch_linear_grad(c, plan, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported && g_force_linear.cg)
    return fail(B200NORM_ERR_UNSUPPORTED, "forced tiling cannot take this call");
  if (e != cudaSuccess) return cuda_fail(e, "gated_linear_grad launch");
  return ok();
}

b200norm_status b200norm_linear_status(b200norm_stream_t stream) {
  unsigned* words = linear_status_words();
  if (!words) return fail(B200NORM_ERR_CUDA, "linear status words not available on this device");
  unsigned v[2] = {0, 0};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(v, words, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && v[0] != 0) e = cudaMemsetAsync(words, 0, sizeof(v), st);
  if (e == cudaSuccess && v[0] != 0) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "linear status read");
  if (v[0] != 0) return fail(static_cast<b200norm_status>(v[0]), "device wait %u gave up", v[1]);
  return ok();
}

// ---- query and key heads -----------------------------------------------------

b200norm_status b200norm_rotary(const b200norm_heads* queries, const b200norm_heads* keys,
                                const b200norm_rotation* rotation, int64_t batch, int64_t seq,
                                int64_t head_size, b200norm_dtype T, int inverse,
                                b200norm_stream_t stream) {
  return heads_forward(queries, keys, rotation, batch, seq, head_size, T, T, false, inverse, 0.0f,
                       stream);
}

b200norm_status b200norm_head_rms_rotary(const b200norm_heads* queries, const b200norm_heads* keys,
                                         const b200norm_rotation* rotation, int64_t batch,
                                         int64_t seq, int64_t head_size, b200norm_dtype T,
                                         b200norm_dtype M, float epsilon,
                                         b200norm_stream_t stream) {
  return heads_forward(queries, keys, rotation, batch, seq, head_size, T, M, true, 0, epsilon,
                       stream);
}

size_t b200norm_head_rms_rotary_grad_workspace_size(int64_t batch, int64_t seq,
                                                    int64_t query_heads, int64_t key_heads,
                                                    int64_t head_size) {
  if (check_heads_shape(batch, seq, query_heads, key_heads, head_size, B200NORM_F32, B200NORM_F32))
    return 0;
  if (batch * seq == 0 || query_heads + key_heads == 0) return 0;
  return head_parts_bytes(head_parts(batch * seq, query_heads, key_heads, head_size), head_size);
}

b200norm_status b200norm_head_rms_rotary_grad(
    const b200norm_heads_grad* queries, const b200norm_heads_grad* keys,
    const b200norm_rotation* rotation, int64_t batch, int64_t seq, int64_t head_size,
    b200norm_dtype T, b200norm_dtype M, float epsilon, void* workspace, size_t workspace_bytes,
    b200norm_stream_t stream) {
  const b200norm_heads_grad* given[2] = {queries, keys};
  if (b200norm_status st = check_heads_shape(batch, seq, queries ? queries->heads : 0,
                                             keys ? keys->heads : 0, head_size, T, M))
    return st;
  if (b200norm_status st = check_rotation(rotation, batch, seq, head_size)) return st;
  if (b200norm_status st = check_eps(epsilon)) return st;
  HeadsCall c = heads_call(rotation, batch, seq, head_size, T, M);
  c.norm = true;
  c.eps = epsilon;
  const size_t es = dtype_size(c.t), ms = dtype_size(c.m), gb = static_cast<size_t>(head_size) * ms;
  static const char* names[2][5] = {
      {"queries dy", "queries x", "queries dx", "queries gamma", "queries dgamma"},
      {"keys dy", "keys x", "keys dx", "keys gamma", "keys dgamma"}};
  const bool empty = batch * seq == 0;
  HeadsArg in[4], out[2];
  Range flat_in[4], flat_out[2];
  int nin = 0, nout = 0, nfin = empty ? 0 : rotation_ranges(c, flat_in), nfout = 0;
  for (int i = 0; i < 2; ++i) {
    const b200norm_heads_grad* h = given[i];
    if (!h || h->heads == 0 || (!h->dx && !h->dgamma)) continue;
    if (!aligned(h->gamma, ms) || !aligned(h->dgamma, ms))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s or %s is not aligned to its element size",
                  names[i][3], names[i][4]);
    if (h->gamma) flat_in[nfin++] = {h->gamma, gb, names[i][3]};
    if (h->dgamma) flat_out[nfout++] = {h->dgamma, gb, names[i][4]};
    auto steps = [&](const int64_t* s) { return to_strides(s, batch, seq, h->heads); };
    c.set[i] = {h->x, h->dy, h->gamma, h->dx, h->dgamma, h->heads, steps(h->x_strides),
                steps(h->dy_strides), steps(h->dx_strides)};
    if (empty) continue;
    in[nin++] = {h->dy, h->heads, h->dy_strides, names[i][0]};
    in[nin++] = {h->x, h->heads, h->x_strides, names[i][1]};
    if (h->dx) out[nout++] = {h->dx, h->heads, h->dx_strides, names[i][2]};
  }
  for (int i = 0; i < nin; ++i)
    if (b200norm_status st = check_heads(in[i], batch, seq, head_size, es)) return st;
  for (int i = 0; i < nout; ++i) {
    if (b200norm_status st = check_heads(out[i], batch, seq, head_size, es)) return st;
    if (!heads_distinct(out[i], batch, seq, head_size))
      return fail(B200NORM_ERR_INVALID_ARGUMENT, "%s overlaps itself", out[i].name);
  }
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (!heads_apart(out[i], in[j], batch, seq, head_size, es))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps %s", out[i].name,
                    in[j].name);
    const Range r = heads_range(out[i], batch, seq, head_size, es);
    for (int j = 0; j < nfin; ++j)
      if (overlaps(r, flat_in[j]))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps %s", r.name,
                    flat_in[j].name);
    for (int j = 0; j < nfout; ++j)
      if (overlaps(r, flat_out[j]))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "outputs %s and %s overlap", r.name,
                    flat_out[j].name);
  }
  if (nout == 2 && !heads_apart(out[0], out[1], batch, seq, head_size, es))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "outputs overlap");
  for (int i = 0; i < nin; ++i)
    for (int j = 0; j < nfout; ++j)
      if (overlaps(heads_range(in[i], batch, seq, head_size, es), flat_out[j]))
        return fail(B200NORM_ERR_INVALID_ARGUMENT, "output %s overlaps %s", flat_out[j].name,
                    in[i].name);
  if (b200norm_status st = check_overlaps(flat_in, nfin, flat_out, nfout)) return st;
  if (!c.set[0].heads && !c.set[1].heads) return ok();
  if (!empty) {
    Tensor all[12];
    int n = 0;
    for (int i = 0; i < nin; ++i) {
      const Range r = heads_range(in[i], batch, seq, head_size, es);
      all[n++] = {r.p, r.bytes, es, r.name, false};
    }
    for (int i = 0; i < nout; ++i) {
      const Range r = heads_range(out[i], batch, seq, head_size, es);
      all[n++] = {r.p, r.bytes, es, r.name, true};
    }
    for (int i = 0; i < nfin; ++i)
      all[n++] = {flat_in[i].p, flat_in[i].bytes, 1, flat_in[i].name, false};
    for (int i = 0; i < nfout; ++i)
      all[n++] = {flat_out[i].p, flat_out[i].bytes, 1, flat_out[i].name, true};
    const HeadParts parts = head_parts(batch * seq, c.set[0].heads, c.set[1].heads, head_size);
    const size_t need = head_parts_bytes(parts, head_size);
    if (b200norm_status st = check_workspace(workspace, workspace_bytes, need, all, n)) return st;
    c.part = static_cast<float*>(workspace);
  }
  cudaError_t e = launch_heads_grad(c, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "head_rms_rotary_grad launch");
  return ok();
}

b200norm_status b200norm_rotary_frequencies(double* inv_freq, int64_t rotary_size, double base,
                                            int scaling, double factor, double original_length,
                                            double low, double high) {
  if (rotary_size < 2 || rotary_size > kMaxHeadSize || rotary_size % 2 || !inv_freq)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "rotary_size must be even, in [2, 1024], and inv_freq given");
  if (!std::isfinite(base) || base <= 0.0)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "base must be > 0 and finite");
  if (scaling < 0 || scaling > 3)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "scaling must be 0 (none), 1 (positions), 2 (base) or 3 (by turns)");
  if (scaling != 0 && (!std::isfinite(factor) || factor <= 0.0))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "factor must be > 0 and finite");
  if (scaling == 2 && rotary_size == 2)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "scaling 2 needs more than one pair");
  if (scaling == 3 && (!std::isfinite(original_length) || original_length <= 0.0 ||
                       !std::isfinite(low) || !std::isfinite(high) || low < 0.0 || low >= high))
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "need original_length > 0 and 0 <= low < high, all finite");
  const double size = static_cast<double>(rotary_size);
  if (scaling == 2) base *= std::pow(factor, size / (size - 2.0));
  constexpr double kTwoPi = 6.283185307179586;
  for (int64_t i = 0; i < rotary_size / 2; ++i) {
    double f = std::pow(base, -2.0 * static_cast<double>(i) / size);
    if (scaling == 1) f /= factor;
    if (scaling == 3) {
      double keep = (original_length * f / kTwoPi - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = f * keep + f / factor * (1.0 - keep);
    }
    inv_freq[i] = f;
  }
  return ok();
}

// ---- testing hooks ---------------------------------------------------------

b200norm_status b200norm_testing_force_linear(int cg, int bn, int splits, int swap) {
  const bool off = cg == 0 && bn == 0 && splits == 0 && swap == 0;
  const bool some = (cg == 1 || cg == 2) && (bn == 16 || bn == 32 || bn == 64 || bn == 128 ||
                                              bn == 256) &&
                    (splits == 1 || splits == 2 || splits == 4 || splits == 8) &&
                    (swap == 0 || swap == 1);
  if (!off && !some) return fail(B200NORM_ERR_INVALID_ARGUMENT, "no such tiling");
  g_force_linear = {cg, bn, splits, swap == 1};
  return ok();
}

b200norm_status b200norm_testing_linear_stall(int on, uint64_t limit_ns) {
  if (on != 0 && on != 1) return fail(B200NORM_ERR_INVALID_ARGUMENT, "on must be 0 or 1");
  if (on && (limit_ns == 0 || limit_ns > 5000000000ull))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "limit_ns must be in (0, 5 s]");
  set_linear_stall(on ? limit_ns : 0);
  return ok();
}

b200norm_status b200norm_testing_layer_withhold(int on, uint64_t limit_ns) {
  if (on != 0 && on != 1) return fail(B200NORM_ERR_INVALID_ARGUMENT, "on must be 0 or 1");
  if (on && (limit_ns == 0 || limit_ns > 100000000ull))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "limit_ns must be in (0, 100 ms]");
  set_layer_withhold(on ? limit_ns : 0);
  return ok();
}

b200norm_status b200norm_testing_linear_withhold(int site, uint64_t limit_ns) {
  if (site && (limit_ns == 0 || limit_ns > 100000000ull))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "limit_ns must be in (0, 100 ms]");
  if (site < 0 ||
      !set_linear_withhold(static_cast<unsigned>(site),
                           site ? static_cast<unsigned>(limit_ns) : 0u))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "no such site");
  return ok();
}

b200norm_status b200norm_testing_barrier_timeout(void* workspace, size_t workspace_bytes,
                                                 uint64_t limit_ns, b200norm_stream_t stream) {
  if (!workspace || workspace_bytes < kControlBytes || !aligned(workspace, 256))
    return fail(B200NORM_ERR_WORKSPACE, "workspace missing, small or misaligned");
  if (limit_ns == 0 || limit_ns > 5000000000ull)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "limit_ns must be in (0, 5 s]");
  cudaError_t e = launch_barrier_timeout_probe(workspace, limit_ns,
                                               reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "timeout probe launch");
  return ok();
}

b200norm_status b200norm_testing_force(int row_mode, int group_route) {
  if (row_mode < 0 || row_mode > 3 || group_route < 0 || group_route == 1 || group_route > 6)
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "row_mode in {0, 1, 2, 3}, group_route in {0, 2, 3, 4, 5, 6}");
  g_force_row_mode = row_mode;
  g_force_group_route = group_route;
  return ok();
}

b200norm_status b200norm_testing_force_split(int csize, int nv) {
  const bool off = csize == 0 && nv == 0;
  const bool pow2_c = csize == 1 || csize == 2 || csize == 4 || csize == 8 || csize == 16;
  const bool pow2_v = nv == 1 || nv == 2 || nv == 4 || nv == 8;
  if (!off && !(pow2_c && pow2_v))
    return fail(B200NORM_ERR_INVALID_ARGUMENT,
                "csize in {1, 2, 4, 8, 16} and nv in {1, 2, 4, 8}, or both 0");
  g_force_csize = csize;
  g_force_nv = nv;
  return ok();
}

b200norm_status b200norm_testing_pipe_stall(int on, uint64_t limit_ns) {
  if ((on != 0 && on != 1) || (on && (limit_ns == 0 || limit_ns > 5000000000ull)))
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "on in {0, 1}; with on, limit_ns in (0, 5 s]");
  set_pipe_stall(on != 0, on ? limit_ns : 0);
  return ok();
}

b200norm_status b200norm_testing_set_pdl(int on) {
  if (on != 0 && on != 1) return fail(B200NORM_ERR_INVALID_ARGUMENT, "on must be 0 or 1");
  set_pdl_enabled(on != 0);
  return ok();
}

static b200norm_status plan_rows_query(int64_t rows, int64_t n, b200norm_dtype T, int aligned16,
                                       RowOp op, int64_t out[8]) {
  if (!dtype_ok(T) || n <= 0 || rows < 0 || !out)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "bad plan query");
  const int ve = static_cast<int>(16 / dtype_size(to_dtype(T)));
  const RowPlan p = plan_rows(rows, n, to_dtype(T), aligned16 && n % ve == 0, op);
  const int64_t v[8] = {p.mode, p.ve, p.tpr, p.nv, p.rpg, p.block, p.csize, p.grid};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
  return ok();
}

b200norm_status b200norm_testing_plan_rows(int64_t rows, int64_t n, b200norm_dtype T,
                                           int aligned16, int64_t out[8]) {
  return plan_rows_query(rows, n, T, aligned16, RowOp::SkipRms, out);
}

b200norm_status b200norm_testing_plan_gated(int64_t rows, int64_t C, b200norm_dtype T,
                                            int aligned16, int64_t out[8]) {
  return plan_rows_query(rows, C, T, aligned16, RowOp::Gated, out);
}

b200norm_status b200norm_testing_plan_group(int64_t N, int64_t C, int64_t H, int64_t W, int groups,
                                            b200norm_dtype T, b200norm_dtype M, int channels_last,
                                            int aligned16, int64_t out[8]) {
  if (!group_types_ok(T, M) || N <= 0 || C <= 0 || H <= 0 || W <= 0 || groups <= 0 ||
      C % groups != 0 || !out)
    return fail(B200NORM_ERR_INVALID_ARGUMENT, "bad plan query");
  SkipGroupCall c{};
  c.N = N;
  c.C = C;
  c.H = H;
  c.W = W;
  c.groups = groups;
  c.t = to_dtype(T);
  c.m = to_dtype(M);
  c.channels_last = channels_last != 0;
  GroupPlan p;
  cudaError_t e = plan_group(c, aligned16 != 0, 0, &p);
  if (e != cudaSuccess) return cuda_fail(e, "plan_group");
  const int64_t v[8] = {p.route, p.ve, p.nv, p.block, p.csize, p.grid, p.ctas_per_item,
                        p.pix_per_cta};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
  return ok();
}

}  // extern "C"
