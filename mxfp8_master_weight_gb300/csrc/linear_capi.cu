// C entry points of the training operators around the MXFP8 weights (declared in
// include/mxfp8_partial.h): argument validation and dispatch.  No entry point allocates
// memory, and only mxfp8_device_status waits for the GPU.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "checks.h"
#include "kernels.h"
#include "linear.h"
#include "mxfp8_partial.h"
#include "status.h"

namespace {

using mxfp8::check_tensor;
using mxfp8::cuda_status;
using mxfp8::device_info;
using mxfp8::DeviceInfo;
using mxfp8::elem_bytes;
using mxfp8::fail;
using mxfp8::is_empty;
using mxfp8::numel;
using mxfp8::ok;

constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1024;  // coordinates fit 32 bits with a tile's slack
constexpr int64_t kMaxElems = int64_t(1) << 40;

int check_extents(int64_t rows, int64_t cols, const char* what) {
  if (rows < 0 || cols < 0) return fail(MXFP8_ERR_INVALID, "%s must not be negative", what);
  if (rows > kMaxExtent || cols > kMaxExtent) return fail(MXFP8_ERR_INVALID, "%s exceed 2^31 - 1024", what);
  if (cols > 0 && rows > kMaxElems / cols) return fail(MXFP8_ERR_INVALID, "%s: more than 2^40 elements", what);
  return MXFP8_OK;
}

// A present matrix argument of at least rows x cols; *ld gets its row stride.
int check_matrix(const mxfp8_tensor* t, const char* name, int64_t rows, int64_t cols, int64_t* ld) {
  if (is_empty(t)) return fail(MXFP8_ERR_MISSING, "%s is required", name);
  if (int rc = check_tensor(t, name)) return rc;
  if (t->ndim == 1) {
    if (t->shape[0] < rows * cols)
      return fail(MXFP8_ERR_SHAPE, "%s holds %lld elements, needs %lld x %lld", name, (long long)t->shape[0],
                  (long long)rows, (long long)cols);
    *ld = cols;
  } else {
    if (t->shape[0] < rows || t->shape[1] < cols)
      return fail(MXFP8_ERR_SHAPE, "%s: shape [%lld, %lld] smaller than [%lld, %lld]", name,
                  (long long)t->shape[0], (long long)t->shape[1], (long long)rows, (long long)cols);
    *ld = t->shape[1];
  }
  return MXFP8_OK;
}

int check_vector(const mxfp8_tensor* t, const char* name, int64_t len) {
  if (is_empty(t)) return fail(MXFP8_ERR_MISSING, "%s is required", name);
  if (int rc = check_tensor(t, name)) return rc;
  if (numel(t) < len)
    return fail(MXFP8_ERR_SHAPE, "%s holds %lld elements, needs %lld", name, (long long)numel(t), (long long)len);
  return MXFP8_OK;
}

int want_dtype(const mxfp8_tensor* t, const char* name, int32_t dtype) {
  return t->dtype == dtype ? MXFP8_OK
                           : fail(MXFP8_ERR_DTYPE, "%s: wrong dtype %d (want %d)", name, int(t->dtype), int(dtype));
}

int want_float(const mxfp8_tensor* t, const char* name) {
  return t->dtype == MXFP8_DTYPE_F32 || t->dtype == MXFP8_DTYPE_BF16
             ? MXFP8_OK
             : fail(MXFP8_ERR_DTYPE, "%s: dtype must be F32 or BF16", name);
}

// Scales of a logical [rows][nblocks] grid in the GEMM layout.
int check_scales(const mxfp8_tensor* t, const char* name, int64_t rows, int64_t nblocks) {
  if (int rc = check_vector(t, name, mxfp8_swizzled_scales_size(rows, nblocks, 0))) return rc;
  if (int rc = want_dtype(t, name, MXFP8_DTYPE_U8)) return rc;
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0)
    return fail(MXFP8_ERR_INVALID, "%s: scales in the GEMM layout must be 16-byte aligned", name);
  return MXFP8_OK;
}

bool aligned(const void* p, int64_t ld, int64_t eb, int64_t to) {
  return reinterpret_cast<uintptr_t>(p) % uintptr_t(to) == 0 && (ld * eb) % to == 0;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int dtype_index(int32_t dtype) { return dtype == MXFP8_DTYPE_F32 ? 0 : 1; }

// Where a matrix lies: bytes [lo, hi), in rows of `width` bytes `pitch` bytes apart.
struct Span {
  uintptr_t lo, hi, width, pitch;
};
Span span_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t eb) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + uintptr_t(((rows - 1) * ld + cols) * eb), uintptr_t(cols * eb), uintptr_t(ld * eb)};
}
// Column ranges of one buffer interleave without sharing a byte: with one pitch, a row of y starts `off` bytes
// after a row of x, behind its end and ending before the next one.
bool overlap(const Span& x, const Span& y) {
  if (x.lo >= y.hi || y.lo >= x.hi) return false;
  if (x.pitch != y.pitch) return true;
  const uintptr_t p = x.pitch, off = y.lo >= x.lo ? (y.lo - x.lo) % p : (p - (x.lo - y.lo) % p) % p;
  return off < x.width || off + y.width > p;
}

}  // namespace

extern "C" {

int mxfp8_checkpoint_save(const mxfp8_tensor* input, mxfp8_tensor* codes_rowwise,
                          mxfp8_tensor* scale_rowwise, mxfp8_tensor* codes_colwise,
                          mxfp8_tensor* scale_colwise, int64_t rows, int64_t cols, void* stream) {
  if (int rc = check_extents(rows, cols, "rows and cols")) return rc;
  if (rows == 0 || cols == 0) return ok();
  mxfp8::CheckpointSaveParams p{};
  if (int rc = check_matrix(input, "input", rows, cols, &p.ld)) return rc;
  if (int rc = want_float(input, "input")) return rc;
  const bool row = !is_empty(codes_rowwise), col = !is_empty(codes_colwise);
  if (!row && !col) return fail(MXFP8_ERR_MISSING, "codes_rowwise or codes_colwise is required");
  if (row) {
    if (int rc = check_matrix(codes_rowwise, "codes_rowwise", rows, cols, &p.ld_r)) return rc;
    if (int rc = want_dtype(codes_rowwise, "codes_rowwise", MXFP8_DTYPE_U8)) return rc;
    if (int rc = check_scales(scale_rowwise, "scale_rowwise", rows, ceil_div(cols, mxfp8::kCkptBlock))) return rc;
    p.q_r = static_cast<uint8_t*>(codes_rowwise->data);
    p.s_r = static_cast<uint8_t*>(scale_rowwise->data);
    p.vec_r = aligned(p.q_r, p.ld_r, 1, 8);
  }
  if (col) {
    if (int rc = check_matrix(codes_colwise, "codes_colwise", rows, cols, &p.ld_c)) return rc;
    if (int rc = want_dtype(codes_colwise, "codes_colwise", MXFP8_DTYPE_U8)) return rc;
    if (int rc = check_scales(scale_colwise, "scale_colwise", cols, ceil_div(rows, mxfp8::kCkptBlock))) return rc;
    p.q_c = static_cast<uint8_t*>(codes_colwise->data);
    p.s_c = static_cast<uint8_t*>(scale_colwise->data);
    p.vec_c = aligned(p.q_c, p.ld_c, 1, 8);
  }
  p.in = input->data;
  p.rows = rows;
  p.cols = cols;
  p.vec_in = aligned(p.in, p.ld, elem_bytes(input->dtype), 8 * elem_bytes(input->dtype));
  return cuda_status(mxfp8::launch_checkpoint_save(p, dtype_index(input->dtype), static_cast<cudaStream_t>(stream)),
                     "checkpoint save launch");
}

int mxfp8_checkpoint_restore(const mxfp8_tensor* codes, const mxfp8_tensor* scale,
                             mxfp8_tensor* output, int64_t rows, int64_t cols, int32_t colwise,
                             void* stream) {
  if (int rc = check_extents(rows, cols, "rows and cols")) return rc;
  if (colwise != 0 && colwise != 1) return fail(MXFP8_ERR_INVALID, "colwise must be 0 or 1");
  if (rows == 0 || cols == 0) return ok();
  mxfp8::CheckpointRestoreParams p{};
  if (int rc = check_matrix(codes, "codes", rows, cols, &p.ld_q)) return rc;
  if (int rc = want_dtype(codes, "codes", MXFP8_DTYPE_U8)) return rc;
  const int64_t lr = colwise ? cols : rows, lc = colwise ? rows : cols;
  if (int rc = check_scales(scale, "scale", lr, ceil_div(lc, mxfp8::kCkptBlock))) return rc;
  if (int rc = check_matrix(output, "output", rows, cols, &p.ld_o)) return rc;
  if (int rc = want_float(output, "output")) return rc;
  p.q = static_cast<const uint8_t*>(codes->data);
  p.s = static_cast<const uint8_t*>(scale->data);
  p.rows = rows;
  p.cols = cols;
  p.out = output->data;
  p.colwise = colwise;
  p.vec_q = aligned(p.q, p.ld_q, 1, 8);
  p.vec_out = aligned(p.out, p.ld_o, elem_bytes(output->dtype), 8 * elem_bytes(output->dtype));
  return cuda_status(mxfp8::launch_checkpoint_restore(p, dtype_index(output->dtype), static_cast<cudaStream_t>(stream)),
                     "checkpoint restore launch");
}

int mxfp8_gemm(const mxfp8_tensor* a, const mxfp8_tensor* a_scale, const mxfp8_tensor* b,
               const mxfp8_tensor* b_scale, const mxfp8_tensor* addend, mxfp8_tensor* out, int64_t m,
               int64_t n, int64_t k, int32_t a_colwise, int32_t b_colwise, int32_t a_block,
               int32_t b_block, void* stream) {
  if (m < 0 || n < 0 || k < 0) return fail(MXFP8_ERR_INVALID, "m, n and k must not be negative");
  if (m > kMaxExtent || n > kMaxExtent || k > kMaxExtent)
    return fail(MXFP8_ERR_INVALID, "m, n or k exceeds 2^31 - 1024");
  if (a_colwise < 0 || a_colwise > 1 || b_colwise < 0 || b_colwise > 1)
    return fail(MXFP8_ERR_INVALID, "a_colwise and b_colwise must be 0 or 1");
  if ((a_block != 128 && a_block != 32) || (b_block != 128 && b_block != 32))
    return fail(MXFP8_ERR_INVALID, "a_block and b_block must be 32 or 128");
  if (m == 0 || n == 0) return ok();
  mxfp8::GemmParams p{};
  p.m = m;
  p.n = n;
  p.k = k;
  auto operand = [&](const mxfp8_tensor* t, const mxfp8_tensor* s, const char* name, const char* sname, int64_t mn,
                     int32_t colwise, int32_t block, mxfp8::GemmOperand* o) {
    o->mn = mn;
    o->colwise = colwise;
    o->block = block;
    if (k == 0) return int(MXFP8_OK);
    if (int rc = check_matrix(t, name, colwise ? k : mn, colwise ? mn : k, &o->ld)) return rc;
    if (int rc = want_dtype(t, name, MXFP8_DTYPE_U8)) return rc;
    if (int rc = check_scales(s, sname, mn, ceil_div(k, block))) return rc;
    o->codes = static_cast<const uint8_t*>(t->data);
    o->scale = static_cast<const uint8_t*>(s->data);
    if ((colwise ? k : mn) == 1) o->ld = (o->ld + 15) / 16 * 16;  // no second row: any stride will do
    o->aligned = aligned(o->codes, o->ld, 1, 16);
    return int(MXFP8_OK);
  };
  if (int rc = operand(a, a_scale, "a", "a_scale", m, a_colwise, a_block, &p.a)) return rc;
  if (int rc = operand(b, b_scale, "b", "b_scale", n, b_colwise, b_block, &p.b)) return rc;
  if (int rc = check_matrix(out, "out", m, n, &p.ld_o)) return rc;
  if (int rc = want_float(out, "out")) return rc;
  p.out = out->data;
  p.out_f32 = out->dtype == MXFP8_DTYPE_F32;
  p.vec_out = aligned(p.out, p.ld_o, elem_bytes(out->dtype), 16);
  if (!is_empty(addend)) {
    if (int rc = check_matrix(addend, "addend", m, n, &p.ld_c)) return rc;
    if (int rc = want_dtype(addend, "addend", MXFP8_DTYPE_F32)) return rc;
    p.addend = static_cast<const float*>(addend->data);
    p.vec_out = p.vec_out && aligned(p.addend, p.ld_c, 4, 16);
    const bool same = p.out_f32 && addend->data == out->data && (p.ld_c == p.ld_o || m == 1);
    if (!same && overlap(span_of(p.addend, m, n, p.ld_c, 4), span_of(p.out, m, n, p.ld_o, elem_bytes(out->dtype))))
      return fail(MXFP8_ERR_INVALID, "addend overlaps out without being the same matrix");
  }
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  const char* what = "gemm launch";
  const cudaError_t e = mxfp8::launch_gemm(p, dev, static_cast<cudaStream_t>(stream), &what);
  return cuda_status(e, what);
}

int mxfp8_device_status(void* stream) {
  unsigned n = 0;
  const cudaError_t e = mxfp8::waits_given_up(static_cast<cudaStream_t>(stream), &n);
  if (e != cudaSuccess) return cuda_status(e, "device status");
  if (n != 0) return fail(MXFP8_ERR_CUDA, "a kernel gave up waiting for its own work: its output is invalid");
  return ok();
}

int mxfp8_layer_norm_forward(const mxfp8_tensor* input, const mxfp8_tensor* weight,
                             const mxfp8_tensor* bias, mxfp8_tensor* output, mxfp8_tensor* mean,
                             mxfp8_tensor* rstd, int64_t rows, int64_t cols, float eps, void* stream) {
  if (int rc = check_extents(rows, cols, "rows and cols")) return rc;
  if (!(eps >= 0.0f)) return fail(MXFP8_ERR_INVALID, "eps must not be negative or NaN");
  if (rows == 0 || cols == 0) return ok();
  mxfp8::NormForwardParams p{};
  if (int rc = check_matrix(input, "input", rows, cols, &p.ld_x)) return rc;
  if (int rc = want_float(input, "input")) return rc;
  if (int rc = check_vector(weight, "weight", cols)) return rc;
  if (int rc = want_float(weight, "weight")) return rc;
  if (!is_empty(bias)) {
    if (int rc = check_vector(bias, "bias", cols)) return rc;
    if (int rc = want_dtype(bias, "bias", weight->dtype)) return rc;
    p.bias = bias->data;
  }
  if (int rc = check_matrix(output, "output", rows, cols, &p.ld_y)) return rc;
  if (int rc = want_dtype(output, "output", input->dtype)) return rc;
  if (int rc = check_vector(mean, "mean", rows)) return rc;
  if (int rc = want_dtype(mean, "mean", MXFP8_DTYPE_F32)) return rc;
  if (int rc = check_vector(rstd, "rstd", rows)) return rc;
  if (int rc = want_dtype(rstd, "rstd", MXFP8_DTYPE_F32)) return rc;
  p.x = input->data;
  p.rows = rows;
  p.cols = cols;
  p.weight = weight->data;
  p.y = output->data;
  p.mean = static_cast<float*>(mean->data);
  p.rstd = static_cast<float*>(rstd->data);
  p.eps = eps;
  const int64_t eb = elem_bytes(input->dtype);
  p.vec = aligned(p.x, p.ld_x, eb, 16) && aligned(p.y, p.ld_y, eb, 16) && aligned(p.weight, 0, 1, 16) &&
          aligned(p.bias, 0, 1, 16);
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  return cuda_status(mxfp8::launch_norm_forward(p, dtype_index(input->dtype), dtype_index(weight->dtype), dev,
                                                static_cast<cudaStream_t>(stream)),
                     "layer norm forward launch");
}

int64_t mxfp8_layer_norm_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxExtent || cols > kMaxExtent) return -1;
  return mxfp8::norm_partials(rows, cols) * 2 * cols * 4;
}

int mxfp8_layer_norm_backward(const mxfp8_tensor* grad_output, const mxfp8_tensor* input,
                              const mxfp8_tensor* input_scale, const mxfp8_tensor* weight,
                              const mxfp8_tensor* mean, const mxfp8_tensor* rstd,
                              mxfp8_tensor* grad_input, mxfp8_tensor* grad_weight,
                              mxfp8_tensor* grad_bias, mxfp8_tensor* workspace, int64_t rows,
                              int64_t cols, void* stream) {
  if (int rc = check_extents(rows, cols, "rows and cols")) return rc;
  if (cols == 0) return ok();
  mxfp8::NormBackwardParams p{};
  if (int rc = check_vector(grad_weight, "grad_weight", cols)) return rc;
  if (int rc = want_dtype(grad_weight, "grad_weight", MXFP8_DTYPE_F32)) return rc;
  p.dweight = static_cast<float*>(grad_weight->data);
  if (!is_empty(grad_bias)) {
    if (int rc = check_vector(grad_bias, "grad_bias", cols)) return rc;
    if (int rc = want_dtype(grad_bias, "grad_bias", MXFP8_DTYPE_F32)) return rc;
    p.dbias = static_cast<float*>(grad_bias->data);
  }
  if (rows == 0) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(p.dweight, 0, size_t(cols) * 4, st);
    if (e == cudaSuccess && p.dbias != nullptr) e = cudaMemsetAsync(p.dbias, 0, size_t(cols) * 4, st);
    return cuda_status(e, "layer norm backward");
  }
  if (int rc = check_matrix(grad_output, "grad_output", rows, cols, &p.ld_dy)) return rc;
  if (int rc = want_float(grad_output, "grad_output")) return rc;
  if (int rc = check_matrix(input, "input", rows, cols, &p.ld_x)) return rc;
  const bool codes = input->dtype == MXFP8_DTYPE_U8;
  if (codes) {
    if (int rc = check_scales(input_scale, "input_scale", rows, ceil_div(cols, mxfp8::kCkptBlock))) return rc;
    p.x_scale = static_cast<const uint8_t*>(input_scale->data);
  } else {
    if (int rc = want_dtype(input, "input", grad_output->dtype)) return rc;
    if (!is_empty(input_scale)) return fail(MXFP8_ERR_INVALID, "input_scale goes with a U8 input only");
  }
  if (int rc = check_vector(weight, "weight", cols)) return rc;
  if (int rc = want_float(weight, "weight")) return rc;
  if (int rc = check_vector(mean, "mean", rows)) return rc;
  if (int rc = want_dtype(mean, "mean", MXFP8_DTYPE_F32)) return rc;
  if (int rc = check_vector(rstd, "rstd", rows)) return rc;
  if (int rc = want_dtype(rstd, "rstd", MXFP8_DTYPE_F32)) return rc;
  if (int rc = check_matrix(grad_input, "grad_input", rows, cols, &p.ld_dx)) return rc;
  if (int rc = want_dtype(grad_input, "grad_input", grad_output->dtype)) return rc;
  const int64_t need = mxfp8_layer_norm_workspace_size(rows, cols);
  if (need > 0) {
    if (int rc = check_vector(workspace, "workspace", need)) return rc;
    if (int rc = want_dtype(workspace, "workspace", MXFP8_DTYPE_U8)) return rc;
    if (reinterpret_cast<uintptr_t>(workspace->data) % 16 != 0)
      return fail(MXFP8_ERR_INVALID, "workspace must be 16-byte aligned");
    p.workspace = static_cast<float*>(workspace->data);
  }
  p.dy = grad_output->data;
  p.rows = rows;
  p.cols = cols;
  p.x = input->data;
  p.weight = weight->data;
  p.mean = static_cast<const float*>(mean->data);
  p.rstd = static_cast<const float*>(rstd->data);
  p.dx = grad_input->data;
  const int64_t eb = elem_bytes(grad_output->dtype);
  p.vec = aligned(p.dy, p.ld_dy, eb, 16) && aligned(p.dx, p.ld_dx, eb, 16) &&
          aligned(p.x, p.ld_x, elem_bytes(input->dtype), codes ? 8 : 16) && aligned(p.weight, 0, 1, 16);
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  return cuda_status(mxfp8::launch_norm_backward(p, dtype_index(grad_output->dtype), dtype_index(weight->dtype), dev,
                                                 static_cast<cudaStream_t>(stream)),
                     "layer norm backward launch");
}

}  // extern "C"
