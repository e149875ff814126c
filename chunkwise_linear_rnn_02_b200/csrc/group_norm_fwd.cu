// Forward of the group norm with an output gate (group_norm.cuh has the mathematics and the kernel).
#include "group_norm.cuh"

using namespace gla::norm;

extern "C" int gla_group_norm_fwd(const void* x, const void* z, const float* w, const float* b, void* y, int B, int H,
                                  int T, int D, int weight_rows, int kind, int act, float eps, int layout, int dtype,
                                  void* stream) {
  NORM_TRY(check_sizes(B, H, T, D, weight_rows));
  NORM_TRY(check_kind(kind, act, eps, layout, dtype));
  if (T == 0) return GLA_OK;
  const size_t es = esize(dtype);
  NORM_TRY(check_ptr(x, es, true));
  NORM_TRY(check_ptr(z, es, false));
  NORM_TRY(check_ptr(w, 4, false));
  NORM_TRY(check_ptr(b, 4, false));
  NORM_TRY(check_ptr(y, es, true));
  Args a = make_args(x, z, w, b, B, H, T, D, weight_rows, kind, eps, layout);
  a.y = y;
  const int grid = row_blocks(a.tokens, H, D, false, es == 4), V = vector_of(a, es);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == GLA_DTYPE_BF16 ? dispatch<gla::bf16, false>(a, V, act, grid, st)
                                 : dispatch<float, false>(a, V, act, grid, st);
}
