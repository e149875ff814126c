// Backward of the group norm with an output gate (group_norm.cuh has the mathematics and the kernel).
#include "group_norm.cuh"

using namespace gla::norm;

namespace {

// out[c] = sum over r < rows of part[r][c], always in the same order, and in pairs, so that the rounding grows with the
// logarithm of the number of rows: 32 groups of 32 threads take every 32nd row of 32 columns, eight of them joined in pairs
// at a time, and then a warp joins the groups' sums of a column.
__global__ void __launch_bounds__(1024) join_kernel(const float* part_w, const float* part_b,
                                                    float* __restrict__ dw, float* __restrict__ db, int rows, int cols) {
  // Launched while the kernel before it still runs: nothing is read before that one has ended.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float s[32][33];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!part) return;
  const int k = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + k;
  float t = 0.f;
  if (c < cols) {
#pragma unroll 2
    for (int first = g; first < rows; first += 32 * 8) {  // sixteen loads in flight: a latency for them all
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = first + 32 * i;
        v[i] = r < rows ? part[(size_t)r * cols + c] : 0.f;
      }
      t += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
  s[g][k] = t;
  __syncthreads();
  t = s[k][g];  // of the group k, column g
#pragma unroll
  for (int d = 1; d < 32; d *= 2) t += __shfl_xor_sync(0xffffffffu, t, d);
  if (k == 0 && blockIdx.x * 32 + g < cols) out[blockIdx.x * 32 + g] = t;
}

}  // namespace

extern "C" size_t gla_group_norm_bwd_workspace(int B, int H, int T, int D, int weight_rows, int need_dw,
                                               int need_db) {
  if (check_sizes(B, H, T, D, weight_rows) != GLA_OK || T == 0) return 0;
  const size_t one = gla::align256((size_t)row_blocks((long long)B * T, H, D, true, false) * H * D * sizeof(float));
  return one * ((need_dw != 0) + (need_db != 0));
}

extern "C" int gla_group_norm_bwd(const void* x, const void* z, const float* w, const float* b, const void* dy,
                                  void* dx, void* dz, float* dw, float* db, int B, int H, int T, int D,
                                  int weight_rows, int kind, int act, float eps, int layout, int dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  NORM_TRY(check_sizes(B, H, T, D, weight_rows));
  NORM_TRY(check_kind(kind, act, eps, layout, dtype));
  const size_t es = esize(dtype);
  NORM_TRY(check_ptr(x, es, T > 0));
  NORM_TRY(check_ptr(z, es, T > 0 && dz));
  NORM_TRY(check_ptr(w, 4, false));
  NORM_TRY(check_ptr(b, 4, false));
  NORM_TRY(check_ptr(dy, es, T > 0));
  NORM_TRY(check_ptr(dx, es, T > 0));
  NORM_TRY(check_ptr(dz, es, false));
  NORM_TRY(check_ptr(dw, 4, false));
  NORM_TRY(check_ptr(db, 4, false));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t n_w = (size_t)weight_rows * D * sizeof(float);
  if (T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, n_w, st) != cudaSuccess) return GLA_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, n_w, st) != cudaSuccess) return GLA_ERR_CUDA;
    return GLA_OK;
  }
  const size_t need = gla_group_norm_bwd_workspace(B, H, T, D, weight_rows, dw != nullptr, db != nullptr);
  if (need > 0 && (!workspace || !gla::aligned_to(workspace, 256) || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  Args a = make_args(x, z, w, b, B, H, T, D, weight_rows, kind, eps, layout);
  a.dy = dy, a.dx = dx, a.dz = dz;
  if (dw) a.part_w = static_cast<float*>(workspace);
  if (db) a.part_b = static_cast<float*>(workspace) + (dw ? need / 2 / sizeof(float) : 0);
  const int grid = row_blocks(a.tokens, H, D, true, false), V = vector_of(a, es);
  NORM_TRY(dtype == GLA_DTYPE_BF16 ? (dispatch<gla::bf16, true>(a, V, act, grid, st))
                                   : (dispatch<float, true>(a, V, act, grid, st)));
  if (!dw && !db) return GLA_OK;
  // A shared weight row also sums over the heads: the partial rows [grid][H][D] are grid * H rows of D.
  const int rows = weight_rows == 1 ? grid * H : grid, cols = weight_rows * D;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((cols + 31) / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const float *part_w = a.part_w, *part_b = a.part_b;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel, part_w, part_b, dw, db, rows, cols);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}
