// Matrix products grouped by expert.  Rows are sorted by group; group e holds rows
// offsets[e] .. offsets[e+1]-1 of X (rows x k) and Y (rows x n) and owns W_e (n x k):
//
//   Y_e = X_e W_e^T      dX_e = dY_e W_e      dW_e = dY_e^T X_e
//
// 16-bit inputs, FP32 accumulation, one rounding.  A group may be empty.
#include "token_common.cuh"

namespace casgd {
namespace {

constexpr int kB = 64, kBK = 16;

// The group's rows, held inside [0, rows] whatever the offsets say.
__device__ __forceinline__ void group_range(const GroupArgs& g, int64_t e, int64_t& r0,
                                            int64_t& r1, bool& bad) {
  const int64_t a = g.offsets[e], b = g.offsets[e + 1];
  r0 = a < 0 ? 0 : a > g.rows ? g.rows : a;
  r1 = b < r0 ? r0 : b > g.rows ? g.rows : b;
  bad = r0 != a || r1 != b || (e == 0 && a != 0);
}

// C[i][j] = sum over t of A[i*ai + t*at] * B[j*bj + t*bt], 64 x 64 per block, 4 x 4 per
// thread, through shared memory.
template <class T, int kDir>
__global__ void __launch_bounds__(256) group_simple_kernel(GroupArgs g, Ctrl* ctrl) {
  __shared__ float sa[kBK][kB + 1], sb[kBK][kB + 1];
  wait_prior_grid();
  allow_next_grid();
  const int64_t e = blockIdx.z;
  int64_t r0, r1;
  bool bad;
  group_range(g, e, r0, r1, bad);
  if (bad && threadIdx.x == 0) set_status(ctrl, ST_BAD_INDEX);
  const T* X = static_cast<const T*>(g.x);
  const T* W = static_cast<const T*>(g.w) + e * g.stride_w;
  const T* Y = static_cast<const T*>(g.y);
  const int64_t I = kDir == GROUP_DW ? g.n : r1 - r0;
  const int64_t J = kDir == GROUP_Y ? g.n : g.k;
  const int64_t D = kDir == GROUP_Y ? g.k : kDir == GROUP_DX ? g.n : r1 - r0;
  const T* A = kDir == GROUP_Y ? X + r0 * g.ldx : Y + r0 * g.ldy;
  const T* B = kDir == GROUP_DW ? X + r0 * g.ldx : W;
  const int64_t ai = kDir == GROUP_Y ? g.ldx : kDir == GROUP_DX ? g.ldy : 1;
  const int64_t at = kDir == GROUP_DW ? g.ldy : 1;
  const int64_t bj = kDir == GROUP_Y ? g.ldw : 1;
  const int64_t bt = kDir == GROUP_Y ? 1 : kDir == GROUP_DX ? g.ldw : g.ldx;
  T* C = kDir == GROUP_Y    ? static_cast<T*>(g.y) + r0 * g.ldy
         : kDir == GROUP_DX ? static_cast<T*>(g.x) + r0 * g.ldx
                            : static_cast<T*>(g.w) + e * g.stride_w;
  const int64_t ldc = kDir == GROUP_Y ? g.ldy : kDir == GROUP_DX ? g.ldx : g.ldw;
  const int64_t j0 = (int64_t)blockIdx.x * kB;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t i0 = (int64_t)blockIdx.y * kB; i0 < I; i0 += (int64_t)gridDim.y * kB) {
    float acc[4][4] = {};
    for (int64_t t0 = 0; t0 < D; t0 += kBK) {
      for (int l = threadIdx.x; l < kB * kBK; l += 256) {
        // consecutive threads along the contiguous direction
        const int ta = at == 1 ? l % kBK : l / kB, ia = at == 1 ? l / kBK : l % kB;
        const int tb = bt == 1 ? l % kBK : l / kB, jb = bt == 1 ? l / kBK : l % kB;
        sa[ta][ia] = i0 + ia < I && t0 + ta < D
                         ? Elem<T>::get(A[(i0 + ia) * ai + (t0 + ta) * at]) : 0.0f;
        sb[tb][jb] = j0 + jb < J && t0 + tb < D
                         ? Elem<T>::get(B[(j0 + jb) * bj + (t0 + tb) * bt]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < kBK; ++t)
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[p][q] += sa[t][ty + 16 * p] * sb[t][tx + 16 * q];
      __syncthreads();
    }
    for (int p = 0; p < 4; ++p)
      for (int q = 0; q < 4; ++q) {
        const int64_t i = i0 + ty + 16 * p, j = j0 + tx + 16 * q;
        if (i < I && j < J) C[i * ldc + j] = Elem<T>::put(acc[p][q]);
      }
  }
}

// Rows outside every group (after the last offset): zeros.
template <class T>
__global__ void group_rest_kernel(GroupArgs g, int dir) {
  wait_prior_grid();
  allow_next_grid();
  int64_t r = g.offsets[g.groups];
  r = r < 0 ? 0 : r;
  T* C = static_cast<T*>(dir == GROUP_Y ? g.y : g.x);
  const int64_t ld = dir == GROUP_Y ? g.ldy : g.ldx, cols = dir == GROUP_Y ? g.n : g.k;
  for (r += blockIdx.x; r < g.rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) C[r * ld + c] = Elem<T>::put(0.0f);
}

template <class T, int kDir>
cudaError_t group_typed(const GroupArgs& g, Ctrl* ctrl, Ctx& c) {
  const int64_t J = kDir == GROUP_Y ? g.n : g.k;
  const int64_t I = kDir == GROUP_DW ? g.n : g.rows;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.stream = c.stream;
  add_pdl_attr(c, cfg, attr);
  cudaError_t e = cudaSuccess;
  if (kDir != GROUP_DW && g.rows > 0) {
    cfg.gridDim = dim3(c.num_sms);
    cfg.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&cfg, group_rest_kernel<T>, g, (int)kDir);
    ++c.launches;
  }
  if (e != cudaSuccess || I == 0) return e;
  const int64_t gy = (I + kB - 1) / kB;
  cfg.gridDim = dim3((unsigned)((J + kB - 1) / kB), (unsigned)(gy < 64 ? gy : 64),
                     (unsigned)g.groups);
  cfg.blockDim = dim3(256);
  ++c.launches;
  return cudaLaunchKernelEx(&cfg, group_simple_kernel<T, kDir>, g, ctrl);
}

template <class T>
cudaError_t group_dir(GroupDir d, const GroupArgs& g, Ctrl* ctrl, Ctx& c) {
  if (d == GROUP_Y) return group_typed<T, GROUP_Y>(g, ctrl, c);
  if (d == GROUP_DX) return group_typed<T, GROUP_DX>(g, ctrl, c);
  return group_typed<T, GROUP_DW>(g, ctrl, c);
}

}  // namespace

cudaError_t launch_group(GroupDir d, const GroupArgs& g, Ctrl* ctrl, Ctx& c) {
  return g.dtype == CASGD_BF16 ? group_dir<__nv_bfloat16>(d, g, ctrl, c)
                               : group_dir<__half>(d, g, ctrl, c);
}

}  // namespace casgd
