// Losses over rows of logits, with their gradients: the preference loss of pairs of
// sequences and the clipped policy loss.
//
// Both need, of each row x, the target's log probability
//   lp = x[target] - max - log(sum of exp(x - max))
// and then write g * (onehot(target) - softmax(x)) for a factor g of the row.  A row's
// exponentials are summed against the largest value the thread has seen (a running
// maximum and sum), and the threads' pairs are joined once per row.  All of it is in
// FP32, rounded once to the logits' type.
#include "token_common.cuh"

namespace casgd {
namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
constexpr int kRowThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

// A maximum m and the sum s of exp2(t - m) over the values t seen (m = -inf, s = 0: none).
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float exp2_diff(float t, float m) {
  return t == m ? 1.0f : exp2f(t - m);  // equal infinities count as one
}
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.s + b.s};
  return {m, a.s * exp2_diff(a.m, m) + b.s * exp2_diff(b.m, m)};
}

template <class T>
__device__ MaxSum row_max_sum(const T* x, int64_t n, float scale2) {
  MaxSum r{-INFINITY, 0.0f};
  for (int64_t i = threadIdx.x; i < n; i += kRowThreads) {
    const float t = Elem<T>::get(x[i]) * scale2;
    if (t > r.m) {
      r.s = r.s * exp2f(r.m - t) + 1.0f;
      r.m = t;
    } else {
      r.s += t == -INFINITY ? 0.0f : exp2_diff(t, r.m);  // NaN stays NaN
    }
  }
  __shared__ MaxSum part[kRowThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o /= 2)
    r = join(r, {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)});
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = r;
  __syncthreads();
  r = part[0];
  for (int w = 1; w < kRowThreads / 32; ++w) r = join(r, part[w]);
  return r;
}

// g * (onehot - softmax) of a row; `zero`: zeros whatever the row holds.
template <class T>
__device__ void row_grad(const T* x, T* out, int64_t n, float scale2, MaxSum r, int64_t target,
                         float g, bool zero) {
  const float inv = 1.0f / r.s;
  for (int64_t i = threadIdx.x; i < n; i += kRowThreads) {
    float v = 0.0f;
    if (!zero) {
      const float p = exp2f(Elem<T>::get(x[i]) * scale2 - r.m) * inv;
      v = g * ((i == target ? 1.0f : 0.0f) - p);
    }
    out[i] = Elem<T>::put(v);
  }
}

// ------------------------------------------------------------------ preference loss
struct PrefLayout {
  size_t off_m, off_s, off_lp, off_coef, off_loss, total;
};
PrefLayout pref_layout(int64_t rows, int64_t pairs) {
  PrefLayout L;
  size_t o = align_up(sizeof(Ctrl));
  auto take = [&](size_t& f, size_t bytes) { f = o; o += align_up(bytes); };
  take(L.off_m, rows * 4);
  take(L.off_s, rows * 4);
  take(L.off_lp, rows * 4);
  take(L.off_coef, rows * 4);
  take(L.off_loss, pairs * 8);
  L.total = o;
  return L;
}
struct PrefWs {
  Ctrl* ctrl;
  float *m, *s, *lp, *coef;
  double* loss;
};

template <class T>
__global__ void __launch_bounds__(kRowThreads) pref_stats_kernel(PrefArgs a, PrefWs w) {
  wait_prior_grid();
  allow_next_grid();
  for (int64_t t = blockIdx.x; t < a.logits.rows; t += gridDim.x) {
    const int64_t target = a.targets.at(t);
    const bool bad = target >= a.logits.cols;
    if (bad && threadIdx.x == 0) set_status(w.ctrl, ST_BAD_INDEX);
    if (target < 0 || bad) {
      if (threadIdx.x == 0) w.coef[t] = w.lp[t] = w.m[t] = w.s[t] = 0.0f;
      continue;
    }
    const T* x = static_cast<const T*>(a.logits.p) + t * a.logits.ld;
    const MaxSum r = row_max_sum(x, a.logits.cols, kLog2e);
    if (threadIdx.x == 0) {
      w.m[t] = r.m;
      w.s[t] = r.s;
      w.coef[t] = 0.0f;
      w.lp[t] = Elem<T>::get(x[target]) - r.m / kLog2e - logf(r.s);
    }
  }
}

// One block per pair: the sequences' sums, the margin, the loss and the rows' factors.
__global__ void __launch_bounds__(256) pref_pair_kernel(PrefArgs a, PrefWs w) {
  __shared__ double ssum[2][8];
  __shared__ int scnt[2][8];
  __shared__ float coef[2];
  __shared__ int last;
  wait_prior_grid();
  allow_next_grid();
  const int64_t p = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t o[3];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    o[e] = a.offsets[2 * p + e];
    const int64_t lo = e > 0 ? o[e - 1] : 0;
    if (o[e] < lo || o[e] > a.logits.rows) bad = true;
    o[e] = o[e] < lo ? lo : o[e];
    o[e] = o[e] > a.logits.rows ? a.logits.rows : o[e];
  }
  if (bad && threadIdx.x == 0) set_status(w.ctrl, ST_BAD_INDEX);
  for (int q = 0; q < 2; ++q) {
    double s = 0.0;
    int n = 0;
    for (int64_t t = o[q] + threadIdx.x; t < o[q + 1]; t += 256) {
      const int64_t target = a.targets.at(t);
      if (target < 0 || target >= a.logits.cols) continue;
      s += w.lp[t];
      ++n;
    }
#pragma unroll
    for (int h = 16; h > 0; h /= 2) {
      s += __shfl_xor_sync(0xffffffffu, s, h);
      n += __shfl_xor_sync(0xffffffffu, n, h);
    }
    if (lane == 0) {
      ssum[q][warp] = s;
      scnt[q][warp] = n;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double lp[2];
    int n[2];
    for (int q = 0; q < 2; ++q) {
      lp[q] = 0.0;
      n[q] = 0;
      for (int i = 0; i < 8; ++i) {
        lp[q] += ssum[q][i];
        n[q] += scnt[q][i];
      }
      if (n[q] < 1 || !a.mean) n[q] = 1;
      lp[q] /= n[q];
      a.logp[2 * p + q] = (float)lp[q];
    }
    const double z = (double)a.beta * ((lp[0] - (double)a.ref[2 * p]) -
                                       (lp[1] - (double)a.ref[2 * p + 1]));
    const float zf = (float)z;
    a.margin[p] = zf;
    w.loss[p] = (1.0 - (double)a.smoothing) * loss_value(a.kind, zf, 1.0f) +
                (double)a.smoothing * loss_value(a.kind, zf, -1.0f);
    const float d = (1.0f - a.smoothing) * loss_deriv(a.kind, zf, 1.0f) +
                    a.smoothing * loss_deriv(a.kind, zf, -1.0f);
    const float g = a.grad_scale * a.beta * d / (float)a.pairs;
    coef[0] = g / n[0];
    coef[1] = -g / n[1];
    __threadfence();
    last = atomicAdd(&w.ctrl->loss_done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  for (int q = 0; q < 2; ++q)
    for (int64_t t = o[q] + threadIdx.x; t < o[q + 1]; t += 256) {
      const int64_t target = a.targets.at(t);
      if (target >= 0 && target < a.logits.cols) w.coef[t] = coef[q];
    }
  if (last && warp == 0) {  // every pair's loss is in: their mean, in a fixed order
    __threadfence();
    double s = 0.0;
    for (int64_t i = lane; i < a.pairs; i += 32) s += __ldcg(&w.loss[i]);
#pragma unroll
    for (int h = 16; h > 0; h /= 2) s += __shfl_xor_sync(0xffffffffu, s, h);
    if (lane == 0) {
      a.loss[0] = (float)(s / (double)a.pairs);
      w.ctrl->loss_done = 0;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kRowThreads) pref_grad_kernel(PrefArgs a, PrefWs w) {
  wait_prior_grid();
  allow_next_grid();
  for (int64_t t = blockIdx.x; t < a.logits.rows; t += gridDim.x) {
    const int64_t target = a.targets.at(t);
    const float g = w.coef[t];
    const bool zero = target < 0 || target >= a.logits.cols || g == 0.0f;
    row_grad(static_cast<const T*>(a.logits.p) + t * a.logits.ld,
             static_cast<T*>(a.grad.p) + t * a.grad.ld, a.logits.cols, kLog2e,
             {w.m[t], w.s[t]}, target, g, zero);
  }
}

// ------------------------------------------------------------------ policy loss
struct PolicyWs {
  Ctrl* ctrl;
  float *loss, *kl, *clipped;  // per row
};

template <class T>
__global__ void __launch_bounds__(kRowThreads) policy_kernel(PolicyArgs a, PolicyWs w) {
  __shared__ float sg;
  __shared__ int last;
  wait_prior_grid();
  allow_next_grid();
  const float inv_t = 1.0f / a.temperature, scale2 = kLog2e * inv_t;
  for (int64_t t = blockIdx.x; t < a.logits.rows; t += gridDim.x) {
    const int64_t target = a.targets.at(t);
    const bool bad = target >= a.logits.cols;
    const bool masked = target < 0 || bad;
    const T* x = static_cast<const T*>(a.logits.p) + t * a.logits.ld;
    MaxSum r{0.0f, 1.0f};
    if (!masked) r = row_max_sum(x, a.logits.cols, scale2);
    if (threadIdx.x == 0) {
      if (bad) set_status(w.ctrl, ST_BAD_INDEX);
      const float wt = masked ? 0.0f : a.weights[t];
      float lp = 0.0f, g = 0.0f, kl = 0.0f, l = 0.0f, clip = 0.0f;
      if (!masked) lp = Elem<T>::get(x[target]) * inv_t - r.m / kLog2e - logf(r.s);
      if (wt != 0.0f) {
        const float adv = a.adv[t], ratio = expf(lp - a.old_logp[t]);
        const float held = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high);
        const bool inside = adv >= 0.0f ? ratio <= 1.0f + a.clip_high : ratio >= 1.0f - a.clip_low;
        l = -fminf(ratio * adv, held * adv);
        g = inside ? -ratio * adv : 0.0f;
        clip = inside ? 0.0f : 1.0f;
        if (a.ref_logp) {
          const float away = a.ref_logp[t] - lp;
          kl = expm1f(away) - away;
          l += a.kl * kl;
          g -= a.kl * expm1f(away);
        }
      }
      a.logp[t] = lp;
      w.loss[t] = wt * l;
      w.kl[t] = wt * kl;
      w.clipped[t] = wt * clip;
      sg = a.grad_scale * g * wt * inv_t;
    }
    __syncthreads();
    const float g = sg;
    const float wt = masked ? 0.0f : a.weights[t];
    if (a.grad.p)
      row_grad(x, static_cast<T*>(a.grad.p) + t * a.grad.ld, a.logits.cols, scale2, r, target, g,
               masked || wt == 0.0f);
    __syncthreads();
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&w.ctrl->loss_done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  __shared__ double red[3][kRowThreads];
  double s[3] = {0, 0, 0};
  for (int64_t t = threadIdx.x; t < a.logits.rows; t += kRowThreads) {
    s[0] += __ldcg(&w.loss[t]);
    s[1] += __ldcg(&w.kl[t]);
    s[2] += __ldcg(&w.clipped[t]);
  }
  for (int e = 0; e < 3; ++e) red[e][threadIdx.x] = s[e];
  for (int h = kRowThreads / 2; h > 0; h /= 2) {
    __syncthreads();
    if (threadIdx.x < h)
      for (int e = 0; e < 3; ++e) red[e][threadIdx.x] += red[e][threadIdx.x + h];
  }
  if (threadIdx.x == 0) {
    for (int e = 0; e < 3; ++e) a.stats[e] = (float)red[e][0];
    w.ctrl->loss_done = 0;
  }
}

template <class... P, class... A>
cudaError_t launch(Ctx& c, unsigned grid, unsigned block, void (*fn)(P...), A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = c.stream;
  add_pdl_attr(c, cfg, attr);
  ++c.launches;
  return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

template <class T>
cudaError_t pref_typed(const PrefArgs& p, const PrefWs& w, Ctx& c) {
  const unsigned grid = (unsigned)(p.logits.rows < 65535 ? p.logits.rows : 65535);
  cudaError_t e = cudaSuccess;
  if (grid) e = launch(c, grid, kRowThreads, pref_stats_kernel<T>, p, w);
  if (e == cudaSuccess) e = launch(c, (unsigned)p.pairs, 256, pref_pair_kernel, p, w);
  if (e == cudaSuccess && grid && p.grad.p)
    e = launch(c, grid, kRowThreads, pref_grad_kernel<T>, p, w);
  return e;
}

template <class T>
cudaError_t policy_typed(const PolicyArgs& p, const PolicyWs& w, Ctx& c) {
  const int64_t rows = p.logits.rows > 0 ? p.logits.rows : 1;
  return launch(c, (unsigned)(rows < 65535 ? rows : 65535), kRowThreads, policy_kernel<T>, p, w);
}

}  // namespace

size_t preference_workspace_bytes(int64_t rows, int64_t pairs) {
  return pref_layout(rows, pairs).total;
}
size_t policy_workspace_bytes(int64_t rows) {
  return align_up(sizeof(Ctrl)) + 3 * align_up((size_t)rows * 4);
}

cudaError_t launch_preference(const PrefArgs& p, void* ws, Ctx& c) {
  const PrefLayout L = pref_layout(p.logits.rows, p.pairs);
  char* b = static_cast<char*>(ws);
  auto f = [&](size_t o) { return reinterpret_cast<float*>(b + o); };
  const PrefWs w{reinterpret_cast<Ctrl*>(b), f(L.off_m), f(L.off_s), f(L.off_lp), f(L.off_coef),
                 reinterpret_cast<double*>(b + L.off_loss)};
  if (p.logits.dtype == CASGD_F32) return pref_typed<float>(p, w, c);
  if (p.logits.dtype == CASGD_BF16) return pref_typed<__nv_bfloat16>(p, w, c);
  return pref_typed<__half>(p, w, c);
}

cudaError_t launch_policy(const PolicyArgs& p, void* ws, Ctx& c) {
  char* b = static_cast<char*>(ws) + align_up(sizeof(Ctrl));
  const size_t step = align_up((size_t)p.logits.rows * 4);
  const PolicyWs w{static_cast<Ctrl*>(ws), reinterpret_cast<float*>(b),
                   reinterpret_cast<float*>(b + step), reinterpret_cast<float*>(b + 2 * step)};
  if (p.logits.dtype == CASGD_F32) return policy_typed<float>(p, w, c);
  if (p.logits.dtype == CASGD_BF16) return policy_typed<__nv_bfloat16>(p, w, c);
  return policy_typed<__half>(p, w, c);
}

}  // namespace casgd
