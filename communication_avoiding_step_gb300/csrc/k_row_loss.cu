// Losses over rows of logits, with their gradients: the preference loss of pairs of
// sequences and the clipped policy loss.
//
// Both need, of each row x, the target's log probability
//   lp = x[target] - max - log(sum of exp(x - max))
// and then write g * (onehot(target) - softmax(x)) for a factor g of the row.  One
// exponential per element and pass, so the bytes of the logits and of the gradient bound
// them.  All of it is in FP32, rounded once to the logits' type.
//
//   Policy loss: g depends on the row alone, so one block reads a row for its sum and at
//   once again for its gradient: the rows in flight (two per SM) stay in L2 between, and
//   memory sees one read and one write (policy_kernel).
//   Preference loss: g depends on every row of both sequences of a pair, which do not fit
//   on chip, so the rows are read twice (pref_stats_kernel, pref_grad_kernel) with the
//   pairs' sums between (pref_pair_kernel).
//
// Rows are handled in 16-byte granules of memory, counted from the granule that holds the
// row's first element, so that rows at any alignment take the same path; the granules that
// hold elements of other rows too (at most the first and the last) go element by element.
#include "token_common.cuh"

namespace casgd {
namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
constexpr float kLog2e = 1.4426950408889634f;

// 2^t; results below the normal range are zero.
__device__ __forceinline__ float fast_exp2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// Of the values x seen: the largest x * scale (m, rounded once) and the sum s of
// 2^(x * scale - m), each exponent one fused multiply-add (m = -inf, s = 0: none seen).
// scale is log2(e) over the temperature.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float rescale(float m, float top) {
  return m == top ? 1.0f : fast_exp2(m - top);
}
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  return {m, a.s * rescale(a.m, m) + b.s * rescale(b.m, m)};
}
template <int kLanes>
__device__ __forceinline__ MaxSum join_lanes(MaxSum r) {
  float m = r.m;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = r.s * rescale(r.m, m);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return {m, s};
}

// A granule: 16 bytes as four words, each kPer elements of the logits' type (kept as
// words so that two 16-bit elements share a register).
struct alignas(16) Granule {
  uint32_t w[4];
};
template <class T>
struct Words;
template <>
struct Words<float> {
  static constexpr int kPer = 1;
  static constexpr uint32_t kLowest = 0xff800000u;  // -inf
  static __device__ __forceinline__ void get(uint32_t w, float (&f)[1]) {
    f[0] = __uint_as_float(w);
  }
  static __device__ __forceinline__ uint32_t put(const float (&f)[1]) {
    return __float_as_uint(f[0]);
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};
template <>
struct Words<__nv_bfloat16> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kLowest = 0xff80ff80u;
  static __device__ __forceinline__ void get(uint32_t w, float (&f)[2]) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t put(const float (&f)[2]) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
    return reinterpret_cast<const uint32_t&>(v);
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v = __hmax2(reinterpret_cast<const __nv_bfloat162&>(a),
                                     reinterpret_cast<const __nv_bfloat162&>(b));
    return reinterpret_cast<const uint32_t&>(v);
  }
};
template <>
struct Words<__half> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kLowest = 0xfc00fc00u;
  static __device__ __forceinline__ void get(uint32_t w, float (&f)[2]) {
    const float2 v = __half22float2(reinterpret_cast<const __half2&>(w));
    f[0] = v.x;
    f[1] = v.y;
  }
  static __device__ __forceinline__ uint32_t put(const float (&f)[2]) {
    const __half2 v = __floats2half2_rn(f[0], f[1]);
    return reinterpret_cast<const uint32_t&>(v);
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __half2 v = __hmax2(reinterpret_cast<const __half2&>(a),
                              reinterpret_cast<const __half2&>(b));
    return reinterpret_cast<const uint32_t&>(v);
  }
};
template <class T>
__device__ __forceinline__ Granule no_granule() {
  return {{Words<T>::kLowest, Words<T>::kLowest, Words<T>::kLowest, Words<T>::kLowest}};
}
// p with element e replaced by x's bits (e a constant after unrolling)
template <class T>
__device__ __forceinline__ void set_element(Granule& p, int e, T x) {
  if (sizeof(T) == 4) {
    p.w[e & 3] = reinterpret_cast<const uint32_t&>(x);
  } else {
    const uint32_t b = reinterpret_cast<const uint16_t&>(x);
    p.w[(e >> 1) & 3] = e & 1 ? (p.w[(e >> 1) & 3] & 0xffffu) | (b << 16)
                              : (p.w[(e >> 1) & 3] & 0xffff0000u) | b;
  }
}
template <class T>
__device__ __forceinline__ T element(const Granule& p, int e) {
  if (sizeof(T) == 4) return reinterpret_cast<const T&>(p.w[e & 3]);
  const uint16_t b = (uint16_t)(p.w[(e >> 1) & 3] >> (16 * (e & 1)));
  return reinterpret_cast<const T&>(b);
}
template <class T>
__device__ __forceinline__ T lowest() {
  const uint32_t w = Words<T>::kLowest;
  return reinterpret_cast<const T&>(w);
}

// Maximum and sum of kN granules (16-bit types compared two at a time).
template <class T, int kN>
__device__ __forceinline__ MaxSum granules_max_sum(const Granule (&p)[kN], float scale) {
  using W = Words<T>;
  uint32_t mw = p[0].w[0];
#pragma unroll
  for (int i = 1; i < 4 * kN; ++i) mw = W::max(mw, p[i / 4].w[i % 4]);
  float mf[W::kPer];
  W::get(mw, mf);
  const float m = fmaxf(mf[0], mf[W::kPer - 1]) * scale;
  const float base = m == -INFINITY ? 0.0f : m;
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < 4 * kN; ++i) {
    float f[W::kPer];
    W::get(p[i / 4].w[i % 4], f);
#pragma unroll
    for (int e = 0; e < W::kPer; ++e)
      s[(i * W::kPer + e) & 3] += fast_exp2(fmaf(f[e], scale, -base));
  }
  return {m, (s[0] + s[1]) + (s[2] + s[3])};
}

// A row as granules of kV elements: element 0 is element `shift` of granule 0, and
// granules whole0 .. whole1-1 hold elements of this row alone.
template <class T>
struct Row {
  static constexpr int kV = 16 / sizeof(T);
  const T* x;  // element 0
  int n, shift, granules, whole0, whole1;
  __device__ __forceinline__ Row(const T* p, int64_t cols)
      : x(p), n((int)cols), shift((int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T))),
        granules((int)((cols + shift + kV - 1) / kV)), whole0(shift ? 1 : 0),
        whole1((int)((cols + shift) / kV)) {}
  __device__ __forceinline__ int64_t first(int g) const { return (int64_t)g * kV - shift; }
  __device__ __forceinline__ bool whole(int g) const { return g >= whole0 && g < whole1; }
  // granule g; -inf in the places of other rows' elements.  kLast: not needed again (the
  // cache may drop it first).
  template <bool kLast = false>
  __device__ __forceinline__ Granule load(int g) const {
    const T* p = x + first(g);
    if (whole(g)) {
      const uint4* q = reinterpret_cast<const uint4*>(p);
      const uint4 v = kLast ? __ldcs(q) : *q;
      return {{v.x, v.y, v.z, v.w}};
    }
    Granule o = no_granule<T>();
    const int64_t i = first(g);
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (i + e >= 0 && i + e < n) set_element(o, e, p[e]);
    return o;
  }
};

template <class T>
__device__ __forceinline__ bool same_phase(const T* a, const T* b) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}
// Granule g of a gradient row (element 0 at `out`), laid over the granules of `r`.
template <class T>
__device__ __forceinline__ void put_granule(const Row<T>& r, T* out, bool aligned, int g,
                                            const Granule& p) {
  constexpr int kV = Row<T>::kV;
  T* dst = out + r.first(g);
  if (aligned && r.whole(g)) {
    __stcs(reinterpret_cast<uint4*>(dst), make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]));
  } else {
    const int64_t i = r.first(g);
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (i + e >= 0 && i + e < r.n) dst[e] = element<T>(p, e);
  }
}

// k * 2^(x * scale - m) of a granule: with k = -g / s, its gradient away from the target.
template <class T>
__device__ __forceinline__ Granule softmax_part(const Granule& x, float scale, float m, float k) {
  using W = Words<T>;
  Granule o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[W::kPer];
    W::get(x.w[i], f);
#pragma unroll
    for (int e = 0; e < W::kPer; ++e) f[e] = k * fast_exp2(fmaf(f[e], scale, -m));
    o.w[i] = W::put(f);
  }
  return o;
}

// Maximum and sum of a row by kT threads (a warp, or a block of kT); every thread gets
// them.  Two groups of granules take turns: one is loaded while the other is summed.
template <class T, int kT>
__device__ MaxSum row_max_sum(const Row<T>& r, int tid, float scale) {
  constexpr int kU = 4;
  MaxSum acc{-INFINITY, 0.0f};
  Granule cur[kU], next[kU];
  auto fetch = [&](Granule(&p)[kU], int g0) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      p[u] = g0 + u * kT < r.granules ? r.load(g0 + u * kT) : no_granule<T>();
  };
  fetch(cur, tid);
  for (int g0 = tid; g0 < r.granules; g0 += kT * kU) {
    const bool more = g0 + kT * kU < r.granules;
    if (more) fetch(next, g0 + kT * kU);
    acc = join(acc, granules_max_sum<T, kU>(cur, scale));
    if (more) {
#pragma unroll
      for (int u = 0; u < kU; ++u) cur[u] = next[u];
    }
  }
  acc = join_lanes<32>(acc);
  if (kT > 32) {
    __shared__ MaxSum part[kT / 32];
    __syncthreads();
    if ((tid & 31) == 0) part[tid >> 5] = acc;
    __syncthreads();
    acc = join_lanes<kT / 32>(part[tid & (kT / 32 - 1)]);
  }
  return acc;
}

// The target's log probability.
__device__ __forceinline__ float log_prob(float xt, MaxSum r, float scale) {
  constexpr float kLn2 = 0.6931471805599453f;
  return fmaf(xt, scale, -r.m) * kLn2 - logf(r.s);
}
// g * (1 - softmax) at the target
__device__ __forceinline__ float target_grad(float g, float xt, MaxSum r, float scale) {
  return g * (1.0f - fast_exp2(fmaf(xt, scale, -r.m)) / r.s);
}

// Writes g * (onehot - softmax), or zeros, for granules g0, g0 + step, .. below g1.
template <class T>
__device__ __forceinline__ void row_grad(const Row<T>& r, T* out, int g0, int g1, int step,
                                         float scale, MaxSum ms, int64_t target,
                                         float g, bool zero) {
  constexpr int kV = Row<T>::kV, kU = 4;
  const bool al = same_phase(r.x, out);
  const float k = -g / ms.s;
  for (int i = g0; i < g1; i += step * kU) {
    Granule v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (!zero && i + u * step < g1) v[u] = r.template load<true>(i + u * step);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int gr = i + u * step;
      if (gr >= g1) break;
      Granule o{{0u, 0u, 0u, 0u}};
      if (!zero) {
        o = softmax_part<T>(v[u], scale, ms.m, k);
        const int64_t t = target - r.first(gr);
        if (t >= 0 && t < kV) {
#pragma unroll
          for (int e = 0; e < kV; ++e)
            if (t == e)
              set_element(o, e, Elem<T>::put(target_grad(
                                    g, Elem<T>::get(element<T>(v[u], e)), ms, scale)));
        }
      }
      put_granule(r, out, al, gr, o);
    }
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

constexpr int kBlock = 256;
// Up to this many columns a warp takes a row, else a block: a block's two barriers cost
// more than a warp's longer loop there.
constexpr int64_t kWarpCols = 2048;
// Up to this many a block of 256 takes a row of the policy loss, else one of 512.
constexpr int64_t kBlockCols = 16384;

// Each row's maximum, sum and log probability; kT threads per row.
template <class T, int kT>
__global__ void __launch_bounds__(kBlock, 4) pref_stats_kernel(PrefArgs a, PrefWs w) {
  wait_prior_grid();
  allow_next_grid();
  const int tid = threadIdx.x % kT;
  constexpr int kRows = kBlock / kT;
  for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / kT; t < a.logits.rows;
       t += (int64_t)gridDim.x * kRows) {
    const int64_t target = a.targets.at(t);
    const bool bad = target >= a.logits.cols;
    if (bad && tid == 0) set_status(w.ctrl, ST_BAD_INDEX);
    if (target < 0 || bad) {
      if (tid == 0) w.coef[t] = w.lp[t] = w.m[t] = w.s[t] = 0.0f;
      continue;
    }
    const Row<T> row(static_cast<const T*>(a.logits.p) + t * a.logits.ld, a.logits.cols);
    const MaxSum r = row_max_sum<T, kT>(row, tid, kLog2e);
    if (tid == 0) {
      w.m[t] = r.m;
      w.s[t] = r.s;
      w.coef[t] = 0.0f;
      w.lp[t] = log_prob(Elem<T>::get(row.x[target]), r, kLog2e);
    }
  }
}

// One block per pair: the sequences' sums, the margin, the loss and the rows' factors.
__global__ void __launch_bounds__(kBlock) pref_pair_kernel(PrefArgs a, PrefWs w) {
  constexpr int kWarps = kBlock / 32;
  __shared__ double ssum[2][kWarps];
  __shared__ int scnt[2][kWarps];
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
    for (int64_t t = o[q] + threadIdx.x; t < o[q + 1]; t += kBlock) {
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
      for (int i = 0; i < kWarps; ++i) {
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
    for (int64_t t = o[q] + threadIdx.x; t < o[q + 1]; t += kBlock) {
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

// The gradient.  kT threads take a segment of 4 granules each of a row; segments (rows for
// warps) are dealt to the blocks in descending order, so that the rows read last by
// pref_stats_kernel, still in L2, come first.
template <class T, int kT>
__global__ void __launch_bounds__(kBlock, 5) pref_grad_kernel(PrefArgs a, PrefWs w, int64_t segs) {
  wait_prior_grid();
  allow_next_grid();
  const int tid = threadIdx.x % kT;
  constexpr int kItems = kBlock / kT, kSeg = kT * 4;
  const int64_t items = a.logits.rows * segs;
  for (int64_t it = (int64_t)blockIdx.x * kItems + threadIdx.x / kT; it < items;
       it += (int64_t)gridDim.x * kItems) {
    const int64_t rev = items - 1 - it;
    const int64_t t = rev / segs, seg = rev - t * segs;
    const int64_t target = a.targets.at(t);
    const float g = w.coef[t];
    const MaxSum ms{w.m[t], w.s[t]};
    const bool zero = target < 0 || target >= a.logits.cols || g == 0.0f;
    const Row<T> row(static_cast<const T*>(a.logits.p) + t * a.logits.ld, a.logits.cols);
    const int g1 = seg == segs - 1 ? row.granules : (int)(seg + 1) * kSeg;
    row_grad(row, static_cast<T*>(a.grad.p) + t * a.grad.ld, (int)seg * kSeg + tid, g1, kT, kLog2e, ms,
             target, g, zero);
  }
}

// ------------------------------------------------------------------ policy loss
struct PolicyWs {
  Ctrl* ctrl;
  float *loss, *kl, *clipped;  // per row
};

// What the loss reads of a row beside its logits.
struct RowInfo {
  int64_t target;  // -1: masked
  float xt, weight, old_logp, ref_logp, adv;
};

__device__ __forceinline__ bool load_info(const PolicyArgs& a, int64_t t, RowInfo& f) {
  f.target = a.targets.at(t);
  const bool bad = f.target >= a.logits.cols;
  if (bad || f.target < 0) f.target = -1;
  f.weight = a.weights[t];
  f.old_logp = a.old_logp[t];
  f.ref_logp = a.ref_logp ? a.ref_logp[t] : 0.0f;
  f.adv = a.adv[t];
  return bad;
}

// The row's loss terms (each times its weight) and g, the factor of its gradient by
// logits / temperature.
struct RowLoss {
  float lp, loss, kl, clipped, g;
  // No gradient: a masked row, one of weight zero, one held by the clip (but not one
  // that is NaN).
  __device__ __forceinline__ bool none() const { return g == 0.0f && lp == lp; }
};
__device__ __forceinline__ RowLoss policy_row(const PolicyArgs& a, const RowInfo& f, MaxSum r,
                                              float inv_t, float scale) {
  RowLoss o{0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (f.target < 0) return o;
  o.lp = log_prob(f.xt, r, scale);
  if (f.weight == 0.0f) return o;
  const float ratio = expf(o.lp - f.old_logp);
  const float held = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high);
  const bool inside =
      f.adv >= 0.0f ? ratio <= 1.0f + a.clip_high : ratio >= 1.0f - a.clip_low;
  float l = -fminf(ratio * f.adv, held * f.adv), d = inside ? -ratio * f.adv : 0.0f;
  if (a.ref_logp) {
    const float away = f.ref_logp - o.lp, em = expm1f(away);
    o.kl = f.weight * (em - away);
    l += a.kl * (em - away);
    d -= a.kl * em;
  }
  o.loss = f.weight * l;
  o.clipped = inside ? 0.0f : f.weight;
  o.g = a.grad_scale * d * f.weight * inv_t;
  return o;
}

// One row per kT threads: its sum, its loss, its gradient.  The last block to finish adds
// the rows' terms in a fixed order.  Blocks take every gridDim-th row: at kT = 512 two
// blocks per SM, so that one's loads cover the other's reduction, and few enough rows in
// flight for L2 to hold them until they are read again.
template <class T, int kT, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 4)
    policy_kernel(PolicyArgs a, PolicyWs w) {
  __shared__ int last;
  __shared__ double red[3][kThreads / 32];
  wait_prior_grid();
  allow_next_grid();
  const int tid = threadIdx.x % kT;
  constexpr int kRows = kThreads / kT;
  const float inv_t = 1.0f / a.temperature, scale = kLog2e * inv_t;
  for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / kT; t < a.logits.rows;
       t += (int64_t)gridDim.x * kRows) {
    RowInfo f;
    if (load_info(a, t, f) && tid == 0) set_status(w.ctrl, ST_BAD_INDEX);
    const Row<T> row(static_cast<const T*>(a.logits.p) + t * a.logits.ld, a.logits.cols);
    MaxSum r{0.0f, 1.0f};
    f.xt = 0.0f;
    if (f.target >= 0) {
      f.xt = Elem<T>::get(row.x[f.target]);
      r = row_max_sum<T, kT>(row, tid, scale);
    }
    const RowLoss o = policy_row(a, f, r, inv_t, scale);
    if (tid == 0) {
      a.logp[t] = o.lp;
      w.loss[t] = o.loss;
      w.kl[t] = o.kl;
      w.clipped[t] = o.clipped;
    }
    if (a.grad.p)
      row_grad(row, static_cast<T*>(a.grad.p) + t * a.grad.ld, tid, row.granules, kT, scale, r,
               f.target, o.g, f.weight == 0.0f || o.none());
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&w.ctrl->loss_done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double s[3] = {0, 0, 0};
  for (int64_t t = threadIdx.x; t < a.logits.rows; t += kThreads) {
    s[0] += __ldcg(&w.loss[t]);
    s[1] += __ldcg(&w.kl[t]);
    s[2] += __ldcg(&w.clipped[t]);
  }
#pragma unroll
  for (int e = 0; e < 3; ++e) {
#pragma unroll
    for (int h = 16; h > 0; h /= 2) s[e] += __shfl_xor_sync(0xffffffffu, s[e], h);
    if ((threadIdx.x & 31) == 0) red[e][threadIdx.x >> 5] = s[e];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double v = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) v += red[threadIdx.x][i];
    a.stats[threadIdx.x] = (float)v;
  }
  if (threadIdx.x == 0) w.ctrl->loss_done = 0;
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

unsigned blocks_for(int64_t items, int64_t most) {
  return (unsigned)(items < 1 ? 1 : items < most ? items : most);
}

template <class T, int kT>
cudaError_t pref_typed(const PrefArgs& p, const PrefWs& w, Ctx& c) {
  constexpr int kV = 16 / sizeof(T), kItems = kBlock / kT;
  const int64_t rows = p.logits.rows;
  cudaError_t e = cudaSuccess;
  if (rows)
    e = launch(c, blocks_for((rows + kItems - 1) / kItems, 1 << 20), kBlock,
               pref_stats_kernel<T, kT>, p, w);
  if (e == cudaSuccess) e = launch(c, (unsigned)p.pairs, kBlock, pref_pair_kernel, p, w);
  if (e == cudaSuccess && rows && p.grad.p) {
    // (one granule more than cols / kV for rows that do not start on one)
    int64_t segs = ((p.logits.cols + kV - 1) / kV + 1 + kT * 4 - 1) / (kT * 4);
    if (kT == 32) segs = 1;
    e = launch(c, blocks_for((rows * segs + kItems - 1) / kItems, 1 << 20), kBlock,
               pref_grad_kernel<T, kT>, p, w, segs);
  }
  return e;
}
template <class T>
cudaError_t pref_by_width(const PrefArgs& p, const PrefWs& w, Ctx& c) {
  return p.logits.cols <= kWarpCols ? pref_typed<T, 32>(p, w, c) : pref_typed<T, kBlock>(p, w, c);
}

template <class T>
cudaError_t policy_typed(const PolicyArgs& p, const PolicyWs& w, Ctx& c) {
  const int64_t rows = p.logits.rows;
  if (p.logits.cols <= kWarpCols)
    return launch(c, blocks_for((rows + 7) / 8, 4 * c.num_sms), kBlock,
                  policy_kernel<T, 32, kBlock>, p, w);
  if (p.logits.cols <= kBlockCols)
    return launch(c, blocks_for(rows, 4 * c.num_sms), kBlock, policy_kernel<T, kBlock, kBlock>, p,
                  w);
  return launch(c, blocks_for(rows, 2 * c.num_sms), 512, policy_kernel<T, 512, 512>, p, w);
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
  if (p.logits.dtype == CASGD_F32) return pref_by_width<float>(p, w, c);
  if (p.logits.dtype == CASGD_BF16) return pref_by_width<__nv_bfloat16>(p, w, c);
  return pref_by_width<__half>(p, w, c);
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
