// Embedding lookup and its gradient.
//
//   lookup    out[i] = scale * table[ids[i]]
//   gradient  grad[v] = scale * sum over i with ids[i] = v of dout[i]   (or grad[v] += ...)
//
// Both are bound by bytes: one multiplication or addition per element read.  The
// gradient sums in a fixed order without floating-point atomics: the tokens are sorted
// by number (a stable counting sort, so equal tokens keep their order), the sorted list
// is cut into chunks of equal length, each chunk sums the runs of equal tokens it holds,
// and a run that crosses chunk borders is joined from the chunks' partial sums in
// ascending order.  Chunks of equal length keep the work even when one token makes up
// most of the batch.
#include "token_common.cuh"

namespace casgd {
namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// ------------------------------------------------------------------ lookup
// One thread per kV consecutive columns (kV = 1 where rows are not 16-byte aligned) and
// kRows rows, so that several independent loads are in flight.
constexpr int kRows = 4;

template <class TI, class TO, int kV>
__global__ void __launch_bounds__(256)
    embed_kernel(const TI* table, int64_t vocab, int64_t dim, int64_t ldt, Ids ids, int64_t rows,
                 float scale, int64_t padding_id, TO* out, int64_t ldo, Ctrl* ctrl) {
  wait_prior_grid();
  allow_next_grid();
  const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * kV;
  for (int64_t r0 = ((int64_t)blockIdx.y * blockDim.y + threadIdx.y) * kRows; r0 < rows;
       r0 += (int64_t)gridDim.y * blockDim.y * kRows) {
    if (col >= dim) continue;
    Pack<TI, kV> v[kRows];
    bool have[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t id = r0 + j < rows ? ids.at(r0 + j) : padding_id;
      have[j] = id != padding_id && id >= 0 && id < vocab;
      if (r0 + j < rows && id != padding_id && !have[j] && col == 0) set_status(ctrl, ST_BAD_INDEX);
      if (have[j]) v[j] = *reinterpret_cast<const Pack<TI, kV>*>(table + id * ldt + col);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (r0 + j >= rows) break;
      Pack<TO, kV> o;
#pragma unroll
      for (int e = 0; e < kV; ++e)
        o.v[e] = Elem<TO>::put(have[j] ? scale * Elem<TI>::get(v[j].v[e]) : 0.0f);
      *reinterpret_cast<Pack<TO, kV>*>(out + (r0 + j) * ldo + col) = o;
    }
  }
}

template <class TI, class TO>
cudaError_t embed_typed(const Mat& t, Ids ids, float scale, int64_t pad, const Mat& o, Ctrl* ctrl,
                        Ctx& c) {
  constexpr int kV = 16 / (sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));
  const bool vec = t.cols % kV == 0 && rows_aligned(t, kV * sizeof(TI)) &&
                   rows_aligned(o, kV * sizeof(TO));
  const int64_t groups = vec ? t.cols / kV : t.cols;
  unsigned tx = 32;
  while (tx < 256 && tx < groups) tx *= 2;
  const unsigned ty = 256 / tx;
  const int64_t gy = (o.rows + ty * kRows - 1) / (ty * kRows);
  const dim3 grid((unsigned)((groups + tx - 1) / tx), (unsigned)(gy < 65535 ? gy : 65535));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(tx, ty);
  cfg.stream = c.stream;
  add_pdl_attr(c, cfg, attr);
  ++c.launches;
  return cudaLaunchKernelEx(&cfg, vec ? embed_kernel<TI, TO, kV> : embed_kernel<TI, TO, 1>,
                            (const TI*)t.p, t.rows, t.cols, t.ld, ids, o.rows, scale, pad,
                            (TO*)o.p, o.ld, ctrl);
}

template <class TI>
cudaError_t embed_from(const Mat& t, Ids ids, float s, int64_t pad, const Mat& o, Ctrl* ctrl,
                       Ctx& c) {
  if (o.dtype == CASGD_F32) return embed_typed<TI, float>(t, ids, s, pad, o, ctrl, c);
  if (o.dtype == CASGD_BF16) return embed_typed<TI, __nv_bfloat16>(t, ids, s, pad, o, ctrl, c);
  return embed_typed<TI, __half>(t, ids, s, pad, o, ctrl, c);
}

// ------------------------------------------------------------------ sort by token
// Stable radix sort of (token, position) pairs, least significant digit first.  A token
// that is dropped (padding, or out of range) sorts last, with the key `vocab`.  Tiles of
// kTile pairs; per pass a tile's scatter base of a digit is the count of smaller digits
// everywhere plus that of the same digit in the tiles before it, summed by the tile
// itself from the per-tile counts (a few hundred KB from L2), so a pass is one launch:
// the scatter of pass p adds each pair to the counts of pass p+1 at its destination.
constexpr int kSortThreads = 256;
constexpr int kSortItems = 8;  // per thread
constexpr int kTile = kSortThreads * kSortItems;
constexpr int kMaxRadix = 512;
constexpr int kMaxPasses = 4;

struct SortPlan {
  int passes, bits;  // digits of `bits` bits
  int radix() const { return 1 << bits; }
};
SortPlan sort_plan(int64_t vocab) {
  int need = 1;
  while (need < 32 && (vocab >> need) != 0) ++need;  // keys 0 .. vocab
  SortPlan p;
  p.passes = (need + 8) / 9;
  p.bits = (need + p.passes - 1) / p.passes;
  return p;
}

struct GradLayout {
  int64_t tiles, chunks, chunk;
  size_t off_count, off_key[2], off_pos[2], off_seen, off_part, off_owner, total;
  size_t count_bytes, seen_bytes;
};

GradLayout grad_layout(int64_t rows, int64_t vocab, int64_t dim) {
  GradLayout L;
  L.tiles = rows > 0 ? (rows + kTile - 1) / kTile : 1;
  // Chunk length: enough chunks to fill the GPU, few enough partial sums for long lists.
  L.chunk = 8;
  while (L.chunk < 64 && rows / L.chunk > 2048) L.chunk *= 2;
  L.chunks = (rows + L.chunk - 1) / L.chunk;
  const SortPlan p = sort_plan(vocab);
  size_t o = align_up(sizeof(Ctrl));
  L.off_count = o;
  L.count_bytes = align_up((size_t)p.passes * L.tiles * p.radix() * 4);
  o += L.count_bytes;
  L.off_seen = o;
  L.seen_bytes = align_up((size_t)(vocab / 32 + 1) * 4);
  o += L.seen_bytes;
  L.off_owner = o;  // word 0: how many; then the first chunk of every run that crosses
  o += align_up((size_t)(L.chunks + 1) * 4);
  for (int i = 0; i < 2; ++i) {
    L.off_key[i] = o;
    o += align_up((size_t)rows * 4);
    L.off_pos[i] = o;
    o += align_up((size_t)rows * 4);
  }
  L.off_part = o;  // per chunk: the sum of its first run, then of its last
  o += align_up((size_t)L.chunks * 2 * dim * 4);
  L.total = o;
  return L;
}

struct SortArgs {
  Ids ids;
  int64_t rows, vocab, padding_id, tiles;
  int bits, passes;
  uint32_t* count;  // [pass][tile][digit]
  uint32_t* seen;   // one bit per table row that receives a gradient
  uint32_t* owner;
  int64_t seen_words;
  Ctrl* ctrl;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int64_t i, bool& bad) {
  const int64_t id = a.ids.at(i);
  bad = id != a.padding_id && (id < 0 || id >= a.vocab);
  return id == a.padding_id || bad ? (uint32_t)a.vocab : (uint32_t)id;
}

// Clears what the later launches add to, and counts the first digit of every tile.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  __shared__ uint32_t cnt[kMaxRadix];
  wait_prior_grid();
  allow_next_grid();
  const int radix = 1 << a.bits;
  const int64_t gid = (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
  const int64_t gn = (int64_t)gridDim.x * kSortThreads;
  for (int64_t i = gid; i < a.seen_words; i += gn) a.seen[i] = 0;
  for (int64_t i = gid; i < (int64_t)(a.passes - 1) * a.tiles * radix; i += gn)
    a.count[a.tiles * radix + i] = 0;
  if (gid == 0) a.owner[0] = 0;
  for (int d = threadIdx.x; d < radix; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  bool any_bad = false;
  for (int j = 0; j < kSortItems; ++j) {
    const int64_t i = t0 + j * kSortThreads + threadIdx.x;
    if (i >= a.rows) break;
    bool bad;
    const uint32_t k = sort_key(a, i, bad);
    any_bad |= bad;
    atomicAdd(&cnt[k & (radix - 1)], 1u);
  }
  if (any_bad) set_status(a.ctrl, ST_BAD_INDEX);
  __syncthreads();
  for (int d = threadIdx.x; d < radix; d += kSortThreads)
    a.count[(int64_t)blockIdx.x * radix + d] = cnt[d];
}

// One pass.  A warp owns kSortItems * 32 consecutive pairs; equal digits within a warp
// are ranked by lane (match), earlier items of the warp by its own counters, earlier
// warps by a sum over the counters.
__global__ void __launch_bounds__(kSortThreads)
    sort_scatter_kernel(SortArgs a, int pass, const uint32_t* key_in, const uint32_t* pos_in,
                        uint32_t* key_out, uint32_t* pos_out) {
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t cnt[kWarps][kMaxRadix];
  __shared__ uint32_t base[kMaxRadix];
  __shared__ uint32_t wsum[kWarps];
  wait_prior_grid();
  allow_next_grid();
  const int radix = 1 << a.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile = blockIdx.x;
  for (int d = threadIdx.x; d < radix; d += kSortThreads)
    for (int w = 0; w < kWarps; ++w) cnt[w][d] = 0;
  // counts: of this digit in earlier tiles, and of every tile
  const uint32_t* cp = a.count + (int64_t)pass * a.tiles * radix;
  uint32_t before[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = 2 * threadIdx.x + h;
    if (d < radix)
      for (int64_t t = 0; t < a.tiles; ++t) {
        const uint32_t v = cp[t * radix + d];
        total[h] += v;
        if (t < tile) before[h] += v;
      }
  }
  // exclusive sum of the totals over the digits
  uint32_t run = total[0] + total[1];
  uint32_t inc = run;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  uint32_t pre = inc - run;
  for (int w = 0; w < warp; ++w) pre += wsum[w];
  if (2 * threadIdx.x < radix) base[2 * threadIdx.x] = pre + before[0];
  if (2 * threadIdx.x + 1 < radix) base[2 * threadIdx.x + 1] = pre + total[0] + before[1];

  const int64_t w0 = tile * kTile + (int64_t)warp * kSortItems * 32;
  uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int64_t i = w0 + j * 32 + lane;
    bool bad;
    key[j] = i >= a.rows ? 0u : key_in ? key_in[i] : sort_key(a, i, bad);
    pos[j] = i >= a.rows ? 0u : pos_in ? pos_in[i] : (uint32_t)i;
  }
  const int sh = pass * a.bits;
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const bool in = w0 + j * 32 + lane < a.rows;
    const uint32_t d = in ? (key[j] >> sh) & (radix - 1) : 0xffffffffu;
    const uint32_t same = __match_any_sync(0xffffffffu, d);
    const int first = __ffs(same) - 1;
    uint32_t old = 0;
    if (in && lane == first) {
      old = cnt[warp][d];
      cnt[warp][d] = old + __popc(same);
    }
    old = __shfl_sync(0xffffffffu, old, first);
    rank[j] = old + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < radix; d += kSortThreads) {
    uint32_t sum = base[d];
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t v = cnt[w][d];
      cnt[w][d] = sum;
      sum += v;
    }
  }
  __syncthreads();
  uint32_t* next = pass + 1 < a.passes ? a.count + (int64_t)(pass + 1) * a.tiles * radix : nullptr;
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    if (w0 + j * 32 + lane >= a.rows) break;
    const uint32_t to = cnt[warp][(key[j] >> sh) & (radix - 1)] + rank[j];
    key_out[to] = key[j];
    pos_out[to] = pos[j];
    if (next)
      atomicAdd(&next[(int64_t)(to / kTile) * radix + ((key[j] >> (sh + a.bits)) & (radix - 1))],
                1u);
    if (pass == 0 && key[j] < (uint32_t)a.vocab)
      atomicOr(&a.seen[key[j] >> 5], 1u << (key[j] & 31));
  }
}

// ------------------------------------------------------------------ sums of the runs
struct GradArgs {
  const uint32_t *key, *pos, *seen;
  uint32_t* owner;
  float* part;
  int64_t rows, vocab, dim, ldd, ldg, chunk, chunks;
  float scale;
  int accumulate;
  unsigned sum_blocks;  // blocks that sum; the others clear rows no token names
};

// kV columns of one table row: grad = scale * sum, or grad += scale * sum.
template <class TG, int kV>
__device__ __forceinline__ void put_row(TG* g, const float (&s)[kV], float scale, bool acc) {
  Pack<TG, kV>* p = reinterpret_cast<Pack<TG, kV>*>(g);
  Pack<TG, kV> o;
  if (acc) o = *p;
#pragma unroll
  for (int e = 0; e < kV; ++e)
    o.v[e] = Elem<TG>::put(acc ? Elem<TG>::get(o.v[e]) + scale * s[e] : scale * s[e]);
  *p = o;
}

// blockDim (tx, ty): tx threads of kV columns each, ty chunks.  Items (chunk group, column
// slab) with the slabs of a chunk group side by side.
template <class TD, class TG, int kV>
__global__ void __launch_bounds__(128) grad_sum_kernel(GradArgs a, const TD* dout, TG* grad) {
  wait_prior_grid();
  allow_next_grid();
  if (blockIdx.x >= a.sum_blocks) {  // rows that no token names: zeros
    const int64_t nb = gridDim.x - a.sum_blocks;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int64_t warp = ((int64_t)(blockIdx.x - a.sum_blocks) * 128 + tid) >> 5;
    const int lane = tid & 31;
    for (int64_t v = warp; v < a.vocab; v += nb * 4) {
      if (a.seen[v >> 5] >> (v & 31) & 1u) continue;
      TG* g = grad + v * a.ldg;
      for (int64_t col = (int64_t)lane * kV; col < a.dim; col += 32 * kV) {
        Pack<TG, kV> z;
#pragma unroll
        for (int e = 0; e < kV; ++e) z.v[e] = Elem<TG>::put(0.0f);
        *reinterpret_cast<Pack<TG, kV>*>(g + col) = z;
      }
    }
    return;
  }
  const int64_t slabs = (a.dim + (int64_t)blockDim.x * kV - 1) / ((int64_t)blockDim.x * kV);
  const int64_t slab = blockIdx.x % slabs;
  const int64_t c = blockIdx.x / slabs * blockDim.y + threadIdx.y;
  const int64_t col = (slab * blockDim.x + threadIdx.x) * kV;
  if (c >= a.chunks || col >= a.dim) return;
  const int64_t i0 = c * a.chunk, i1 = i0 + a.chunk < a.rows ? i0 + a.chunk : a.rows;
  const uint32_t before = i0 > 0 ? a.key[i0 - 1] : 0xffffffffu;
  const uint32_t after = i1 < a.rows ? a.key[i1] : 0xffffffffu;
  float s[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) s[e] = 0.0f;
  int64_t start = i0;  // of the run being summed
  constexpr int kU = 4;
  for (int64_t i = i0; i < i1; i += kU) {
    Pack<TD, kV> v[kU];
    uint32_t k[kU + 1];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      k[j] = i + j < i1 ? a.key[i + j] : (uint32_t)a.vocab;
      if (k[j] < (uint32_t)a.vocab)
        v[j] = *reinterpret_cast<const Pack<TD, kV>*>(dout + (int64_t)a.pos[i + j] * a.ldd + col);
    }
    k[kU] = i + kU < i1 ? a.key[i + kU] : after;
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      if (k[j] >= (uint32_t)a.vocab) break;  // dropped tokens sort last
#pragma unroll
      for (int e = 0; e < kV; ++e) s[e] += Elem<TD>::get(v[j].v[e]);
      const uint32_t nk = i + j + 1 < i1 ? k[j + 1] : after;
      const bool last = i + j + 1 == i1;
      if (!last && nk == k[j]) continue;
      // the run ends here, or the chunk does
      const bool from = start == i0 && before == k[j];
      const bool on = last && after == k[j];
      if (!from && !on) {
        put_row<TG, kV>(grad + (int64_t)k[j] * a.ldg + col, s, a.scale, a.accumulate != 0);
      } else {
        Pack<float, kV> o;
#pragma unroll
        for (int e = 0; e < kV; ++e) o.v[e] = s[e];
        *reinterpret_cast<Pack<float, kV>*>(a.part + (2 * c + (from ? 0 : 1)) * a.dim + col) = o;
        if (!from && slab == 0 && threadIdx.x == 0)
          a.owner[1 + atomicAdd(&a.owner[0], 1u)] = (uint32_t)c;
      }
#pragma unroll
      for (int e = 0; e < kV; ++e) s[e] = 0.0f;
      start = i + j + 1;
    }
  }
}

// Runs that cross chunk borders: the last partial of the chunk that the run starts in,
// then the first partials of the chunks it goes on into, ascending.  A block joins 64
// columns of one run: four groups of threads each add every fourth chunk in order, and
// the four sums are added in a fixed order.
template <class TG>
__global__ void __launch_bounds__(256) grad_join_kernel(GradArgs a, TG* grad) {
  __shared__ float red[4][64];
  wait_prior_grid();
  allow_next_grid();
  const int64_t n = a.owner[0];
  const int64_t slabs = (a.dim + 63) / 64;
  const int x = threadIdx.x & 63, q = threadIdx.x >> 6;
  for (int64_t it = blockIdx.x; it < n * slabs; it += gridDim.x) {
    const int64_t c = a.owner[1 + it / slabs];
    const int64_t col = it % slabs * 64 + x;
    const uint32_t k = a.key[(c + 1) * a.chunk];
    // chunks c+1 .. e-1 start with this run
    int64_t lo = c + 1, hi = a.chunks;
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (a.key[mid * a.chunk] == k) lo = mid + 1; else hi = mid;
    }
    float s = 0.0f;
    if (col < a.dim) {
      if (q == 0) s = a.part[(2 * c + 1) * a.dim + col];
#pragma unroll 4
      for (int64_t j = c + 1 + q; j < lo; j += 4) s += a.part[2 * j * a.dim + col];
    }
    red[q][x] = s;
    __syncthreads();
    if (q == 0 && col < a.dim) {
      const float t[1] = {(red[0][x] + red[1][x]) + (red[2][x] + red[3][x])};
      put_row<TG, 1>(grad + (int64_t)k * a.ldg + col, t, a.scale, a.accumulate != 0);
    }
    __syncthreads();
  }
}

template <class... P, class... A>
cudaError_t launch(Ctx& c, unsigned grid, dim3 block, void (*fn)(P...), A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.stream = c.stream;
  add_pdl_attr(c, cfg, attr);
  ++c.launches;
  return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

template <class TD, class TG>
cudaError_t sum_typed(const Mat& d, const Mat& g, GradArgs a, Ctx& c) {
  constexpr int kV = 16 / sizeof(TD);
  const bool vec = rows_aligned(d, 16) && rows_aligned(g, kV * sizeof(TG));
  const int v = vec ? kV : 1;
  const int64_t groups = (a.dim + v - 1) / v;
  unsigned tx = 8;
  while (tx < 128 && tx < groups) tx *= 2;
  const unsigned ty = 128 / tx;
  const int64_t slabs = (groups + tx - 1) / tx;
  a.sum_blocks = (unsigned)((a.chunks + ty - 1) / ty * slabs);
  // clearing blocks: enough warps to fill the GPU beside the summing ones
  const int64_t want = (a.vocab + 3) / 4;
  const unsigned clear =
      a.accumulate ? 0u : (unsigned)(want < 8 * c.num_sms ? want : 8 * (int64_t)c.num_sms);
  cudaError_t e = cudaSuccess;
  if (a.sum_blocks + clear > 0)
    e = launch(c, a.sum_blocks + clear, dim3(tx, ty),
               vec ? grad_sum_kernel<TD, TG, kV> : grad_sum_kernel<TD, TG, 1>, a,
               (const TD*)d.p, (TG*)g.p);
  if (e != cudaSuccess || a.chunks < 2) return e;
  return launch(c, 2 * c.num_sms, dim3(256), grad_join_kernel<TG>, a, (TG*)g.p);
}

template <class TD>
cudaError_t sum_from(const Mat& d, const Mat& g, const GradArgs& a, Ctx& c) {
  if (g.dtype == CASGD_F32) return sum_typed<TD, float>(d, g, a, c);
  if (g.dtype == CASGD_BF16) return sum_typed<TD, __nv_bfloat16>(d, g, a, c);
  return sum_typed<TD, __half>(d, g, a, c);
}

}  // namespace

size_t embed_workspace_bytes(int64_t rows, int64_t vocab, int64_t dim) {
  return grad_layout(rows, vocab, dim).total;
}

cudaError_t launch_embed(const Mat& t, Ids ids, float scale, int64_t pad, const Mat& o, Ctrl* ctrl,
                         Ctx& c) {
  if (o.rows == 0) return cudaSuccess;
  if (t.dtype == CASGD_F32) return embed_from<float>(t, ids, scale, pad, o, ctrl, c);
  if (t.dtype == CASGD_BF16) return embed_from<__nv_bfloat16>(t, ids, scale, pad, o, ctrl, c);
  return embed_from<__half>(t, ids, scale, pad, o, ctrl, c);
}

cudaError_t launch_embed_grad(const Mat& d, Ids ids, float scale, int64_t pad, bool accumulate,
                              const Mat& g, void* ws, Ctx& c) {
  const GradLayout L = grad_layout(d.rows, g.rows, d.cols);
  const SortPlan sp = sort_plan(g.rows);
  char* base = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<uint32_t*>(base + o); };
  SortArgs s{ids, d.rows, g.rows, pad, L.tiles, sp.bits, sp.passes, at(L.off_count),
             at(L.off_seen), at(L.off_owner), (int64_t)(L.seen_bytes / 4),
             reinterpret_cast<Ctrl*>(ws)};
  cudaError_t e = launch(c, (unsigned)L.tiles, dim3(kSortThreads), sort_count_kernel, s);
  const uint32_t *kin = nullptr, *pin = nullptr;
  for (int p = 0; p < sp.passes && d.rows > 0 && e == cudaSuccess; ++p) {
    uint32_t *ko = at(L.off_key[p & 1]), *po = at(L.off_pos[p & 1]);
    e = launch(c, (unsigned)L.tiles, dim3(kSortThreads), sort_scatter_kernel, s, p, kin, pin, ko,
               po);
    kin = ko;
    pin = po;
  }
  if (e != cudaSuccess) return e;
  GradArgs a{kin, pin, s.seen, s.owner, reinterpret_cast<float*>(base + L.off_part), d.rows,
             g.rows, d.cols, d.ld, g.ld, L.chunk, L.chunks, scale, accumulate ? 1 : 0, 0};
  if (d.dtype == CASGD_F32) return sum_from<float>(d, g, a, c);
  if (d.dtype == CASGD_BF16) return sum_from<__nv_bfloat16>(d, g, a, c);
  return sum_from<__half>(d, g, a, c);
}

}  // namespace casgd
