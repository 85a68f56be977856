// Matrix products grouped by expert.  Rows are sorted by group; group e holds rows
// offsets[e] .. offsets[e+1]-1 of X (rows x k) and Y (rows x n) and owns W_e (n x k):
//
//   Y_e = X_e W_e^T      dX_e = dY_e W_e      dW_e = dY_e^T X_e
//
// 16-bit inputs, FP32 accumulation in tensor memory, one rounding.  One persistent launch
// for all groups: every CTA reads the offsets (they live on the device, so no host has to
// know the groups' sizes), lays the groups' output tiles of 128 x BN out in one list and
// takes every gridDim-th tile.
//
//   warp 0     TMA producer: 64-deep slices of both operands into a ring of stages;
//   warp 1     issues tcgen05.mma (128 x BN x 16) into one of two TMEM accumulators, so
//              that a tile's epilogue overlaps the next tile's products;
//   warps 2-5  epilogue: TMEM -> registers -> one rounding -> shared memory (to turn rows
//              per lane into 128-byte row segments) -> masked stores.
//
// Tiles at a group's ragged end.  In Y and dX the rows are the tile's M side: rows past
// the end are other groups' and are computed and dropped (a row of the accumulator depends
// on its own row of A alone).  In dW they are the summed side: only whole steps of 16 rows
// are issued, and the rows past the end in the last step are set to zero in both operands
// in shared memory first, since zero times another group's infinity would not be zero.
// The operand layouts: k runs along the 128-byte rows of both operands in Y; in dX the
// weights are summed over their rows (n), in dW both operands are summed over their rows,
// which the MMA takes as MN-major operands, so nothing is transposed in memory.
//
// TMA needs rows on 16-byte boundaries.  Inputs without them (odd widths or pitches) are
// copied once into the workspace with padded rows; outputs without them are stored element
// by element.
#include <cstring>

#include "tc_tile.cuh"
#include "token_common.cuh"

namespace casgd {
namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

constexpr int BM = 128, BK = 64;
constexpr int kThreads = 192;
constexpr int kABytes = BM * BK * 2;
constexpr int kMaxGroups = CASGD_MAX_GROUPS;
constexpr uint64_t kTimeoutNs = 1000000000ull;
constexpr int kOutBytes = 4 * 32 * 128;  // per epilogue warp: 32 rows of 64 16-bit values

template <int BN>
struct Ring {
  static constexpr int kBBytes = BN * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr uint32_t kTmemCols = 2 * BN;
};

struct Shared {
  uint64_t full[8], empty[8], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  volatile uint32_t abort;
  int32_t tiles;
  int32_t row0[kMaxGroups + 2];   // first row of each group, held ascending
  int32_t tile0[kMaxGroups + 2];  // first tile of each group
};

template <int BN>
constexpr size_t smem_bytes() {
  return (size_t)Ring<BN>::kStages * Ring<BN>::kStageBytes + kOutBytes + sizeof(Shared) + 1024;
}

struct GroupTc {
  const int32_t* offsets;
  int rows, groups, k, n;
  uint16_t* out;
  int64_t ldo, stride_o;
  bool vec_out;  // output rows on 16-byte boundaries
  Ctrl* ctrl;
};

// Bounded wait: false (and the CTA's abort word set) if the phase does not complete in
// time or another role of this CTA gave up.
__device__ bool wait_on(uint64_t* bar, uint32_t parity, Shared* sh, Ctrl* ctrl) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (sh->abort) return false;
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      sh->abort = 1;
      atomicOr(&ctrl->status, ST_TIMEOUT);
      return false;
    }
  }
}

// Groups' first rows (each at least the one before, inside [0, rows]) and first tiles.
// Y and dX have one more group: the rows after the last offset, which receive zeros.
template <int kDir, int BN>
__device__ void lay_out_tiles(const GroupTc& a, Shared* sh) {
  const int E = a.groups;
  for (int e = threadIdx.x; e <= E; e += kThreads) sh->row0[e] = a.offsets[e];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int nt = ((kDir == GROUP_Y ? a.n : a.k) + BN - 1) / BN;
    const int per_dw = (a.n + BM - 1) / BM * nt;
    int top = 0, tiles = 0;
    bool bad = false;
    // row0 for e = 0 .. E, then (below) row0[E+1] = rows
    for (int e0 = 0; e0 <= E; e0 += 32) {
      const int e = e0 + lane;
      const int raw = e <= E ? sh->row0[e] : 0;
      int r = raw < 0 ? 0 : raw > a.rows ? a.rows : raw;
      r = r < top ? top : r;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, r, o);
        if (lane >= o && v > r) r = v;
      }
      if (e <= E) {
        if (r != raw || (e == 0 && raw != 0)) bad = true;
        sh->row0[e] = r;
      }
      top = __shfl_sync(0xffffffffu, r, 31);
    }
    if (lane == 0) sh->row0[E + 1] = a.rows;
    __syncwarp();
    const int last = kDir == GROUP_DW ? E : E + 1;
    for (int e0 = 0; e0 < last; e0 += 32) {
      const int e = e0 + lane;
      int t = 0;
      if (e < last)
        t = kDir == GROUP_DW ? per_dw : (sh->row0[e + 1] - sh->row0[e] + BM - 1) / BM * nt;
      int inc = t;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (e < last) sh->tile0[e] = tiles + inc - t;
      tiles += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      sh->tile0[last] = tiles;
      sh->tiles = tiles;
    }
    if (bad && blockIdx.x == 0) set_status(a.ctrl, ST_BAD_INDEX);
  }
  __syncthreads();
}

struct Tile {
  int e, m0, n0;   // group, first row / column of the tile (dW: of W_e)
  int row0, rows;  // the group's rows
  int nkb;         // 64-deep slices to sum (0: the tile is zeros)
};

template <int kDir, int BN>
__device__ __forceinline__ Tile tile_at(const GroupTc& a, const Shared* sh, int t) {
  int lo = 0, hi = kDir == GROUP_DW ? a.groups : a.groups + 1;  // the last e with tile0 <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sh->tile0[mid] <= t) lo = mid; else hi = mid;
  }
  Tile r;
  r.e = lo;
  r.row0 = sh->row0[lo];
  r.rows = sh->row0[lo + 1] - r.row0;
  const int local = t - sh->tile0[lo];
  const int mt = ((kDir == GROUP_DW ? a.n : r.rows) + BM - 1) / BM;
  r.n0 = local / mt * BN;
  r.m0 = local % mt * BM;
  const int depth = kDir == GROUP_Y ? a.k : kDir == GROUP_DX ? a.n : r.rows;
  r.nkb = kDir != GROUP_DW && lo == a.groups ? 0 : (depth + BK - 1) / BK;
  return r;
}

template <class T>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return reinterpret_cast<const uint32_t&>(v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(uint32_t lo, uint32_t hi) {
  const __half2 v = __floats2half2_rn(__uint_as_float(lo), __uint_as_float(hi));
  return reinterpret_cast<const uint32_t&>(v);
}

// One warp's 32 rows of a tile: 64 columns at a time, one row per lane into a staging
// buffer (16-byte chunk c of row r at slot c ^ (r % 8), so neither side has bank
// conflicts), then four rows of 128 bytes per store instruction.
template <class T, int BN>
__device__ __forceinline__ void store_tile(const GroupTc& a, uint16_t* out, int rows, int cols,
                                           uint32_t taddr, bool zero, uint8_t* stage, int lane) {
  for (int c0 = 0; c0 < BN; c0 += 64) {
    if (c0 >= cols) break;
    uint32_t lo[32], hi[32];
    if (!zero) {
      __syncwarp();
      tile::tmem_load32(taddr + c0, lo);
      tile::tmem_load32(taddr + c0 + 32, hi);
      tile::tmem_wait(lo);
      tile::tmem_wait(hi);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) lo[e] = hi[e] = 0u;
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint4 v;
      const uint32_t* s = c < 4 ? lo + 8 * c : hi + 8 * (c - 4);
      v.x = pack2<T>(s[0], s[1]);
      v.y = pack2<T>(s[2], s[3]);
      v.z = pack2<T>(s[4], s[5]);
      v.w = pack2<T>(s[6], s[7]);
      *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) * 16)) = v;
    }
    __syncwarp();
    const int c = lane & 7, col = c0 + 8 * c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (r >= rows || col >= cols) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) * 16));
      uint16_t* dst = out + (int64_t)r * a.ldo + col;
      if (a.vec_out && col + 8 <= cols) {
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int j = 0; j < 8 && col + j < cols; ++j)
          dst[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
}

// mapA: X (Y), dY (dX, dW); mapA16: the same in boxes of 16 rows (Y, dX); mapB: W (Y, dX),
// X (dW).
template <class T, int kDir, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    group_kernel(const __grid_constant__ CUtensorMap mapA,
                 const __grid_constant__ CUtensorMap mapA16,
                 const __grid_constant__ CUtensorMap mapB, const GroupTc a) {
  using R = Ring<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* out_stage = smem + (size_t)R::kStages * R::kStageBytes;
  Shared* sh = reinterpret_cast<Shared*>(out_stage + kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::kStages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->tfull[i], 1);
      mbar_init(&sh->tempty[i], 4);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tile::tmem_alloc(&sh->tmem_base, R::kTmemCols);
  wait_prior_grid();
  allow_next_grid();
  tile::fence_before();
  lay_out_tiles<kDir, BN>(a, sh);  // (synchronises the block)
  tile::fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int tiles = sh->tiles;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const Tile c = tile_at<kDir, BN>(a, sh, t);
        const int valid = c.rows - c.m0;
        // few rows (decoding): only the 16-row boxes that hold some
        const int boxes16 = kDir != GROUP_DW && valid <= 64 ? (valid + 15) / 16 : 0;
        for (int kb = 0; kb < c.nkb; ++kb) {
          if (!wait_on(&sh->empty[stage], phase ^ 1u, sh, a.ctrl)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + (size_t)stage * R::kStageBytes);
          const uint32_t sb = sa + kABytes;
          uint64_t* bar = &sh->full[stage];
          mbar_expect_tx(bar, (boxes16 ? boxes16 * 2048 : kABytes) + R::kBBytes);
          const int d = kb * BK;
          if (kDir == GROUP_DW) {
            for (int i = 0; i < BM / 64; ++i)
              tile::tma_load_2d(sa + i * 8192, &mapA, bar, c.m0 + i * 64, c.row0 + d);
            for (int i = 0; i < BN / 64; ++i)
              tile::tma_load_2d(sb + i * 8192, &mapB, bar, c.n0 + i * 64, c.row0 + d);
          } else {
            if (boxes16)
              for (int i = 0; i < boxes16; ++i)
                tile::tma_load_2d(sa + i * 2048, &mapA16, bar, d, c.row0 + c.m0 + i * 16);
            else
              tile::tma_load_2d(sa, &mapA, bar, d, c.row0 + c.m0);
            if (kDir == GROUP_Y)
              tile::tma_load_3d(sb, &mapB, bar, d, c.n0, c.e);
            else
              for (int i = 0; i < BN / 64; ++i)
                tile::tma_load_3d(sb + i * 8192, &mapB, bar, c.n0 + i * 64, d, c.e);
          }
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == R::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every copy has landed before the CTA may exit
      for (int st = 0; st < R::kStages; ++st)
        if (issued & (1u << st)) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(&sh->full[st], (last_par >> st) & 1u) &&
                 globaltimer_ns() - t0 < kTimeoutNs) {
          }
        }
    }
  } else if (warp == 1) {
    constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
    constexpr uint32_t kIdesc =
        tile::instr_desc(BM, BN, kBf16, kDir == GROUP_DW, kDir != GROUP_Y);
    constexpr uint32_t kAStep = kDir == GROUP_DW ? 128 : 2;   // 16 of the depth, >> 4
    constexpr uint32_t kBStep = kDir == GROUP_Y ? 2 : 128;
    int stage = 0, iter = 0;
    uint32_t phase = 0, tphase[2] = {0, 0};
    bool ok = true, any = false;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile c = tile_at<kDir, BN>(a, sh, t);
      if (c.nkb == 0) continue;
      const int acc = iter++ & 1;
      ok = __shfl_sync(0xffffffffu,
                       lane == 0 ? (int)wait_on(&sh->tempty[acc], tphase[acc] ^ 1u, sh, a.ctrl)
                                 : 0, 0) != 0;
      if (!ok) break;
      tphase[acc] ^= 1u;
      tile::fence_after();
      const int depth = kDir == GROUP_Y ? a.k : kDir == GROUP_DX ? a.n : c.rows;
      for (int kb = 0; kb < c.nkb; ++kb) {
        ok = __shfl_sync(0xffffffffu,
                         lane == 0 ? (int)wait_on(&sh->full[stage], phase, sh, a.ctrl) : 0,
                         0) != 0;
        if (!ok) break;
        const int left = depth - kb * BK;
        const int steps = left >= BK ? BK / 16 : (left + 15) / 16;
        uint8_t* sp = smem + (size_t)stage * R::kStageBytes;
        if (kDir == GROUP_DW && left < BK && (left & 15)) {
          // rows left .. of the last step are other groups': zero in every 64-column block
          __syncwarp();
          const int zr = steps * 16 - left;
          for (int i = lane; i < zr * 8 * (BM + BN) / 64; i += 32) {
            const int blk = i / (zr * 8), r = i / 8 % zr, ch = i & 7;
            *reinterpret_cast<uint4*>(sp + blk * 8192 + (left + r) * 128 + ch * 16) =
                make_uint4(0, 0, 0, 0);
          }
          tile::fence_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          tile::fence_after();
          const uint32_t sa = smem_u32(sp), sb = sa + kABytes;
          const uint64_t ad = tile::smem_desc(sa, kDir == GROUP_DW ? 8192 : 16, 1024);
          const uint64_t bd = tile::smem_desc(sb, kDir == GROUP_Y ? 16 : 8192, 1024);
          for (int s = 0; s < steps; ++s)
            tile::mma_16bit(tmem + (uint32_t)(acc * BN), ad + (uint64_t)(s * kAStep),
                            bd + (uint64_t)(s * kBStep), kIdesc, (kb | s) ? 1u : 0u);
          tile::mma_commit(&sh->empty[stage]);
        }
        any = true;
        if (++stage == R::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) tile::mma_commit(&sh->tfull[acc]);
    }
    if (any && lane == 0) {  // every MMA has completed before TMEM is freed
      tile::mma_commit(&sh->drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&sh->drain, 0) && globaltimer_ns() - t0 < kTimeoutNs) {
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;  // TMEM lanes 32 * quarter .. + 31
    uint8_t* stage = out_stage + (warp - 2) * (32 * 128);
    int iter = 0;
    uint32_t tphase[2] = {0, 0};
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile c = tile_at<kDir, BN>(a, sh, t);
      const int m_end = kDir == GROUP_DW ? a.n : c.rows;
      const int cols = (kDir == GROUP_Y ? a.n : a.k) - c.n0;
      const int rows = m_end - c.m0 - quarter * 32;
      uint16_t* out = a.out + (kDir == GROUP_DW
                                   ? c.e * a.stride_o + (int64_t)(c.m0 + quarter * 32) * a.ldo
                                   : (int64_t)(c.row0 + c.m0 + quarter * 32) * a.ldo) + c.n0;
      int acc = 0;
      if (c.nkb > 0) {
        acc = iter++ & 1;
        int ok = 1;
        if (lane == 0) ok = wait_on(&sh->tfull[acc], tphase[acc], sh, a.ctrl) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        tphase[acc] ^= 1u;
        tile::fence_after();
      }
      if (rows > 0)
        store_tile<T, BN>(a, out, rows, cols,
                          tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * BN),
                          c.nkb == 0, stage, lane);
      if (c.nkb > 0) {
        tile::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->tempty[acc]);
      }
    }
  }
  tile::fence_before();
  __syncthreads();
  tile::fence_after();
  if (warp == 1) tile::tmem_free(tmem, R::kTmemCols);
}

// dst (rows x cols8, cols padded to a multiple of 8 with zeros) = src; `parts` matrices.
__global__ void __launch_bounds__(256)
    group_pad_kernel(const uint16_t* src, int64_t ld, int64_t stride, int64_t rows, int64_t cols,
                     int64_t parts, uint16_t* dst) {
  wait_prior_grid();
  allow_next_grid();
  const int64_t groups = (cols + 7) / 8;
  const int64_t total = parts * rows * groups;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t g = i % groups, r = i / groups;
    const uint16_t* s = src + r / rows * stride + r % rows * ld + g * 8;
    Pack<uint16_t, 8> v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.v[j] = g * 8 + j < cols ? s[j] : (uint16_t)0;
    *reinterpret_cast<Pack<uint16_t, 8>*>(dst + i * 8) = v;
  }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn = reinterpret_cast<EncodeFn>(p);
  }
  return fn;
}

// A 16-bit operand: cols x rows (x parts), rows on 16-byte boundaries.
struct Operand {
  const void* p;
  int64_t rows, cols, ld, parts, stride;  // parts = 0: two dimensions
};

bool encode(CUtensorMap* map, const Operand& o, uint32_t box_cols, uint32_t box_rows, bool bf16) {
  EncodeFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)o.parts};
  const cuuint64_t str[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.stride * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             o.parts ? 3 : 2, const_cast<void*>(o.p), dim, str, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_ok(const Operand& o) {
  return reinterpret_cast<uintptr_t>(o.p) % 16 == 0 && o.ld % 8 == 0 &&
         (o.parts <= 1 || o.stride % 8 == 0);
}
size_t pad_bytes(const Operand& o) {
  if (tma_ok(o)) return 0;
  return align_up((size_t)(o.parts ? o.parts : 1) * o.rows * ((o.cols + 7) / 8 * 8) * 2);
}

// The operand itself, or its padded copy at `at` (advanced past it).
cudaError_t pad(Operand& o, char*& at, Ctx& c) {
  const size_t bytes = pad_bytes(o);
  if (!bytes) {
    if (o.parts == 1) o.stride = (o.rows * o.ld + 7) / 8 * 8;  // never used, but checked
    return cudaSuccess;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(8 * c.num_sms);
  cfg.blockDim = dim3(256);
  cfg.stream = c.stream;
  add_pdl_attr(c, cfg, attr);
  ++c.launches;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, group_pad_kernel, (const uint16_t*)o.p, o.ld,
                                           o.stride, o.rows, o.cols,
                                           o.parts ? o.parts : (int64_t)1, (uint16_t*)at);
  o.p = at;
  o.ld = (o.cols + 7) / 8 * 8;
  o.stride = o.rows * o.ld;
  at += bytes;
  return e;
}

Operand rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return {p, rows, cols, ld, 0, 0};
}
Operand weights_of(const GroupArgs& g) {
  return {g.w, g.n, g.k, g.ldw, g.groups, g.stride_w};
}

template <class T, int kDir, int BN>
cudaError_t launch_tiles(const GroupArgs& g, Operand A, Operand B, void* ws, Ctx& c) {
  constexpr bool kBf16 = !__is_same(T, __half);
  char* at = static_cast<char*>(ws) + align_up(sizeof(Ctrl));
  cudaError_t e = cudaSuccess;
  CUtensorMap ma, ma16, mb;
  memset(&ma, 0, sizeof(ma));
  memset(&ma16, 0, sizeof(ma16));
  memset(&mb, 0, sizeof(mb));
  if (g.rows > 0) {  // (without rows only zeros are stored: no map is used)
    if ((e = pad(A, at, c)) != cudaSuccess || (e = pad(B, at, c)) != cudaSuccess) return e;
    const bool ok = kDir == GROUP_DW
                        ? encode(&ma, A, 64, BK, kBf16) && encode(&mb, B, 64, BK, kBf16)
                        : encode(&ma, A, BK, BM, kBf16) && encode(&ma16, A, BK, 16, kBf16) &&
                              encode(&mb, B, 64, kDir == GROUP_Y ? BN : BK, kBf16);
    if (!ok) return cudaErrorInvalidValue;
  }
  GroupTc a;
  a.offsets = g.offsets;
  a.rows = (int)g.rows;
  a.groups = (int)g.groups;
  a.k = (int)g.k;
  a.n = (int)g.n;
  a.out = static_cast<uint16_t*>(kDir == GROUP_Y ? g.y : kDir == GROUP_DX ? g.x : g.w);
  a.ldo = kDir == GROUP_Y ? g.ldy : kDir == GROUP_DX ? g.ldx : g.ldw;
  a.stride_o = kDir == GROUP_DW && g.groups > 1 ? g.stride_w : 0;
  a.vec_out = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.ldo % 8 == 0 &&
              a.stride_o % 8 == 0;
  a.ctrl = static_cast<Ctrl*>(ws);
  const int64_t nt = ((kDir == GROUP_Y ? g.n : g.k) + BN - 1) / BN;
  const int64_t most = kDir == GROUP_DW ? g.groups * ((g.n + BM - 1) / BM) * nt
                                        : (g.rows / BM + (g.rows < g.groups ? g.rows : g.groups)
                                           + 1) * nt;
  const auto fn = group_kernel<T, kDir, BN>;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<BN>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)(most < c.num_sms ? most : c.num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<BN>();
  cfg.stream = c.stream;
  add_pdl_attr(c, cfg, attr);
  ++c.launches;
  return cudaLaunchKernelEx(&cfg, fn, ma, ma16, mb, a);
}

template <class T, int kDir>
cudaError_t group_typed(const GroupArgs& g, void* ws, Ctx& c) {
  const Operand A = kDir == GROUP_Y ? rows_of(g.x, g.rows, g.k, g.ldx)
                                    : rows_of(g.y, g.rows, g.n, g.ldy);
  const Operand B = kDir == GROUP_DW ? rows_of(g.x, g.rows, g.k, g.ldx) : weights_of(g);
  return launch_tiles<T, kDir, 256>(g, A, B, ws, c);
}

template <class T>
cudaError_t group_dir(GroupDir d, const GroupArgs& g, void* ws, Ctx& c) {
  if (d == GROUP_Y) return group_typed<T, GROUP_Y>(g, ws, c);
  if (d == GROUP_DX) return group_typed<T, GROUP_DX>(g, ws, c);
  return group_typed<T, GROUP_DW>(g, ws, c);
}

}  // namespace

size_t group_workspace_bytes(const GroupArgs& g) {
  return align_up(sizeof(Ctrl)) + pad_bytes(rows_of(g.x, g.rows, g.k, g.ldx)) +
         pad_bytes(rows_of(g.y, g.rows, g.n, g.ldy)) + pad_bytes(weights_of(g));
}

cudaError_t launch_group(GroupDir d, const GroupArgs& g, void* ws, Ctx& c) {
  if (d != GROUP_DW && g.rows == 0) return cudaSuccess;
  return g.dtype == CASGD_BF16 ? group_dir<__nv_bfloat16>(d, g, ws, c)
                               : group_dir<__half>(d, g, ws, c);
}

}  // namespace casgd
