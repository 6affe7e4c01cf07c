// act(x W^T + bias) + residual (gdn_linear): tcgen05.mma fed by TMA, f32
// accumulators in TMEM, the epilogue on the accumulators' way out.
//
// Two kernels. Many rows: CTA pairs (cta_group::2) on 256 x BN output tiles,
// bound by the tensor cores. Few rows (up to 128): the weight rows take the
// MMA's M and the x rows its N, so no tensor-core row is spent on rows that are
// not there, and K is split over a cluster of CTAs so that every SM streams
// weights; bound by their bandwidth.
//
// Both read x and W through tile maps with zero fill, so odd M, N and K need no
// care in the main loop: what is outside either matrix is zero in both operands.
//
// Measured (us): 8192 x 20480 x 8192 1376 by itself (2.0 PFLOP/s, 104% of the measured
// library product) and 1485 to 1674 back to back, where the power limit holds the clock down;
// 4100 x 8192 x 1024 with a residual 61, of which 36 are the products and 24 the bytes:
// 17 x 32 tiles, the last row of them with 4 rows of 256, on 76 pairs leave 8 rounds for
// 7.2, and each pair reads 1 MB of tiles from L2 in the 7 us it has for a round; 5 x 2560 x
// 8192 8.0 in a graph, the weights' bytes being 6.2, and 128 rows of it 15.4. 129 to 512
// rows of it take 30 to 32: 40 tiles on 76 pairs, 128 steps in a row.
#include <algorithm>
#include <atomic>

#include "gdn_prefill.cuh"
#include "gdn_tc_pair.cuh"

namespace gdn {
namespace {

using namespace tc;

// Set by a kernel whose wait passed its limit (gdn_linear_check reads it).
__device__ unsigned int g_linear_error;

constexpr int kBK = 64;  // K columns of a stage: 128 bytes, one swizzle row

// SiLU(y) = y sigmoid(y); GELU's tanh form is y sigmoid(2 u), u = sqrt(2/pi) (y +
// 0.044715 y^3). The fast exponential and division (a few 2^-22) are far below the
// rounding to bf16, and short: with expf and tanhf inlined for every value the epilogue
// outgrew the instruction cache.
template <bool ACT>
__device__ __forceinline__ float act_f(float y, int act) {
  if (!ACT) return y;
  const float s = act == 1 ? y : y * fmaf(0.07135481627f, y * y, 1.595769122f);
  return __fdividef(y, 1.0f + __expf(-s));
}

// ------------------------------------------------------------- many rows

// Stages of the ring: what the 227 KB hold beside the epilogue's staging.
template <int BN>
constexpr int pair_stages() {
  return BN == 256 ? 5 : BN == 128 ? 7 : 8;
}
// Producer, MMA, TMEM, -; eight epilogue warps (with four, each with all the columns of 32
// rows, 4100 x 8192 x 1024 took 74 us).
constexpr int kPairThreads = 384;
constexpr int kStageStride = 36;  // floats a staged row takes: 32 and four, against bank conflicts

template <int BN>
struct alignas(1024) PairSmem {
  static constexpr int kStages = pair_stages<BN>();
  unsigned char a[kStages][128 * 128];
  unsigned char b[kStages][BN / 2 * 128];
  float stage[8][32 * kStageStride];
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
};

struct PairTiles {
  int tiles_m, tiles_n, total;
};

// Tile order: groups of 8 row tiles, column tiles within them, so the tiles in
// flight share both operands in L2.
__device__ __forceinline__ void tile_at(const PairTiles& t, int i, int* m, int* n) {
  const int per = 8 * t.tiles_n, g = i / per, rows = min(8, t.tiles_m - 8 * g), r = i - g * per;
  *m = 8 * g + r % rows;
  *n = r / rows;
}

// Eight columns of one output row, 16 bytes of residual in and of output out.
template <bool ACT>
__device__ __forceinline__ void put8(const LinearParams& p, long long m, int n, const float* v, const float (&bias)[8],
                                     const uint4& res) {
  const uint32_t r[4] = {res.x, res.y, res.z, res.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = pack_bf16x2(act_f<ACT>(v[2 * j] + bias[2 * j], p.act) + bf16_lo(r[j]),
                       act_f<ACT>(v[2 * j + 1] + bias[2 * j + 1], p.act) + bf16_hi(r[j]));
  *reinterpret_cast<uint4*>(p.out + m * p.ldo + n) = make_uint4(o[0], o[1], o[2], o[3]);
}

// Two columns of one output row (any alignment): the residual, and the output.
__device__ __forceinline__ float2 get2(const LinearParams& p, long long m, int n, bool wide) {
  const __nv_bfloat16* r = p.residual + m * p.ldr + n;
  if (wide && n + 1 < p.N) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(r);
    return make_float2(bf16_lo(v), bf16_hi(v));
  }
  return make_float2(bf16_to_f(r[0]), n + 1 < p.N ? bf16_to_f(r[1]) : 0.f);
}
template <bool ACT>
__device__ __forceinline__ void put2(const LinearParams& p, long long m, int n, float2 v, float2 bias, float2 res, bool wide) {
  const float a = act_f<ACT>(v.x + bias.x, p.act) + res.x, b = act_f<ACT>(v.y + bias.y, p.act) + res.y;
  __nv_bfloat16* o = p.out + m * p.ldo + n;
  if (wide && n + 1 < p.N) {
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(a, b);
  } else {
    o[0] = __float2bfloat16_rn(a);
    if (n + 1 < p.N) o[1] = __float2bfloat16_rn(b);
  }
}

template <int BN, bool ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const LinearParams p,
                const PairTiles tiles) {
  extern __shared__ unsigned char raw[];
  constexpr int kStages = pair_stages<BN>();
  static_assert(sizeof(PairSmem<BN>) + 1024 <= 232448, "227 KB of shared memory a CTA");
  PairSmem<BN>& s = *reinterpret_cast<PairSmem<BN>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  constexpr uint32_t kBytes = 128 * 128 + BN / 2 * 128;  // one CTA's share of a stage
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 16);  // eight epilogue warps of both CTAs
    }
    fence_mbar_init();
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&wmap);
  }
  if (warp == 2) tmem_alloc_pair(&s.tmem, 512);
  __syncthreads();
  cluster_sync();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int ksteps = (p.K + kBK - 1) / kBK;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // producer: this CTA's 128 rows of x and half of the tile's weight rows
    int st = 0;
    uint32_t ph = 0;
    for (int i = pair; i < tiles.total && ok; i += pairs) {
      int tm, tn;
      tile_at(tiles, i, &tm, &tn);
      const int m0 = tm * 256 + (int)rank * 128, n0 = tn * BN + (int)rank * (BN / 2);
      for (int k = 0; k < ksteps; ++k) {
        if (!(ok = mbar_wait(&s.empty[st], ph ^ 1))) break;
        if (rank == 0) mbar_arrive_expect_tx(&s.full[st], 2 * kBytes);
        const uint32_t bar = map_rank(&s.full[st], 0);
        tma_load_2d_pair(s.a[st], &xmap, k * kBK, m0, bar);
        tma_load_2d_pair(s.b[st], &wmap, k * kBK, n0, bar);
        if (++st == kStages) st = 0, ph ^= 1;
      }
    }
    // every stage consumed: no copy is in flight when the CTAs leave
    const int next = st;
    const uint32_t round = ph;
    for (int k = 0; k < kStages && ok; ++k) {
      ok = mbar_wait(&s.empty[st], ph ^ 1);
      if (++st == kStages) st = 0, ph ^= 1;
    }
    // nor where a wait has failed: stages from the next one on were last filled a round before
    if (!ok && rank == 0)
      for (int k = 0; k < kStages; ++k) mbar_wait(&s.full[k], k < next ? round : round ^ 1);
  } else if (warp == 1 && rank == 0) {
    constexpr uint32_t idesc = idesc_bf16_f32(256, BN);
    int st = 0, buf = 0;
    uint32_t ph = 0, aph = 0;
    for (int i = pair; i < tiles.total && ok; i += pairs) {
      if (!(ok = mbar_wait(&s.acc_empty[buf], aph ^ 1))) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * 256;
      for (int k = 0; k < ksteps; ++k) {
        if (!(ok = mbar_wait(&s.full[st], ph))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = sdesc_k_sw128(smem_u32(s.a[st])), b = sdesc_k_sw128(smem_u32(s.b[st]));
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j) mma_bf16_pair(d, a + 2 * j, b + 2 * j, idesc, (k | j) != 0);
          mma_commit_pair(&s.empty[st]);
        }
        __syncwarp();
        if (++st == kStages) st = 0, ph ^= 1;
      }
      if (elect_one()) mma_commit_pair(&s.acc_full[buf]);
      __syncwarp();
      if (++buf == 2) buf = 0, aph ^= 1;
    }
  } else if (warp >= 4) {
    // Two warps share each 32 rows (TMEM lanes 32 q ..), in turns of kCols columns.
    constexpr int kCols = 32;
    constexpr int kLanes8 = kCols / 8, kRows8 = 32 / kLanes8;  // 16-byte rows: lanes a row, rows a turn
    constexpr int kLanes2 = kCols / 2, kRows2 = 32 / kLanes2;  // two columns a lane
    const int q = warp & 3, half = (warp - 4) >> 2;
    float* sm = s.stage[warp - 4];
    const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.residual)) & 3) == 0 &&
                      p.ldo % 2 == 0 && (!p.residual || p.ldr % 2 == 0);
    // rows of 16 bytes throughout
    const bool vec = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.residual)) & 15) == 0 &&
                     p.N % 8 == 0 && p.ldo % 8 == 0 && (!p.residual || p.ldr % 8 == 0);
    int buf = 0;
    uint32_t aph = 0;
    for (int i = pair; i < tiles.total && ok; i += pairs) {
      int tm, tn;
      tile_at(tiles, i, &tm, &tn);
      const int m0 = tm * 256 + (int)rank * 128 + q * 32;
      const int rows = min(32, p.M - m0);
      for (int c = half * kCols; c < BN; c += 2 * kCols) {
        // the residual's loads are in flight while the tile is multiplied
        const int n8 = tn * BN + c + (lane % kLanes8) * 8;
        const bool mine = vec && n8 < p.N;
        uint4 res[kLanes8];
#pragma unroll
        for (int r = 0; r < kLanes8; ++r) {
          res[r] = make_uint4(0, 0, 0, 0);
          const int row = kRows8 * r + lane / kLanes8;
          if (mine && p.residual && row < rows)
            res[r] = *reinterpret_cast<const uint4*>(p.residual + (long long)(m0 + row) * p.ldr + n8);
        }
        if (c < 2 * kCols) {
          ok = mbar_wait(&s.acc_full[buf], aph);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t t = tmem + buf * 256 + c + ((uint32_t)(q * 32) << 16);
#pragma unroll
        for (int h = 0; h < kCols; h += 32) {
          float v[32];
          tmem_ld32(t + h, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(sm + lane * kStageStride + h + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        if (c + 2 * kCols >= BN) {
          // this warp's part of the accumulator is out: the next tile but one may take it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_rank(&s.acc_empty[buf], 0));
        }
        __syncwarp();
        if (vec) {
          if (mine) {
            float bias[8] = {};
            if (p.bias) {
#pragma unroll
              for (int j = 0; j < 8; ++j) bias[j] = bf16_to_f(p.bias[n8 + j]);
            }
#pragma unroll
            for (int r = 0; r < kLanes8; ++r) {
              const int row = kRows8 * r + lane / kLanes8;
              if (row < rows) put8<ACT>(p, m0 + row, n8, sm + row * kStageStride + (lane % kLanes8) * 8, bias, res[r]);
            }
          }
        } else {
          const int n = tn * BN + c + 2 * (lane % kLanes2);
          if (n < p.N) {
            float2 bias = make_float2(0.f, 0.f);
            if (p.bias) bias = make_float2(bf16_to_f(p.bias[n]), n + 1 < p.N ? bf16_to_f(p.bias[n + 1]) : 0.f);
#pragma unroll 1
            for (int r0 = lane / kLanes2; r0 < rows; r0 += 8 * kRows2) {
              float2 rs[8];
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                rs[r] = make_float2(0.f, 0.f);
                if (p.residual && r0 + r * kRows2 < rows) rs[r] = get2(p, m0 + r0 + r * kRows2, n, wide);
              }
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                const int row = r0 + r * kRows2;
                if (row < rows)
                  put2<ACT>(p, m0 + row, n, *reinterpret_cast<const float2*>(sm + row * kStageStride + 2 * (lane % kLanes2)),
                            bias, rs[r], wide);
              }
            }
          }
        }
        __syncwarp();
      }
      if (++buf == 2) buf = 0, aph ^= 1;
    }
  }
  if (!ok) atomicCAS(&g_linear_error, 0u, (kStatusDeadline << 24) | (kWhatWait << 16) | (blockIdx.x & 0xffff));
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------- few rows

constexpr int kFewThreads = 192;  // producer, MMA, four epilogue warps
constexpr int kFewMaxStages = 8;
constexpr int kFewRing = 98304;   // bytes of a CTA's ring: two CTAs share an SM

struct FewParams {
  LinearParams p;
  int split;   // CTAs of the cluster, along K
  int stages;
};

// TOK: x rows the MMA takes (its N).
template <int TOK>
__global__ void __launch_bounds__(kFewThreads) linear_few(const __grid_constant__ CUtensorMap xmap,
                                                          const __grid_constant__ CUtensorMap wmap, const FewParams f) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[kFewMaxStages], empty[kFewMaxStages], done;
  __shared__ uint32_t tmem_base;
  const LinearParams& p = f.p;
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  constexpr uint32_t kBytes = 128 * 128 + TOK * 128;
  constexpr uint32_t kCols = TOK < 32 ? 32 : TOK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % f.split, n0 = blockIdx.x / f.split * 128;
  const int ksteps = (p.K + kBK - 1) / kBK;
  const int k0 = (int)((long long)ksteps * rank / f.split), k1 = (int)((long long)ksteps * (rank + 1) / f.split);
  if (threadIdx.x == 0) {
    for (int i = 0; i < f.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    fence_mbar_init();
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&wmap);
  }
  if (warp == 1) tmem_alloc(&tmem_base, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool ok = true;
  if (warp == 0 && lane == 0) {
    int st = 0;
    uint32_t ph = 0;
    for (int k = k0; k < k1; ++k) {
      if (!(ok = mbar_wait(&empty[st], ph ^ 1))) break;
      unsigned char* w = ring + st * kBytes;
      mbar_arrive_expect_tx(&full[st], kBytes);
      tma_load_2d_plain(w, &wmap, k * kBK, n0, &full[st]);
      tma_load_2d_plain(w + 128 * 128, &xmap, k * kBK, 0, &full[st]);
      if (++st == f.stages) st = 0, ph ^= 1;
    }
    // A wait has failed: no copy is in flight when the CTA leaves (stages from st on were last
    // filled a round before).
    if (!ok)
      for (int i = 0; i < f.stages; ++i) mbar_wait(&full[i], i < st ? ph : ph ^ 1);
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, TOK);
    int st = 0, k = k0;
    uint32_t ph = 0;
    for (; k < k1; ++k) {
      if (!(ok = mbar_wait(&full[st], ph))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t a = sdesc_k_sw128(smem_u32(ring + st * kBytes)), b = sdesc_k_sw128(smem_u32(ring + st * kBytes + 128 * 128));
#pragma unroll
        for (int j = 0; j < kBK / 16; ++j) mma_bf16(tmem, a + 2 * j, b + 2 * j, idesc, (k > k0) | (j > 0));
        mma_commit(&empty[st]);
      }
      __syncwarp();
      if (++st == f.stages) st = 0, ph ^= 1;
    }
    // a wait has failed: nor the copies that the producer goes on to make before it waits itself
    for (int left = ok ? 0 : min(f.stages, k1 - k); left > 0; --left) {
      mbar_wait(&full[st], ph);
      if (++st == f.stages) st = 0, ph ^= 1;
    }
    if (elect_one()) mma_commit(&done);
  } else if (warp >= 2) {
    ok = mbar_wait(&done, 0);
    ok = __all_sync(0xffffffffu, ok);
  }
  __syncwarp();
  if (!ok) atomicCAS(&g_linear_error, 0u, (kStatusDeadline << 24) | (kWhatWait << 16) | (blockIdx.x & 0xffff));
  // The MMAs are done, so the ring is free: this CTA's sums, [row of x][128 weight rows].
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2 && ok) {
    tc_fence_after();
    const int q = warp & 3;  // the TMEM lanes this warp may read
#pragma unroll
    for (int c = 0; c < TOK; c += 16) {
      if (c >= p.M) break;
      float v[16];
      tmem_ld16(tmem + c + ((uint32_t)(q * 32) << 16), v);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = v[j];
    }
    tc_fence_before();
  }
  if (f.split > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
  // The cluster's CTAs share the outputs; every one is the sum of the parts in
  // rank order, so it does not depend on who arrives first.
  const int total = p.M * 128;
  for (int i = rank * kFewThreads + threadIdx.x; i < total; i += f.split * kFewThreads) {
    const int m = i >> 7, n = n0 + (i & 127);
    float y = 0.f;
    if (f.split > 1)
      for (int r = 0; r < f.split; ++r) y += ld_cluster_f(map_rank(part + i, r));
    else
      y = part[i];
    if (n >= p.N) continue;
    y += p.bias ? bf16_to_f(p.bias[n]) : 0.f;
    if (p.act) y = act_f<true>(y, p.act);
    if (p.residual) y += bf16_to_f(p.residual[m * p.ldr + n]);
    p.out[m * p.ldo + n] = __float2bfloat16_rn(y);
  }
  if (f.split > 1) cluster_sync();  // no CTA leaves while its part is read
}

// ------------------------------------------------------------- host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeTiledFn)f;
  }();
  return fn;
}

// Tile map of a row-major [rows][cols] bf16 matrix: boxes of 64 columns x
// `box` rows, 128-byte swizzle, zero outside.
bool encode_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t boxes[2] = {(cuuint32_t)kBK, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's shared memory opt-in (the most any launch of it takes), once a
// device.
template <auto* KERNEL>
cudaError_t opt_in(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t f = cudaFuncSetAttribute((const void*)KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (f == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return f;
}

int sm_count() {
  static int count[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (!count[dev]) cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev);
  return count[dev] > 0 ? count[dev] : 152;
}

template <int BN>
cudaError_t launch_pair(const LinearParams& p, cudaStream_t s) {
  CUtensorMap xm, wm;
  if (!encode_map(&xm, p.x, p.M, p.K, p.ldx, 128) || !encode_map(&wm, p.w, p.N, p.K, p.ldw, BN / 2)) return cudaErrorInvalidValue;
  const size_t smem = sizeof(PairSmem<BN>) + 1024;
  const cudaError_t e = p.act ? opt_in<linear_pair<BN, true>>(smem) : opt_in<linear_pair<BN, false>>(smem);
  if (e != cudaSuccess) return e;
  PairTiles t;
  t.tiles_m = (p.M + 255) / 256;
  t.tiles_n = (p.N + BN - 1) / BN;
  t.total = t.tiles_m * t.tiles_n;
  const int pairs = std::min(t.total, sm_count() / 2);
  if (p.act)
    linear_pair<BN, true><<<2 * pairs, kPairThreads, smem, s>>>(xm, wm, p, t);
  else
    linear_pair<BN, false><<<2 * pairs, kPairThreads, smem, s>>>(xm, wm, p, t);
  return cudaGetLastError();
}

template <int TOK>
cudaError_t launch_few(const LinearParams& p, cudaStream_t s) {
  CUtensorMap xm, wm;
  if (!encode_map(&xm, p.x, p.M, p.K, p.ldx, TOK) || !encode_map(&wm, p.w, p.N, p.K, p.ldw, 128)) return cudaErrorInvalidValue;
  FewParams f;
  f.p = p;
  const int stage = 128 * 128 + TOK * 128, tiles = (p.N + 127) / 128, ksteps = (p.K + kBK - 1) / kBK;
  // Split K while the CTAs fit two to an SM and each keeps two stages' worth.
  f.split = std::max(1, std::min({8, 2 * sm_count() / tiles, ksteps / 2}));
  f.stages = std::min(kFewMaxStages, kFewRing / stage);
  const size_t smem = std::max((size_t)f.stages * stage, (size_t)TOK * 512) + 1024;
  const cudaError_t e = opt_in<linear_few<TOK>>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(f.split * tiles);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = f.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_few<TOK>, xm, wm, f);
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, cudaStream_t s) {
  if (p.M <= 16) return launch_few<16>(p, s);
  if (p.M <= 32) return launch_few<32>(p, s);
  if (p.M <= 64) return launch_few<64>(p, s);
  if (p.M <= 128) return launch_few<128>(p, s);
  // The tile width that takes the fewest waves x (width + a fixed part a tile).
  const int pairs = sm_count() / 2, tm = (p.M + 255) / 256;
  int best = 256;
  long long least = 0;
  for (int bn : {256, 128, 64}) {
    const long long tiles = (long long)tm * ((p.N + bn - 1) / bn), cost = (tiles + pairs - 1) / pairs * (bn + 32);
    if (!least || cost < least) least = cost, best = bn;
  }
  return best == 256 ? launch_pair<256>(p, s) : best == 128 ? launch_pair<128>(p, s) : launch_pair<64>(p, s);
}

cudaError_t linear_error(unsigned int* word, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_linear_error, 4, 0, cudaMemcpyDeviceToHost, s);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || !*word) return e;
  const unsigned int zero = 0;
  e = cudaMemcpyToSymbolAsync(g_linear_error, &zero, 4, 0, cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace gdn
