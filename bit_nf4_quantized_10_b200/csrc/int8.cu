// 8-bit integer linear: rows quantized to int8 with one scale each, and the
// product of two such operands on the tensor cores (tcgen05 kind::i8):
//   s_m = fl32(max_k |x[m, k]| / 127),  a[m, k] = rint(fl32(x[m, k] / s_m))
//   Y[m, n] = fl32(acc) * fl32(s_a[m] s_b[n]),  acc = sum_k a[m, k] b[n, k]
// acc is exact (int32), so it does not depend on how K is split.
//
// Product.  The weight rows n are the M side of the MMA and the tokens m its N
// side: a tile is 256 weight rows x tn tokens (tn a multiple of 32, at most
// 256, chosen so that the token tiles are even), so a handful of tokens costs
// no more tensor-core time than it has to and the weight streams through
// unchanged.  Two CTAs on two SMs share a tile (cta_group::2): each loads its
// 128 weight rows and half of the tokens, 128 bytes of K per stage.
//   warp 0      TMA producer (both CTAs); the copies of both complete on the even
//               CTA's barrier of the stage (a thread of the odd CTA that passed
//               its own barriers on took 1100 cycles a stage, twice the MMAs)
//   warp 1      one thread of the even CTA issues the MMAs
//   warps 2-5   drain one of the two accumulators (TMEM columns 0-255 and
//               256-511) while the next tile fills the other
// In the accumulator a TMEM lane is a weight row, so the 32 lanes of a warp
// write 32 neighbouring values of a token's output row.
//
// Work.  The pairs walk the tiles in rounds, token tiles fastest (the pairs at
// work at a time share a few weight tiles in L2).  The tiles left over after
// the whole rounds are cut along K into equal ranges, one per pair; a range
// that is not a whole tile leaves its int32 sums in the workspace, and a second
// kernel adds them.  Every wait is bounded (QL_ERR_TIMEOUT).
#include <cudaTypedefs.h>

#include <algorithm>

#include "common.cuh"
#include "sm100.cuh"
#include "trace.cuh"

namespace ql {
using namespace sm100;

QL_DEFINE_STATUS_ACCESSOR(status_word_int8)

bool make_map_2d(CUtensorMap* map, CUtensorMapDataType dt, int elem_bytes, const void* base, uint64_t cols,
                 uint64_t rows, uint64_t ld, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swz);

namespace i8 {

// ------------------------------------------------------------------ quantize
constexpr int kQThreads = 256;

__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[8 * i + 2 * k] = bf16_lo(w[k]);
      v[8 * i + 2 * k + 1] = bf16_hi(w[k]);
    }
  }
}

// Codes of 16 values.  q = x (1/s) is within 2.3e-5 of fl32(x / s) (three
// roundings of a value up to 127), so both round to the same integer unless q
// is that close to halfway; those few values (and rows whose 1/s leaves the
// normal range) take the division.  Adding 1.5 2^23 rounds to the nearest even
// integer and leaves it in the low mantissa bits.
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float s, float inv, bool divide) {
  constexpr float kMagic = 12582912.0f;
  float r[16], far = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = __fmul_rn(v[i], inv);
    r[i] = __fadd_rn(q, kMagic);
    far = fmaxf(far, fabsf(__fsub_rn(q, __fsub_rn(r[i], kMagic))));
  }
  if (divide || far > 0.4999f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __fadd_rn(fminf(fmaxf(__fdiv_rn(v[i], s), -127.0f), 127.0f), kMagic);
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __byte_perm(__float_as_uint(r[4 * i]), __float_as_uint(r[4 * i + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(r[4 * i + 2]), __float_as_uint(r[4 * i + 3]), 0x0040);
    o[i] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One row per block.  VPT groups of 16 values per thread stay in registers
// between the maximum and the codes; wider rows are read a second time.
template <typename T, int VPT>
__global__ void __launch_bounds__(1024) int8_quant_kernel(const T* __restrict__ x, int64_t K, int8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  __shared__ uint32_t red[32];
  pdl_wait();
  pdl_trigger();
  const int64_t m = blockIdx.x;
  const T* row = x + m * K;
  const int groups = (int)(K / 16), t = threadIdx.x, nt = blockDim.x;
  float v[VPT][16];
  uint32_t top = 0;   // largest |x| as bits: a NaN or infinity is above every finite value
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = t + k * nt;
    if (g < groups) {
      load16(row + (int64_t)g * 16, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[k][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[k][i]) & 0x7FFFFFFFu);
  }
  for (int g = t + VPT * nt; g < groups; g += nt) {
    float w[16];
    load16(row + (int64_t)g * 16, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(w[i]) & 0x7FFFFFFFu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((t & 31) == 0) red[t >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, (t & 31) < (nt >> 5) ? red[t & 31] : 0u);
  const bool finite = top < 0x7F800000u;
  const float s = finite ? __fdiv_rn(__uint_as_float(top), 127.0f) : __uint_as_float(0x7FC00000u);
  if (t == 0) {
    scales[m] = s;
    if (!finite) raise_status(ST_NONFINITE);
  }
  uint4* out = reinterpret_cast<uint4*>(codes + m * K);
  const bool zero = !finite || s == 0.0f, divide = s < 1e-30f;
  const float inv = divide ? 0.0f : __fdiv_rn(1.0f, s);
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int g = t + k * nt;
    if (g < groups) out[g] = zero ? make_uint4(0, 0, 0, 0) : codes16(v[k], s, inv, divide);
  }
  for (int g = t + VPT * nt; g < groups; g += nt) {
    float w[16];
    load16(row + (int64_t)g * 16, w);
    out[g] = zero ? make_uint4(0, 0, 0, 0) : codes16(w, s, inv, divide);
  }
}

template <typename T>
ql_status run_quant(const void* x, int64_t rows, int64_t K, int8_t* codes, float* scales, cudaStream_t st) {
  const int64_t groups = K / 16;
  // one group per thread up to 1024 threads' worth, then two per thread
  const unsigned threads = (unsigned)std::min<int64_t>((groups + 31) / 32 * 32, 512);
  const bool two = groups > 512;
  TraceScope ts(TK_INT8, st);
  if (two)
    QL_CUDA_TRY(launch(int8_quant_kernel<T, 2>, dim3((unsigned)rows), dim3(threads), 0, st, 1, 1, (const T*)x, K, codes,
                       scales));
  else
    QL_CUDA_TRY(launch(int8_quant_kernel<T, 1>, dim3((unsigned)rows), dim3(threads), 0, st, 1, 1, (const T*)x, K, codes,
                       scales));
  QL_LAUNCH_CHECK();
  return QL_OK;
}

// ------------------------------------------------------------------- product
constexpr int BW = 256;                    // weight rows of a tile (128 per CTA)
constexpr int BT = 256;                    // most tokens of a tile
constexpr int BK = 128;                    // K values (bytes) of a stage
constexpr int A_BYTES = BW / 2 * BK;       // 16 KB: a CTA's weight rows of a stage
constexpr int MAX_STAGES = 8;
constexpr int RING_BYTES = 7 * 32768;      // 7 stages at tn = 256
constexpr int THREADS = 6 * 32;
constexpr int TMEM_COLS = 512;
constexpr size_t SMEM_BYTES = RING_BYTES + 2 * BT * 4 + 256;   // 226.25 of the 227 KB that a block can have

// Instruction descriptor, kind::i8: int32 D (2 at bit 4), int8 A and B (1 at
// bits 7 and 10), both K-major, N >> 3 at bit 17, M >> 4 at bit 24, K = 32.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// TMA load of one CTA of a pair into its own shared memory that completes on a
// barrier of the even CTA (no multicast).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t even_bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(even_bar), "r"(x), "r"(y)
      : "memory");
}

// Arrive on this CTA's barrier alone once every pair MMA issued so far has completed.
__device__ __forceinline__ void mma_commit_pair_local(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// How the tiles are dealt to the pairs; the same on host and device.
struct Plan {
  int tn;              // tokens of a tile
  int token_tiles;
  int tiles;           // weight tiles x token tiles, token tiles fastest
  int ksteps;
  int pairs;
  int whole;           // tiles done in whole rounds (a multiple of `pairs`)
  int rem_pairs;       // pairs that share the remaining tiles
  int64_t rem_steps;   // stages of the remaining tiles together
};

struct Work {
  int tile, k0, k1;
  int slot;            // where the part sums go, or -1: the whole of K is here
};

__host__ __device__ inline bool work_at(const Plan& p, int pair, int i, Work& w) {
  const int rounds = p.whole / p.pairs;
  if (i < rounds) {
    w.tile = pair + i * p.pairs;
    w.k0 = 0;
    w.k1 = p.ksteps;
    w.slot = -1;
    return true;
  }
  i -= rounds;
  if (pair >= p.rem_pairs || i > 1) return false;
  const int64_t b = p.rem_steps * pair / p.rem_pairs, e = p.rem_steps * (pair + 1) / p.rem_pairs;
  const int64_t t0 = b / p.ksteps + i, base = t0 * p.ksteps;
  if (base >= e) return false;
  w.tile = p.whole + (int)t0;
  w.k0 = i ? 0 : (int)(b - base);
  w.k1 = (int)(e - base < p.ksteps ? e - base : p.ksteps);
  w.slot = w.k0 == 0 && w.k1 == p.ksteps ? -1 : pair * 2 + i;
  return true;
}

struct Params {
  Plan plan;
  int M, N;
  int stages, stage_bytes;
  const float* sa;
  const float* sb;
  void* Y;
  int32_t* parts;      // [2 rem_pairs][tn][BW]
  bool y_bf16;
  uint32_t wait_limit;
};

__device__ __forceinline__ void put_y(const Params& p, int64_t at, float v) {
  if (p.y_bf16)
    reinterpret_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float*>(p.Y)[at] = v;
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// Up to 16 tokens' values of one output channel (y points at the first; rows are N apart).
template <typename T>
__device__ __forceinline__ void put_column(T* y, int N, const float (&v)[16], int count) {
  if (count >= 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) put(y + (int64_t)j * N, v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < count) put(y + (int64_t)j * N, v[j]);
  }
}

__global__ void __launch_bounds__(THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                     const Params p) {
  extern __shared__ __align__(1024) uint8_t ring[];                  // the swizzle's atoms start on 1024 bytes
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + RING_BYTES);   // even CTA: a stage has landed in both
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* acc_full = empty + MAX_STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drained = acc_empty + 2;
  float* sa_tile = reinterpret_cast<float*>(drained + 2);            // [2][BT]
  uint32_t* tmem_addr = reinterpret_cast<uint32_t*>(sa_tile + 2 * BT);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_addr + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1;
  const int S = p.stages, tn = p.plan.tn;

  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);   // four warps of each CTA
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc2(tmem_addr, TMEM_COLS);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are initialised and TMEM is allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_addr;
  pdl_wait();
  pdl_trigger();

  Work w;
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&map_w);
      prefetch_tmap(&map_x);
      int n = 0;       // stages issued
      bool ok = true;
      for (int i = 0; ok && work_at(p.plan, pair, i, w); ++i) {
        const int wrow = w.tile / p.plan.token_tiles * BW + rank * (BW / 2);
        const int xrow = w.tile % p.plan.token_tiles * tn + rank * (tn / 2);
        for (int k = w.k0; k < w.k1; ++k) {
          const int s = n % S, use = n / S;
          if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1, abort_flag, p.wait_limit)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + s * p.stage_bytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * (uint32_t)p.stage_bytes);
          const uint32_t bar = cluster_map(smem_u32(&full[s]), 0);
          tma_load_pair(st, &map_w, bar, k * BK, wrow);
          tma_load_pair(st + A_BYTES, &map_x, bar, k * BK, xrow);
          ++n;
        }
      }
      // a stage is empty once its copies have landed and the MMAs have read it:
      // no copy may still be landing, and no commit arriving, when the CTA exits
      for (int i = n > S ? n - S : 0; i < n; ++i) mbar_wait(&empty[i % S], (i / S) & 1, abort_flag, p.wait_limit);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_i8(BW, tn);
      int n = 0;
      bool ok = true;
      for (int i = 0; ok && work_at(p.plan, pair, i, w); ++i) {
        const int b = i & 1, use_b = i >> 1;
        if (use_b > 0) {
          ok = mbar_wait_cluster(&acc_empty[b], (use_b - 1) & 1, abort_flag, p.wait_limit);
          tc_fence_after();
        }
        for (int k = w.k0; ok && k < w.k1; ++k, ++n) {
          const int s = n % S;
          ok = mbar_wait_cluster(&full[s], (n / S) & 1, abort_flag, p.wait_limit);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_addr = smem_u32(ring + s * p.stage_bytes), b_addr = a_addr + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma_i8_pair(tmem + b * BT, sdesc_sw128(a_addr + kk * 32, 16, 1024), sdesc_sw128(b_addr + kk * 32, 16, 1024),
                        idesc, (k > w.k0 || kk > 0) ? 1u : 0u);
          mma_commit_pair(&empty[s]);
        }
        if (ok) mma_commit_pair(&acc_full[b]);
      }
      // every MMA issued has completed before the pair frees its memory
      mma_commit_pair_local(drained);
      for (int i = 0; i < 4 && !mbar_try_wait(drained, 0); ++i) mbar_wait(drained, 0, abort_flag, p.wait_limit);
    }
  } else {
    const int quad = warp & 3, et = threadIdx.x - 64;
    const int in_tile = rank * (BW / 2) + quad * 32 + lane;   // weight row within the tile
    for (int i = 0; work_at(p.plan, pair, i, w); ++i) {
      const int b = i & 1;
      const int n = w.tile / p.plan.token_tiles * BW + in_tile;
      const int m0 = w.tile % p.plan.token_tiles * tn;
      const int cols = min(tn, p.M - m0);
      // the tokens' scales, while the accumulator fills; a warp comes here again
      // for the same half only after the barrier of the other
      float* sa = sa_tile + b * BT;
      for (int c = et; c < tn; c += 128) sa[c] = c < cols ? p.sa[m0 + c] : 0.0f;
      const float sb = n < p.N ? p.sb[n] : 0.0f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[b], (i >> 1) & 1, abort_flag, p.wait_limit) && !*abort_flag);
      if (!ok) *abort_flag = 1;     // the barrier above needs all four warps: keep going, without writing
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(b * BT);
      uint32_t next[16];
      tmem_ld16(acc, next);
      for (int c0 = 0; c0 < cols && ok; c0 += 16) {
        uint32_t v[16];
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = next[j];
        if (c0 + 16 < cols) tmem_ld16(acc + (uint32_t)(c0 + 16), next);
        if (w.slot >= 0) {
          int32_t* dst = p.parts + ((int64_t)w.slot * tn + c0) * BW + in_tile;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c0 + j < cols) dst[(int64_t)j * BW] = (int32_t)v[j];
        } else if (n < p.N) {
          float y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = __fmul_rn(__int2float_rn((int32_t)v[j]), __fmul_rn(sa[c0 + j], sb));
          const int64_t at = (int64_t)(m0 + c0) * p.N + n;
          if (p.y_bf16)
            put_column(reinterpret_cast<__nv_bfloat16*>(p.Y) + at, p.N, y, cols - c0);
          else
            put_column(reinterpret_cast<float*>(p.Y) + at, p.N, y, cols - c0);
        }
      }
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(&acc_empty[b], 0);
    }
  }
  tc_fence_before();
  cluster_sync();   // neither CTA leaves while the pair's MMAs or arrivals may still touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, TMEM_COLS);
  }
}

// Adds the part sums of the tiles that several pairs shared: a thread is a
// weight row, blockIdx.x the tile, blockIdx.y deals the token columns.
__global__ void __launch_bounds__(BW) int8_join_kernel(const Params p) {
  pdl_wait();
  pdl_trigger();
  const Plan& q = p.plan;
  const int64_t lo = (int64_t)blockIdx.x * q.ksteps, hi = lo + q.ksteps;   // this tile's stages
  int first = (int)(lo * q.rem_pairs / q.rem_steps);
  while (first > 0 && q.rem_steps * first / q.rem_pairs > lo) --first;
  while (q.rem_steps * (first + 1) / q.rem_pairs <= lo) ++first;
  const int64_t b0 = q.rem_steps * first / q.rem_pairs, e0 = q.rem_steps * (first + 1) / q.rem_pairs;
  if (b0 <= lo && e0 >= hi) return;     // one pair had the whole tile and has written it
  const int tile = q.whole + blockIdx.x;
  const int n = tile / q.token_tiles * BW + threadIdx.x, m0 = tile % q.token_tiles * q.tn;
  if (n >= p.N) return;
  const int cols = min(q.tn, p.M - m0);
  const float sb = p.sb[n];
  for (int c = blockIdx.y; c < cols; c += gridDim.y) {
    int32_t acc = 0;
    for (int r = first; r < q.rem_pairs; ++r) {
      const int64_t b = q.rem_steps * r / q.rem_pairs;
      if (b >= hi) break;
      const int slot = r * 2 + (b < lo ? 1 : 0);
      acc += p.parts[((int64_t)slot * q.tn + c) * BW + threadIdx.x];
    }
    const int64_t m = m0 + c;
    put_y(p, m * p.N + n, __fmul_rn(__int2float_rn(acc), __fmul_rn(p.sa[m], sb)));
  }
}

Plan make_plan(int64_t M, int64_t N, int64_t K) {
  Plan p;
  p.token_tiles = (int)((M + BT - 1) / BT);
  p.tn = (int)(((M + p.token_tiles - 1) / p.token_tiles + 31) / 32 * 32);
  p.tiles = (int)((N + BW - 1) / BW) * p.token_tiles;
  p.ksteps = (int)((K + BK - 1) / BK);
  p.pairs = std::max(1, (device_sm_count() > 0 ? device_sm_count() : 148) / 2);
  p.whole = p.tiles / p.pairs * p.pairs;
  const int rem = p.tiles - p.whole;
  p.rem_steps = (int64_t)rem * p.ksteps;
  // a range of under 4 stages costs more to join than it saves
  p.rem_pairs = (int)std::min<int64_t>(p.pairs, std::max<int64_t>(rem, p.rem_steps / 4));
  return p;
}

}  // namespace i8

int64_t int8_max_k() { return 131056; }   // the largest multiple of 16 whose sum of 128^2 stays in int32

size_t int8_gemm_ws(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M >= ((int64_t)1 << 31) || N >= ((int64_t)1 << 31) || K > int8_max_k()) return 0;
  const i8::Plan p = i8::make_plan(M, N, K);
  const int rem = p.tiles - p.whole;
  if (rem == 0 || p.rem_pairs == rem) return 0;   // every remaining tile has a pair to itself
  return (size_t)p.rem_pairs * 2 * p.tn * i8::BW * 4;
}

ql_status launch_int8_quantize(const void* x, ql_dtype dt, int64_t rows, int64_t K, int8_t* codes, float* scales,
                               cudaStream_t st) {
  return dt == QL_F32 ? i8::run_quant<float>(x, rows, K, codes, scales, st)
                      : i8::run_quant<__nv_bfloat16>(x, rows, K, codes, scales, st);
}

ql_status launch_int8_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb, int64_t M, int64_t N,
                           int64_t K, void* Y, ql_dtype y_dt, void* ws, cudaStream_t st) {
  using namespace i8;
  if (per_device(reinterpret_cast<const void*>(int8_gemm_kernel), 0, [] {
        if (cudaFuncSetAttribute(int8_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES) !=
            cudaSuccess) {
          cudaGetLastError();
          return -1;
        }
        return 1;
      }) < 0)
    return QL_ERR_CUDA;
  Params p;
  p.plan = make_plan(M, N, K);
  CUtensorMap map_w, map_x;
  if (!make_map_2d(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b, (uint64_t)K, (uint64_t)N, (uint64_t)K, BK, BW / 2,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&map_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a, (uint64_t)K, (uint64_t)M, (uint64_t)K, BK,
                   (uint32_t)p.plan.tn / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return QL_ERR_CUDA;
  p.M = (int)M;
  p.N = (int)N;
  p.stage_bytes = A_BYTES + p.plan.tn / 2 * BK;
  p.stages = std::min(MAX_STAGES, RING_BYTES / p.stage_bytes);
  p.sa = sa;
  p.sb = sb;
  p.Y = Y;
  p.parts = reinterpret_cast<int32_t*>(ws);
  p.y_bf16 = y_dt == QL_BF16;
  p.wait_limit = 1u << 22;
  const int active = p.plan.whole > 0 ? p.plan.pairs : p.plan.rem_pairs;
  {
    TraceScope ts(TK_INT8GEMM, st);
    QL_CUDA_TRY(launch(int8_gemm_kernel, dim3(2u * (unsigned)active), dim3(THREADS), SMEM_BYTES, st, 2, 1, map_w, map_x, p));
    QL_LAUNCH_CHECK();
  }
  const int rem = p.plan.tiles - p.plan.whole;
  if (rem == 0 || p.plan.rem_pairs == rem) return QL_OK;
  const unsigned deal = (unsigned)std::max(1, std::min(p.plan.tn, 592 / rem));
  TraceScope ts(TK_INT8GEMM, st);
  QL_CUDA_TRY(launch(int8_join_kernel, dim3((unsigned)rem, deal), dim3(BW), 0, st, 1, 1, p));
  QL_LAUNCH_CHECK();
  return QL_OK;
}

}  // namespace ql
