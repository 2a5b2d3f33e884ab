// Products of E4M3 codes whose scales are fp32 numbers for blocks of 128: rows with a scale
// for each 128 values along the contraction, times weights with a scale for each 128 x 128
// block (forward, input gradients), or times rows again (weight gradients).
//
//   C[m][n] = sum_kb sa[kb][m] * sb[..] * (sum_{k in block kb} a[m][k] b[n][k])
//
// The scales are no powers of two, so the block-scaled MMA cannot apply them: each 128-deep
// block is its own tcgen05 product (kind::f8f6f4, M = 128, N = BN, four K = 32 steps), and
// eight warps take it out of tensor memory and add it, scaled, to sums in fp32 registers.
// Tensor memory holds two such block products, so that the next one is multiplied while one
// is taken out.  Bounds, a 128 x 256 x 128 block: the MMA 512 cycles at its nominal rate, the
// tensor-memory reads 256, the multiply-adds 256 (column scales: 512), operands 48 KB.
//
// Schedules and tile order are those of the other grouped products (gemm.cuh): SCHED_ROWS
// multiplies each expert's rows by its own weights, SCHED_KGROUP sums over each expert's rows.
// Rows and columns past the operands' ends are read as zeros and not stored.
#include "fp8.cuh"
#include "kernels.h"

namespace moe {

constexpr int F8_K = 128;                                   // codes a stage, a scale block
constexpr int F8_A_BYTES = BM * F8_K;                       // 16 KB
constexpr int F8_B_BOX = 128;                               // rows of a B tensor load
constexpr int F8_EPI_WARPS = 8;                             // two a lane quarter, half of the columns each
constexpr int F8_THREADS = 64 + 32 * F8_EPI_WARPS;
__host__ __device__ constexpr int f8_stages(int bn) { return bn == 256 ? 4 : 6; }
__host__ __device__ constexpr int f8_stage_bytes(int bn) { return F8_A_BYTES + bn * F8_K; }
// operand stages, column scales a stage (SCHED_KGROUP), a 2 KB staging box a warp, alignment
__host__ __device__ constexpr int f8_smem(int bn) {
  return f8_stages(bn) * (f8_stage_bytes(bn) + bn * 4) + F8_EPI_WARPS * 2048 + 1024;
}

struct Fp8Params {
  int rows;                    // rows of A (SCHED_ROWS), or along the contraction (SCHED_KGROUP)
  int M, N, K;                 // SCHED_KGROUP: out [E][M][N]; SCHED_ROWS: out [rows][N], K long
  int E;
  const int32_t* row_offsets;  // [E + 1] multiples of 128, or NULL: one group
  const float* sa;             // [kb][rows or M]
  long long sa_ld;
  const float* sb;             // SCHED_ROWS: block scales with these strides; SCHED_KGROUP: [kb][N]
  long long sb_e, sb_n, sb_k;
  GemmParams g;                // what the shared schedules read
  int32_t* status;
};

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f8f6f4, E4M3 A and B, both K-major, fp32 D: bits 4-5 D format (1 = f32), 7-9 and
// 10-12 the operands' formats (0 = E4M3), 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// 32 lanes x 16 consecutive fp32 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The wait for such a load; it hands the registers on, so that nothing uses them before it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

template <int SCHED, int BN>
__global__ void __launch_bounds__(F8_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const Fp8Params p) {
  constexpr int STAGES = f8_stages(BN), STAGE_BYTES = f8_stage_bytes(BN);
  constexpr int WC = BN / 2;       // columns of an epilogue warp
  constexpr int NC = WC / 32;      // its 32-column boxes of the output
  extern __shared__ uint8_t dyn_smem[];
  __shared__ __align__(8) uint64_t full_bar[STAGES];
  __shared__ __align__(8) uint64_t empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ int s_ro[MAX_EXPERTS + 1];
  __shared__ int s_order[SCHED == SCHED_KGROUP ? MAX_EXPERTS : 1];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  float* s_sb = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);   // [STAGES][BN] column scales
  uint8_t* s_stage = smem + STAGES * (STAGE_BYTES + BN * 4);

  const int E = p.row_offsets ? p.E : 1;
  const int all_rows = (p.rows + F8_K - 1) / F8_K * F8_K;
  for (int i = threadIdx.x; i <= E; i += blockDim.x)
    s_ro[i] = p.row_offsets ? min(max(p.row_offsets[i], 0), all_rows) : (i == 0 ? 0 : all_rows);
  const int n_tiles = (p.N + BN - 1) / BN;
  bool snake = false;
  if (SCHED == SCHED_KGROUP) {
    __syncthreads();
    snake = kgroup_order(s_ro, E, (p.g.M / BM) * n_tiles, gridDim.x, s_order);  // complete at the barrier below
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], SCHED == SCHED_KGROUP ? F8_EPI_WARPS : 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&tfull_bar[a], 1); mbar_init(&tempty_bar[a], F8_EPI_WARPS); }
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) { tmem_alloc(&s_tmem_base, TMEM_COLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int total = (SCHED == SCHED_ROWS) ? (s_ro[E] / BM) * n_tiles : E * (p.g.M / BM) * n_tiles;
  volatile int* abort_flag = &s_abort;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      for (int rnd = 0, tile = sched_tile(0, blockIdx.x, gridDim.x, snake); ok && tile < total;
           tile = sched_tile(++rnd, blockIdx.x, gridDim.x, snake)) {
        const TileCoord c = tile_coord<SCHED, EPI_STORE, false, F8_K>(p.g, s_ro, s_order, E, n_tiles, tile);
        const uint32_t sb_bytes = SCHED == SCHED_KGROUP ? static_cast<uint32_t>(min(BN, p.N - c.out_col)) * 4u : 0u;
        for (int kb = 0; kb < c.kblocks; ++kb) {
          if (!mbar_wait_bounded(&empty_bar[stage], phase ^ 1, abort_flag, p.status, WAIT_LIMIT_CYCLES)) { ok = false; break; }
          uint8_t* sa = smem + stage * STAGE_BYTES;
          uint8_t* sb = sa + F8_A_BYTES;
          uint64_t* bar = &full_bar[stage];
          mbar_arrive_expect_tx(bar, STAGE_BYTES + sb_bytes);
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          tma_load_2d(sa, &tmA, bar, c.a_k + kb * F8_K, c.a_m);
#pragma unroll
          for (int i = 0; i < BN / F8_B_BOX; ++i)
            tma_load_2d(sb + i * F8_B_BOX * F8_K, &tmB, bar, c.b_k + kb * F8_K, c.b_n + i * F8_B_BOX);
          if (SCHED == SCHED_KGROUP)
            bulk_load(s_sb + stage * BN, p.sb + static_cast<long long>(c.b_k / F8_K + kb) * p.sb_k + c.out_col, sb_bytes, bar);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      for (int s = 0; s < STAGES; ++s)
        if ((armed >> s) & 1u) mbar_drain(&full_bar[s], (armed_parity >> s) & 1u, WAIT_LIMIT_CYCLES);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f8(BM, BN);
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int rnd = 0, tile = sched_tile(0, blockIdx.x, gridDim.x, snake); ok && tile < total;
           tile = sched_tile(++rnd, blockIdx.x, gridDim.x, snake)) {
        const TileCoord c = tile_coord<SCHED, EPI_STORE, false, F8_K>(p.g, s_ro, s_order, E, n_tiles, tile);
        for (int kb = 0; kb < c.kblocks; ++kb, ++it) {
          const uint32_t buf = it & 1u;
          if (!mbar_wait_bounded(&tempty_bar[buf], ((it >> 1) & 1u) ^ 1u, abort_flag, p.status, WAIT_LIMIT_CYCLES) ||
              !mbar_wait_bounded(&full_bar[stage], phase, abort_flag, p.status, WAIT_LIMIT_CYCLES)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
          const uint32_t sb = sa + F8_A_BYTES;
#pragma unroll
          for (int kk = 0; kk < F8_K / 32; ++kk)
            tc_mma_f8(tmem_base + buf * 256, smem_desc_sw128(sa + kk * 32, 16, 1024), smem_desc_sw128(sb + kk * 32, 16, 1024),
                      idesc, kk != 0 ? 1u : 0u);
          // SCHED_KGROUP: the epilogue reads the stage's column scales, so it frees the stage
          if (SCHED == SCHED_ROWS) tc_commit(&empty_bar[stage]);
          tc_commit(&tfull_bar[buf]);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      tc_commit(&drain_bar);
      mbar_drain(&drain_bar, 0, WAIT_LIMIT_CYCLES);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums and stores
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = s_stage + (warp - 2) * 2048;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * WC;
    int stage = 0;
    uint32_t it = 0;
    for (int rnd = 0, tile = sched_tile(0, blockIdx.x, gridDim.x, snake); tile < total;
         tile = sched_tile(++rnd, blockIdx.x, gridDim.x, snake)) {
      const TileCoord c = tile_coord<SCHED, EPI_STORE, false, F8_K>(p.g, s_ro, s_order, E, n_tiles, tile);
      const int row = c.a_m + q * 32 + lane;
      const int col = c.out_col + half * WC;
      const bool row_ok = row < (SCHED == SCHED_ROWS ? p.rows : p.M);
      const float* pa = p.sa + (row_ok ? row : 0) + static_cast<long long>(c.a_k / F8_K) * p.sa_ld;
      const float* pb = p.sb;
      if (SCHED == SCHED_ROWS) pb += c.e * p.sb_e + min(col / 128, (p.N - 1) / 128) * p.sb_n;
      // this row's and (SCHED_ROWS) these columns' scales, two blocks ahead of their use
      float sa0 = 0.f, sa1 = 0.f, sb0 = 1.f, sb1 = 1.f;
      if (c.kblocks > 0) { sa0 = pa[0]; if (SCHED == SCHED_ROWS) sb0 = pb[0]; }
      if (c.kblocks > 1) { sa1 = pa[p.sa_ld]; if (SCHED == SCHED_ROWS) sb1 = pb[p.sb_k]; }
      f32x2 acc[WC / 2];
#pragma unroll
      for (int j = 0; j < WC / 2; ++j) acc[j] = 0;
      bool ok = true;
      for (int kb = 0; kb < c.kblocks; ++kb, ++it) {
        const uint32_t buf = it & 1u;
        const float s = row_ok ? sa0 * sb0 : 0.f;
        const f32x2 s2 = pair(s, s);
        sa0 = sa1;
        sb0 = sb1;
        if (kb + 2 < c.kblocks) {
          sa1 = pa[(kb + 2) * p.sa_ld];
          if (SCHED == SCHED_ROWS) sb1 = pb[(kb + 2) * p.sb_k];
        }
        if (!mbar_wait_bounded(&tfull_bar[buf], (it >> 1) & 1u, abort_flag, p.status, WAIT_LIMIT_CYCLES)) { ok = false; break; }
        tc_fence_after();
        const ulonglong2* cs = reinterpret_cast<const ulonglong2*>(s_sb + stage * BN + half * WC);
        // 16 columns at a time: beside 128 sums a thread 32 would not fit its 168 registers
#pragma unroll
        for (int i = 0; i < WC / 16; ++i) {
          uint32_t r[16];
          tmem_ld16(lane_base + buf * 256 + 16 * i, r);
          tmem_wait_ld16(r);
          if (i == WC / 16 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty_bar[buf]);
          }
          if (SCHED == SCHED_ROWS) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[8 * i + j] = fma2(pair(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), s2, acc[8 * i + j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const ulonglong2 v = cs[4 * i + j];
              acc[8 * i + 2 * j] = fma2(pair(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])), mul2(s2, v.x),
                                        acc[8 * i + 2 * j]);
              acc[8 * i + 2 * j + 1] = fma2(pair(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                                            mul2(s2, v.y), acc[8 * i + 2 * j + 1]);
            }
          }
        }
        if (SCHED == SCHED_KGROUP) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty_bar[stage]);
          if (++stage == STAGES) stage = 0;
        }
      }
      if (!ok) break;
      // bf16 through the warp's staging box; 32-row and 32-column boxes past the ends are skipped
      const int y0 = static_cast<int>(c.out_row) + q * 32;
      const int y_end = SCHED == SCHED_ROWS ? min(s_ro[c.e + 1], p.rows) : p.M;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
        float v[32];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 x = unpair(acc[16 * i + j]);
          v[2 * j] = x.x;
          v[2 * j + 1] = x.y;
        }
        stage_row_bf16(stg, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && y0 < y_end && col + 32 * i < p.N) {
          tma_store_3d(&tmC, stg, col + 32 * i, y0, SCHED == SCHED_KGROUP ? c.e : 0);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

template <int SCHED, int BN>
static cudaError_t launch_fp8_t(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const Fp8Params& p,
                                cudaStream_t stream) {
  auto kern = fp8_gemm_kernel<SCHED, BN>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, f8_smem(BN));
  if (err != cudaSuccess) return err;
  kern<<<num_sms(), F8_THREADS, f8_smem(BN), stream>>>(a, b, c, p);
  count_launch();
  return cudaGetLastError();
}


}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_fp8_gemm(const uint8_t* a, const float* a_scales, int64_t rows, int32_t K, const uint8_t* b,
                        const float* b_scales, int32_t b_transposed, int32_t N, int32_t E, const int32_t* row_offsets,
                        moe_bf16* out, int32_t* dev_status, void* stream) {
  if (rows < 0 || K <= 0 || N <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (E > 1 && !row_offsets) return MOE_ERR_INVALID_ARG;
  if (E > MAX_EXPERTS || K % 16 != 0 || N % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (rows > (1ll << 31) - 256 || static_cast<int64_t>(E) * N >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  if (!b || !b_scales || !dev_status || (rows > 0 && (!a || !a_scales || !out))) return MOE_ERR_INVALID_ARG;
  if (!f8_aligned(a) || !f8_aligned(b) || !f8_aligned(out)) return MOE_ERR_ALIGNMENT;
  if (rows == 0) return MOE_OK;
  const int64_t tiles = up128(rows) / 128;
  // BN = 128 where the rows make too few 256-wide tiles to fill the SMs evenly
  const int64_t wide = tiles * ((N + 255) / 256);
  const int bn = (N <= 128 || wide < num_sms()) ? 128 : 256;
  CUtensorMap ta, tb, tc;
  if (!make_tensor_map_u8(&ta, a, K, rows, F8_K, BM) ||
      !make_tensor_map_u8(&tb, b, K, static_cast<uint64_t>(E) * N, F8_K, F8_B_BOX) ||
      !make_tensor_map_store3(&tc, out, N, rows, 1))
    return MOE_ERR_CUDA;
  Fp8Params p{};
  p.rows = static_cast<int>(rows); p.N = N; p.K = K; p.E = E; p.row_offsets = row_offsets;
  p.sa = a_scales; p.sa_ld = rows;
  const long long nb = (N + 127) / 128, kb = (K + 127) / 128;
  p.sb = b_scales; p.sb_e = nb * kb; p.sb_n = b_transposed ? 1 : kb; p.sb_k = b_transposed ? nb : 1;
  p.g.BN = bn; p.g.K = static_cast<int>(up128(K)); p.g.b_rows_per_expert = N; p.g.m_fastest = ORDER_PER_GROUP;
  p.g.band_krows = BAND_KROWS_E4M3;
  p.status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bn == 256 ? launch_fp8_t<SCHED_ROWS, 256>(ta, tb, tc, p, s) : launch_fp8_t<SCHED_ROWS, 128>(ta, tb, tc, p, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp8_wgrad(const uint8_t* dy_t, const float* dy_scales, const uint8_t* x_t, const float* x_scales, int64_t rows,
                         int32_t N, int32_t K, int32_t E, const int32_t* row_offsets, moe_bf16* out, int32_t* dev_status,
                         void* stream) {
  if (rows < 0 || K <= 0 || N <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (E > 1 && !row_offsets) return MOE_ERR_INVALID_ARG;
  if (E > MAX_EXPERTS || K % 8 != 0 || rows % 128 != 0 || rows >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  if (!out || !dev_status || (rows > 0 && (!dy_t || !dy_scales || !x_t || !x_scales))) return MOE_ERR_INVALID_ARG;
  if (!f8_aligned(dy_t) || !f8_aligned(x_t) || !f8_aligned(x_scales) || !f8_aligned(out)) return MOE_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0)
    return cudaMemsetAsync(out, 0, static_cast<size_t>(E) * N * K * sizeof(moe_bf16), s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  const int bn = K <= 128 || E * up128(N) / 128 * ((K + 255) / 256) < num_sms() ? 128 : 256;
  CUtensorMap ta, tb, tc;
  if (!make_tensor_map_u8(&ta, dy_t, rows, N, F8_K, BM) || !make_tensor_map_u8(&tb, x_t, rows, K, F8_K, F8_B_BOX) ||
      !make_tensor_map_store3(&tc, out, K, N, E))
    return MOE_ERR_CUDA;
  Fp8Params p{};
  p.rows = static_cast<int>(rows); p.M = N; p.N = K; p.E = E; p.row_offsets = row_offsets;
  p.sa = dy_scales; p.sa_ld = N; p.sb = x_scales; p.sb_k = K;
  p.g.BN = bn; p.g.M = static_cast<int>(up128(N)); p.g.N = K; p.g.m_fastest = N <= K ? 1 : 0;
  p.status = dev_status;
  const cudaError_t e = bn == 256 ? launch_fp8_t<SCHED_KGROUP, 256>(ta, tb, tc, p, s) : launch_fp8_t<SCHED_KGROUP, 128>(ta, tb, tc, p, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
