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
// Measured, 32768 rows over 32 experts, 4096 x 7168: 719 us where they are equal (2.68 PFLOP/s; 562 with operands that are
// already there, 708 with codes of 0 at a higher clock: operands from L2, 52 bytes a cycle and SM, and the way of a block
// through two buffers bound, under the power limit), 822 to 850 where they are skewed.  Weight gradients, 7168 x 2048: 585
// to 600 us, about 1400 cycles a block where the MMA and the multiply-adds take 512 each and nothing is full (tensor
// pipe 37 %, issue 47 %): a chunk's load from tensor memory, the wait for it and its arithmetic follow one another.  (CTA pairs with 32 KB of operands a block: 675 and 831 us, as odd numbers of
// 128-row tiles leave half a pair idle.)
//
// Schedules and tile order are those of the other grouped products (gemm.cuh): SCHED_ROWS
// multiplies each expert's rows by its own weights, SCHED_KGROUP sums over each expert's rows.
// Rows and columns past the operands' ends are read as zeros and not stored.
#include "fp8.cuh"
#include "kernels.h"
#include "pipe.cuh"

namespace moe {

constexpr int F8_K = 128;                                   // codes a stage, a scale block
constexpr int F8_A_BYTES = BM * F8_K;                       // 16 KB
constexpr int F8_B_BOX = 128;                               // rows of a B tensor load
constexpr int F8_EPI_WARPS = 8;                             // two a lane quarter, half of the columns each
// Warp 0 loads operands, warps 1 and 2 multiply every other block (a block's issue, its waits and commits
// take one warp longer than its MMA takes), warp 3 loads scales.  The four hand registers to
// those that hold the sums: 128 x 64 + 256 x 216 of the 384 x 168 of the launch.
constexpr int F8_EPI_WARP0 = 4;
constexpr int F8_THREADS = 32 * (F8_EPI_WARP0 + F8_EPI_WARPS);
constexpr int F8_REGS_FEW = 64, F8_REGS_MANY = 216;
static_assert(128 * F8_REGS_FEW + 256 * F8_REGS_MANY <= 384 * 168, "registers of the block at launch");
// Operand stages: as many as shared memory holds beside boxes for a whole tile of the output (with boxes of a
// quarter and a fourth stage, a tile's store took 3700 cycles instead of 1300).
__host__ __device__ constexpr int f8_stages(int bn) { return bn == 256 ? 3 : 5; }
__host__ __device__ constexpr int f8_stage_bytes(int bn) { return F8_A_BYTES + bn * F8_K; }
__host__ __device__ constexpr int f8_box_bytes(int bn) { return 32 * bn / 2 * 2; }
// Scales of a block: the tile's 128 rows, then its columns (SCHED_KGROUP) or the columns' blocks.  The
// loader is at most the operand stages ahead of the MMAs, these two blocks ahead of the sums, so
// that with three slots more than stages it never writes one that is still read.
__host__ __device__ constexpr int f8_slots(int bn) { return f8_stages(bn) + 3; }
__host__ __device__ constexpr int f8_slot_floats(int bn, bool col_scales) { return BM + (col_scales ? bn : 4); }
__host__ __device__ constexpr int f8_smem(int bn, bool col_scales) {
  return f8_stages(bn) * f8_stage_bytes(bn) + F8_EPI_WARPS * f8_box_bytes(bn) +
         f8_slots(bn) * f8_slot_floats(bn, col_scales) * 4 + 1024;
}

constexpr int F8_INFOS = 4;
constexpr int F8_SPLIT_LD = 128 + 4;     // floats of a row of a part

struct Fp8Params {
  int rows;                    // rows of A (SCHED_ROWS), or along the contraction (SCHED_KGROUP)
  int M, N;                    // SCHED_KGROUP: out [E][M][N]; SCHED_ROWS: out [rows][N]
  int E;
  const int32_t* row_offsets;  // [E + 1] multiples of 128, or NULL: one group
  const float* sa;             // [kb][rows or M]
  long long sa_ld;
  const float* sb;             // SCHED_ROWS: block scales with these strides; SCHED_KGROUP: [kb][N]
  long long sb_e, sb_n, sb_k;
  int split;                   // SPLIT: CTAs of a tile, a power of two
  moe_bf16* out;               // SPLIT
  GemmParams g;                // what the shared schedules read
  int32_t* status;
};

// kind::f8f6f4, E4M3 A and B, both K-major, fp32 D: bits 4-5 D format (1 = f32), 7-9 and
// 10-12 the operands' formats (0 = E4M3), 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// The wait for loads of 32 columns; it hands the registers on, so that nothing uses them before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29])::"memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31])::"memory");
}
// 16 lanes x 32 columns, spread as an MMA's result: registers 4 g and the next are columns 8 g + 2 (lane % 4) and
// the next of row lane / 4, registers 4 g + 2 and the next those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_rows4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ f32x2 ld_shared_pair(uint32_t addr) {
  f32x2 v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
// acc += (x, y) * s, kept in its place among the loads: moved past the next ones, the registers that they
// hold would not fit beside the sums.
__device__ __forceinline__ void add_scaled(f32x2& acc, uint32_t x, uint32_t y, f32x2 s) {
  asm volatile("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(acc) : "r"(x), "r"(y), "l"(s));
}
// One fp32 to shared memory, asynchronously; zero where it is not valid.
__device__ __forceinline__ void scale_async(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// The experts' rows from 0 to all_rows; none where the offsets are out of order, which would make tiles of rows
// before an operand's first.  (Inlined, it took registers from the sums: 840 us became 1000.)
__device__ __noinline__ void f8_offsets(const int32_t* offsets, int E, int all_rows, int* s_ro, int32_t* status) {
  bool bad = false;
  for (int i = threadIdx.x; i <= E; i += blockDim.x) {
    const int r = offsets[i];
    bad = bad || r % BM != 0 || (i == 0 ? r != 0 : r < offsets[i - 1]);
    s_ro[i] = min(r, all_rows);
  }
  if (!__syncthreads_or(bad)) return;
  for (int i = threadIdx.x; i <= E; i += blockDim.x) s_ro[i] = 0;
  set_status(status, MOE_ERR_INVARIANT);
}

// SPLIT: one tile a cluster of CTAs, each a part of the contraction; their sums meet in shared memory.
template <int SCHED, int BN, bool SPLIT>
__global__ void __launch_bounds__(F8_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const Fp8Params p) {
  constexpr int STAGES = f8_stages(BN), STAGE_BYTES = f8_stage_bytes(BN);
  constexpr int WC = BN / 2;       // columns of an epilogue warp
  extern __shared__ uint8_t dyn_smem[];
  __shared__ __align__(8) uint64_t full_bar[STAGES];
  __shared__ __align__(8) uint64_t empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar[2];
  __shared__ __align__(8) uint64_t ifull_bar[F8_INFOS];
  __shared__ __align__(8) uint64_t iempty_bar[F8_INFOS];
  __shared__ int4 s_info[F8_INFOS];       // of the tiles on their way to the sums: see below
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;
  __shared__ int s_ro[MAX_EXPERTS + 1];
  __shared__ int s_order[SCHED == SCHED_KGROUP ? MAX_EXPERTS : 1];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int SLOTS = f8_slots(BN), SLOT = f8_slot_floats(BN, SCHED == SCHED_KGROUP);
  uint8_t* s_box = smem + STAGES * STAGE_BYTES;
  float* s_scales = reinterpret_cast<float*>(s_box + F8_EPI_WARPS * f8_box_bytes(BN));

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full_bar[s], 1 + 32); mbar_init(&empty_bar[s], 1); }   // full: the tensor loads, the scale loader's lanes
    for (int a = 0; a < 2; ++a) { mbar_init(&tfull_bar[a], 1); mbar_init(&tempty_bar[a], F8_EPI_WARPS); }
    for (int a = 0; a < 2; ++a) mbar_init(&drain_bar[a], 1);
    for (int i = 0; i < F8_INFOS; ++i) { mbar_init(&ifull_bar[i], 1); mbar_init(&iempty_bar[i], F8_EPI_WARPS); }
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) { tmem_alloc(&s_tmem_base, TMEM_COLS); tmem_relinquish(); }
  wait_for_previous();
  launch_dependents();
  const int E = p.row_offsets ? p.E : 1;
  const int all_rows = (p.rows + F8_K - 1) / F8_K * F8_K;
  if (p.row_offsets) f8_offsets(p.row_offsets, E, all_rows, s_ro, p.status);
  else if (threadIdx.x < 2) s_ro[threadIdx.x] = threadIdx.x * all_rows;
  const int n_tiles = (p.N + BN - 1) / BN;
  bool snake = false;
  if (SCHED == SCHED_KGROUP) {
    __syncthreads();
    snake = kgroup_order(s_ro, E, (p.g.M / BM) * n_tiles, gridDim.x, s_order);  // complete at the barrier below
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  const int total = (SCHED == SCHED_ROWS) ? (s_ro[E] / BM) * n_tiles : E * (p.g.M / BM) * n_tiles;
  volatile int* const aborted = &s_abort;
  // tiles of this CTA: every `step`-th from its own; a split tile's contraction from block kb0 on
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int mine = SPLIT ? blockIdx.x / p.split : blockIdx.x, step = SPLIT ? total : gridDim.x;
  auto coord = [&](int tile) {
    TileCoord c = tile_coord<SCHED, EPI_STORE, false, F8_K>(p.g, s_ro, s_order, E, n_tiles, tile);
    if (SPLIT) {
      const int per = (c.kblocks + p.split - 1) / p.split, kb0 = min(rank * per, c.kblocks);
      c.a_k += kb0 * F8_K;
      c.b_k += kb0 * F8_K;
      c.kblocks = min(per, c.kblocks - kb0);
    }
    return c;
  };
  const uint32_t leader = lane == 0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8_REGS_FEW));
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    for (int rnd = 0, tile = sched_tile(0, mine, step, snake); tile < total && !*aborted;
         tile = sched_tile(++rnd, mine, step, snake)) {
      const TileCoord c = coord(tile);
#pragma unroll 1
      for (int kb = 0; kb < c.kblocks; ++kb) {
        pipe_wait(&empty_bar[stage], phase ^ 1, &s_abort, p.status);
        uint8_t* sa = smem + stage * STAGE_BYTES;
        uint8_t* sb = sa + F8_A_BYTES;
        uint64_t* bar = &full_bar[stage];
        pipe_expect(bar, STAGE_BYTES, leader);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        pipe_load_2d(sa, &tmA, bar, c.a_k + kb * F8_K, c.a_m, leader);
#pragma unroll
        for (int i = 0; i < BN / F8_B_BOX; ++i)
          pipe_load_2d(sb + i * F8_B_BOX * F8_K, &tmB, bar, c.b_k + kb * F8_K, c.b_n + i * F8_B_BOX, leader);
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
    if (lane == 0)
      for (int s = 0; s < STAGES; ++s)
        if ((armed >> s) & 1u) mbar_drain(&full_bar[s], (armed_parity >> s) & 1u, WAIT_LIMIT_CYCLES);
    __syncwarp();
    if (SPLIT) { cluster_sync_all(); cluster_sync_all(); }   // the summing warps' two
  } else if (warp <= 2) {
    // ------------------------------------------------------------ MMA issuers, a buffer each
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8_REGS_FEW));
    constexpr uint32_t idesc = idesc_f8(BM, BN);
    const uint64_t desc0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint32_t buf = warp - 1, d_tmem = tmem_base + buf * 256;
    int stage = 0;
    uint32_t phase = 0, it = 0;
    for (int rnd = 0, tile = sched_tile(0, mine, step, snake); tile < total && !*aborted;
         tile = sched_tile(++rnd, mine, step, snake)) {
      const TileCoord c = coord(tile);
#pragma unroll 1
      for (int kb = 0; kb < c.kblocks; ++kb, ++it) {
        if ((it & 1u) == buf) {
          pipe_wait(&tempty_bar[buf], ((it >> 1) & 1u) ^ 1u, &s_abort, p.status);
          pipe_wait(&full_bar[stage], phase, &s_abort, p.status);
          tc_fence_after();
          const uint64_t ad = desc0 + static_cast<uint32_t>(stage * (STAGE_BYTES >> 4)), bd = ad + (F8_A_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < F8_K / 32; ++kk) pipe_mma_f8(d_tmem, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u, leader);
          pipe_commit(&tfull_bar[buf], leader);
          pipe_commit(&empty_bar[stage], leader);
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
    if (lane == 0) {
      tc_commit(&drain_bar[buf]);
      mbar_drain(&drain_bar[buf], 0, WAIT_LIMIT_CYCLES);
    }
    __syncwarp();
    if (SPLIT) { cluster_sync_all(); cluster_sync_all(); }   // the summing warps' two
  } else if (warp == 3) {
    // ------------------------------------------------------------ scale loader
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8_REGS_FEW));
    int stage = 0, slot = 0, info = 0;
    uint32_t phase = 0, info_phase = 0;
    for (int rnd = 0, tile = sched_tile(0, mine, step, snake); tile < total && !*aborted;
         tile = sched_tile(++rnd, mine, step, snake)) {
      const TileCoord c = coord(tile);
      const int rows = SCHED == SCHED_ROWS ? p.rows : p.M;
      // the tile for the summing warps, to whom its coordinates would cost 1100 cycles a tile: columns, rows
      // and their end, blocks, expert
      pipe_wait(&iempty_bar[info], info_phase ^ 1, &s_abort, p.status);
      if (lane == 0) {
        s_info[info] = make_int4(c.out_col, static_cast<int>(c.out_row), SCHED == SCHED_ROWS ? min(s_ro[c.e + 1], p.rows) : c.e, c.kblocks);
        mbar_arrive(&ifull_bar[info]);
      }
      __syncwarp();
      if (++info == F8_INFOS) { info = 0; info_phase ^= 1; }
      const float* pa = p.sa + static_cast<long long>(c.a_k / F8_K) * p.sa_ld;
      // SCHED_ROWS: lanes 0 and 1 take the two halves' block scale
      const float* pb = SCHED == SCHED_ROWS ? p.sb + c.e * p.sb_e + min(c.out_col / 128 + (lane & 1), (p.N - 1) / 128) * p.sb_n + c.b_k / F8_K * p.sb_k
                                            : p.sb + static_cast<long long>(c.b_k / F8_K) * p.sb_k;
#pragma unroll 1
      for (int kb = 0; kb < c.kblocks; ++kb) {
        pipe_wait(&empty_bar[stage], phase ^ 1, &s_abort, p.status);
        float* to = s_scales + slot * SLOT;
#pragma unroll
        for (int i = 0; i < BM / 32; ++i) {
          const int r = c.a_m + 32 * i + lane;
          scale_async(to + 32 * i + lane, r < rows ? pa + r : p.sa, r < rows);
        }
        if (SCHED == SCHED_ROWS) {
          if (lane < 2) scale_async(to + BM + lane, pb, true);
        } else {
#pragma unroll
          for (int i = 0; i < BN / 32; ++i) {
            const int n = c.out_col + 32 * i + lane;
            scale_async(to + BM + 32 * i + lane, n < p.N ? pb + n : p.sb, n < p.N);
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full_bar[stage])) : "memory");
        pa += p.sa_ld;
        pb += p.sb_k;
        if (++slot == SLOTS) slot = 0;
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (SPLIT) { cluster_sync_all(); cluster_sync_all(); }   // the summing warps' two
  } else {
    // ------------------------------------------------------------ sums and stores
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F8_REGS_MANY));
    const int q = warp & 3, part = (warp - F8_EPI_WARP0) >> 2;
    uint8_t* box = s_box + (warp - F8_EPI_WARP0) * f8_box_bytes(BN);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + part * WC;
    int slot = 0, info = 0;
    uint32_t it = 0, info_phase = 0;
    for (int rnd = 0, tile = sched_tile(0, mine, step, snake); tile < total && !*aborted;
         tile = sched_tile(++rnd, mine, step, snake)) {
      pipe_wait(&ifull_bar[info], info_phase, &s_abort, p.status);
      const int4 c = s_info[info];
      __syncwarp();
      pipe_arrive(&iempty_bar[info], leader);
      if (++info == F8_INFOS) { info = 0; info_phase ^= 1; }
      const int col = c.x + part * WC, kblocks = c.w;
      f32x2 acc[WC / 2];
#pragma unroll
      for (int j = 0; j < WC / 2; ++j) acc[j] = 0;
#pragma unroll 1
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const uint32_t buf = it & 1u;
        pipe_wait(&tfull_bar[buf], (it >> 1) & 1u, &s_abort, p.status);
        tc_fence_after();
        const float* sc = s_scales + slot * SLOT;
        if (++slot == SLOTS) slot = 0;
        if constexpr (SCHED == SCHED_ROWS) {
          // a thread has a row: 64 columns at a time, the last out of tensor memory before they are added
          const float s = sc[q * 32 + lane] * sc[BM + (part * WC) / 128];
          const f32x2 s2 = pair(s, s);
#pragma unroll
          for (int i = 0; i < WC / 64; ++i) {
            uint32_t r[2][32];
            tmem_ld32(lane_base + buf * 256 + 64 * i, r[0]);
            tmem_ld32(lane_base + buf * 256 + 64 * i + 32, r[1]);
            tmem_wait_ld32(r[0]);
            tmem_wait_ld32(r[1]);
            if (i == WC / 64 - 1) {
              tc_fence_before();
              __syncwarp();
              pipe_arrive(&tempty_bar[buf], leader);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) add_scaled(acc[32 * i + j], r[j >> 4][2 * (j & 15)], r[j >> 4][2 * (j & 15) + 1], s2);
          }
        } else {
          // a thread has columns 2 (lane % 4) and the next of every eight, in rows lane / 4 + 0, 8, 16, 24: a
          // column's scale serves four rows.  With a row a thread it served one, and the scales' way from shared
          // memory to the registers bound (1600 cycles a block).
          f32x2 rs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = sc[q * 32 + 8 * i + (lane >> 2)];
            rs[i] = pair(v, v);
          }
          // scales of the next 32 columns are read ahead: each read where it is used, their latencies add up
          const uint32_t cs = smem_u32(sc + BM + part * WC + 2 * (lane & 3));
          f32x2 c2[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) c2[g] = ld_shared_pair(cs + 32 * g);
#pragma unroll
          for (int i = 0; i < WC / 32; ++i) {
            uint32_t r[2][16];
            tmem_ld_rows4(lane_base + buf * 256 + 32 * i, r[0]);
            tmem_ld_rows4(lane_base + (16u << 16) + buf * 256 + 32 * i, r[1]);
            tmem_wait_ld16(r[0]);
            tmem_wait_ld16(r[1]);
            if (i == WC / 32 - 1) {
              tc_fence_before();
              __syncwarp();
              pipe_arrive(&tempty_bar[buf], leader);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              f32x2 s4[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) s4[k] = mul2(rs[k], c2[g]);
              if (i + 1 < WC / 32) c2[g] = ld_shared_pair(cs + 32 * (4 * (i + 1) + g));
#pragma unroll
              for (int k = 0; k < 4; ++k)
                add_scaled(acc[4 * (4 * i + g) + k], r[k >> 1][4 * g + 2 * (k & 1)], r[k >> 1][4 * g + 2 * (k & 1) + 1], s4[k]);
            }
          }
        }
      }
      if (SPLIT) {                        // the part's sums, for the cluster
        float* to = reinterpret_cast<float*>(smem) + (q * 32 + lane) * F8_SPLIT_LD + part * WC;
        // the stage that this overwrites is read: every block's product has been taken out
#pragma unroll
        for (int j = 0; j < WC / 4; ++j) *reinterpret_cast<ulonglong2*>(to + 4 * j) = make_ulonglong2(acc[2 * j], acc[2 * j + 1]);
        break;
      }
      if (*aborted) break;
      // bf16 through the warp's boxes of 64 columns (16-byte pieces swizzled as the tensor store expects
      // them); boxes past the ends are skipped
      const int y0 = c.y + q * 32, y_end = SCHED == SCHED_ROWS ? c.z : p.M;
      const uint32_t at = smem_u32(box) + lane * 128;
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      if constexpr (SCHED == SCHED_KGROUP) {
#pragma unroll
        for (int g = 0; g < WC / 8; ++g) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 8 * k + (lane >> 2);
            const float2 v = unpair(acc[4 * g + k]);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(smem_u32(box) + (g >> 3) * 4096 + row * 128 + (((g & 7) ^ (row & 7)) << 4) + 4 * (lane & 3)),
                         "r"(pack_bf16(v.x, v.y))
                         : "memory");
          }
        }
      } else
#pragma unroll
      for (int j = 0; j < WC / 8; ++j) {
        float2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = unpair(acc[4 * j + i]);
        st_shared_v4(at + (j >> 3) * 4096 + (((j & 7) ^ (lane & 7)) << 4), pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y),
                     pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && y0 < y_end) {
#pragma unroll
        for (int j = 0; j < WC / 64; ++j)
          if (col + 64 * j < p.N) tma_store_3d(&tmC, box + j * 4096, col + 64 * j, y0, SCHED == SCHED_KGROUP ? c.z : 0);
        bulk_commit();
      }
    }
    if (lane == 0) bulk_wait_all();
    if (SPLIT) {
      // each CTA adds the parts of its share of the tile's columns, in the order of the contraction
      __syncwarp();
      cluster_sync_all();
      const TileCoord c = tile_coord<SCHED, EPI_STORE, false, F8_K>(p.g, s_ro, s_order, E, n_tiles, mine);
      const int rows = min(BM, p.rows - c.a_m), cols = BN / p.split, col0 = rank * cols;
      for (int i = threadIdx.x - 32 * F8_EPI_WARP0; i < rows * (cols / 4) && !*aborted; i += 32 * F8_EPI_WARPS) {
        const int r = i / (cols / 4), n = col0 + (i - r * (cols / 4)) * 4;
        if (c.out_col + n >= p.N) continue;
        const uint32_t at = smem_u32(smem) + (r * F8_SPLIT_LD + n) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < p.split; ++k) {
          float x[4];
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                       : "r"(mapa_shared(at, k))
                       : "memory");
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += x[j];
        }
        *reinterpret_cast<uint2*>(p.out + static_cast<long long>(c.a_m + r) * p.N + c.out_col + n) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      }
      __syncwarp();
      cluster_sync_all();        // no CTA leaves while another may read its parts
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

template <int SCHED, int BN, bool SPLIT = false>
static cudaError_t launch_fp8_t(const CUtensorMap& a, const CUtensorMap& b, const void* out, int groups, int out_rows, const Fp8Params& p,
                                cudaStream_t stream, int tiles = 0) {
  CUtensorMap c;
  if (!make_tensor_map_store3(&c, out, p.N, out_rows, groups)) return cudaErrorInvalidValue;
  constexpr int smem = f8_smem(BN, SCHED == SCHED_KGROUP);
  const cudaError_t err = allow_smem<fp8_gemm_kernel<SCHED, BN, SPLIT>>(smem);
  if (err != cudaSuccess) return err;
  return launch_early_clusters(fp8_gemm_kernel<SCHED, BN, SPLIT>, dim3(SPLIT ? tiles * p.split : num_sms()), dim3(F8_THREADS), smem, stream,
                      SPLIT ? p.split : 0, a, b, c, p);
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
  // 256 columns a tile; 128 where those are too few to fill the SMs, and where experts have about a tile of rows or
  // less: reading the weights bounds those, and tiles of half the width spread over the SMs more evenly (4 tokens
  // through a layer of 256 experts: 268 us with 256, 249 with 128).
  const int64_t wide = tiles * ((N + 255) / 256);
  const int bn = N <= 128 || wide < num_sms() || rows <= 256ll * E ? 128 : 256;
  CUtensorMap ta, tb;
  if (!make_tensor_map_u8(&ta, a, K, rows, F8_K, BM) ||
      !make_tensor_map_u8(&tb, b, K, static_cast<uint64_t>(E) * N, F8_K, F8_B_BOX))
    return MOE_ERR_CUDA;
  Fp8Params p{};
  p.rows = static_cast<int>(rows); p.N = N; p.E = E; p.row_offsets = row_offsets;
  p.sa = a_scales; p.sa_ld = rows;
  const long long nb = (N + 127) / 128, kb = (K + 127) / 128;
  p.sb = b_scales; p.sb_e = nb * kb; p.sb_n = b_transposed ? 1 : kb; p.sb_k = b_transposed ? nb : 1;
  p.g.BN = bn; p.g.K = static_cast<int>(up128(K)); p.g.b_rows_per_expert = N; p.g.m_fastest = ORDER_PER_GROUP;
  p.g.band_krows = BAND_KROWS_E4M3;
  p.status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int R = p.rows;
  // One matrix and few tiles: the contraction over up to eight SMs a tile, four blocks each or more but for the last
  // ones, which take what is left (33 blocks over eight: five each, three, none).  (5 x 4096 x 7168,
  // bound by reading the weights: 13 us on 128 SMs, 22 on 32).
  const int64_t few = tiles * ((N + 127) / 128);
  if (!row_offsets) {
    p.split = 1;
    while (p.split < 8 && few * p.split * 2 <= num_sms() && kb >= 8ll * p.split) p.split *= 2;
    p.out = out;
    if (p.split > 1) return status_of(launch_fp8_t<SCHED_ROWS, 128, true>(ta, tb, out, 1, R, p, s, static_cast<int>(few)));
  }
  const cudaError_t e = bn == 128 ? launch_fp8_t<SCHED_ROWS, 128>(ta, tb, out, 1, R, p, s) : launch_fp8_t<SCHED_ROWS, 256>(ta, tb, out, 1, R, p, s);
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
  CUtensorMap ta, tb;
  if (!make_tensor_map_u8(&ta, dy_t, rows, N, F8_K, BM) || !make_tensor_map_u8(&tb, x_t, rows, K, F8_K, F8_B_BOX)) return MOE_ERR_CUDA;
  Fp8Params p{};
  p.rows = static_cast<int>(rows); p.M = N; p.N = K; p.E = E; p.row_offsets = row_offsets;
  p.sa = dy_scales; p.sa_ld = N; p.sb = x_scales; p.sb_k = K;
  p.g.BN = bn; p.g.M = static_cast<int>(up128(N)); p.g.N = K; p.g.m_fastest = N <= K ? 1 : 0;
  p.status = dev_status;
  const cudaError_t e = bn == 256 ? launch_fp8_t<SCHED_KGROUP, 256>(ta, tb, out, E, N, p, s)
                                  : launch_fp8_t<SCHED_KGROUP, 128>(ta, tb, out, E, N, p, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
