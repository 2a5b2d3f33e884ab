// An update orthogonalised by Newton-Schulz products, for batches of matrices.
//
//   X_0 = U / max(|U|_F, floor);   A = X X^T;  B = b A + c A A;  X' = a X + B X      (a, b, c of each step)
//
// on the side with fewer rows: X is [s][l], s <= l, in the workspace, transposed where the
// tensor is tall, and padded with zeros to multiples of 128 (which the products keep at zero).
//
// Arithmetic: tensor-core products of fp16 operands with fp32 sums.  Every matrix here is bounded (singular
// values below 1.3), so fp16's 11 bits serve better than bf16's 8.  The caller chooses between
//   SPLIT: X, A and B each in two fp16 parts, 22 bits, and three products (lo hi + hi lo + hi hi) for each.  The roundings
//     cost 3e-6 of the factor's norm at 1024 x 1024 and less for smaller matrices; what tensor-core sums lose comes on
//     top of it with long contractions (1e-6 to 2e-6 off up to 128 x 256, where fp32 products are too, 7e-6 at 1024 x 1024,
//     4e-5 at 1536 x 4096);
//   one part, a third of the multiplying: on gaussian matrices with 128 rows or more the result is 0.8e-3 to 1.2e-3 off,
//     relative to its norm (bf16 operands: 1.1e-2); with fewer, up to 3e-3, and up to 8e-3 below 16.
// X is held times a power of two near sqrt(l), so that its entries stay normal numbers.  The addend a X would carry X's
// rounding past the products straight into the small singular values, which later steps amplify by up to a each; X is
// therefore kept in two fp16 parts also where its products take one (low-rank plus noise: 3.4e-3 off without, 2.4e-4 with it).
// In the last two steps X is near orthogonal, A near a multiple of I and B near a negative one; taking the
// multiples off first, A' = A - u I and X' = (a - t) X + (B + t I) X with u = 1/2, t = a - 1, leaves fp16 less to
// round (the same polynomial in other terms: 1.3e-3 -> 5.2e-4 on strong directions under noise, 300 x 700).  (A second
// part of A for its addend alone does not help: A's rounding in b A and in c A A partly cancels.)
// A and B are symmetric: only tiles on and above the diagonal are computed, the others mirrored.
//
// Bound: tensor cores, s s l / 2 + s s s / 2 + s s l multiply-adds a step and matrix.  48 matrices of 1536 x 4096, five
// steps: 18.2 ms, of which the products 16.4 (73 % of the measured bf16 rate for three products each; operands from shared
// memory and the power limit), the passes over momenta, weights and X 1.8; with one part 7.9 to 8.0 ms, 6.3 (64 %) and 1.6.
#include "around.cuh"
#include "kernels.h"
#include "pipe.cuh"
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

namespace moe {

constexpr int NS_STAGES = 5;
constexpr int NS_EPI_WARPS = 8;
constexpr int NS_THREADS = 64 + 32 * NS_EPI_WARPS;
constexpr int NS_BOX = 2048;                       // a 32 x 32 box of 16-bit values
constexpr int NS_EPI_BYTES = 4 * NS_BOX;           // a warp's boxes: two read, two written
constexpr int NS_SMEM = NS_STAGES * P_STAGE_BYTES + NS_EPI_WARPS * NS_EPI_BYTES + 1024;

enum { NS_GRAM = 0, NS_POLY = 1, NS_APPLY = 2 };   // A = X X^T; B = b A + c A A; X' = a X + B X

struct NsParams {
  int batch, s, n, k;       // a matrix's padded rows, output columns, contraction
  float alpha, beta, diag;  // out = alpha * product + beta * in + diag I (not NS_APPLY)
  int lo_out;               // NS_APPLY: X's second part is written
  int32_t* status;
};

// kind::f16 with fp16 A and B, fp32 D; see idesc_bf16.
__host__ __device__ constexpr uint32_t idesc_fp16(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half_pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

struct NsTile {
  int e, m, n;   // matrix, 256-row block, 256-column block
};
template <int KIND>
__device__ __forceinline__ NsTile ns_tile(const NsParams& p, int t) {
  const int mt = (p.s + 255) / 256, nt = (p.n + 255) / 256;
  NsTile o;
  if (KIND == NS_APPLY) {
    const int per = mt * nt;
    o.e = t / per;
    const int r = t - o.e * per;
    o.n = r / mt;
    o.m = r - o.n * mt;
  } else {                                          // n >= m, column by column
    const int per = mt * (mt + 1) / 2;
    o.e = t / per;
    int r = t - o.e * per, n = 0;
    while (r > n) r -= ++n;
    o.n = n;
    o.m = r;
  }
  return o;
}

// One CTA pair computes a 256 x 256 tile (tcgen05 cta_group::2), as in gemm2.cuh: warp 0 of each
// CTA loads its halves, warp 1 of the leader multiplies, eight warps of each take its 128 rows out.
// What the sum is added to arrives by tensor loads in a warp's boxes, a chunk of 32 columns ahead, across
// tiles.  The MMA warp looks for two stages at a time: a wait's latency, 130 cycles, comes on top of the
// 512 that a stage's MMAs take.
// SPLIT: the contraction runs three times into one sum, over A's second parts and B's first, A's first and B's second, and
// both first; results leave in two parts.  The first parts come last: tensor-core sums lose up to a unit in the last place
// at each step of 16, which counts for most where the sum is large.
template <int KIND, bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NS_THREADS, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmALo, const __grid_constant__ CUtensorMap tmBLo,
                   const __grid_constant__ CUtensorMap tmIn, const __grid_constant__ CUtensorMap tmInLo,
                   const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmOutLo, const NsParams p) {
  constexpr bool B_MN = KIND == NS_APPLY;
  constexpr bool TWO_IN = KIND == NS_APPLY || (SPLIT && KIND == NS_POLY);   // what is added is in two parts
  extern __shared__ uint8_t dyn_smem[];
  __shared__ __align__(8) uint64_t full_bar[NS_STAGES];
  __shared__ __align__(8) uint64_t empty_bar[NS_STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(8) uint64_t in_bar[NS_EPI_WARPS];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair_id = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS_STAGES; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&tfull_bar[a], 1); mbar_init(&tempty_bar[a], 2 * NS_EPI_WARPS); }
    for (int w = 0; w < NS_EPI_WARPS; ++w) mbar_init(&in_bar[w], 1);
    mbar_init(&drain_bar, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc_pair(&s_tmem_base, TMEM_COLS); tmem_relinquish_pair(); }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  wait_for_previous();
  launch_dependents();
  const uint32_t tmem_base = s_tmem_base;
  const int mt = (p.s + 255) / 256;
  const int total = p.batch * (KIND == NS_APPLY ? mt * ((p.n + 255) / 256) : mt * (mt + 1) / 2);
  const int kblocks = p.k / BK, all_kblocks = SPLIT ? 3 * kblocks : kblocks;
  volatile int* const aborted = &s_abort;
  const uint32_t leader = lane == 0;

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    for (int t = pair_id; t < total && !*aborted; t += npairs) {
      const NsTile c = ns_tile<KIND>(p, t);
      // a half past the matrix's rows (or columns) reads the zero fill past the tensor
      const int a_local = c.m * 256 + rank * 128, b_local = c.n * 256 + rank * 128;
      const int a_row = a_local < p.s ? c.e * p.s + a_local : DEAD_ROW;
      const int b_row = b_local < p.n ? c.e * p.s + b_local : DEAD_ROW;
      int part = 0, kb = 0;
#pragma unroll 1
      for (int i = 0; i < all_kblocks; ++i) {
        const CUtensorMap* ma = SPLIT && part == 0 ? &tmALo : &tmA;
        const CUtensorMap* mb = SPLIT && part == 1 ? &tmBLo : &tmB;
        pipe_wait(&empty_bar[stage], phase ^ 1, &s_abort, p.status);
        uint8_t* sa = smem + stage * P_STAGE_BYTES;
        uint8_t* sb = sa + P_A_BYTES;
        const uint32_t bar = mapa_shared(smem_u32(&full_bar[stage]), 0);
        pipe_expect(&full_bar[stage], 2 * P_STAGE_BYTES, leader && rank == 0);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        pipe_load_2d_pair(sa, ma, bar, kb * BK, a_row, leader);
        if (!B_MN) {
          pipe_load_2d_pair(sb, mb, bar, kb * BK, b_row, leader);
        } else {
          pipe_load_2d_pair(sb, mb, bar, b_local, c.e * p.s + kb * BK, leader);
          pipe_load_2d_pair(sb + 8192, mb, bar, b_local + 64, c.e * p.s + kb * BK, leader);
        }
        if (++kb == kblocks) { kb = 0; ++part; }
        if (++stage == NS_STAGES) { stage = 0; phase ^= 1; }
      }
    }
    if (lane == 0 && rank == 0)
      for (int s = 0; s < NS_STAGES; ++s)
        if ((armed >> s) & 1u) mbar_drain(&full_bar[s], (armed_parity >> s) & 1u, WAIT_LIMIT_CYCLES);
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_fp16(256, 256, B_MN ? 1 : 0);
      const uint64_t desc_a = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t desc_b = B_MN ? smem_desc_sw128(smem_u32(smem) + P_A_BYTES, 8192, 1024) : smem_desc_sw128(smem_u32(smem) + P_A_BYTES, 16, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int t = pair_id; t < total && !*aborted; t += npairs) {
        pipe_wait(&tempty_bar[acc], acc_phase ^ 1, &s_abort, p.status);
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_STRIDE;
#pragma unroll 1
        for (int kb = 0; kb < all_kblocks; kb += 2) {    // the contraction is a multiple of 128
          const int next = stage + 1 == NS_STAGES ? 0 : stage + 1;
          pipe_wait_two(&full_bar[stage], phase, &full_bar[next], phase ^ (next == 0), &s_abort, p.status);
          tc_fence_after();
#pragma unroll
          for (int two = 0; two < 2; ++two) {
            const uint32_t at = static_cast<uint32_t>(stage * (P_STAGE_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk)
              pipe_mma_f16_pair(d_tmem, desc_a + at + 2 * kk, desc_b + at + (B_MN ? 128 : 2) * kk, idesc, (kb | two | kk) != 0 ? 1u : 0u, leader);
            pipe_commit_pair_mc(&empty_bar[stage], 0x3, leader);
            if (++stage == NS_STAGES) { stage = 0; phase ^= 1; }
          }
        }
        pipe_commit_pair_mc(&tfull_bar[acc], 0x3, leader);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (lane == 0) {
        tc_commit_pair(&drain_bar);
        mbar_drain(&drain_bar, 0, WAIT_LIMIT_CYCLES);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* in = smem + NS_STAGES * P_STAGE_BYTES + (warp - 2) * NS_EPI_BYTES;
    uint8_t* out = in + 2 * NS_BOX;
    uint64_t* ibar = &in_bar[warp - 2];
    const int sw = (lane >> 1) & 3;                  // 64-byte swizzle of this lane's row of a box
    const uint32_t in_row = smem_u32(in) + lane * 64, out_row = smem_u32(out) + lane * 64;
    int acc = 0;
    uint32_t acc_phase = 0, taken = 0, asked = 0;    // chunks
    // the chunks to ask for: of this warp's tiles (a warp whose rows or columns lie past a matrix has none there)
    struct Place {
      int row0, col0, y;
      bool live;
    };
    auto place = [&](int t) {
      const NsTile c = ns_tile<KIND>(p, t);
      Place o;
      o.row0 = c.m * 256 + rank * 128 + q * 32;      // of the matrix
      o.col0 = c.n * 256 + half * 128;
      o.live = o.row0 < p.s && o.col0 < p.n;         // 128-row and 128-column halves are whole
      o.y = c.e * p.s + o.row0;
      return o;
    };
    int ask_t = pair_id, ask_i = 0;
    Place ask{0, 0, 0, false};
    auto next_live = [&]() {
      while (ask_t < total && !(ask = place(ask_t)).live) ask_t += npairs;
    };
    auto issue = [&]() {                             // the next chunk's boxes
      if (KIND == NS_GRAM || ask_t >= total) return;
      const int x = ask.col0 + 32 * ask_i;
      if (lane == 0) fence_proxy_async_smem();
      pipe_expect(ibar, TWO_IN ? 2 * NS_BOX : NS_BOX, leader);
      pipe_load_2d(in, &tmIn, ibar, x, ask.y, leader);
      if (TWO_IN) pipe_load_2d(in + NS_BOX, &tmInLo, ibar, x, ask.y, leader);
      ++asked;
      if (++ask_i == 4) {
        ask_i = 0;
        ask_t += npairs;
        next_live();
      }
    };
    if (KIND != NS_GRAM) {
      next_live();
      issue();
    }
    for (int t = pair_id; t < total && !*aborted; t += npairs) {
      const NsTile c = ns_tile<KIND>(p, t);
      const Place at = place(t);
      const int row0 = at.row0, col0 = at.col0, y = at.y;
      pipe_wait(&tfull_bar[acc], acc_phase, &s_abort, p.status);
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * ACC_STRIDE + half * 128;
      if (at.live) {
        for (int i = 0; i < 4; ++i) {
          uint32_t r[32];
          tmem_ld32(tbase + 32 * i, r);
          uint32_t hi[16], lo[16];
          if (KIND != NS_GRAM) {
            pipe_wait(ibar, taken & 1u, &s_abort, p.status);
            if (*aborted) break;
            ++taken;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const uint4 x = ld_shared_v4(in_row + ((v ^ sw) << 4));
              const uint4 z = TWO_IN ? ld_shared_v4(in_row + NS_BOX + ((v ^ sw) << 4)) : make_uint4(0, 0, 0, 0);
              hi[4 * v] = x.x; hi[4 * v + 1] = x.y; hi[4 * v + 2] = x.z; hi[4 * v + 3] = x.w;
              lo[4 * v] = z.x; lo[4 * v + 1] = z.y; lo[4 * v + 2] = z.z; lo[4 * v + 3] = z.w;
            }
            __syncwarp();
            issue();
          }
          tmem_wait_ld();
          uint32_t oh[16], ol[16];
          const float diag = KIND != NS_APPLY && row0 == col0 + 32 * i ? p.diag : 0.0f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a = p.alpha * __uint_as_float(r[2 * j]), b = p.alpha * __uint_as_float(r[2 * j + 1]);
            if (KIND != NS_APPLY) {
              a += lane == 2 * j ? diag : 0.0f;
              b += lane == 2 * j + 1 ? diag : 0.0f;
            }
            if (KIND != NS_GRAM) {
              const float2 x = half_pair(hi[j]), z = half_pair(lo[j]);
              a = fmaf(p.beta, x.x + z.x, a);
              b = fmaf(p.beta, x.y + z.y, b);
            }
            oh[j] = pack_half(a, b);
            if (KIND == NS_APPLY || SPLIT) {
              const float2 h = half_pair(oh[j]);
              ol[j] = pack_half(a - h.x, b - h.y);
            }
          }
          const bool mirror = KIND != NS_APPLY && c.n > c.m;
#pragma unroll
          for (int part = 0; part < (SPLIT && KIND != NS_APPLY ? 2 : 1); ++part) {   // A and B in two parts: one after the other
            uint32_t(&o)[16] = part == 0 ? oh : ol;
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              st_shared_v4(out_row + ((v ^ sw) << 4), o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
              if (KIND == NS_APPLY && p.lo_out)
                st_shared_v4(out_row + NS_BOX + ((v ^ sw) << 4), ol[4 * v], ol[4 * v + 1], ol[4 * v + 2], ol[4 * v + 3]);
            }
            if (mirror) {
              // the box's transpose: two rows' values of a column meet in one word
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, o[j], 1);
                // even lanes take column 2j of rows (lane, lane + 1), odd ones column 2j + 1 of (lane - 1, lane)
                const uint32_t w = lane & 1 ? __byte_perm(other, o[j], 0x7632) : __byte_perm(o[j], other, 0x5410);
                const int col = 2 * j + (lane & 1);
                *reinterpret_cast<uint32_t*>(out + NS_BOX + col * 64 + (((lane >> 3) ^ ((col >> 1) & 3)) << 4) + ((lane >> 1) & 3) * 4) = w;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const CUtensorMap* to = part == 0 ? &tmOut : &tmOutLo;
              tma_store_2d(to, out, col0 + 32 * i, y);
              if (KIND == NS_APPLY && p.lo_out) tma_store_2d(&tmOutLo, out + NS_BOX, col0 + 32 * i, y);
              if (mirror) tma_store_2d(to, out + NS_BOX, row0, c.e * p.s + col0 + 32 * i);
              bulk_commit();
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      pipe_arrive_cluster(mapa_shared(smem_u32(&tempty_bar[acc]), 0), leader);
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    for (; taken < asked; ++taken) mbar_drain(ibar, taken & 1u, WAIT_LIMIT_CYCLES);   // after an abort
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// ------------------------------------------------------------------------ around the products

constexpr int NS_TENSORS = 32;       // of a launch
constexpr int NS_PARTS = 64;         // blocks, and partial sums of squares, a matrix at most

// A step as the kernels take it: A' = X X^T - u I;  B = c A' A' + b A' + d I;  X' = a X + B X.
struct NsStep {
  float u, a, b, c, d;
};
struct NsSteps {
  int steps;
  NsStep s[MOE_MUON_MAX_STEPS];
};
static NsSteps ns_steps(const moe_muon_hyper& h) {
  NsSteps o{};
  o.steps = h.steps;
  for (int k = 0; k < h.steps; ++k) {
    const double a = h.coefficients[3 * k], b = h.coefficients[3 * k + 1], c = h.coefficients[3 * k + 2];
    const bool late = k >= 1 && k >= h.steps - 2;
    const double u = late ? 0.5 : 0.0, t = late ? a - 1.0 : 0.0;
    o.s[k] = NsStep{static_cast<float>(u), static_cast<float>(a - t), static_cast<float>(b + 2 * u * c), static_cast<float>(c),
                    static_cast<float>(b * u + c * u * u + t)};
  }
  return o;
}

// Tensors of one shape, their matrices numbered through.
struct NsTensors {
  const void* grad[NS_TENSORS];
  float* m[NS_TENSORS];              // NULL: the gradient itself is orthogonalised
  float* w[NS_TENSORS];
  moe_bf16* w16[NS_TENSORS];
  void* out[NS_TENSORS];
  float decay[NS_TENSORS];
  int first[NS_TENSORS + 1];         // its first matrix
  int skip0;                         // matrices of the first tensor that an earlier chunk had
  int count;
  int grad_type, out_type;
  int rows, cols;                    // of a matrix
  int vec;                           // every tensor starts at 16 bytes
  float momentum;
  int nesterov;
  const moe_adamw_control* control;
};
__device__ __forceinline__ int ns_find(const NsTensors& p, int e) {
  int i = 0;
  while (i + 1 < p.count && p.first[i + 1] <= e) ++i;
  return i;
}
__device__ __forceinline__ long long ns_base(const NsTensors& p, int i, int e) {
  return static_cast<long long>(e - p.first[i] + (i == 0 ? p.skip0 : 0)) * p.rows * p.cols;
}
// Eight values from element i on, one by one where rows do not start at whole vectors (`n` of them are there).
__device__ __forceinline__ void ns_get8(float (&v)[8], const void* g, int type, long long i, bool vec, int n) {
  if (vec) {
    if (type == MOE_TYPE_BF16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) { v[2 * j] = bf16_lo(u[j]); v[2 * j + 1] = bf16_hi(u[j]); }
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
      const float4 x = f[0], y = f[1];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = j >= n ? 0.0f : type == MOE_TYPE_BF16 ? bf16_lo(static_cast<const uint16_t*>(g)[i + j]) : static_cast<const float*>(g)[i + j];
  }
}
__device__ __forceinline__ void ns_put8(const float (&v)[8], void* o, int type, long long i, bool vec, int n) {
  if (vec) {
    if (type == MOE_TYPE_BF16) store8(static_cast<moe_bf16*>(o) + i, v);
    else store8(static_cast<float*>(o) + i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= n) continue;
      if (type == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(o)[i + j] = __float2bfloat16_rn(v[j]);
      else static_cast<float*>(o)[i + j] = v[j];
    }
  }
}

// |U|_F from two sums of squares: of U, and of U times 2^100, which keeps what underflows in the first. The second
// serves where the first is below 2^-80: there no element reaches 2^-40 and the second cannot overflow (2^120), and above it
// the squares lost below 2^-149 are no part of the sum (2^32 of them are 2^-37 of it). fp32's smallest numbers
// are 2^-49 times 2^100, their squares normal numbers.
constexpr float NS_TINY = 8.271806125530277e-25f;          // 2^-80
constexpr float NS_UP = 1.2676506002282294e30f;            // 2^100
__device__ __forceinline__ void ns_add_square(float (&s)[2], float u) {
  const float t = u * NS_UP;
  s[0] = fmaf(u, u, s[0]);
  s[1] = fmaf(t, t, s[1]);
}
// What takes U to X_0, over a norm of at least `floor`: times `up`, a power of two, then times `inv`. Zeros stay zeros; a
// sum that overflowed, or a NaN in it, makes NaNs rather than a silent zero.
struct NsNorm {
  float up, inv;
};
__device__ __forceinline__ NsNorm ns_norm(const float (&s)[2], float scale, float floor) {
  if (!(s[0] < __int_as_float(0x7f800000))) return {1.0f, __int_as_float(0x7fc00000)};
  const bool tiny = s[0] < NS_TINY;
  const float up = tiny ? NS_UP : 1.0f, norm = fmaxf(sqrtf(tiny ? s[1] : s[0]), floor * up);
  return {up, norm > 0.0f ? scale / norm : 0.0f};
}

// m = momentum m + scale g; the sums of squares of what is orthogonalised, in at most NS_PARTS parts a matrix.
__global__ void __launch_bounds__(256) ns_momentum_kernel(const NsTensors p, float* parts) {
  wait_for_previous();
  launch_dependents();
  __shared__ float buf[64];
  const int e = blockIdx.y, i = ns_find(p, e);
  const bool skip = p.control && p.control->skip;
  const float gs = p.control ? p.control->grad_scale : 1.0f;
  const long long n = static_cast<long long>(p.rows) * p.cols, base = ns_base(p, i, e);
  const bool vec = p.vec && n % 8 == 0;
  float s[2] = {0.0f, 0.0f};
  float* m = p.m[i];
#pragma unroll 2
  for (long long j = (blockIdx.x * 256ll + threadIdx.x) * 8; j < n && !skip; j += gridDim.x * 2048ll) {
    const int left = static_cast<int>(n - j < 8 ? n - j : 8);
    float g[8], v[8];
    ns_get8(g, p.grad[i], p.grad_type, base + j, vec, left);
    if (m) ns_get8(v, m, MOE_TYPE_FP32, base + j, vec, left);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float u = gs * g[k];
      if (m) {
        v[k] = fmaf(p.momentum, v[k], u);
        u = p.nesterov ? fmaf(p.momentum, v[k], u) : v[k];
      }
      ns_add_square(s, u);
    }
    if (m) ns_put8(v, m, MOE_TYPE_FP32, base + j, vec, left);
  }
  row_sums<false>(s, buf);
  if (threadIdx.x == 0) {
    parts[2 * e * NS_PARTS + blockIdx.x] = s[0];
    parts[(2 * e + 1) * NS_PARTS + blockIdx.x] = s[1];
  }
}

// The two kernels below move 64 x 64 tiles between a tensor and X, a thread eight columns of two rows on
// either side, through shared memory where the tensor is tall and X its transpose.
constexpr int NS_LD = 65;
template <bool TALL>
__device__ __forceinline__ void ns_turn(float (&v)[2][8], float* tile, int r, int c) {
  if (!TALL) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[(r + 32 * k) * NS_LD + c + j] = v[k][j];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = tile[(c + j) * NS_LD + r + 32 * k];
}

// X = scale U / max(|U|, floor) in two fp16 parts, [s][l] with zeros in the padding.
template <bool TALL>
__global__ void __launch_bounds__(256) ns_load_kernel(const NsTensors p, const float* parts, int nparts, int s, int l, float scale,
                                                      float floor, __half* hi, __half* lo) {
  wait_for_previous();
  launch_dependents();
  __shared__ float tile[TALL ? 64 * NS_LD : 1];
  const int e = blockIdx.z, i = ns_find(p, e);
  const float gs = p.control ? p.control->grad_scale : 1.0f;
  float sum[2] = {0.0f, 0.0f};
  for (int j = 0; j < nparts; ++j) sum[0] += parts[2 * e * NS_PARTS + j];
  if (sum[0] < NS_TINY)                                          // the other sum serves (always added: 58 us became 74)
    for (int j = 0; j < nparts; ++j) sum[1] += parts[(2 * e + 1) * NS_PARTS + j];
  const NsNorm norm = ns_norm(sum, scale, floor);
  const long long base = ns_base(p, i, e);
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
  const int x0 = blockIdx.x * 64, y0 = blockIdx.y * 64;          // of X
  float v[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = (TALL ? x0 : y0) + r + 32 * k, col = (TALL ? y0 : x0) + c;
    const int left = row < p.rows ? max(0, min(8, p.cols - col)) : 0;
    const bool vec = p.vec && p.cols % 8 == 0 && left == 8;
    const long long at = base + static_cast<long long>(row) * p.cols + col;
    float g[8], m[8];
    ns_get8(g, p.grad[i], p.grad_type, at, vec, left);
    if (p.m[i]) ns_get8(m, p.m[i], MOE_TYPE_FP32, at, vec, left);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float u = gs * g[j];
      if (p.m[i]) u = p.nesterov ? fmaf(p.momentum, m[j], u) : m[j];
      v[k][j] = u * norm.up * norm.inv;
    }
  }
  ns_turn<TALL>(v, tile, r, c);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const long long at = (static_cast<long long>(e) * s + y0 + r + 32 * k) * l + x0 + c;
    uint32_t h[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = pack_half(v[k][2 * j], v[k][2 * j + 1]);
      const float2 f = half_pair(h[j]);
      w[j] = pack_half(v[k][2 * j] - f.x, v[k][2 * j + 1] - f.y);
    }
    *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// w = w - lr (decay w + rms sqrt(max side) X), or out = X; lo: X's second part, or NULL.
template <bool TALL>
__global__ void __launch_bounds__(256) ns_update_kernel(const NsTensors p, const __half* x, const __half* lo, int s, int l, float unscale,
                                                        float lr, float rms) {
  wait_for_previous();
  launch_dependents();
  __shared__ float tile[TALL ? 64 * NS_LD : 1];
  const int e = blockIdx.z, i = ns_find(p, e);
  if (p.control && p.control->skip) return;
  const float rate = p.control ? lr * p.control->lr_scale : lr;
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
  const int x0 = blockIdx.x * 64, y0 = blockIdx.y * 64;          // of the tensor
  float v[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {                                  // X's padding holds whole tiles
    const long long at = (static_cast<long long>(e) * s + (TALL ? x0 : y0) + r + 32 * k) * l + (TALL ? y0 : x0) + c;
    const uint4 h = *reinterpret_cast<const uint4*>(x + at);
    const uint4 g = lo ? *reinterpret_cast<const uint4*>(lo + at) : make_uint4(0, 0, 0, 0);
    const uint32_t u[4] = {h.x, h.y, h.z, h.w}, d[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = half_pair(u[j]), z = lo ? half_pair(d[j]) : make_float2(0.0f, 0.0f);
      v[k][2 * j] = unscale * (f.x + z.x);
      v[k][2 * j + 1] = unscale * (f.y + z.y);
    }
  }
  ns_turn<TALL>(v, tile, r, c);
  const long long base = ns_base(p, i, e);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = y0 + r + 32 * k, col = x0 + c;
    const int left = row < p.rows ? max(0, min(8, p.cols - col)) : 0;
    if (left == 0) continue;
    const bool vec = p.vec && p.cols % 8 == 0 && left == 8;
    const long long at = base + static_cast<long long>(row) * p.cols + col;
    if (p.out[i]) {
      ns_put8(v[k], p.out[i], p.out_type, at, vec, left);
    } else {
      float w[8];
      ns_get8(w, p.w[i], MOE_TYPE_FP32, at, vec, left);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = fmaf(-rate, fmaf(p.decay[i], w[j], rms * v[k][j]), w[j]);
      ns_put8(w, p.w[i], MOE_TYPE_FP32, at, vec, left);
      if (p.w16[i]) ns_put8(w, p.w16[i], MOE_TYPE_BF16, at, vec, left);
    }
  }
}

// ------------------------------------------------------------------------ small matrices
//
// A matrix of at most 128 x 256 goes through the whole step in one block: X in fp32 registers (a thread has a
// row, half of the columns), its fp16 form, A and B in shared memory, products in tensor memory.  Fifteen products of
// one tile each are latency: 39 us for six matrices of 131 x 72 (one part: 26; 98 with 18 launches).
// X's fp16 form lies in blocks of 64 columns, 128 rows of 128 bytes each (128-byte swizzle), which the MMA reads
// K-major in X X^T and MN-major in B X.

constexpr int SM_BLOCK = 128 * 128;                  // bytes of 128 rows x 64 columns
// X, A and B lie where X's fp32 form was before them and is after.  SPLIT: two parts of X, then two of A, which B's
// take the place of.
__host__ __device__ constexpr int small_smem(int l, bool split) {
  const int stage = 128 * (l + 1) * 4, operands = (split ? 2 * (l / 64) + 4 : l / 64 + 4) * SM_BLOCK;
  return (stage > operands ? stage : operands) + 1024;
}

__device__ __forceinline__ void small_put(uint32_t block0, int row, int col, const float* v) {   // eight columns
  const uint32_t at = block0 + (col >> 6) * SM_BLOCK + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
  st_shared_v4(at, pack_half(v[0], v[1]), pack_half(v[2], v[3]), pack_half(v[4], v[5]), pack_half(v[6], v[7]));
}

// The same in two fp16 parts.
__device__ __forceinline__ void small_put_split(uint32_t hi0, uint32_t lo0, int row, int col, const float* v) {
  const uint32_t at = (col >> 6) * SM_BLOCK + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
  uint32_t h[4], d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = pack_half(v[2 * j], v[2 * j + 1]);
    const float2 f = half_pair(h[j]);
    d[j] = pack_half(v[2 * j] - f.x, v[2 * j + 1] - f.y);
  }
  st_shared_v4(hi0 + at, h[0], h[1], h[2], h[3]);
  st_shared_v4(lo0 + at, d[0], d[1], d[2], d[3]);
}

template <int L, bool SPLIT>
__global__ void __launch_bounds__(256, 1) ns_small_kernel(const NsTensors p, const NsSteps h, float scale, float floor, float lr, float rms,
                                                          int32_t* status) {
  constexpr int HALF = L / 2;                        // X's columns of a thread
  extern __shared__ uint8_t dyn_smem[];
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float buf[64];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(&bar, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) { tmem_alloc(&s_tmem, TMEM_COLS); tmem_relinquish(); }
  float* stage = reinterpret_cast<float*>(smem);     // [128][L + 1]
  for (int i = tid; i < 128 * (L + 1); i += 256) stage[i] = 0.0f;
  tc_fence_before();
  wait_for_previous();
  launch_dependents();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  const int e = blockIdx.x, ti = ns_find(p, e);
  const bool skip = p.control && p.control->skip;
  const float gs = p.control ? p.control->grad_scale : 1.0f;
  const bool tall = p.rows > p.cols;
  const int n = p.rows * p.cols;
  const long long base = ns_base(p, ti, e);
  float* m = p.m[ti];
  float sq[2] = {0.0f, 0.0f};
  constexpr int WAYS = 8;                            // elements of a thread on their way together
  for (int i0 = tid; i0 < n && !skip; i0 += 256 * WAYS) {
    float g[WAYS], v[WAYS];
    if (p.grad_type == MOE_TYPE_BF16) {
      const uint16_t* from = static_cast<const uint16_t*>(p.grad[ti]) + base;
      uint16_t b[WAYS];
#pragma unroll
      for (int j = 0; j < WAYS; ++j) b[j] = from[min(i0 + 256 * j, n - 1)];
#pragma unroll
      for (int j = 0; j < WAYS; ++j) g[j] = bf16_lo(b[j]);
    } else {
      const float* from = static_cast<const float*>(p.grad[ti]) + base;
#pragma unroll
      for (int j = 0; j < WAYS; ++j) g[j] = from[min(i0 + 256 * j, n - 1)];
    }
    if (m) {
#pragma unroll
      for (int j = 0; j < WAYS; ++j) v[j] = m[base + min(i0 + 256 * j, n - 1)];
    }
#pragma unroll
    for (int j = 0; j < WAYS; ++j) {
      const int i = i0 + 256 * j;
      if (i >= n) break;
      float u = gs * g[j];
      if (m) {
        const float w = fmaf(p.momentum, v[j], u);
        m[base + i] = w;
        u = p.nesterov ? fmaf(p.momentum, w, u) : w;
      }
      ns_add_square(sq, u);
      const int r = i / p.cols, c = i - r * p.cols;
      stage[(tall ? c : r) * (L + 1) + (tall ? r : c)] = u;
    }
  }
  row_sums<false>(sq, buf);
  __syncthreads();
  const NsNorm norm = ns_norm(sq, scale, floor);
  const int row = (warp & 3) * 32 + lane, col0 = (warp >> 2) * HALF;
  float x[HALF];
#pragma unroll
  for (int j = 0; j < HALF; ++j) x[j] = stage[row * (L + 1) + col0 + j] * norm.up * norm.inv;
  __syncthreads();

  const uint32_t sx = smem_u32(smem), sx_lo = sx + (L / 64) * SM_BLOCK, sa = sx_lo + (SPLIT ? (L / 64) * SM_BLOCK : 0), sa_lo = sa + 2 * SM_BLOCK;
  const uint32_t sb = SPLIT ? sa : sa_lo, sb_lo = sa_lo;   // one part: A's second place is B's
  constexpr int PART0 = SPLIT ? 0 : 2;               // lo hi, hi lo, hi hi
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  // steps of 16 that the matrix's own rows and columns reach; what lies past them is not multiplied, and what
  // tensor memory and X's registers hold there is not used
  const int ks = (min(p.rows, p.cols) + 15) / 16, kl = (max(p.rows, p.cols) + 15) / 16;
  uint32_t phase = 0;
  // products: the writers' shared memory is handed to the tensor core, one thread issues, all wait
  auto hand = [&]() {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  auto take = [&]() {
    mbar_wait_bounded(&bar, phase, &s_abort, status, WAIT_LIMIT_CYCLES);
    phase ^= 1u;
    __syncwarp();
    tc_fence_after();
  };
#pragma unroll 1
  for (int k = 0; k < h.steps; ++k) {
    const NsStep q = h.s[k];
#pragma unroll
    for (int j = 0; j < HALF; j += 8)
      if (col0 + j < 16 * kl) {
        if (SPLIT) small_put_split(sx, sx_lo, row, col0 + j, x + j);
        else small_put(sx, row, col0 + j, x + j);
      }
    hand();
    if (tid == 0) {                                  // A = X X^T
#pragma unroll
      for (int part = PART0; part < 3; ++part)
#pragma unroll
        for (int kk = 0; kk < L / 16; ++kk) {
          if (kk >= kl) break;
          const uint32_t at = (kk >> 2) * SM_BLOCK + (kk & 3) * 32;
          tc_mma_f16(tmem, smem_desc_sw128((part == 0 ? sx_lo : sx) + at, 16, 1024), smem_desc_sw128((part == 1 ? sx_lo : sx) + at, 16, 1024),
                     idesc_fp16(128, 128, 0), part != PART0 || kk != 0);
        }
      tc_commit(&bar);
    }
    __syncwarp();
    take();
    const int ac = (warp >> 2) * 64;                 // A's and B's columns of a thread
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (ac + 32 * i >= 16 * ks) break;
      uint32_t r[32];
      tmem_ld32(tmem + lanes + ac + 32 * i, r);
      tmem_wait_ld();
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * (1.0f / (scale * scale)) - (row == ac + 32 * i + j ? q.u : 0.0f);
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        if (SPLIT) small_put_split(sa, sa_lo, row, ac + 32 * i + j, v + j);
        else small_put(sa, row, ac + 32 * i + j, v + j);
      }
    }
    hand();
    if (tid == 0) {                                  // A A
#pragma unroll
      for (int part = PART0; part < 3; ++part)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          if (kk >= ks) break;
          const uint32_t at = (kk >> 2) * SM_BLOCK + (kk & 3) * 32;
          tc_mma_f16(tmem + 128, smem_desc_sw128((part == 0 ? sa_lo : sa) + at, 16, 1024), smem_desc_sw128((part == 1 ? sa_lo : sa) + at, 16, 1024),
                     idesc_fp16(128, 128, 0), part != PART0 || kk != 0);
        }
      tc_commit(&bar);
    }
    __syncwarp();
    take();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (ac + 32 * i >= 16 * ks) break;
      uint32_t r[32];
      tmem_ld32(tmem + lanes + 128 + ac + 32 * i, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        const int col = ac + 32 * i + j;
        const uint32_t at = (col >> 6) * SM_BLOCK + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
        const uint4 w = ld_shared_v4(sa + at), z = SPLIT ? ld_shared_v4(sa_lo + at) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w}, d[4] = {z.x, z.y, z.z, z.w};
        float v[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float2 f = half_pair(u[t]);
          if (SPLIT) {
            const float2 g = half_pair(d[t]);
            f.x += g.x;
            f.y += g.y;
          }
          v[2 * t] = fmaf(q.b, f.x, q.c * __uint_as_float(r[j + 2 * t])) + (row == col + 2 * t ? q.d : 0.0f);
          v[2 * t + 1] = fmaf(q.b, f.y, q.c * __uint_as_float(r[j + 2 * t + 1])) + (row == col + 2 * t + 1 ? q.d : 0.0f);
        }
        if (SPLIT) small_put_split(sb, sb_lo, row, col, v);   // over the elements of A that this thread alone reads
        else small_put(sb, row, col, v);
      }
    }
    hand();
    if (tid == 0) {                                  // B X
#pragma unroll
      for (int part = PART0; part < 3; ++part)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          if (kk >= ks) break;
          tc_mma_f16(tmem + 256, smem_desc_sw128((part == 0 ? sb_lo : sb) + (kk >> 2) * SM_BLOCK + (kk & 3) * 32, 16, 1024),
                     smem_desc_sw128((part == 1 ? sx_lo : sx) + kk * 2048, SM_BLOCK, 1024), idesc_fp16(128, 16 * kl, 1), part != PART0 || kk != 0);
        }
      tc_commit(&bar);
    }
    __syncwarp();
    take();
#pragma unroll
    for (int i = 0; i < HALF / 32; ++i) {
      if (col0 + 32 * i >= 16 * kl) break;
      uint32_t r[32];
      tmem_ld32(tmem + lanes + 256 + col0 + 32 * i, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) x[32 * i + j] = fmaf(q.a, x[32 * i + j], __uint_as_float(r[j]));
    }
  }
  tc_fence_before();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < HALF; ++j) stage[row * (L + 1) + col0 + j] = x[j] * (1.0f / scale);
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
  if (skip) return;
  const float rate = p.control ? lr * p.control->lr_scale : lr;
  float* const weights = p.w[ti];
  for (int i0 = tid; i0 < n; i0 += 256 * WAYS) {
    float w[WAYS];
#pragma unroll
    for (int j = 0; j < WAYS; ++j) w[j] = weights ? weights[base + min(i0 + 256 * j, n - 1)] : 0.0f;
#pragma unroll
    for (int j = 0; j < WAYS; ++j) {
      const int i = i0 + 256 * j;
      if (i >= n) break;
      const int r = i / p.cols, c = i - r * p.cols;
      const float v = stage[(tall ? c : r) * (L + 1) + (tall ? r : c)];
      const long long at = base + i;
      if (!weights) {
        if (p.out_type == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(p.out[ti])[at] = __float2bfloat16_rn(v);
        else static_cast<float*>(p.out[ti])[at] = v;
      } else {
        const float nw = fmaf(-rate, fmaf(p.decay[ti], w[j], rms * v), w[j]);
        weights[at] = nw;
        if (p.w16[ti]) reinterpret_cast<__nv_bfloat16*>(p.w16[ti])[at] = __float2bfloat16_rn(nw);
      }
    }
  }
}

// ------------------------------------------------------------------------ host

struct NsShape {
  int s, l;                    // padded sides, s <= l
  size_t x, a;                 // bytes of X (one part) and of A, a matrix
};
static NsShape ns_shape(int rows, int cols) {
  NsShape o;
  o.s = (std::min(rows, cols) + 127) / 128 * 128;
  o.l = (std::max(rows, cols) + 127) / 128 * 128;
  o.x = static_cast<size_t>(o.s) * o.l * 2;
  o.a = static_cast<size_t>(o.s) * o.s * 2;
  return o;
}
// X twice (a step reads one and writes the other), its second part, A, B, the partial sums; split: the second parts of
// both X, of A and of B
static size_t ns_matrix_bytes(const NsShape& o, bool split) {
  return (split ? 4 * o.x + 4 * o.a : 3 * o.x + 2 * o.a) + 2 * NS_PARTS * sizeof(float);
}

// A matrix in the workspace and its second part, as operands (K-major, MN-major) and in 32 x 32 boxes.
struct NsMaps {
  CUtensorMap k[2], n[2], box[2];
};
static bool ns_maps(NsMaps& m, const void* hi, const void* lo, uint64_t cols, uint64_t rows) {
  for (int i = 0; i < 2; ++i) {
    const void* at = i == 0 ? hi : lo;
    if (!make_tensor_map_bf16(&m.k[i], at, cols, rows, 64, 128) || !make_tensor_map_bf16(&m.n[i], at, cols, rows, 64, 64) ||
        !make_tensor_map_store(&m.box[i], at, cols, cols, rows))
      return false;
  }
  return true;
}

template <int KIND, bool SPLIT>
static cudaError_t launch_ns(const CUtensorMap (&a)[2], const CUtensorMap (&b)[2], const NsMaps& in, const NsMaps& out, const NsParams& p,
                             cudaStream_t s) {
  auto kern = ns_gemm_kernel<KIND, SPLIT>;
  const cudaError_t err = allow_smem<ns_gemm_kernel<KIND, SPLIT>>(NS_SMEM);
  if (err != cudaSuccess) return err;
  static const int most = pair_grid(reinterpret_cast<const void*>(kern), NS_THREADS, NS_SMEM);
  const int mt = (p.s + 255) / 256;
  const long long tiles = static_cast<long long>(p.batch) * (KIND == NS_APPLY ? mt * ((p.n + 255) / 256) : mt * (mt + 1) / 2);
  const int grid = static_cast<int>(2 * tiles < most ? 2 * tiles : most);
  return launch_early(kern, dim3(grid), dim3(NS_THREADS), NS_SMEM, s, a[0], b[0], a[1], b[1], in.box[0], in.box[1], out.box[0], out.box[1], p);
}
template <int L, bool SPLIT>
static cudaError_t launch_small(const NsTensors& t, int batch, const NsSteps& steps, float scale, float floor, float lr, float rms,
                                int32_t* status, cudaStream_t st) {
  const cudaError_t err = allow_smem<ns_small_kernel<L, SPLIT>>(small_smem(L, SPLIT));
  if (err != cudaSuccess) return err;
  return launch_early(ns_small_kernel<L, SPLIT>, dim3(batch), dim3(256), small_smem(L, SPLIT), st, t, steps, scale, floor, lr, rms, status);
}

// What X is multiplied by in an update.
static float ns_rms(const moe_muon_hyper& h, int rows, int cols) {
  return static_cast<float>(h.rms * std::sqrt(static_cast<double>(std::max(rows, cols))));
}

// `batch` matrices of one shape: products, update.
template <bool SPLIT>
static cudaError_t ns_chunk(NsTensors& t, int batch, const moe_muon_hyper& h, float floor, float lr, void* workspace, int32_t* status,
                            cudaStream_t st) {
  const NsShape o = ns_shape(t.rows, t.cols);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  const auto take = [&](size_t bytes) {
    uint8_t* at = w;
    w += batch * bytes;
    return at;
  };
  // X's second part is an operand where it is split, so that a step may not write over it; A and B have none otherwise
  uint8_t* const x[2] = {take(o.x), take(o.x)};
  uint8_t* const lo0 = take(o.x);
  uint8_t* const lo[2] = {lo0, SPLIT ? take(o.x) : lo0};
  uint8_t* const A = take(o.a);
  uint8_t* const B = take(o.a);
  uint8_t* const A_lo = SPLIT ? take(o.a) : A;
  uint8_t* const B_lo = SPLIT ? take(o.a) : B;
  float* parts = reinterpret_cast<float*>(w);
  const long long n = static_cast<long long>(t.rows) * t.cols;
  const int nparts = static_cast<int>(std::min<long long>(NS_PARTS, (n + 2047) / 2048));
  float scale = 1.0f;
  while (scale * scale * 4.0f <= o.l) scale *= 2.0f;
  const bool tall = t.rows > t.cols;
  const NsSteps steps = ns_steps(h);
  const float rms = ns_rms(h, t.rows, t.cols);
  if (o.s == 128 && o.l <= 256)
    return o.l == 128 ? launch_small<128, SPLIT>(t, batch, steps, scale, floor, lr, rms, status, st)
                      : launch_small<256, SPLIT>(t, batch, steps, scale, floor, lr, rms, status, st);
  t.vec = 1;
  for (int i = 0; i < t.count; ++i)
    for (const void* q : {t.grad[i], static_cast<const void*>(t.m[i]), static_cast<const void*>(t.w[i]), static_cast<const void*>(t.w16[i]),
                          static_cast<const void*>(t.out[i])})
      t.vec = t.vec && ptr_aligned16(q);
  cudaError_t err = launch_early(ns_momentum_kernel, dim3(nparts, batch), dim3(256), 0, st, t, parts);
  if (err != cudaSuccess) return err;
  const dim3 tiles_x(o.l / 64, o.s / 64, batch), tiles_t((t.cols + 63) / 64, (t.rows + 63) / 64, batch);
  const auto load = tall ? ns_load_kernel<true> : ns_load_kernel<false>;
  err = launch_early(load, tiles_x, dim3(256), 0, st, t, parts, nparts, o.s, o.l, scale, floor, reinterpret_cast<__half*>(x[0]),
                     reinterpret_cast<__half*>(lo[0]));
  if (err != cudaSuccess) return err;
  const uint64_t rows = static_cast<uint64_t>(batch) * o.s;
  NsMaps mx[2], ma, mb;
  if (!ns_maps(mx[0], x[0], lo[0], o.l, rows) || !ns_maps(mx[1], x[1], lo[1], o.l, rows) || !ns_maps(ma, A, A_lo, o.s, rows) ||
      !ns_maps(mb, B, B_lo, o.s, rows))
    return cudaErrorInvalidValue;
  int cur = 0;
  for (int k = 0; k < h.steps; ++k, cur ^= 1) {
    const NsStep& q = steps.s[k];
    NsParams p{batch, o.s, o.s, o.l, 1.0f / (scale * scale), 0.0f, -q.u, 0, status};
    err = launch_ns<NS_GRAM, SPLIT>(mx[cur].k, mx[cur].k, ma, ma, p, st);
    if (err != cudaSuccess) return err;
    p.k = o.s; p.alpha = q.c; p.beta = q.b; p.diag = q.d;
    err = launch_ns<NS_POLY, SPLIT>(ma.k, ma.k, ma, mb, p, st);
    if (err != cudaSuccess) return err;
    p.n = o.l; p.alpha = 1.0f; p.beta = q.a;
    p.lo_out = SPLIT || k + 1 < h.steps;
    err = launch_ns<NS_APPLY, SPLIT>(mb.k, mx[cur].n, mx[cur], mx[cur ^ 1], p, st);
    if (err != cudaSuccess) return err;
  }
  const auto update = tall ? ns_update_kernel<true> : ns_update_kernel<false>;
  return launch_early(update, tiles_t, dim3(256), 0, st, t, reinterpret_cast<const __half*>(x[cur]),
                      SPLIT ? reinterpret_cast<const __half*>(lo[cur]) : nullptr, o.s, o.l, 1.0f / scale, lr, rms);
}

}  // namespace moe

using namespace moe;

extern "C" {

static moe_status muon_check(const moe_muon_tensor* ts, int32_t count) {
  if (count < 0 || (count > 0 && !ts)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const moe_muon_tensor& t = ts[i];
    if (t.batch < 0 || t.rows <= 0 || t.cols <= 0) return MOE_ERR_INVALID_ARG;
    if (t.rows > 65536 || t.cols > 65536 || static_cast<int64_t>(t.batch) * ns_shape(t.rows, t.cols).s >= (1ll << 30)) return MOE_ERR_UNSUPPORTED;
    if (t.grad_type != MOE_TYPE_BF16 && t.grad_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (t.out_type != MOE_TYPE_BF16 && t.out_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

size_t moe_muon_workspace_size(const moe_muon_tensor* tensors, int32_t count, size_t limit) {
  return moe_muon_workspace_size_with(tensors, count, limit, MOE_MUON_FP16);
}

size_t moe_muon_workspace_size_with(const moe_muon_tensor* tensors, int32_t count, size_t limit, int32_t products) {
  if (muon_check(tensors, count) != MOE_OK || (products != MOE_MUON_FP16 && products != MOE_MUON_FP32)) return 0;
  size_t most = 0;
  for (int i = 0; i < count; ++i) {
    // tensors of one shape run together
    size_t batch = 0;
    for (int j = 0; j < count; ++j)
      if (tensors[j].rows == tensors[i].rows && tensors[j].cols == tensors[i].cols) batch += tensors[j].batch;
    const size_t one = ns_matrix_bytes(ns_shape(tensors[i].rows, tensors[i].cols), products == MOE_MUON_FP32);
    most = std::max(most, one * std::min(batch, std::max<size_t>(1, limit / one)));
  }
  return most;
}

moe_status moe_muon_step(const moe_muon_hyper* hyper, const moe_muon_tensor* tensors, int32_t count, void* workspace,
                         size_t workspace_bytes, const moe_adamw_control* control, int32_t* dev_status, void* stream) {
  return moe_muon_step_with(hyper, tensors, count, 0.0, MOE_MUON_FP16, workspace, workspace_bytes, control, dev_status, stream);
}

moe_status moe_muon_step_with(const moe_muon_hyper* hyper, const moe_muon_tensor* tensors, int32_t count, double norm_floor,
                              int32_t products, void* workspace, size_t workspace_bytes, const moe_adamw_control* control,
                              int32_t* dev_status, void* stream) {
  if (!hyper || !dev_status) return MOE_ERR_INVALID_ARG;
  const moe_muon_hyper& h = *hyper;
  const float lr = static_cast<float>(h.lr), floor = static_cast<float>(norm_floor);
  if (!(floor >= 0.0f) || !std::isfinite(floor) || (products != MOE_MUON_FP16 && products != MOE_MUON_FP32)) return MOE_ERR_INVALID_ARG;
  const bool split = products == MOE_MUON_FP32;
  if (!(lr >= 0.0f) || !std::isfinite(lr) || !(h.momentum >= 0.0 && static_cast<float>(h.momentum) < 1.0f) || !(h.rms >= 0.0) ||
      !std::isfinite(h.rms) || h.steps < 1 || h.steps > MOE_MUON_MAX_STEPS)
    return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * h.steps; ++i)
    if (!std::isfinite(h.coefficients[i])) return MOE_ERR_INVALID_ARG;
  moe_status stc = muon_check(tensors, count);
  if (stc != MOE_OK) return stc;
  size_t need = 0;
  for (int i = 0; i < count; ++i) {
    const moe_muon_tensor& t = tensors[i];
    if (t.batch == 0) continue;
    if (!t.grad || (!t.out == !t.w) || (!t.w != !t.m) || (t.w16 && !t.w)) return MOE_ERR_INVALID_ARG;
    if (t.w && (!std::isfinite(t.weight_decay) || !std::isfinite(ns_rms(h, t.rows, t.cols)))) return MOE_ERR_INVALID_ARG;
    need = std::max(need, ns_matrix_bytes(ns_shape(t.rows, t.cols), split));
  }
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (!ptr_aligned16(workspace)) return MOE_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto alike = [&](int i, int j) {
    const moe_muon_tensor &f = tensors[i], &g = tensors[j];
    return g.batch > 0 && g.rows == f.rows && g.cols == f.cols && g.grad_type == f.grad_type && g.out_type == f.out_type && !g.out == !f.out;
  };
  for (int i = 0; i < count; ++i) {
    bool done = tensors[i].batch == 0;
    for (int j = 0; j < i && !done; ++j) done = alike(i, j);
    if (done) continue;
    // the tensors like this one, in order, in chunks that fit the workspace
    const moe_muon_tensor& f = tensors[i];
    const int fit = static_cast<int>(std::min<size_t>(workspace_bytes / ns_matrix_bytes(ns_shape(f.rows, f.cols), split), 65535));
    NsTensors t{};
    t.rows = f.rows; t.cols = f.cols; t.grad_type = f.grad_type; t.out_type = f.out_type;
    t.momentum = static_cast<float>(h.momentum); t.nesterov = h.nesterov != 0; t.control = control;
    int batch = 0;
    auto flush = [&]() -> cudaError_t {
      if (batch == 0) return cudaSuccess;
      t.first[t.count] = batch;
      const cudaError_t e = split ? ns_chunk<true>(t, batch, h, floor, lr, workspace, dev_status, s)
                                  : ns_chunk<false>(t, batch, h, floor, lr, workspace, dev_status, s);
      t.count = 0; t.skip0 = 0; batch = 0;
      return e;
    };
    for (int j = i; j < count; ++j) {
      const moe_muon_tensor& g = tensors[j];
      if (!alike(i, j)) continue;
      for (int at = 0; at < g.batch;) {
        if (batch == fit || t.count == NS_TENSORS) {
          if (flush() != cudaSuccess) return MOE_ERR_CUDA;
        }
        const int take = std::min(g.batch - at, fit - batch), k = t.count++;
        t.grad[k] = g.grad; t.m[k] = g.m; t.w[k] = g.w; t.w16[k] = g.w16; t.out[k] = g.out; t.decay[k] = g.weight_decay;
        t.first[k] = batch;
        if (k == 0) t.skip0 = at;
        batch += take;
        at += take;
      }
    }
    if (flush() != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
