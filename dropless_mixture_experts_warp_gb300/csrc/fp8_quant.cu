// The quantiser of the 8-bit products with blocks of 128: bf16 rows to E4M3 codes with fp32
// scales, blocks along rows, down columns (codes transposed, the operand of weight gradients)
// or square (weights); and the SwiGLU between the experts' two products, quantised as it is
// computed.  The row forms and the weights are bound by memory (SwiGLU of 131072 rows of 768: 93 us,
// 5.4 TB/s; 128 x 1536 x 2048 weights both ways: 291 us, 5.5 TB/s); the column forms fill neither memory nor
// the issue slots: a tile's steps follow one another.
#include "fp8.cuh"
#include "kernels.h"

namespace moe {

// Rows that a call works on: *nrows_dev of them, where it is given; none where that is negative.
__device__ __forceinline__ int rows_in_use(int rows, const int32_t* nrows_dev) {
  return nrows_dev ? max(0, min(rows, *nrows_dev)) : rows;
}

// ------------------------------------------------------------------------ rows

constexpr int QR_ROWS = 4;   // rows under way in a warp

// Eight values of 16 lanes (one block of 128): scale, codes.
__device__ __forceinline__ uint2 f8_block16(const f32x2 (&v)[4], float amax, float& scale) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const F8Scale f = f8_scale(amax);
  scale = f.s;
  const f32x2 ns = pair(-f.s, -f.s), inv = pair(f.inv, f.inv);
  return make_uint2(f8_codes4(v[0], v[1], ns, inv), f8_codes4(v[2], v[3], ns, inv));
}

// A warp takes QR_ROWS rows x 256 columns: 16 lanes of 16 bytes a block, every row's load
// issued before the first is used.  row_map: row r reads src row row_map[r], zeros where that
// is negative.
__global__ void __launch_bounds__(256) f8_rows_kernel(const uint16_t* src, int rows, int C,
                                                      const int32_t* row_map,
                                                      const int32_t* nrows_dev, uint8_t* codes,
                                                      float* scales) {
  wait_for_previous();
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int limit = rows_in_use(rows, nrows_dev);
  const int groups = (C + 255) / 256;
  const long long total = static_cast<long long>((limit + QR_ROWS - 1) / QR_ROWS) * groups;
  for (long long t = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < total; t += gridDim.x * 8ll) {
    const int r0 = static_cast<int>(t / groups) * QR_ROWS;
    const int col = static_cast<int>(t % groups) * 256 + lane * 8;
    const bool in = col < C;
    uint4 w[QR_ROWS];
#pragma unroll
    for (int i = 0; i < QR_ROWS; ++i) {
      const int r = r0 + i;
      const int from = r >= limit ? -1 : (row_map ? row_map[r] : r);
      w[i] = in && from >= 0 ? *reinterpret_cast<const uint4*>(src + static_cast<long long>(from) * C + col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < QR_ROWS; ++i) {
      const uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, w[i].x), w[i].y), w[i].z), w[i].w);
      const f32x2 v[4] = {bf16_pair(w[i].x), bf16_pair(w[i].y), bf16_pair(w[i].z), bf16_pair(w[i].w)};
      float s;
      const uint2 c = f8_block16(v, max_halves(m), s);
      if (in && r0 + i < limit) {
        *reinterpret_cast<uint2*>(codes + static_cast<long long>(r0 + i) * C + col) = c;
        if ((lane & 15) == 0) scales[static_cast<long long>(col >> 7) * rows + r0 + i] = s;
      }
    }
  }
}

// Each token's row quantised once, its codes written to the k rows that the routing gave it: a
// warp takes 256 columns of a token.  Rows without a token are left as they were.
__global__ void __launch_bounds__(256) f8_scatter_kernel(const uint16_t* x, int T, int C, int k, const int32_t* token_to_row, int rows,
                                                         uint8_t* codes, float* scales) {
  wait_for_previous();
  launch_dependents();
  const int lane = threadIdx.x & 31, groups = (C + 255) / 256;
  const long long total = static_cast<long long>(T) * groups;
  for (long long t = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < total; t += gridDim.x * 8ll) {
    const int tok = static_cast<int>(t / groups), col = static_cast<int>(t - static_cast<long long>(tok) * groups) * 256 + lane * 8;
    const bool in = col < C;
    const int mine = lane < k ? token_to_row[static_cast<long long>(tok) * k + lane] : -1;
    const uint4 w = in ? *reinterpret_cast<const uint4*>(x + static_cast<long long>(tok) * C + col) : make_uint4(0, 0, 0, 0);
    const uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, w.x), w.y), w.z), w.w);
    const f32x2 v[4] = {bf16_pair(w.x), bf16_pair(w.y), bf16_pair(w.z), bf16_pair(w.w)};
    float s;
    const uint2 c = f8_block16(v, max_halves(m), s);
    for (int j = 0; j < k; ++j) {
      const int r = __shfl_sync(0xffffffffu, mine, j);
      if (in && r >= 0 && r < rows) {
        *reinterpret_cast<uint2*>(codes + static_cast<long long>(r) * C + col) = c;
        if ((lane & 15) == 0) scales[static_cast<long long>(col >> 7) * rows + r] = s;
      }
    }
  }
}

// ------------------------------------------------------------------------ tiles

constexpr int QT_IN_LD = 128 + 8;     // padded bf16 input rows
constexpr int QT_LD = 128 + 16;       // padded code rows (bytes)
constexpr int QT_IN_BYTES = 128 * QT_IN_LD * 2;
constexpr int QT_SMEM = QT_IN_BYTES + 2 * 128 * QT_LD + (4 * 128 + 2 * 128 + 8) * 4;

// What a tile kernel writes.  Rows: codes [batch][R][C] and scales; columns: codes_t
// [batch][C][R_t] (R_t >= R: rows from R on are zeros) and scales_t.  Either may be NULL.
struct F8Tiles {
  const uint16_t* src;         // [batch][R][C]
  const int32_t* row_map;      // batch 1
  const int32_t* nrows_dev;    // batch 1: 128-row tiles from *nrows_dev on are left out
  int batch, R, C, R_t;
  uint8_t* codes;
  float* scales;               // [ceil(C / 128)][R]; SQUARE: [batch][ceil(R / 128)][ceil(C / 128)]
  uint8_t* codes_t;
  float* scales_t;             // [ceil(R / 128)][C]; SQUARE: not used
};

// 128 x 128 tiles, three persistent blocks an SM; a tile's rows are asked for (cp.async) as soon as the codes of the
// one before have left its buffer.  A thread takes 32 rows of two columns and 64 columns of one row,
// first for the maxima, then for the codes, which are assembled in shared memory and leave as whole lines.  16384 x 7168,
// both forms: 94 us, 5.06 TB/s (75 % of a copy) and 60 % of the issue slots; three blocks an SM cover each other's barriers and
// loads, but not all of them.  SQUARE: one scale a tile.
template <bool SQUARE>
__global__ void __launch_bounds__(256, 3) f8_tiles_kernel(const F8Tiles p) {
  extern __shared__ __align__(16) uint8_t sm[];
  uint8_t* ct = sm + QT_IN_BYTES;              // column codes [128 columns][QT_LD]
  uint8_t* rt = ct + 128 * QT_LD;                  // row codes [128 rows][QT_LD]
  float* cmax = reinterpret_cast<float*>(rt + 128 * QT_LD);   // [4][128]
  float* rmax = cmax + 4 * 128;                    // [2][128]
  float* tmax = rmax + 2 * 128;                    // [8]
  const int tid = threadIdx.x;
  wait_for_previous();
  launch_dependents();
  const int limit = rows_in_use(p.R, p.nrows_dev);
  const unsigned ctiles = (p.C + 127) / 128, rtiles = (limit + 127) / 128;
  const unsigned total = p.batch * rtiles * ctiles;

  auto rows_of = [&](unsigned t, int (&sr)[8]) {
    const unsigned rti = t < total ? (t / ctiles) % rtiles : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = static_cast<int>(rti) * 128 + (tid >> 4) + 16 * j;
      sr[j] = (t >= total || r >= limit) ? -1 : (p.row_map ? p.row_map[r] : r);
    }
  };
  auto fetch = [&](unsigned t, const int (&sr)[8]) {
    if (t < total) {
      const unsigned q = t / ctiles;
      const int col = static_cast<int>(t - q * ctiles) * 128 + (tid & 15) * 8;
      const uint16_t* s = p.src + static_cast<long long>(q / rtiles) * p.R * p.C;
      uint8_t* dst = sm + (tid >> 4) * QT_IN_LD * 2 + (tid & 15) * 16;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool ok = sr[j] >= 0 && col < p.C;
        const uint16_t* from = s + (ok ? static_cast<long long>(sr[j]) * p.C + col : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + 16 * j * QT_IN_LD * 2)), "l"(from),
                     "r"(ok ? 16 : 0)
                     : "memory");
      }
    }
    copy_commit();
  };

  unsigned t = blockIdx.x;
  int next[8];
  rows_of(t, next);
  fetch(t, next);
  rows_of(t + gridDim.x, next);
  for (; t < total; t += gridDim.x) {
    copy_wait<0>();
    __syncthreads();
    const uint16_t(*tile)[QT_IN_LD] = reinterpret_cast<const uint16_t(*)[QT_IN_LD]>(sm);
    const unsigned qq = t / ctiles;
    const int c0 = static_cast<int>(t - qq * ctiles) * 128, r0 = static_cast<int>(qq % rtiles) * 128;
    const long long b = qq / rtiles;
    // columns 2 cp and 2 cp + 1, rows 32 g to 32 g + 31; row rr, columns 64 hh to 64 hh + 63
    const int cp = tid & 63, g = tid >> 6, rr = tid & 127, hh = tid >> 7;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      m = absmax_bf16x2(m, *reinterpret_cast<const uint32_t*>(&tile[g * 32 + i][2 * cp]));
    }
    float amax = max_halves(m);
    if (!SQUARE) {
      cmax[g * 128 + 2 * cp] = fabsf(bf16_lo(m));
      cmax[g * 128 + 2 * cp + 1] = fabsf(bf16_hi(m));
    }
    if (SQUARE) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      if ((tid & 31) == 0) tmax[tid >> 5] = amax;
    } else {
      m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(&tile[rr][hh * 64 + 8 * i]);
        m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, u.x), u.y), u.z), u.w);
      }
      rmax[hh * 128 + rr] = max_halves(m);
    }
    __syncthreads();
    {
      // one column's (the first 128 threads) or row's scale a thread, - scale and 1 / scale over two of the maxima that
      // only this thread reads
      float top;
      if (SQUARE) {
        top = tmax[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, tmax[i]);
      } else if (tid < 128) {
        top = fmaxf(fmaxf(cmax[tid], cmax[128 + tid]), fmaxf(cmax[256 + tid], cmax[384 + tid]));
      } else {
        top = fmaxf(rmax[tid - 128], rmax[tid]);
      }
      const F8Scale f = f8_scale(top);
      float* ends = tid < 128 ? cmax + tid : rmax + tid - 128;
      ends[0] = -f.s;
      ends[128] = f.inv;
      if (SQUARE) {
        if (tid == 0) p.scales[(b * rtiles + (r0 >> 7)) * ctiles + (c0 >> 7)] = f.s;
      } else if (tid < 128) {
        if (p.codes_t && c0 + tid < p.C) p.scales_t[static_cast<long long>(r0 >> 7) * p.C + c0 + tid] = f.s;
      } else {
        if (p.codes && r0 + tid - 128 < p.R) p.scales[static_cast<long long>(c0 >> 7) * p.R + r0 + tid - 128] = f.s;
      }
    }
    __syncthreads();
    if (p.codes_t) {
      const f32x2 ns = *reinterpret_cast<const f32x2*>(cmax + 2 * cp), inv = *reinterpret_cast<const f32x2*>(cmax + 128 + 2 * cp);
      uint32_t k0[8], k1[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = unpair(f8_quotient(bf16_pair(*reinterpret_cast<const uint32_t*>(&tile[g * 32 + 4 * i + j][2 * cp])), ns, inv));
        k0[i] = cvt_e4m3x4(x[0].x, x[1].x, x[2].x, x[3].x);
        k1[i] = cvt_e4m3x4(x[0].y, x[1].y, x[2].y, x[3].y);
      }
      // line cp holds column 2 cp, line 64 + cp column 2 cp + 1
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint4*>(ct + cp * QT_LD + g * 32 + 16 * i) = make_uint4(k0[4 * i], k0[4 * i + 1], k0[4 * i + 2], k0[4 * i + 3]);
        *reinterpret_cast<uint4*>(ct + (64 + cp) * QT_LD + g * 32 + 16 * i) = make_uint4(k1[4 * i], k1[4 * i + 1], k1[4 * i + 2], k1[4 * i + 3]);
      }
    }
    if (p.codes) {
      const f32x2 ns = pair(rmax[rr], rmax[rr]), inv = pair(rmax[128 + rr], rmax[128 + rr]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t k[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 u = *reinterpret_cast<const uint4*>(&tile[rr][hh * 64 + 16 * i + 8 * j]);
          k[2 * j] = f8_codes4(bf16_pair(u.x), bf16_pair(u.y), ns, inv);
          k[2 * j + 1] = f8_codes4(bf16_pair(u.z), bf16_pair(u.w), ns, inv);
        }
        *reinterpret_cast<uint4*>(rt + rr * QT_LD + hh * 64 + 16 * i) = make_uint4(k[0], k[1], k[2], k[3]);
      }
    }
    __syncthreads();
    fetch(t + gridDim.x, next);
    rows_of(t + 2 * gridDim.x, next);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int line = (tid + 256 * j) >> 3, at = (tid & 7) * 16;
      if (p.codes_t) {
        const int col = c0 + (line < 64 ? 2 * line : 2 * (line - 64) + 1);
        if (col < p.C && r0 + at < p.R_t)
          *reinterpret_cast<uint4*>(p.codes_t + (b * p.C + col) * static_cast<long long>(p.R_t) + r0 + at) =
              *reinterpret_cast<const uint4*>(ct + line * QT_LD + at);
      }
      if (p.codes && r0 + line < p.R && c0 + at < p.C)
        *reinterpret_cast<uint4*>(p.codes + (b * p.R + r0 + line) * static_cast<long long>(p.C) + c0 + at) =
            *reinterpret_cast<const uint4*>(rt + line * QT_LD + at);
    }
  }
}

template <bool SQUARE>
static cudaError_t launch_f8_tiles(const F8Tiles& p, cudaStream_t s) {
  const cudaError_t err = allow_smem<f8_tiles_kernel<SQUARE>>(QT_SMEM);
  if (err != cudaSuccess) return err;
  const long long tiles = static_cast<long long>(p.batch) * ((p.R + 127) / 128) * ((p.C + 127) / 128);
  if (tiles >= (1ll << 31) - (1 << 20)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(tiles < 3ll * num_sms() ? tiles : 3ll * num_sms());
  return launch_early(f8_tiles_kernel<SQUARE>, dim3(grid), dim3(256), QT_SMEM, s, p);
}

// ------------------------------------------------------------------------ SwiGLU

// The sigmoid of a gate: a fast exponential and an approximate reciprocal.  The exponential is off by 2 + 1.2 |g| units
// in the last place: 2^-19 of silu(g) at g = -12, 2^-16 at -88, where half a step of a code is 2^-4.  The forward and the
// gradient compute silu(g) = g sigmoid(g) and h = (w silu(g)) u with these operations in this order, so that both quantise the
// same numbers.
__device__ __forceinline__ float f8_sigmoid(float g) { return rcp_fast(1.0f + __expf(-g)); }

// h = w silu(G) U of gu [rows][2f], a block of 128 columns of h on 16 lanes, quantised.
__global__ void __launch_bounds__(256) f8_swiglu_kernel(const uint16_t* gu, const float* w_rows, int rows,
                                                        int f, const int32_t* nrows_dev,
                                                        uint8_t* codes, float* scales) {
  wait_for_previous();
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int limit = rows_in_use(rows, nrows_dev);
  const int groups = (f + 255) / 256;
  const long long total = static_cast<long long>((limit + 1) / 2) * groups;
  for (long long t = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < total; t += gridDim.x * 8ll) {
    const int r0 = static_cast<int>(t / groups) * 2;
    const int col = static_cast<int>(t % groups) * 256 + lane * 8;
    const bool in = col < f;
    uint4 g[2], u[2];
    float w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = r0 + i >= limit ? 0.0f : (w_rows ? w_rows[r0 + i] : 1.0f);
      const bool ok = in && w[i] != 0.0f;       // padding rows weigh 0
      const uint16_t* at = gu + static_cast<long long>(r0 + i) * 2 * f + col;
      g[i] = ok ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
      u[i] = ok ? *reinterpret_cast<const uint4*>(at + f) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w}, uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      f32x2 v[4];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 gate = bf16_pair(gw[j]), sg = pair(f8_sigmoid(bf16_lo(gw[j])), f8_sigmoid(bf16_hi(gw[j])));
        v[j] = mul2(mul2(pair(w[i], w[i]), mul2(gate, sg)), bf16_pair(uw[j]));
        const float2 x = unpair(v[j]);
        amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
      float s;
      const uint2 c = f8_block16(v, amax, s);
      if (in && r0 + i < limit) {
        *reinterpret_cast<uint2*>(codes + static_cast<long long>(r0 + i) * f + col) = c;
        if ((lane & 15) == 0) scales[static_cast<long long>(col >> 7) * rows + r0 + i] = s;
      }
    }
  }
}

// The gradient of the SwiGLU, quantised both ways, and h again for the down weights' gradient:
//   dA = w dH;  dG = dA U silu'(G);  dU = dA silu(G);  dw = sum silu(G) U dH
// One 128 x 128 tile of h's columns at a time; the next one's operands come (cp.async) while a tile's columns are
// quantised.  A thread holds dG, dU and h of four rows and eight columns in registers, so that nothing is computed
// twice.  A row's block is on 16 lanes, as in the forward; columns take their maxima through shared memory and their
// codes leave through transposing tiles whose four-byte units are permuted so that neither side has bank conflicts.
// 131072 rows of 768: 332 us, 3.3 TB/s.  Bound by latency: the one block of an SM stands still at each of a tile's four
// barriers (issue slots 50 %, DRAM 35 %).  (A pass for each
// of the three, with its sigmoids and the next tile's operands in registers: 653 us.)
struct F8SwigluBwd {
  const uint16_t *gu, *dh;    // [rows][2f], [rows][f]
  const float* w_rows;        // NULL = 1
  const int32_t* nrows_dev;
  int rows, f, R_t;
  uint8_t* dgu;               // [rows][2f]
  float* dgu_s;               // [2f / 128][rows]
  uint8_t* dgu_t;             // [2f][R_t]
  float* dgu_ts;              // [R_t / 128][2f]
  uint8_t* h_t;               // [f][R_t]
  float* h_ts;                // [R_t / 128][f]
  float* dw_part;             // [rows][f / 128], or NULL
};
constexpr int SB_THREADS = 512;
constexpr int SB_IN = 128 * 256;                     // bytes of a tile's G, U or dH
constexpr int SB_SMEM = 3 * SB_IN + 3 * 16 * 128 * 4 + 3 * 128 * 128 + 3 * 128 * 8 + 128 * 4;

__global__ void __launch_bounds__(SB_THREADS, 1) f8_swiglu_bwd_kernel(const F8SwigluBwd p) {
  extern __shared__ __align__(16) uint8_t sm[];      // G, U, dH
  float* const cmax = reinterpret_cast<float*>(sm + 3 * SB_IN);               // [3][16][128] columns' maxima by a warp's eight rows
  uint32_t* const ct = reinterpret_cast<uint32_t*>(cmax + 3 * 16 * 128);      // [3][128][32] codes of the columns
  float2* const cscale = reinterpret_cast<float2*>(ct + 3 * 128 * 32);        // [3][128] -scale, 1 / scale
  float* const ws = reinterpret_cast<float*>(cscale + 3 * 128);               // [128] rows' weights
  wait_for_previous();
  launch_dependents();
  const int tid = threadIdx.x, c = tid & 15, u = tid >> 4;
  const int limit = rows_in_use(p.rows, p.nrows_dev);
  const unsigned ctiles = p.f / 128, total = static_cast<unsigned>((limit + 127) / 128) * ctiles;

  auto fetch = [&](unsigned t) {
    if (t < total) {
      const int r0 = static_cast<int>(t / ctiles) * 128, col = static_cast<int>(t % ctiles) * 128 + 8 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + u + 32 * i;
        const bool ok = r < limit;
        const uint16_t* gu = p.gu + (ok ? 2ll * r * p.f + col : 0);
        const uint16_t* dh = p.dh + (ok ? static_cast<long long>(r) * p.f + col : 0);
        const uint32_t to = smem_u32(sm) + (u + 32 * i) * 256 + c * 16, n = ok ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(gu), "r"(n) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + SB_IN), "l"(gu + p.f), "r"(n) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 2 * SB_IN), "l"(dh), "r"(n) : "memory");
      }
      if (tid < 128) {
        if (p.w_rows) {
          const bool ok = r0 + tid < limit;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(ws + tid)), "l"(p.w_rows + (ok ? r0 + tid : 0)),
                       "r"(ok ? 4 : 0)
                       : "memory");
        } else {
          ws[tid] = 1.0f;
        }
      }
    }
    copy_commit();
  };
  fetch(blockIdx.x);
  for (unsigned t = blockIdx.x; t < total; t += gridDim.x) {
    copy_wait<0>();
    __syncthreads();
    const int r0 = static_cast<int>(t / ctiles) * 128, c0 = static_cast<int>(t % ctiles) * 128;
    f32x2 v[3][4][4];                                // dG, dU, h
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* at = sm + (4 * u + i) * 256 + c * 16;
      const uint4 G = *reinterpret_cast<const uint4*>(at), U = *reinterpret_cast<const uint4*>(at + SB_IN),
                  H = *reinterpret_cast<const uint4*>(at + 2 * SB_IN);
      const uint32_t gw[4] = {G.x, G.y, G.z, G.w}, uw[4] = {U.x, U.y, U.z, U.w}, dw[4] = {H.x, H.y, H.z, H.w};
      const float w = ws[4 * u + i];
      const f32x2 w2 = pair(w, w);
      f32x2 sum2 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 g = bf16_pair(gw[j]), uu = bf16_pair(uw[j]), dh = bf16_pair(dw[j]);
        const f32x2 sg = pair(f8_sigmoid(bf16_lo(gw[j])), f8_sigmoid(bf16_hi(gw[j])));
        const f32x2 silu = mul2(g, sg), a = mul2(w2, dh);
        const f32x2 slope = fma2(silu, fma2(sg, pair(-1.0f, -1.0f), pair(1.0f, 1.0f)), sg);     // sg (1 + g (1 - sg))
        const f32x2 su = mul2(silu, uu);
        v[0][i][j] = mul2(mul2(a, uu), slope);
        v[1][i][j] = mul2(a, silu);
        v[2][i][j] = mul2(mul2(w2, silu), uu);   // as the forward: (w silu) u
        sum2 = fma2(su, dh, sum2);
      }
      if (w == 0.0f) {                               // as the forward, which does not read such a row
#pragma unroll
        for (int j = 0; j < 12; ++j) v[j >> 2][i][j & 3] = 0;
      }
      const int r = r0 + 4 * u + i;
#pragma unroll
      for (int what = 0; what < 2; ++what) {         // the row's own blocks
        float rmax = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpair(v[what][i][j]);
          rmax = fmaxf(rmax, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
        float s;
        const uint2 k = f8_block16(v[what][i], rmax, s);
        const int col = what * p.f + c0 + 8 * c;
        if (r < limit) {
          *reinterpret_cast<uint2*>(p.dgu + 2ll * r * p.f + col) = k;
          if (c == 0) p.dgu_s[static_cast<long long>(col >> 7) * p.rows + r] = s;
        }
      }
      if (p.dw_part) {
        const float2 x = unpair(sum2);
        float sum = x.x + x.y;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (c == 0 && r < limit) p.dw_part[static_cast<long long>(r) * ctiles + (c0 >> 7)] = sum;
      }
    }
#pragma unroll
    for (int what = 0; what < 3; ++what) {
      float m[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpair(v[what][i][j]);
          a = fmaxf(a, fabsf(x.x));
          b = fmaxf(b, fabsf(x.y));
        }
        m[2 * j] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
        m[2 * j + 1] = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 16));
      }
      // each half of the warp writes half of the eight columns
      float* to = cmax + (what * 16 + (u >> 1)) * 128 + 8 * c;
      if (u & 1) *reinterpret_cast<float4*>(to + 4) = make_float4(m[4], m[5], m[6], m[7]);
      else *reinterpret_cast<float4*>(to) = make_float4(m[0], m[1], m[2], m[3]);
    }
    __syncthreads();
    fetch(t + gridDim.x);
    if (tid < 384) {
      const int what = tid >> 7, col = tid & 127;
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) a = fmaxf(a, cmax[(what * 16 + i) * 128 + col]);
      const F8Scale f = f8_scale(a);
      cscale[tid] = make_float2(-f.s, f.inv);
      const int width = what < 2 ? 2 * p.f : p.f, out_c = (what == 1 ? p.f : 0) + c0;
      (what < 2 ? p.dgu_ts : p.h_ts)[static_cast<long long>(r0 >> 7) * width + out_c + col] = f.s;
    }
    __syncthreads();
#pragma unroll
    for (int what = 0; what < 3; ++what) {
      uint32_t* to = ct + what * 128 * 32 + 8 * c * 32 + (u ^ (2 * c));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 s = *reinterpret_cast<const float4*>(cscale + what * 128 + 8 * c + 2 * j);
        const f32x2 ns = pair(s.x, s.z), inv = pair(s.y, s.w);
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = unpair(f8_quotient(v[what][i][j], ns, inv));
        to[2 * j * 32] = cvt_e4m3x4(x[0].x, x[1].x, x[2].x, x[3].x);
        to[(2 * j + 1) * 32] = cvt_e4m3x4(x[0].y, x[1].y, x[2].y, x[3].y);
      }
    }
    __syncthreads();
#pragma unroll
    for (int what = 0; what < 3; ++what) {
      uint8_t* const out_t = what < 2 ? p.dgu_t : p.h_t;
      const int out_c = (what == 1 ? p.f : 0) + c0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = tid + SB_THREADS * j, line = i >> 3, q = i & 7, cc = line >> 3;
        uint4 k = *reinterpret_cast<const uint4*>(ct + what * 128 * 32 + line * 32 + 4 * (q ^ (cc >> 1)));
        if (cc & 1) k = make_uint4(k.z, k.w, k.x, k.y);
        *reinterpret_cast<uint4*>(out_t + static_cast<long long>(out_c + line) * p.R_t + r0 + 16 * q) = k;
      }
    }
  }
}

// dw [r] = its parts' sum, in order.
__global__ void f8_dw_kernel(const float* part, int parts, int rows, const int32_t* nrows_dev,
                             float* dw) {
  wait_for_previous();
  launch_dependents();
  const int limit = rows_in_use(rows, nrows_dev);
  for (int r = blockIdx.x * blockDim.x + threadIdx.x; r < limit; r += gridDim.x * blockDim.x) {
    float s = 0.0f;
    for (int i = 0; i < parts; ++i) s += part[static_cast<long long>(r) * parts + i];
    dw[r] = s;
  }
}

static int f8_row_grid(long long warps) {
  const long long blocks = (warps + 7) / 8, most = 8ll * num_sms();
  return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_fp8_quantize(const moe_bf16* src, int64_t rows, int32_t C, const int32_t* row_map, const int32_t* nrows_dev,
                            uint8_t* codes, float* scales, uint8_t* codes_t, float* scales_t, void* stream) {
  if (rows < 0 || C <= 0 || (rows > 0 && !src)) return MOE_ERR_INVALID_ARG;
  if (!codes != !scales || !codes_t != !scales_t || (rows > 0 && !codes && !codes_t)) return MOE_ERR_INVALID_ARG;
  if (C % 16 != 0 || rows > (1ll << 31) - 256) return MOE_ERR_UNSUPPORTED;
  if (!f8_aligned(src) || !f8_aligned(codes) || !f8_aligned(codes_t)) return MOE_ERR_ALIGNMENT;
  if (rows == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!codes_t) {
    const long long warps = (rows + QR_ROWS - 1) / QR_ROWS * ((C + 255) / 256);
    return status_of(launch_early(f8_rows_kernel, dim3(f8_row_grid(warps)), dim3(256), 0, s, src, static_cast<int>(rows), C, row_map,
                                  nrows_dev, codes, scales));
  }
  const F8Tiles p{src, row_map, nrows_dev, 1, static_cast<int>(rows), C, static_cast<int>(up128(rows)), codes, scales, codes_t, scales_t};
  return status_of(launch_f8_tiles<false>(p, s));
}

moe_status moe_fp8_quantize_weights(const moe_bf16* src, int32_t E, int32_t N, int32_t K, uint8_t* codes, uint8_t* codes_t,
                                    float* scales, void* stream) {
  if (E <= 0 || N <= 0 || K <= 0 || !src || !scales || (!codes && !codes_t)) return MOE_ERR_INVALID_ARG;
  if (N % 16 != 0 || K % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (!f8_aligned(src) || !f8_aligned(codes) || !f8_aligned(codes_t)) return MOE_ERR_ALIGNMENT;
  const F8Tiles p{src, nullptr, nullptr, E, N, K, N, codes, scales, codes_t, nullptr};
  return status_of(launch_f8_tiles<true>(p, static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_swiglu(const moe_bf16* gu, const float* w_rows, int64_t rows, int32_t f, const int32_t* nrows_dev, uint8_t* codes,
                          float* scales, void* stream) {
  if (rows < 0 || f <= 0 || (rows > 0 && (!gu || !codes || !scales))) return MOE_ERR_INVALID_ARG;
  if (f % 16 != 0 || rows > (1ll << 31) - 256) return MOE_ERR_UNSUPPORTED;
  if (!f8_aligned(gu) || !f8_aligned(codes)) return MOE_ERR_ALIGNMENT;
  if (rows == 0) return MOE_OK;
  const long long warps = (rows + 1) / 2 * ((f + 255) / 256);
  return status_of(launch_early(f8_swiglu_kernel, dim3(f8_row_grid(warps)), dim3(256), 0, static_cast<cudaStream_t>(stream), gu, w_rows,
                                static_cast<int>(rows), f, nrows_dev, codes, scales));
}

moe_status moe_fp8_swiglu_bwd(const moe_bf16* gu, const moe_bf16* dh, const float* w_rows, int64_t rows, int32_t f,
                              const int32_t* nrows_dev, uint8_t* dgu_codes, float* dgu_scales, uint8_t* dgu_codes_t,
                              float* dgu_scales_t, uint8_t* h_codes_t, float* h_scales_t, float* dw_rows, float* dw_part,
                              void* stream) {
  if (rows < 0 || f <= 0 || !dw_rows != !dw_part) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!gu || !dh || !dgu_codes || !dgu_scales || !dgu_codes_t || !dgu_scales_t || !h_codes_t || !h_scales_t))
    return MOE_ERR_INVALID_ARG;
  if (f % 128 != 0 || rows > (1ll << 31) - 256 || up128(rows) / 128 * (f / 128) >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  if (!f8_aligned(gu) || !f8_aligned(dh) || !f8_aligned(dgu_codes) || !f8_aligned(dgu_codes_t) || !f8_aligned(h_codes_t))
    return MOE_ERR_ALIGNMENT;
  if (rows == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const F8SwigluBwd p{gu, dh, w_rows, nrows_dev, static_cast<int>(rows), f, static_cast<int>(up128(rows)), dgu_codes, dgu_scales,
                      dgu_codes_t, dgu_scales_t, h_codes_t, h_scales_t, dw_part};
  const long long tiles = up128(rows) / 128 * (f / 128);
  const int grid = static_cast<int>(tiles < num_sms() ? tiles : num_sms());
  if (allow_smem<f8_swiglu_bwd_kernel>(SB_SMEM) != cudaSuccess ||
      launch_early(f8_swiglu_bwd_kernel, dim3(grid), dim3(SB_THREADS), SB_SMEM, s, p) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (!dw_rows) return MOE_OK;
  const long long blocks = (rows + 255) / 256;
  return status_of(launch_early(f8_dw_kernel, dim3(static_cast<int>(blocks < 4 * num_sms() ? blocks : 4 * num_sms())), dim3(256), 0, s,
                                dw_part, f / 128, static_cast<int>(rows), nrows_dev, dw_rows));
}

moe_status moe_permute_fp8(const moe_dims* dims, const moe_bf16* x, const int32_t* topk_idx, const float* topk_w,
                           const int32_t* split_sizes, const int32_t* row_offsets, const void* workspace, uint8_t* codes,
                           float* scales, uint8_t* codes_t, float* scales_t, int32_t* row_to_token, int32_t* token_to_row,
                           float* w_rows, int32_t* dev_status, void* stream) {
  const moe_status st = moe_check_dims(dims);
  if (st != MOE_OK) return st;
  const moe_dims& d = *dims;
  if (!split_sizes || !row_offsets || !codes || !scales || !row_to_token || !w_rows || !dev_status) return MOE_ERR_INVALID_ARG;
  if (!codes_t != !scales_t || (d.T > 0 && (!x || !topk_idx || !topk_w || !token_to_row))) return MOE_ERR_INVALID_ARG;
  if (!workspace) return MOE_ERR_WORKSPACE;
  if (!f8_aligned(x) || !f8_aligned(codes) || !f8_aligned(codes_t)) return MOE_ERR_ALIGNMENT;
  const int64_t rows = moe_row_capacity(dims);
  const RouteScratch rs = route_scratch(d, const_cast<void*>(workspace));
  if (launch_route_maps(d.T, d.E, d.k, topk_idx, topk_w, split_sizes, row_offsets, rs, row_to_token, token_to_row, w_rows,
                        static_cast<int>(rows), dev_status, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (d.T == 0) return MOE_OK;
  if (!codes_t) {
    const long long warps = static_cast<long long>(d.T) * ((d.d + 255) / 256);
    return status_of(launch_early(f8_scatter_kernel, dim3(f8_row_grid(warps)), dim3(256), 0, static_cast<cudaStream_t>(stream), x, d.T, d.d,
                                  d.k, token_to_row, static_cast<int>(rows), codes, scales));
  }
  return moe_fp8_quantize(x, rows, d.d, row_to_token, row_offsets + d.E, codes, scales, codes_t, scales_t, stream);
}

}  // extern "C"
