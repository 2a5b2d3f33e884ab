// Block norms: the norm before a block, the merge after it (norm of its output, gate,
// scaled residual, the next block's norm) and their gradients.  Every kernel reads each
// row of its inputs once, keeps it in registers between the sums over the row and the
// outputs, and does its arithmetic in fp32; all are bound by HBM bandwidth.
#include "around.cuh"

namespace moe {

constexpr int NORM_MAX_D = 16384;
// Rows in progress at once in the backward, each with its own partial column sums:
// blocks of a row each, or (narrow rows) warps of a row each.
constexpr int NORM_BLOCK_WORKERS = 304;
constexpr int NORM_WARP_WORKERS = 2432;
constexpr int NORM_WARP_VECTORS = 64;  // rows of up to 64 8-element vectors take one warp

struct NormArgs {
  int T, d;
  int weight_type, gate_kind, gate_sigmoid;
  float eps, offset, alpha, beta;
  const void* h;        // stream (backward of the merge: the stream after it)
  const moe_bf16* y;
  const void* w_post;
  const void* gate;
  const void* w_next;   // the norm's weight
  void* h_out;
  moe_bf16* x;
  // backward
  const void* d_stream;     // gradient of the stream by what follows (NULL = 0)
  const moe_bf16* dx;
  void* dh;
  moe_bf16* dy;
  float* dgate_rows;    // token gate: its gradient
  float* part;          // [worker][3][d] partial sums of dw_next, dw_post, dgate
};

__device__ __forceinline__ float gate_act(float g, int sigmoid) { return sigmoid ? 1.0f / (1.0f + __expf(-g)) : g; }

// One row per block (or per warp).  MERGE: h_out and, with w_next, its norm; else the
// norm of h.
template <typename ST, int VPT, bool MERGE, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_fwd_kernel(const NormArgs a) {
  __shared__ float buf[2][32];
  const int tpr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const long long row = WARP ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.T) return;
  const int nvec = a.d >> 3;
  const long long base = row * a.d;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float h[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * tpr;
    if (v < nvec) load8(static_cast<const ST*>(a.h) + base + v * 8, h[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
  }
  if (MERGE) {
    float y[VPT][8];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * tpr;
      if (v < nvec) load8(a.y + base + v * 8, y[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(y[i][j], y[i][j], s[0]);
    }
    float r = 1.0f;
    if (a.w_post) {
      row_sums<WARP, 1>(s, buf[0]);
      r = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
    }
    float g = a.beta;
    if (a.gate_kind == MOE_GATE_TOKEN) g *= gate_act(static_cast<const float*>(a.gate)[row], a.gate_sigmoid);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * tpr;
      if (v >= nvec) continue;
      float w[8];
      if (a.w_post) {
        load8_as(a.w_post, a.weight_type, v * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * r * (w[j] + a.offset);
      }
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        load8_as(a.gate, a.weight_type, v * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] *= gate_act(w[j], a.gate_sigmoid);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = fmaf(g, y[i][j], a.alpha * h[i][j]);
      store8(static_cast<ST*>(a.h_out) + base + v * 8, h[i]);
    }
    if (!a.w_next) return;
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] = fmaf(h[i][j], h[i][j], s[0]);
  row_sums<WARP, 1>(s, buf[1]);
  const float r = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * tpr;
    if (v >= nvec) continue;
    float w[8];
    load8_as(a.w_next, a.weight_type, v * 8, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = h[i][j] * r * (w[j] + a.offset);
    store8(a.x + base + v * 8, w);
  }
}

// Gradients.  A worker (block or warp) takes rows worker, worker + workers, ...; a thread
// keeps its columns' sums over the worker's rows in registers and writes them as the
// worker's partial sums, which norm_reduce_kernel adds in worker order.
//   D = d_stream + r (n - h r^2 mean(n h)),  n = dx (w_next + offset)
//   dz = beta a D,  q = dz (w_post + offset),  dy = r (q - y r^2 mean(q y))
template <typename ST, int VPT, bool MERGE, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512) norm_bwd_kernel(const NormArgs a) {
  __shared__ float buf[2][3 * 32];
  const int tpr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int per = WARP ? (blockDim.x >> 5) : 1;
  const int worker = WARP ? blockIdx.x * per + (threadIdx.x >> 5) : blockIdx.x;
  const int workers = gridDim.x * per;
  const int nvec = a.d >> 3;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const bool next = a.w_next != nullptr, post = MERGE && a.w_post != nullptr;
  const int gate = MERGE ? a.gate_kind : MOE_GATE_NONE;
  const bool need_y = post || gate != MOE_GATE_NONE;
  float dw_next[VPT][8], dw_post[VPT][8], dgate[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw_next[i][j] = dw_post[i][j] = dgate[i][j] = 0.0f;

  int flip = 0;  // the buffer of the next sum over the row
  for (long long row = worker; row < a.T; row += workers) {
    const long long base = row * a.d;
    float D[VPT][8], h[VPT][8], n[VPT][8], y[VPT][8];
    float s[3] = {0.0f, 0.0f, 0.0f};  // sums of h^2, n h, y^2
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * tpr;
#pragma unroll
      for (int j = 0; j < 8; ++j) D[i][j] = h[i][j] = n[i][j] = y[i][j] = 0.0f;
      if (v >= nvec) continue;
      if (a.d_stream) load8(static_cast<const ST*>(a.d_stream) + base + v * 8, D[i]);
      if (next) {
        load8(static_cast<const ST*>(a.h) + base + v * 8, h[i]);
        load8(a.dx + base + v * 8, n[i]);
      }
      if (MERGE && need_y) load8(a.y + base + v * 8, y[i]);
    }
    if (next) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * tpr;
        if (v >= nvec) continue;
        float w[8];
        load8_as(a.w_next, a.weight_type, v * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[0] = fmaf(h[i][j], h[i][j], s[0]);
          s[1] = fmaf(n[i][j] * (w[j] + a.offset), h[i][j], s[1]);
        }
      }
    }
    if (post) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[2] = fmaf(y[i][j], y[i][j], s[2]);
    }
    row_sums<WARP, 3>(s, buf[flip]);
    flip ^= 1;
    if (next) {
      const float r = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
      const float c = r * r * s[1] * inv_d;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * tpr;
        if (v >= nvec) continue;
        float w[8];
        load8_as(a.w_next, a.weight_type, v * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw_next[i][j] = fmaf(n[i][j], h[i][j] * r, dw_next[i][j]);
          D[i][j] = fmaf(r, n[i][j] * (w[j] + a.offset) - h[i][j] * c, D[i][j]);
        }
      }
    }
    float out[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * tpr;
      if (v >= nvec) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) out[i][j] = MERGE ? a.alpha * D[i][j] : D[i][j];
      store8(static_cast<ST*>(a.dh) + base + v * 8, out[i]);
    }
    if (!MERGE) continue;
    const float ry = post ? 1.0f / sqrtf(fmaf(s[2], inv_d, a.eps)) : 1.0f;
    float tg = a.beta, tact = 1.0f;  // beta * a for the row
    if (gate == MOE_GATE_TOKEN) {
      tact = gate_act(static_cast<const float*>(a.gate)[row], a.gate_sigmoid);
      tg *= tact;
    }
    float s2[2] = {0.0f, 0.0f};  // sums of q y, D z
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * tpr;
      if (v >= nvec) continue;
      float wp[8], wg[8];
      if (post) load8_as(a.w_post, a.weight_type, v * 8, wp);
      if (gate == MOE_GATE_CHANNEL) load8_as(a.gate, a.weight_type, v * 8, wg);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float w = post ? wp[j] + a.offset : 1.0f;
        const float yh = y[i][j] * ry;
        const float Dv = D[i][j];
        float dz = tg * Dv;
        if (gate == MOE_GATE_CHANNEL) {
          const float act = gate_act(wg[j], a.gate_sigmoid);
          const float slope = a.gate_sigmoid ? act * (1.0f - act) : 1.0f;
          dgate[i][j] = fmaf(dz * slope, yh * w, dgate[i][j]);
          dz *= act;
        } else if (gate == MOE_GATE_TOKEN) {
          s2[1] = fmaf(Dv, yh * w, s2[1]);
        }
        dw_post[i][j] = fmaf(dz, yh, dw_post[i][j]);
        const float q = dz * w;
        s2[0] = fmaf(q, y[i][j], s2[0]);
        D[i][j] = q;
      }
    }
    float c = 0.0f;
    if (post || gate == MOE_GATE_TOKEN) {
      row_sums<WARP, 2>(s2, buf[flip]);
      flip ^= 1;
      c = ry * ry * s2[0] * inv_d;
      if (gate == MOE_GATE_TOKEN && tid == 0)
        a.dgate_rows[row] = a.beta * s2[1] * (a.gate_sigmoid ? tact * (1.0f - tact) : 1.0f);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * tpr;
      if (v >= nvec) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = post ? ry * (D[i][j] - y[i][j] * c) : D[i][j];
      store8(a.dy + base + v * 8, o);
    }
  }
  float* part = a.part + static_cast<long long>(worker) * 3 * a.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * tpr;
    if (v >= nvec) continue;
    if (next) store8(part + v * 8, dw_next[i]);
    if (post) store8(part + a.d + v * 8, dw_post[i]);
    if (gate == MOE_GATE_CHANNEL) store8(part + 2 * a.d + v * 8, dgate[i]);
  }
}

// Column sums of the workers' partial sums, in worker order within each of the 8 lanes of
// a column, then over the lanes.  blockIdx.y picks the sum; a NULL output is skipped.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* __restrict__ part, int workers, int d,
                                                          float* __restrict__ o0, float* __restrict__ o1,
                                                          float* __restrict__ o2) {
  __shared__ float4 buf[8][32];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < d) {
#pragma unroll 4
    for (int w = grp; w < workers; w += 8) {
      const float4 p = *reinterpret_cast<const float4*>(part + (static_cast<long long>(w) * 3 + blockIdx.y) * d + c);
      s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
    }
  }
  buf[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && c < d) {
    for (int g = 1; g < 8; ++g) {
      const float4 p = buf[g][lane];
      s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
    }
    *reinterpret_cast<float4*>(out + c) = s;
  }
}

// ------------------------------------------------------------------ launchers

static int norm_workers(int d) { return (d >> 3) <= NORM_WARP_VECTORS ? NORM_WARP_WORKERS : NORM_BLOCK_WORKERS; }

// Threads of a block that shares a row of nvec vectors, VPT of them a thread.
static int row_threads(int nvec, int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; }

template <typename ST, bool MERGE>
static cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int nvec = a.d >> 3;
  if (nvec <= NORM_WARP_VECTORS) norm_fwd_kernel<ST, 2, MERGE, true><<<(a.T + 7) / 8, 256, 0, s>>>(a);
  else if (nvec <= 1024) norm_fwd_kernel<ST, 2, MERGE, false><<<a.T, row_threads(nvec, 2), 0, s>>>(a);
  else norm_fwd_kernel<ST, 4, MERGE, false><<<a.T, row_threads(nvec, 4), 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename ST, bool MERGE>
static cudaError_t launch_norm_bwd(const NormArgs& a, float* dw_next, float* dw_post, float* dgate_cols, cudaStream_t s) {
  const int nvec = a.d >> 3;
  int workers = 0;
  if (a.T > 0) {
    if (nvec <= NORM_WARP_VECTORS) {
      const int grid = min((a.T + 7) / 8, NORM_WARP_WORKERS / 8);
      workers = grid * 8;
      norm_bwd_kernel<ST, 2, MERGE, true><<<grid, 256, 0, s>>>(a);
    } else {
      workers = min(a.T, NORM_BLOCK_WORKERS);
      if (nvec <= 1024) norm_bwd_kernel<ST, 2, MERGE, false><<<workers, row_threads(nvec, 2), 0, s>>>(a);
      else norm_bwd_kernel<ST, 4, MERGE, false><<<workers, row_threads(nvec, 4), 0, s>>>(a);
    }
    count_launch();
  }
  if (dw_next || dw_post || dgate_cols) {
    norm_reduce_kernel<<<dim3((a.d + 127) / 128, 3), 256, 0, s>>>(a.part, workers, a.d, dw_next, dw_post, dgate_cols);
    count_launch();
  }
  return cudaGetLastError();
}

static NormArgs norm_args(const moe_norm_dims& m) {
  NormArgs a{};
  a.T = m.T; a.d = m.d; a.weight_type = m.weight_type; a.gate_kind = m.gate;
  a.gate_sigmoid = m.gate_act == MOE_GATE_SIGMOID;
  a.eps = m.eps; a.offset = m.weight_offset; a.alpha = m.alpha; a.beta = m.beta;
  return a;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_check_dims(const moe_norm_dims* dims) {
  if (!dims) return MOE_ERR_INVALID_ARG;
  const moe_norm_dims& m = *dims;
  if (m.T < 0 || m.d <= 0) return MOE_ERR_INVALID_ARG;
  if (m.stream_type != MOE_TYPE_BF16 && m.stream_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (m.weight_type != MOE_TYPE_BF16 && m.weight_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (m.gate < MOE_GATE_NONE || m.gate > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
  if (m.gate_act != MOE_GATE_IDENTITY && m.gate_act != MOE_GATE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!(m.eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  if (m.d % 8 != 0 || m.d > NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t moe_norm_workspace_size(const moe_norm_dims* dims) {
  if (moe_norm_check_dims(dims) != MOE_OK) return 0;
  return static_cast<size_t>(norm_workers(dims->d)) * 3 * dims->d * sizeof(float);
}

moe_status moe_norm_fwd(const moe_norm_dims* dims, const void* h, const void* w, moe_bf16* x, void* stream) {
  const moe_status st = moe_norm_check_dims(dims);
  if (st != MOE_OK) return st;
  if (!w || (dims->T > 0 && (!h || !x))) return MOE_ERR_INVALID_ARG;
  if (!ptr_aligned16(h) || !ptr_aligned16(w) || !ptr_aligned16(x)) return MOE_ERR_ALIGNMENT;
  NormArgs a = norm_args(*dims);
  a.h = h; a.w_next = w; a.x = x;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(dims->stream_type == MOE_TYPE_BF16 ? launch_norm_fwd<moe_bf16, false>(a, s)
                                                      : launch_norm_fwd<float, false>(a, s));
}

moe_status moe_norm_bwd(const moe_norm_dims* dims, const moe_bf16* dx, const void* h, const void* w,
                        const void* dh_add, void* dh, float* dw, void* workspace, void* stream) {
  const moe_status st = moe_norm_check_dims(dims);
  if (st != MOE_OK) return st;
  if (!w || !dw || (dims->T > 0 && (!dx || !h || !dh))) return MOE_ERR_INVALID_ARG;
  if (!workspace) return MOE_ERR_WORKSPACE;
  if (!ptr_aligned16(dx) || !ptr_aligned16(h) || !ptr_aligned16(w) || !ptr_aligned16(dh_add) || !ptr_aligned16(dh) ||
      !ptr_aligned16(dw) || !ptr_aligned16(workspace))
    return MOE_ERR_ALIGNMENT;
  NormArgs a = norm_args(*dims);
  a.dx = dx; a.h = h; a.w_next = w; a.d_stream = dh_add; a.dh = dh; a.part = static_cast<float*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(dims->stream_type == MOE_TYPE_BF16 ? launch_norm_bwd<moe_bf16, false>(a, dw, nullptr, nullptr, s)
                                                      : launch_norm_bwd<float, false>(a, dw, nullptr, nullptr, s));
}

moe_status moe_merge_fwd(const moe_norm_dims* dims, const void* h, const moe_bf16* y, const void* w_post,
                         const void* gate, const void* w_next, void* h_out, moe_bf16* x_next, void* stream) {
  const moe_status st = moe_norm_check_dims(dims);
  if (st != MOE_OK) return st;
  if (dims->T > 0 && (!h || !y || !h_out || (dims->gate != MOE_GATE_NONE && !gate) || (w_next && !x_next)))
    return MOE_ERR_INVALID_ARG;
  if ((dims->gate == MOE_GATE_NONE && gate) || (!w_next && x_next)) return MOE_ERR_INVALID_ARG;
  if (!ptr_aligned16(h) || !ptr_aligned16(y) || !ptr_aligned16(w_post) || !ptr_aligned16(gate) ||
      !ptr_aligned16(w_next) || !ptr_aligned16(h_out) || !ptr_aligned16(x_next))
    return MOE_ERR_ALIGNMENT;
  NormArgs a = norm_args(*dims);
  a.h = h; a.y = y; a.w_post = w_post; a.gate = gate; a.w_next = w_next; a.h_out = h_out; a.x = x_next;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(dims->stream_type == MOE_TYPE_BF16 ? launch_norm_fwd<moe_bf16, true>(a, s)
                                                      : launch_norm_fwd<float, true>(a, s));
}

moe_status moe_merge_bwd(const moe_norm_dims* dims, const void* dh_out, const moe_bf16* dx_next, const void* h_out,
                         const moe_bf16* y, const void* w_post, const void* gate, const void* w_next, void* dh,
                         moe_bf16* dy, float* dw_post, float* dgate, float* dw_next, void* workspace, void* stream) {
  const moe_status st = moe_norm_check_dims(dims);
  if (st != MOE_OK) return st;
  const moe_norm_dims& m = *dims;
  if ((w_post != nullptr) != (dw_post != nullptr) || (w_next != nullptr) != (dw_next != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (m.gate == MOE_GATE_NONE && (gate || dgate)) return MOE_ERR_INVALID_ARG;
  if (m.gate == MOE_GATE_CHANNEL && (!gate || !dgate)) return MOE_ERR_INVALID_ARG;
  if (!w_next && dx_next) return MOE_ERR_INVALID_ARG;
  if (m.T > 0) {
    if (!dh || !dy || (m.gate == MOE_GATE_TOKEN && (!gate || !dgate))) return MOE_ERR_INVALID_ARG;
    if (w_next ? (!dx_next || !h_out) : !dh_out) return MOE_ERR_INVALID_ARG;
    if ((w_post || m.gate != MOE_GATE_NONE) && !y) return MOE_ERR_INVALID_ARG;
  }
  if (!workspace) return MOE_ERR_WORKSPACE;
  const void* every[] = {dh_out, dx_next, h_out, y, w_post, gate, w_next, dh, dy, dw_post, dgate, dw_next, workspace};
  for (const void* p : every)
    if (!ptr_aligned16(p)) return MOE_ERR_ALIGNMENT;
  NormArgs a = norm_args(m);
  a.d_stream = dh_out; a.dx = dx_next; a.h = h_out; a.y = y; a.w_post = w_post; a.gate = gate; a.w_next = w_next;
  a.dh = dh; a.dy = dy; a.part = static_cast<float*>(workspace);
  a.dgate_rows = m.gate == MOE_GATE_TOKEN ? dgate : nullptr;
  float* dgate_cols = m.gate == MOE_GATE_CHANNEL ? dgate : nullptr;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(m.stream_type == MOE_TYPE_BF16 ? launch_norm_bwd<moe_bf16, true>(a, dw_next, dw_post, dgate_cols, s)
                                                  : launch_norm_bwd<float, true>(a, dw_next, dw_post, dgate_cols, s));
}

}  // extern "C"
