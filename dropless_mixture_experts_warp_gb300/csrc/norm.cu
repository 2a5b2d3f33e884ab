// Block norms: the norm before a block, the merge after it (norm of its output, gate,
// scaled residual, the next block's norm) and their gradients.  Every kernel reads each
// row of its inputs once, keeps it in shared memory and registers between the sums over
// the row and the outputs, and does its arithmetic in fp32; all are bound by HBM.
//
// One block an SM, its threads in groups that each have a row: tpr threads (a multiple of
// 32) with UPT units of U columns each, a unit being 16 bytes of the stream (8 or 16 of a
// bf16 array).  Groups walk the rows worker, worker + workers, ...; a row's units arrive by
// asynchronous copies in the group's ring of `stages` rows in shared memory, each thread
// copying and reading its own units only, so that the next rows are on their way while one
// is computed.  The weights are shared by the block's rows: as fp32, offsets added and
// gates activated, in shared memory where that has room beside two rows a group.
//
// Measured (GB300, bf16 stream, 16384 x 7168): the norm 73 us, its gradients 142 us; the merge
// with every weight and a channel gate 138 us (6.8 TB/s, the rate of a copy), its gradients
// 222 us (6.35 TB/s); fp32 stream, 16384 x 4096: merge 120 us, gradients 215 us (5.65 TB/s).
//
// KNOWN variants know at compile time that a call has every weight and the gradient of the
// stream, and the kind of gate GATE (asked element by element at run time these choices took
// half of the instructions); EXACT ones also that the weights are in shared memory and that
// the row's units fill the threads.  A merge without an output norm, or of more than 8192
// columns, asks at run time: 16384 x 7168 bf16 with the next norm alone 151 us, gradients
// 364 us (a copy's rate would be 141 and 176).
#include "around.cuh"

#include <algorithm>

namespace moe {

constexpr int NORM_MAX_D = 16384;
constexpr int NORM_SMEM = 225 * 1024;  // dynamic shared memory of a block: of the 227 KB, static buffers aside
constexpr int NORM_MAX_SMS = 160;      // blocks at most
// Threads of a block: the forward of the merge needs 96 registers a thread (spills with 64
// cost 12 %), the backward those of three weights' column sums, 128 with 16 columns a thread.
constexpr int norm_fwd_threads(bool merge) { return merge ? 640 : 1024; }
constexpr int norm_bwd_threads(int cols) { return cols == 8 ? 768 : 512; }

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

enum { RING_D, RING_H, RING_DX, RING_Y, RING_ARRAYS };
enum { W_NEXT, W_POST, W_GATE, W_SLOPE, W_ARRAYS };
constexpr int GATE_SLOPE = 3;  // a sigmoid channel gate, for the backward's variants

// How the threads and the shared memory of a block are split.
struct NormPlan {
  int grid, groups, tpr, cols;
  bool staged;            // every weight has a place
  int off[RING_ARRAYS];   // each array's place in a ring row (-1: not read)
  int weight[W_ARRAYS];   // each weight's place, in floats (-1: read from global memory)
  int row_bytes, weight_bytes, stages;
  int smem_bytes;
  bool join;              // backward: the groups' column sums are added in the block
  int y_bytes;            // backward: y has a ring of its own, of stages + 1 rows
  bool late_y;            // of stages rows instead, for two stages (the LATE form)
};

// The activated gate and its slope.  With e = exp(-|g|) the sigmoid is 1 / (1 + e) or
// e / (1 + e) and its slope e / (1 + e)^2, all within a few units of fp32.  (As a (1 - a) the
// slope would be 17 % off at g = 15 and 0 from 17 on, where a rounds to 1.)
__device__ __forceinline__ float gate_act(float g, int sigmoid) {
  if (!sigmoid) return g;
  const float e = expf(-fabsf(g));
  return (g < 0.0f ? e : 1.0f) / (1.0f + e);
}
__device__ __forceinline__ float gate_slope(float g, int sigmoid) {
  if (!sigmoid) return 1.0f;
  const float e = expf(-fabsf(g));
  return e / ((1.0f + e) * (1.0f + e));
}

// Until at most n (0 .. 3) of the thread's groups of copies are under way.
__device__ __forceinline__ void copy_wait_but(int n) {
  switch (n) {
    case 0: copy_wait<0>(); break;
    case 1: copy_wait<1>(); break;
    case 2: copy_wait<2>(); break;
    default: copy_wait<3>(); break;
  }
}

// Units of U columns as U / 2 pairs.
template <int U>
__device__ __forceinline__ void unpack(const moe_bf16* p, f32x2 (&v)[U / 2]) {
  if (U == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    v[0] = pair(bf16_lo(q.x), bf16_hi(q.x));
    v[1] = pair(bf16_lo(q.y), bf16_hi(q.y));
    v[U / 2 - 2] = pair(bf16_lo(q.z), bf16_hi(q.z));
    v[U / 2 - 1] = pair(bf16_lo(q.w), bf16_hi(q.w));
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = pair(bf16_lo(q.x), bf16_hi(q.x));
    v[1] = pair(bf16_lo(q.y), bf16_hi(q.y));
  }
}
template <int U>
__device__ __forceinline__ void unpack(const float* p, f32x2 (&v)[U / 2]) {
#pragma unroll
  for (int j = 0; j < U / 4; ++j) {
    const ulonglong2 q = reinterpret_cast<const ulonglong2*>(p)[j];
    v[2 * j] = q.x;
    v[2 * j + 1] = q.y;
  }
}
template <int U>
__device__ __forceinline__ void pack(moe_bf16* p, const f32x2 (&v)[U / 2]) {
  uint32_t w[U / 2];
#pragma unroll
  for (int j = 0; j < U / 2; ++j) {
    const float2 f = unpair(v[j]);
    w[j] = pack_bf16(f.x, f.y);
  }
  if (U == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[U / 2 - 2], w[U / 2 - 1]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int U>
__device__ __forceinline__ void pack(float* p, const f32x2 (&v)[U / 2]) {
#pragma unroll
  for (int j = 0; j < U / 4; ++j) reinterpret_cast<ulonglong2*>(p)[j] = make_ulonglong2(v[2 * j], v[2 * j + 1]);
}
template <int U>
__device__ __forceinline__ void fill(f32x2 (&v)[U / 2], float x) {
#pragma unroll
  for (int j = 0; j < U / 2; ++j) v[j] = pair(x, x);
}

// What a weight array holds for the kernels: weight + offset, the activated gate, its slope.
__device__ __forceinline__ float weight_value(const NormArgs& a, int kind, float w) {
  if (kind == W_NEXT || kind == W_POST) return w + a.offset;
  return kind == W_GATE ? gate_act(w, a.gate_sigmoid) : gate_slope(w, a.gate_sigmoid);
}
template <int U>
__device__ __forceinline__ void raw_weights(const NormArgs& a, int kind, int u, f32x2 (&v)[U / 2]) {
  const void* w = kind == W_NEXT ? a.w_next : kind == W_POST ? a.w_post : a.gate;
  if (a.weight_type == MOE_TYPE_BF16) unpack<U>(static_cast<const moe_bf16*>(w) + u * U, v);
  else unpack<U>(static_cast<const float*>(w) + u * U, v);
}
template <int U>
__device__ __forceinline__ void weight_values(const NormArgs& a, int kind, f32x2 (&v)[U / 2]) {
#pragma unroll
  for (int j = 0; j < U / 2; ++j) {
    const float2 f = unpair(v[j]);
    v[j] = pair(weight_value(a, kind, f.x), weight_value(a, kind, f.y));
  }
}
// Unit u of a weight array.  In shared memory a unit's 16-byte pieces lie `units` apart: at
// 32-byte strides every access would take two passes.
template <int U, bool STAGED>
__device__ __forceinline__ void weights(const NormArgs& a, const NormPlan& plan, const float* smem, int kind, int units,
                                        int u, f32x2 (&v)[U / 2]) {
  if (STAGED || plan.weight[kind] >= 0) {
    const float* w = smem + plan.weight[kind];
#pragma unroll
    for (int j = 0; j < U / 4; ++j) {
      const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(w + (j * units + u) * 4);
      v[2 * j] = q.x;
      v[2 * j + 1] = q.y;
    }
  } else {
    raw_weights<U>(a, kind, u, v);
    weight_values<U>(a, kind, v);
  }
}
// Copies the weights that have a place into shared memory (the caller synchronises).  All
// arrays' loads come before the first use of one: they wait for memory together.
template <int U>
__device__ __forceinline__ void stage_weights(const NormArgs& a, const NormPlan& plan, float* smem, int units) {
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    f32x2 v[W_ARRAYS][U / 2];
#pragma unroll
    for (int kind = 0; kind < W_SLOPE; ++kind)
      if (plan.weight[kind] >= 0 || (kind == W_GATE && plan.weight[W_SLOPE] >= 0)) raw_weights<U>(a, kind, u, v[kind]);
#pragma unroll
    for (int j = 0; j < U / 2; ++j) v[W_SLOPE][j] = v[W_GATE][j];
#pragma unroll
    for (int kind = 0; kind < W_ARRAYS; ++kind) {
      if (plan.weight[kind] < 0) continue;
      weight_values<U>(a, kind, v[kind]);
#pragma unroll
      for (int j = 0; j < U / 4; ++j)
        *reinterpret_cast<ulonglong2*>(smem + plan.weight[kind] + (j * units + u) * 4) =
            make_ulonglong2(v[kind][2 * j], v[kind][2 * j + 1]);
    }
  }
}

// Sums of up to 4 values over a warp: lanes give half of the values away while they add (4
// values: 6 shuffles instead of 20).  The sum of value i stands in lanes i * WIDTH and on.
template <int N>
struct SumLanes {
  static constexpr int WIDTH = N == 1 ? 32 : N == 2 ? 16 : 8;
};
template <int N>
__device__ __forceinline__ float lane_sums(const float* s, int lane) {
  constexpr unsigned ALL = 0xffffffffu;
  float v = s[0];
  if (N == 2) {
    const bool up = lane & 16;
    v = (up ? s[1] : s[0]) + __shfl_xor_sync(ALL, up ? s[0] : s[1], 16);
  } else if (N >= 3) {
    const bool up = lane & 16, odd = lane & 8;
    const float last = N == 4 ? s[3] : 0.0f;
    const float x = (up ? s[2] : s[0]) + __shfl_xor_sync(ALL, up ? s[0] : s[2], 16);
    const float y = (up ? last : s[1]) + __shfl_xor_sync(ALL, up ? s[1] : last, 16);
    v = (odd ? y : x) + __shfl_xor_sync(ALL, odd ? x : y, 8);
  }
#pragma unroll
  for (int off = SumLanes<N>::WIDTH / 2; off > 0; off >>= 1) v += __shfl_xor_sync(ALL, v, off);
  return v;
}

// Sums of N values (at most SUMS_MAX) over the threads of a group, in a fixed order; every thread
// gets them.  Two buffers taken in turn need one barrier a sum: whoever writes a buffer
// again has passed the barrier of the other, which its readers reach after reading.
constexpr int SUMS_MAX = 5;
constexpr int MAX_WARPS = 24;  // of a group
struct GroupSums {
  float* buf;   // the group's 2 * SUMS_MAX * tpr / 32 floats
  int tpr, group, tid, flip;
  template <int N>
  __device__ __forceinline__ void write(const float* s, float* b) {
    const int lane = tid & 31, value = lane / SumLanes<N>::WIDTH;
    const float v = lane_sums<N>(s, lane);
    if ((lane & (SumLanes<N>::WIDTH - 1)) == 0 && value < N) b[value * (tpr >> 5) + (tid >> 5)] = v;
  }
  template <int N>
  __device__ __forceinline__ void read(float* s, const float* b) {
    constexpr int WIDTH = SumLanes<N>::WIDTH;
    const int lane = tid & 31, warps = tpr >> 5, first = lane & (WIDTH - 1), value = lane / WIDTH;
    const float* r = b + (value < N ? value : 0) * warps;
    float v = first < warps ? r[first] : 0.0f;
#pragma unroll
    for (int more = WIDTH; more < MAX_WARPS; more += WIDTH) v += first + more < warps ? r[first + more] : 0.0f;
#pragma unroll
    for (int off = WIDTH / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = N == 1 ? v : __shfl_sync(0xffffffffu, v, i * WIDTH);
  }
  template <int N>
  __device__ __forceinline__ void warp_only(float* s) {
    const float v = lane_sums<N>(s, tid & 31);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = N == 1 ? v : __shfl_sync(0xffffffffu, v, i * SumLanes<N>::WIDTH);
  }
  template <int N>
  __device__ __forceinline__ void operator()(float (&s)[N]) {
    static_assert(N <= SUMS_MAX, "more sums than the buffers hold");
    constexpr int A = N < 4 ? N : 4, B = N - A;
    if (tpr == 32) {
      warp_only<A>(s);
      if (B) warp_only<B ? B : 1>(s + (B ? A : 0));
      return;
    }
    float* b = buf + flip * SUMS_MAX * (tpr >> 5);
    flip ^= 1;
    write<A>(s, b);
    if (B) write<B ? B : 1>(s + (B ? A : 0), b + A * (tpr >> 5));
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    read<A>(s, b);
    if (B) read<B ? B : 1>(s + (B ? A : 0), b + A * (tpr >> 5));
  }
};

// 1 / sqrt(mean + eps) of a sum of squares; within 2 units.
__device__ __forceinline__ float inv_rms(float sum, float inv_d, float eps) { return rsqrtf(fmaf(sum, inv_d, eps)); }

// MERGE: h_out and, with w_next, its norm; else the norm of h.  Two rows are under way in a
// group: the sum that the next row's first norm needs (of y^2, or of h^2) is added up
// together with this row's sum of h_out^2, so that a row takes one barrier and its waits are
// filled with the other row's work.
template <typename ST, int UPT, bool MERGE, bool KNOWN, bool EXACT, int GATE>
__global__ void __launch_bounds__(norm_fwd_threads(MERGE)) norm_fwd_kernel(const NormArgs a, const NormPlan plan) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[2 * SUMS_MAX * 32];
  constexpr int U = 16 / sizeof(ST);
  const int tpr = plan.tpr, group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr;
  const int worker = group * gridDim.x + blockIdx.x, workers = plan.groups * gridDim.x;
  const int units = a.d / U;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  GroupSums sums{buf + group * 2 * SUMS_MAX * (tpr >> 5), tpr, group, tid, 0};
  const float* s_w = reinterpret_cast<const float*>(smem);
  uint8_t* my_ring = smem + plan.weight_bytes + group * plan.stages * plan.row_bytes;
  auto fetch = [&](long long row, int stage) {
    if (row < a.T) {
      const uint32_t dst = smem_u32(my_ring + stage * plan.row_bytes);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tid + i * tpr;
        if (!EXACT && u >= units) continue;
        const long long at = row * a.d + u * U;
        copy_async<16>(dst + plan.off[RING_H] + u * 16, static_cast<const ST*>(a.h) + at);
        if (MERGE) copy_async<U * 2>(dst + plan.off[RING_Y] + u * U * 2, a.y + at);
      }
    }
    copy_commit();
  };
  wait_for_previous();
  launch_dependents();
  // one group of copies a row: `stages` of them are open when a row is waited for
  for (int s = 0; s < plan.stages; ++s) fetch(worker + static_cast<long long>(s) * workers, s);
  stage_weights<U>(a, plan, reinterpret_cast<float*>(smem), units);
  __syncthreads();
  const int gate = !MERGE ? MOE_GATE_NONE : KNOWN ? GATE : a.gate_kind;
  const bool post = MERGE && (KNOWN || a.w_post != nullptr), next = KNOWN || a.w_next != nullptr;
  const bool channel = gate == MOE_GATE_CHANNEL;

  // A row's sum of y^2 (MERGE) or h^2, this thread's part.
  auto first_sum = [&](const uint8_t* at) {
    f32x2 ss = pair(0.0f, 0.0f);
    if (MERGE && !post) return 0.0f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tid + i * tpr;
      if (!EXACT && u >= units) continue;
      f32x2 v[U / 2];
      if (MERGE) unpack<U>(reinterpret_cast<const moe_bf16*>(at + plan.off[RING_Y]) + u * U, v);
      else unpack<U>(reinterpret_cast<const ST*>(at + plan.off[RING_H]) + u * U, v);
#pragma unroll
      for (int j = 0; j < U / 2; ++j) ss = fma2(v[j], v[j], ss);
    }
    return sum_pair(ss);
  };
  int stage = 0;
  float first = 0.0f;  // the row's first sum, over all its columns
  if (worker < a.T) {
    copy_wait_but(plan.stages - 1);
    float s[1] = {first_sum(my_ring)};
    sums(s);
    first = s[0];
  }
  for (long long row = worker; row < a.T; row += workers) {
    const uint8_t* at = my_ring + stage * plan.row_bytes;
    const long long base = row * a.d;
    const float r1 = inv_rms(first, inv_d, a.eps);
    float g = MERGE ? a.beta : r1;
    if (gate == MOE_GATE_TOKEN) g *= gate_act(static_cast<const float*>(a.gate)[row], a.gate_sigmoid);
    if (post) g *= r1;
    const f32x2 g2 = pair(g, g);
    f32x2 h[UPT][U / 2], ss = pair(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tid + i * tpr;
      if (!EXACT && u >= units) continue;
      f32x2 w[U / 2];
      unpack<U>(reinterpret_cast<const ST*>(at + plan.off[RING_H]) + u * U, h[i]);
      if (MERGE) {
        f32x2 y[U / 2];
        unpack<U>(reinterpret_cast<const moe_bf16*>(at + plan.off[RING_Y]) + u * U, y);
        if (post) {
          weights<U, EXACT>(a, plan, s_w, W_POST, units, u, w);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) y[j] = mul2(y[j], w[j]);
        }
        if (channel) {
          weights<U, EXACT>(a, plan, s_w, W_GATE, units, u, w);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) y[j] = mul2(y[j], w[j]);
        }
#pragma unroll
        for (int j = 0; j < U / 2; ++j) {
          const float2 f = unpair(h[i][j]);
          h[i][j] = fma2(g2, y[j], pair(a.alpha * f.x, a.alpha * f.y));
          ss = fma2(h[i][j], h[i][j], ss);
        }
        pack<U>(static_cast<ST*>(a.h_out) + base + u * U, h[i]);
      } else {
        weights<U, EXACT>(a, plan, s_w, W_NEXT, units, u, w);
#pragma unroll
        for (int j = 0; j < U / 2; ++j) w[j] = mul2(mul2(h[i][j], g2), w[j]);
        pack<U>(a.x + base + u * U, w);
      }
    }
    // every value of the row was used above: its place in the ring is free
    fetch(row + static_cast<long long>(plan.stages) * workers, stage);
    stage = stage + 1 == plan.stages ? 0 : stage + 1;
    float s[MERGE ? 2 : 1] = {};
    if (row + workers < a.T) {
      copy_wait_but(plan.stages - 1);
      s[0] = first_sum(my_ring + stage * plan.row_bytes);
    }
    if (MERGE) s[MERGE ? 1 : 0] = sum_pair(ss);
    sums(s);
    first = s[0];
    if (!MERGE || !next) continue;
    const float r = inv_rms(s[MERGE ? 1 : 0], inv_d, a.eps);
    const f32x2 r2 = pair(r, r);
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tid + i * tpr;
      if (!EXACT && u >= units) continue;
      f32x2 w[U / 2];
      weights<U, EXACT>(a, plan, s_w, W_NEXT, units, u, w);
#pragma unroll
      for (int j = 0; j < U / 2; ++j) w[j] = mul2(mul2(h[i][j], r2), w[j]);
      pack<U>(a.x + base + u * U, w);
    }
  }
}

// Gradients.  A thread keeps its columns' sums over the worker's rows in registers and
// writes them as the worker's partial sums, which norm_reduce_kernel adds in worker order.
//   D = d_stream + r (n - h r^2 mean(n h)),  n = dx (w_next + offset)
//   dz = beta a D,  q = dz (w_post + offset),  dy = r (q - y r^2 mean(q y))
// Two rows are under way in a group: the sums that D of the next row needs are added up
// together with those that dy of this row needs, so that a row takes one barrier and its
// waits are filled with the other row's work (355 us with two barriers a row, for 16384 x
// 7168 bf16 with everything).  So y has one place more in the ring than the others; where
// that leaves a weight no room (it would come from L2 for each row) LATE takes none more and
// fetches y when the row that used its place is done (8192 x 7168 fp32 stream without a gate:
// 173 us, 219 without; 16384 x 8192 bf16 with a channel gate: 287, 316 without).
// What a call lacks (weights, gate) takes its neutral value, a unit at a time.
template <typename ST, int UPT, bool MERGE, bool KNOWN, bool EXACT, int GATE, bool LATE>
__global__ void __launch_bounds__(norm_bwd_threads(UPT * 16 / static_cast<int>(sizeof(ST)))) norm_bwd_kernel(const NormArgs a, const NormPlan plan) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[2 * SUMS_MAX * 32];
  constexpr int U = 16 / sizeof(ST);
  const int tpr = plan.tpr, group = threadIdx.x / tpr, tid = threadIdx.x - group * tpr;
  const int worker = group * gridDim.x + blockIdx.x, workers = plan.groups * gridDim.x;
  const int units = a.d / U;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  GroupSums sums{buf + group * 2 * SUMS_MAX * (tpr >> 5), tpr, group, tid, 0};
  const float* s_w = reinterpret_cast<const float*>(smem);
  const int last_y = plan.stages - (LATE ? 1 : 0);  // of the places of y
  uint8_t* my_ring = smem + plan.weight_bytes + group * (plan.stages * plan.row_bytes + (last_y + 1) * plan.y_bytes);
  uint8_t* my_y = my_ring + plan.stages * plan.row_bytes;
  auto fetch_y = [&](long long row, int y_stage) {
    if (row < a.T) {
      const uint32_t dst_y = smem_u32(my_y + y_stage * plan.y_bytes);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tid + i * tpr;
        if (EXACT || u < units) copy_async<U * 2>(dst_y + u * U * 2, a.y + row * a.d + u * U);
      }
    }
    copy_commit();
  };
  auto fetch = [&](long long row, int stage, int y_stage) {
    if (row < a.T) {
      const uint32_t dst = smem_u32(my_ring + stage * plan.row_bytes), dst_y = smem_u32(my_y + y_stage * plan.y_bytes);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tid + i * tpr;
        if (!EXACT && u >= units) continue;
        const long long at = row * a.d + u * U;
        if (KNOWN || plan.off[RING_D] >= 0) copy_async<16>(dst + plan.off[RING_D] + u * 16, static_cast<const ST*>(a.d_stream) + at);
        if (KNOWN || plan.off[RING_H] >= 0) copy_async<16>(dst + plan.off[RING_H] + u * 16, static_cast<const ST*>(a.h) + at);
        if (KNOWN || plan.off[RING_DX] >= 0) copy_async<U * 2>(dst + plan.off[RING_DX] + u * U * 2, a.dx + at);
        if (MERGE && !LATE && (KNOWN || plan.y_bytes > 0)) copy_async<U * 2>(dst_y + u * U * 2, a.y + at);
      }
    }
    copy_commit();
  };
  wait_for_previous();
  launch_dependents();
  // one group of copies a row, or two where LATE (the row's other arrays, its y): those of
  // `stages` rows are open when a row is waited for
  for (int s = 0; s < plan.stages; ++s) {
    fetch(worker + static_cast<long long>(s) * workers, s, s);
    if (LATE) fetch_y(worker + static_cast<long long>(s) * workers, s);
  }
  stage_weights<U>(a, plan, reinterpret_cast<float*>(smem), units);
  __syncthreads();
  const bool next = KNOWN || a.w_next != nullptr, post = MERGE && (KNOWN || a.w_post != nullptr);
  const int gate = !MERGE ? MOE_GATE_NONE : !KNOWN ? a.gate_kind : GATE == GATE_SLOPE ? MOE_GATE_CHANNEL : GATE;
  const bool channel = gate == MOE_GATE_CHANNEL, token = gate == MOE_GATE_TOKEN;
  const bool slope = KNOWN ? GATE == GATE_SLOPE : channel && a.gate_sigmoid, has_y = post || gate != MOE_GATE_NONE;
  const f32x2 zero = pair(0.0f, 0.0f);

  // A row's sums of h^2, n h and y^2.
  auto first_sums = [&](const uint8_t* at, const uint8_t* y_at, float& hh, float& nh, float& yy) {
    f32x2 shh = zero, snh = zero, syy = zero;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int u = tid + i * tpr;
      if (!EXACT && u >= units) continue;
      if (next) {
        f32x2 h[U / 2], n[U / 2], w[U / 2];
        unpack<U>(reinterpret_cast<const ST*>(at + plan.off[RING_H]) + u * U, h);
        unpack<U>(reinterpret_cast<const moe_bf16*>(at + plan.off[RING_DX]) + u * U, n);
        weights<U, EXACT>(a, plan, s_w, W_NEXT, units, u, w);
#pragma unroll
        for (int j = 0; j < U / 2; ++j) {
          shh = fma2(h[j], h[j], shh);
          snh = fma2(mul2(n[j], w[j]), h[j], snh);
        }
      }
      if (post) {
        f32x2 y[U / 2];
        unpack<U>(reinterpret_cast<const moe_bf16*>(y_at) + u * U, y);
#pragma unroll
        for (int j = 0; j < U / 2; ++j) syy = fma2(y[j], y[j], syy);
      }
    }
    hh = sum_pair(shh);
    nh = sum_pair(snh);
    yy = sum_pair(syy);
  };

  f32x2 dw_next[UPT][U / 2], dw_post[UPT][U / 2], dgate[UPT][U / 2];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    fill<U>(dw_next[i], 0.0f);
    fill<U>(dw_post[i], 0.0f);
    fill<U>(dgate[i], 0.0f);
  }
  int stage = 0, y_stage = 0;
  float hh = 0.0f, nh = 0.0f, yy = 0.0f;  // of the row, over all its columns
  if (worker < a.T) {
    copy_wait_but(LATE ? 2 : plan.stages - 1);
    float s[3];
    first_sums(my_ring, my_y, s[0], s[1], s[2]);
    sums(s);
    hh = s[0];
    nh = s[1];
    yy = s[2];
  }
  for (long long row = worker; row < a.T; row += workers) {
    const long long base = row * a.d;
    const uint8_t* at = my_ring + stage * plan.row_bytes;
    const moe_bf16* r_y = reinterpret_cast<const moe_bf16*>(my_y + y_stage * plan.y_bytes);
    const float r = next ? inv_rms(hh, inv_d, a.eps) : 0.0f;
    const float c = -r * r * nh * inv_d;
    const float ry = post ? inv_rms(yy, inv_d, a.eps) : 1.0f;
    float tg = a.beta, tslope = 1.0f;  // beta * a for the row
    if (token) {
      const float gate = static_cast<const float*>(a.gate)[row];
      tg *= gate_act(gate, a.gate_sigmoid);
      tslope = gate_slope(gate, a.gate_sigmoid);
    }
    f32x2 sqy = zero, sdz = zero;
    f32x2 q[UPT][U / 2];
    {
      const f32x2 r2 = pair(r, r), c2 = pair(c, c), ry2 = pair(ry, ry), tg2 = pair(tg, tg);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tid + i * tpr;
        if (!EXACT && u >= units) continue;
        f32x2 D[U / 2];
        if (KNOWN || a.d_stream) unpack<U>(reinterpret_cast<const ST*>(at + plan.off[RING_D]) + u * U, D);
        else fill<U>(D, 0.0f);
        if (next) {
          f32x2 h[U / 2], n[U / 2], w[U / 2];
          unpack<U>(reinterpret_cast<const ST*>(at + plan.off[RING_H]) + u * U, h);
          unpack<U>(reinterpret_cast<const moe_bf16*>(at + plan.off[RING_DX]) + u * U, n);
          weights<U, EXACT>(a, plan, s_w, W_NEXT, units, u, w);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) {
            dw_next[i][j] = fma2(n[j], mul2(h[j], r2), dw_next[i][j]);
            D[j] = fma2(r2, fma2(h[j], c2, mul2(n[j], w[j])), D[j]);
          }
        }
        f32x2 o[U / 2];
#pragma unroll
        for (int j = 0; j < U / 2; ++j) {
          const float2 f = unpair(D[j]);
          o[j] = MERGE ? pair(a.alpha * f.x, a.alpha * f.y) : D[j];
        }
        pack<U>(static_cast<ST*>(a.dh) + base + u * U, o);
        if (MERGE) {
          f32x2 y[U / 2], wp[U / 2], wg[U / 2], ds[U / 2];
          if (has_y) unpack<U>(r_y + u * U, y);
          else fill<U>(y, 0.0f);
          if (post) weights<U, EXACT>(a, plan, s_w, W_POST, units, u, wp);
          else fill<U>(wp, 1.0f);
          if (channel) weights<U, EXACT>(a, plan, s_w, W_GATE, units, u, wg);
          else fill<U>(wg, 1.0f);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) q[i][j] = ds[j] = mul2(tg2, D[j]);
          if (slope) {
            f32x2 sl[U / 2];
            weights<U, EXACT>(a, plan, s_w, W_SLOPE, units, u, sl);
#pragma unroll
            for (int j = 0; j < U / 2; ++j) ds[j] = mul2(ds[j], sl[j]);
          }
#pragma unroll
          for (int j = 0; j < U / 2; ++j) {
            const f32x2 yh = mul2(y[j], ry2), z = mul2(yh, wp[j]);
            dgate[i][j] = fma2(ds[j], z, dgate[i][j]);
            if (!KNOWN || token) sdz = fma2(D[j], z, sdz);
            const f32x2 dz = mul2(q[i][j], wg[j]);
            dw_post[i][j] = fma2(dz, yh, dw_post[i][j]);
            q[i][j] = mul2(dz, wp[j]);
            sqy = fma2(q[i][j], y[j], sqy);
          }
        }
      }
    }
    // the row's D, h and dx were used above and y of the row before in its dy: their places
    // are free for the row `stages` further on (where LATE, this row's y is, below)
    const int y_after = LATE ? y_stage : y_stage + plan.stages > plan.stages ? y_stage - 1 : plan.stages;
    fetch(row + static_cast<long long>(plan.stages) * workers, stage, y_after);
    stage = stage + 1 == plan.stages ? 0 : stage + 1;
    y_stage = y_stage == last_y ? 0 : y_stage + 1;
    float s[!MERGE ? 2 : KNOWN && GATE != MOE_GATE_TOKEN ? 4 : 5] = {};
    if (row + workers < a.T) {
      copy_wait_but(plan.stages - 1);
      float y2;
      first_sums(my_ring + stage * plan.row_bytes, my_y + y_stage * plan.y_bytes, s[0], s[1], y2);
      if (MERGE) s[MERGE ? 2 : 0] = y2;
    }
    if (MERGE) {
      s[MERGE ? 3 : 0] = sum_pair(sqy);
      if (!KNOWN || token) s[sizeof(s) / 4 - 1] = sum_pair(sdz);
    }
    sums(s);
    hh = s[0];
    nh = s[1];
    if (MERGE) {
      yy = s[MERGE ? 2 : 0];
      if (token && tid == 0)
        a.dgate_rows[row] = a.beta * s[sizeof(s) / 4 - 1] * tslope;
      if (post) {
        const float cy = -ry * ry * s[MERGE ? 3 : 0] * inv_d;
        const f32x2 cy2 = pair(cy, cy), ry2 = pair(ry, ry);
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          const int u = tid + i * tpr;
          if (!EXACT && u >= units) continue;
          f32x2 y[U / 2];
          unpack<U>(r_y + u * U, y);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) q[i][j] = mul2(ry2, fma2(y[j], cy2, q[i][j]));
        }
      }
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tid + i * tpr;
        if (EXACT || u < units) pack<U>(a.dy + base + u * U, q[i]);
      }
      if (LATE) fetch_y(row + static_cast<long long>(plan.stages) * workers, y_after);
    }
  }
  // the groups' column sums, added in order through the rings' room where that suffices
  const bool wanted[3] = {next, post, channel};
  if (plan.join) {
    copy_wait<0>();
    __syncthreads();
    float* room = reinterpret_cast<float*>(smem + plan.weight_bytes);
    const int stride = plan.groups * a.d;
    int k = 0;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      if (!wanted[which]) continue;
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int u = tid + i * tpr;
        if (!EXACT && u >= units) continue;
        pack<U>(room + k * stride + group * a.d + u * U, which == 0 ? dw_next[i] : which == 1 ? dw_post[i] : dgate[i]);
      }
      ++k;
    }
    __syncthreads();
    k = 0;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      if (!wanted[which]) continue;
      float* part = a.part + (static_cast<long long>(blockIdx.x) * 3 + which) * a.d;
      for (int c = threadIdx.x * 4; c < a.d; c += blockDim.x * 4) {
        float4 v = *reinterpret_cast<const float4*>(room + k * stride + c);
        for (int g = 1; g < plan.groups; ++g) {
          const float4 p = *reinterpret_cast<const float4*>(room + k * stride + g * a.d + c);
          v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
        }
        *reinterpret_cast<float4*>(part + c) = v;
      }
      ++k;
    }
    return;
  }
  float* part = a.part + static_cast<long long>(worker) * 3 * a.d;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tid + i * tpr;
    if (!EXACT && u >= units) continue;
    if (next) pack<U>(part + u * U, dw_next[i]);
    if (post) pack<U>(part + a.d + u * U, dw_post[i]);
    if (channel) pack<U>(part + 2 * a.d + u * U, dgate[i]);
  }
}

// Column sums of the workers' partial sums, 32 columns a block: 32 threads a column, each
// adding every 32nd worker in order, then the 32 in order.  blockIdx.y picks the sum; a NULL
// output is skipped.  (It is resident while `part` is still being written: plain pointers.)
constexpr int REDUCE_COLS = 32;
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* part, int workers, int d, float* o0, float* o1, float* o2) {
  __shared__ float buf[32][REDUCE_COLS + 1];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  wait_for_previous();
  launch_dependents();
  if (!out) return;
  const int quad = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int c = blockIdx.x * REDUCE_COLS + quad * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < d) {
#pragma unroll 8
    for (int w = grp; w < workers; w += 32) {
      const float4 p = *reinterpret_cast<const float4*>(part + (static_cast<long long>(w) * 3 + blockIdx.y) * d + c);
      s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
    }
  }
  float* b = &buf[grp][quad * 4];
  b[0] = s.x; b[1] = s.y; b[2] = s.z; b[3] = s.w;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int col = warp * 4 + k;
    float v = buf[lane][col];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0 && blockIdx.x * REDUCE_COLS + col < d) out[blockIdx.x * REDUCE_COLS + col] = v;
  }
}

// ------------------------------------------------------------------ launchers

static int row_threads(int d, int cols) { return ((d + cols - 1) / cols + 31) / 32 * 32; }

// The plan for rows of d columns with `cols` a thread and up to max_threads a block; rows[]
// and w[] tell the arrays and weights of the call, may_late whether the kernel has a LATE form.
static NormPlan norm_plan_for(int T, int d, int cols, int stream_size, bool bwd, bool may_late, int max_threads,
                              const bool (&rows)[RING_ARRAYS], const bool (&w)[W_ARRAYS]) {
  NormPlan p{};
  p.cols = cols;
  p.tpr = row_threads(d, cols);
  p.groups = max_threads / p.tpr;
  if (p.tpr > 32 && p.groups > 15) p.groups = 15;  // named barriers 1 .. 15
  const int sms = num_sms() < NORM_MAX_SMS ? num_sms() : NORM_MAX_SMS;
  p.grid = T < sms ? T : sms;
  const int each = (T + p.grid - 1) / p.grid;  // rows of a block
  if (p.groups > each) p.groups = each;
  const int size[RING_ARRAYS] = {stream_size, stream_size, 2, 2};
  for (int i = 0; i < RING_ARRAYS; ++i) {
    const bool apart = bwd && i == RING_Y;
    p.off[i] = rows[i] && !apart ? p.row_bytes : -1;
    if (rows[i]) (apart ? p.y_bytes : p.row_bytes) += d * size[i];
  }
  auto ring = [&](int stages) { return p.groups * (stages * p.row_bytes + (stages + (p.late_y ? 0 : 1)) * p.y_bytes); };
  // groups as far as each has room for two rows (one row fits always: 16384 columns take at
  // most 224 KB), then the weights, then up to four rows a group
  while (p.groups > 1 && ring(2) > NORM_SMEM) --p.groups;
  p.stages = ring(2) <= NORM_SMEM ? 2 : 1;
  int wanted = 0;
  for (int k = 0; k < W_ARRAYS; ++k) wanted += w[k];
  auto places = [&] { return std::min(wanted, (NORM_SMEM - ring(p.stages)) / (d * 4)); };
  if (may_late && p.stages == 2 && places() < wanted) {
    const int before = places();
    p.late_y = true;
    p.late_y = places() > before;
  }
  int left = places();
  p.staged = left == wanted;
  for (int k = 0; k < W_ARRAYS; ++k) {
    p.weight[k] = w[k] && left > 0 ? p.weight_bytes / 4 : -1;
    if (p.weight[k] < 0) continue;
    p.weight_bytes += d * 4;
    --left;
  }
  if (p.late_y) {
    p.smem_bytes = ring(p.stages) + p.weight_bytes;
    p.join = p.groups > 1 && p.groups * (w[W_NEXT] + w[W_POST] + w[W_GATE]) * d * 4 <= ring(p.stages);
    return p;
  }
  while (p.stages > 1 && p.stages < 4 && ring(p.stages + 1) + p.weight_bytes <= NORM_SMEM) ++p.stages;
  p.smem_bytes = ring(p.stages) + p.weight_bytes;
  p.join = bwd && p.groups > 1 && p.groups * (w[W_NEXT] + w[W_POST] + w[W_GATE]) * d * 4 <= ring(p.stages);
  return p;
}

// Columns of a thread: 16 where that fills the block (narrow rows: 8, beyond 8192 columns 32).
static NormPlan norm_fwd_plan(int T, int d, int stream_size, bool merge, const bool (&rows)[RING_ARRAYS], const bool (&w)[W_ARRAYS]) {
  return norm_plan_for(T, d, d <= 256 ? 8 : d <= 8192 ? 16 : 32, stream_size, false, false, norm_fwd_threads(merge), rows, w);
}
// In the backward 8 also where 16 leave most of the block without threads (4472 columns: one
// group of 288) or more groups' rings leave no room for the weights (4096 columns of an fp32
// stream: two groups of 256, weights read from global memory for each row).
static NormPlan norm_bwd_plan(int T, int d, int stream_size, const bool (&rows)[RING_ARRAYS], const bool (&w)[W_ARRAYS]) {
  if (d > 8192) return norm_plan_for(T, d, 32, stream_size, true, false, norm_bwd_threads(32), rows, w);
  const bool known = rows[RING_D] && w[W_NEXT] && w[W_POST];  // the variants that have a LATE form
  const NormPlan wide = norm_plan_for(T, d, 16, stream_size, true, known, norm_bwd_threads(16), rows, w);
  if (row_threads(d, 8) > norm_bwd_threads(8)) return wide;
  if (d > 256 && wide.staged && norm_bwd_threads(16) / wide.tpr * wide.tpr >= 384) return wide;
  const NormPlan narrow = norm_plan_for(T, d, 8, stream_size, true, false, norm_bwd_threads(8), rows, w);
  return wide.staged && !narrow.staged ? wide : narrow;
}

// Whether the KNOWN variants take the call (see the top of the file).
static bool norm_known(const NormPlan& p, const NormArgs& a, bool merge) { return p.cols < 32 && a.w_next && (!merge || a.w_post); }
template <auto KERN>
static cudaError_t launch_rows(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
  const cudaError_t err = allow_smem<KERN>(NORM_SMEM);
  if (err != cudaSuccess) return err;
  return launch_early(KERN, dim3(p.grid), dim3(p.groups * p.tpr), p.smem_bytes, s, a, p);
}

template <typename ST, int COLS, bool MERGE, bool EXACT>
static cudaError_t launch_fwd_known(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
  constexpr int N = COLS * sizeof(ST) / 16, CH = MERGE ? MOE_GATE_CHANNEL : MOE_GATE_NONE, TK = MERGE ? MOE_GATE_TOKEN : MOE_GATE_NONE;
  if (!MERGE || a.gate_kind == MOE_GATE_NONE) return launch_rows<norm_fwd_kernel<ST, N, MERGE, true, EXACT, MOE_GATE_NONE>>(a, p, s);
  if (a.gate_kind == MOE_GATE_TOKEN) return launch_rows<norm_fwd_kernel<ST, N, MERGE, true, EXACT, TK>>(a, p, s);
  return launch_rows<norm_fwd_kernel<ST, N, MERGE, true, EXACT, CH>>(a, p, s);
}

template <typename ST, int COLS, bool MERGE>
static cudaError_t launch_fwd_cols(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
  if (COLS == 16 && norm_known(p, a, MERGE)) {
    constexpr int C = COLS == 16 ? 16 : 8;
    // where one row fills the block (16384 x 7168: 139 us, 164 without); with two groups or
    // more the guarded form is faster (16384 x 4096: 87 us, 95 with)
    constexpr bool EXACT = MERGE && sizeof(ST) == 2 && C == 16;
    return p.staged && a.d == p.tpr * COLS && 2 * p.tpr > norm_fwd_threads(MERGE) ? launch_fwd_known<ST, C, MERGE, EXACT>(a, p, s) : launch_fwd_known<ST, C, MERGE, false>(a, p, s);
  }
  return launch_rows<norm_fwd_kernel<ST, COLS * static_cast<int>(sizeof(ST)) / 16, MERGE, false, false, MOE_GATE_NONE>>(a, p, s);
}

template <typename ST, bool MERGE>
static cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const NormPlan p = norm_fwd_plan(a.T, a.d, sizeof(ST), MERGE, {false, true, false, MERGE},
                                   {a.w_next != nullptr, a.w_post != nullptr, MERGE && a.gate_kind == MOE_GATE_CHANNEL, false});
  return p.cols == 8 ? launch_fwd_cols<ST, 8, MERGE>(a, p, s)
                     : p.cols == 16 ? launch_fwd_cols<ST, 16, MERGE>(a, p, s) : launch_fwd_cols<ST, 32, MERGE>(a, p, s);
}

template <typename ST, int COLS, bool MERGE, bool EXACT, bool LATE>
static cudaError_t launch_bwd_known(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
  constexpr int N = COLS * sizeof(ST) / 16, CH = MERGE ? MOE_GATE_CHANNEL : MOE_GATE_NONE, TK = MERGE ? MOE_GATE_TOKEN : MOE_GATE_NONE;
  constexpr int SL = MERGE ? GATE_SLOPE : MOE_GATE_NONE;
  if (!MERGE || a.gate_kind == MOE_GATE_NONE) return launch_rows<norm_bwd_kernel<ST, N, MERGE, true, EXACT, MOE_GATE_NONE, LATE>>(a, p, s);
  if (a.gate_kind == MOE_GATE_TOKEN) return launch_rows<norm_bwd_kernel<ST, N, MERGE, true, EXACT, TK, LATE>>(a, p, s);
  if (a.gate_sigmoid) return launch_rows<norm_bwd_kernel<ST, N, MERGE, true, EXACT, SL, LATE>>(a, p, s);
  return launch_rows<norm_bwd_kernel<ST, N, MERGE, true, EXACT, CH, LATE>>(a, p, s);
}

template <typename ST, int COLS, bool MERGE>
static cudaError_t launch_bwd_cols(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
  if (COLS < 32 && norm_known(p, a, MERGE) && a.d_stream) {
    constexpr int C = COLS < 32 ? COLS : 16;
    // (16384 x 7168 bf16 with a channel gate: 222 us, 276 without.  Not for an fp32 stream and 8
    // columns, where it spills; the form for a sigmoid channel gate spills 28 bytes in the row loop:
    // 369 us)
    constexpr bool EXACT = sizeof(ST) == 2 && C == 16, LATE = MERGE && C == 16;
    const bool exact = p.staged && a.d == p.tpr * COLS;
    if (p.late_y) return exact ? launch_bwd_known<ST, C, MERGE, EXACT, LATE>(a, p, s) : launch_bwd_known<ST, C, MERGE, false, LATE>(a, p, s);
    return exact ? launch_bwd_known<ST, C, MERGE, EXACT, false>(a, p, s) : launch_bwd_known<ST, C, MERGE, false, false>(a, p, s);
  }
  return launch_rows<norm_bwd_kernel<ST, COLS * static_cast<int>(sizeof(ST)) / 16, MERGE, false, false, MOE_GATE_NONE, false>>(a, p, s);
}

template <typename ST, bool MERGE>
static cudaError_t launch_norm_bwd(const NormArgs& a, float* dw_next, float* dw_post, float* dgate_cols, cudaStream_t s) {
  const bool next = a.w_next, post = MERGE && a.w_post, channel = MERGE && a.gate_kind == MOE_GATE_CHANNEL;
  int workers = 0;
  if (a.T > 0) {
    const NormPlan p = norm_bwd_plan(a.T, a.d, sizeof(ST),
                                     {a.d_stream != nullptr, next, next, post || (MERGE && a.gate_kind != MOE_GATE_NONE)},
                                     {next, post, channel, channel && a.gate_sigmoid});
    workers = p.join ? p.grid : p.grid * p.groups;
    const cudaError_t err = p.cols == 8 ? launch_bwd_cols<ST, 8, MERGE>(a, p, s)
                                        : p.cols == 16 ? launch_bwd_cols<ST, 16, MERGE>(a, p, s) : launch_bwd_cols<ST, 32, MERGE>(a, p, s);
    if (err != cudaSuccess) return err;
  }
  if (dw_next || dw_post || dgate_cols) {
    return launch_early(norm_reduce_kernel, dim3((a.d + REDUCE_COLS - 1) / REDUCE_COLS, 3), dim3(256), 0, s,
                        static_cast<const float*>(a.part), workers, a.d, dw_next, dw_post, dgate_cols);
  }
  return cudaSuccess;
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
  // blocks times the most groups of a block, as if none added their sums in the block
  const int d = dims->d, most = std::max({1, norm_bwd_threads(8) / row_threads(d, 8), norm_bwd_threads(16) / row_threads(d, 16)});
  return static_cast<size_t>(NORM_MAX_SMS) * most * 3 * d * sizeof(float);
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
