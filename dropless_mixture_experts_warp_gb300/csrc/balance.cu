// Balance loss of the router over ragged sequences, per-expert counts, the z-loss, and
// their gradient by the logits.
#include "around.cuh"

namespace moe {

constexpr int BAL_MAX_E = 1024;
constexpr int BAL_MAX_S = 65535;
constexpr int BAL_CHUNK = 128;  // tokens of a forward block
constexpr int BAL_WARPS = 8;

struct BalanceArgs {
  int T, E, k, S;
  float coef, z_coef;
  const float* logits;
  const int32_t* topk_idx;
  const int32_t* seq_offsets;  // NULL: one sequence of T tokens
  const uint8_t* mask;
  // forward
  float* losses;
  int32_t* counts;
  float* prob_mean;
  int32_t* seq_tokens;
  int32_t* status;
  // partial sums of the part of a sequence that lies in a chunk: slot chunk + sequence
  // (along the tokens either number grows, so no two parts share a slot)
  float* part_p;       // [slots][E]
  int32_t* part_c;     // [slots][E]
  float* part_z;       // [slots] sums of logsumexp^2
  int32_t* part_n;     // [slots] kept tokens
  float* seq_loss;     // [S][2] a sequence's sum f P and sum logsumexp^2
  int32_t* counter;
  // backward
  const int32_t* counts_in;
  const int32_t* tokens_in;
  const float* grad_losses;
  int accumulate;
  float* d_logits;
};

// Start of sequence s, whatever the array holds inside [0, T].
__device__ __forceinline__ int seq_at(const BalanceArgs& a, int s) {
  if (!a.seq_offsets) return s == 0 ? 0 : a.T;
  return min(max(a.seq_offsets[s], 0), a.T);
}

// The last sequence that starts at or before token t (0 if none does).
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int t) {
  int lo = 0, hi = a.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_at(a, mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A row of E logits over the lanes of a warp: expert lane + 32 c in slot c.
template <int PL>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&l)[PL]) {
#pragma unroll
  for (int c = 0; c < PL; ++c) l[c] = lane + 32 * c < E ? row[lane + 32 * c] : -INFINITY;
}

// The row's largest logit.
template <int PL>
__device__ __forceinline__ float row_top(const float (&l)[PL]) {
  float top = l[0];
#pragma unroll
  for (int c = 1; c < PL; ++c) top = fmaxf(top, l[c]);
  return warp_max(top);
}

// Softmax of the row and its logsumexp; p = 0 and lse = 0 for a row of -inf.
template <int PL>
__device__ __forceinline__ void row_softmax(const float (&l)[PL], float top, float (&p)[PL], float& lse) {
  if (top == -INFINITY) top = 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < PL; ++c) {
    p[c] = expf(l[c] - top);
    sum += p[c];
  }
  sum = warp_sum(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int c = 0; c < PL; ++c) p[c] *= inv;
  lse = sum == 0.0f ? 0.0f : top + logf(sum);
}

// p = sigmoid(l) / sum, each sigmoid taken times e^-c with c = min(top, 0): 1 / (e^c +
// e^(c - l)).  The largest is then at least 1/2, so that a row of far negative logits,
// whose sigmoids fp32 cannot hold, keeps its shares.  p = 0 for a row of -inf.
template <int PL>
__device__ __forceinline__ void row_sigmoid(const float (&l)[PL], float top, float (&p)[PL]) {
  const float c0 = top == -INFINITY ? 0.0f : fminf(top, 0.0f);
  const float ec = expf(c0);
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < PL; ++c) {
    p[c] = 1.0f / (ec + expf(c0 - l[c]));
    sum += p[c];
  }
  sum = warp_sum(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int c = 0; c < PL; ++c) p[c] *= inv;
}

// A block takes a chunk of tokens, sequence by sequence: its warps take the tokens in
// turn and keep the sums of p in registers; the counts are integer sums in shared memory.
template <int PL, bool SIGMOID>
__global__ void __launch_bounds__(BAL_WARPS * 32) balance_fwd_kernel(const BalanceArgs a) {
  __shared__ float s_p[BAL_WARPS][PL * 32];
  __shared__ int s_c[PL * 32];
  __shared__ float s_z[BAL_WARPS];
  __shared__ int s_n[BAL_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x * BAL_CHUNK, c1 = min(a.T, c0 + BAL_CHUNK);
  for (int s = seq_of(a, c0); s < a.S; ++s) {
    const int b = max(c0, seq_at(a, s)), e = min(c1, seq_at(a, s + 1));
    if (seq_at(a, s) >= c1) break;
    if (b >= e) continue;
    for (int i = threadIdx.x; i < PL * 32; i += blockDim.x) s_c[i] = 0;
    __syncthreads();
    float acc[PL], z = 0.0f;
    int n = 0;
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] = 0.0f;
    for (int t = b + warp; t < e; t += BAL_WARPS) {
      if (a.mask && !a.mask[t]) continue;
      ++n;
      float l[PL], p[PL], lse = 0.0f;
      load_row(a.logits + static_cast<long long>(t) * a.E, a.E, lane, l);
      const float top = row_top(l);
      if (!SIGMOID || a.z_coef != 0.0f) row_softmax(l, top, p, lse);
      if (SIGMOID) row_sigmoid(l, top, p);
      if (a.z_coef != 0.0f) z = fmaf(lse, lse, z);
#pragma unroll
      for (int c = 0; c < PL; ++c) acc[c] += p[c];
      if (lane < a.k) {
        const int x = a.topk_idx[static_cast<long long>(t) * a.k + lane];
        if (x >= 0 && x < a.E) atomicAdd(&s_c[x], 1);
        else set_status(a.status, MOE_ERR_INVARIANT);
      }
    }
#pragma unroll
    for (int c = 0; c < PL; ++c) s_p[warp][lane + 32 * c] = acc[c];
    if (lane == 0) {
      s_z[warp] = z;
      s_n[warp] = n;
    }
    __syncthreads();
    const long long slot = blockIdx.x + s;
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < BAL_WARPS; ++w) v += s_p[w][i];
      a.part_p[slot * a.E + i] = v;
      a.part_c[slot * a.E + i] = s_c[i];
    }
    if (threadIdx.x == 0) {
      float zs = 0.0f;
      int ns = 0;
      for (int w = 0; w < BAL_WARPS; ++w) {
        zs += s_z[w];
        ns += s_n[w];
      }
      a.part_z[slot] = zs;
      a.part_n[slot] = ns;
    }
    __syncthreads();
  }
}

// A block per sequence adds its parts in token order; the last block to finish turns the
// sequences' sums into the losses, in sequence order.
__global__ void __launch_bounds__(256) balance_join_kernel(const BalanceArgs a) {
  __shared__ float buf[32 * 2];
  __shared__ int s_last;
  const int s = blockIdx.x;
  const int b = seq_at(a, s), e = seq_at(a, s + 1);
  if (threadIdx.x == 0 && a.seq_offsets) {
    const int x = a.seq_offsets[s], y = a.seq_offsets[s + 1];
    if (x > y || (s == 0 && x != 0) || (s == a.S - 1 && y != a.T)) set_status(a.status, MOE_ERR_INVARIANT);
  }
  int first = 0, last = -1;  // slots
  if (b < e) {
    first = b / BAL_CHUNK + s;
    last = (e - 1) / BAL_CHUNK + s;
  }
  int n = 0;
  float z = 0.0f;
  for (int i = first; i <= last; ++i) {
    n += a.part_n[i];
    z += a.part_z[i];
  }
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  const float fs = inv_n * static_cast<float>(a.E) / static_cast<float>(a.k);
  float sum[1] = {0.0f};
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
    float p = 0.0f;
    int c = 0;
    for (int j = first; j <= last; ++j) {
      p += a.part_p[static_cast<long long>(j) * a.E + i];
      c += a.part_c[static_cast<long long>(j) * a.E + i];
    }
    a.counts[static_cast<long long>(s) * a.E + i] = c;
    a.prob_mean[static_cast<long long>(s) * a.E + i] = p * inv_n;
    sum[0] = fmaf(static_cast<float>(c) * fs, p * inv_n, sum[0]);
  }
  row_sums<false, 1>(sum, buf);
  if (threadIdx.x == 0) {
    a.seq_tokens[s] = n;
    a.seq_loss[2 * s] = sum[0];
    a.seq_loss[2 * s + 1] = z;
    __threadfence();
    s_last = atomicAdd(a.counter, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // losses, sequences and tokens that count
  __shared__ float buf4[32 * 4];
  for (int i = threadIdx.x; i < a.S; i += blockDim.x) {
    const int c = __ldcg(&a.seq_tokens[i]);
    t[0] += __ldcg(&a.seq_loss[2 * i]);
    t[1] += __ldcg(&a.seq_loss[2 * i + 1]);
    t[2] += c > 0 ? 1.0f : 0.0f;
    t[3] += static_cast<float>(c);
  }
  row_sums<false, 4>(t, buf4);
  if (threadIdx.x == 0) {
    a.losses[0] = t[2] > 0.0f ? a.coef * t[0] / t[2] : 0.0f;
    a.losses[1] = t[3] > 0.0f ? a.z_coef * t[1] / t[3] : 0.0f;
  }
}

// A warp takes a run of consecutive tokens.  dl_j = g0 coef / (S' n_s) p_j (f_j - sum f p)
// [(1 - sigmoid(l_j)) for sigmoid scores] + g1 z_coef 2 / N lse softmax(l)_j.
template <int PL, bool SIGMOID>
__global__ void __launch_bounds__(256) balance_bwd_kernel(const BalanceArgs a, int run) {
  __shared__ float buf[32 * 2];
  const int lane = threadIdx.x & 31;
  float tot[2] = {0.0f, 0.0f};  // sequences and tokens that count
  for (int i = threadIdx.x; i < a.S; i += blockDim.x) {
    const int c = a.tokens_in[i];
    tot[0] += c > 0 ? 1.0f : 0.0f;
    tot[1] += static_cast<float>(c);
  }
  row_sums<false, 2>(tot, buf);
  const float g0 = (a.grad_losses ? a.grad_losses[0] : 1.0f) * a.coef / fmaxf(tot[0], 1.0f);
  const float g1 = (a.grad_losses ? a.grad_losses[1] : 1.0f) * a.z_coef * 2.0f / fmaxf(tot[1], 1.0f);
  const long long t0 = (static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * run;
  if (t0 >= a.T) return;
  const int t1 = static_cast<int>(min(static_cast<long long>(a.T), t0 + run));
  int s = seq_of(a, static_cast<int>(t0));
  int end = -1;
  float f[PL], gs = 0.0f;
  for (int t = static_cast<int>(t0); t < t1; ++t) {
    if (t >= end) {  // first token of the run, or of a sequence
      while (s + 1 < a.S && seq_at(a, s + 1) <= t) ++s;
      end = s + 1 < a.S ? seq_at(a, s + 1) : a.T;
      const int n = a.tokens_in[s];
      const float inv = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
      gs = g0 * inv;
      const float fs = inv * static_cast<float>(a.E) / static_cast<float>(a.k);
#pragma unroll
      for (int c = 0; c < PL; ++c)
        f[c] = lane + 32 * c < a.E ? static_cast<float>(a.counts_in[static_cast<long long>(s) * a.E + lane + 32 * c]) * fs : 0.0f;
    }
    float* out = a.d_logits + static_cast<long long>(t) * a.E;
    if (a.mask && !a.mask[t]) {
      if (!a.accumulate)
        for (int i = lane; i < a.E; i += 32) out[i] = 0.0f;
      continue;
    }
    float l[PL], p[PL], q[PL], lse = 0.0f;
    load_row(a.logits + static_cast<long long>(t) * a.E, a.E, lane, l);
    const float top = row_top(l);
    if (!SIGMOID || a.z_coef != 0.0f) row_softmax(l, top, q, lse);
    else
#pragma unroll
      for (int c = 0; c < PL; ++c) q[c] = 0.0f;
    if (SIGMOID) row_sigmoid(l, top, p);
    else
#pragma unroll
      for (int c = 0; c < PL; ++c) p[c] = q[c];
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < PL; ++c) m = fmaf(f[c], p[c], m);
    m = warp_sum(m);
#pragma unroll
    for (int c = 0; c < PL; ++c) {
      const int i = lane + 32 * c;
      if (i >= a.E) continue;
      float d = gs * p[c] * (f[c] - m);
      if (SIGMOID) d *= 1.0f / (1.0f + expf(l[c]));
      d = fmaf(g1 * lse, q[c], d);
      out[i] = a.accumulate ? out[i] + d : d;
    }
  }
}

// ------------------------------------------------------------------ launchers

static size_t al256(size_t x) { return (x + 255) / 256 * 256; }

static long long balance_slots(const moe_balance_dims& m) {
  return (static_cast<long long>(m.T) + BAL_CHUNK - 1) / BAL_CHUNK + m.S;
}

static size_t balance_carve(const moe_balance_dims& m, void* ws, BalanceArgs* a) {
  const size_t slots = balance_slots(m);
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = p + at;
    at += al256(bytes);
    return r;
  };
  uint8_t* counter = take(4);
  uint8_t* pp = take(slots * m.E * 4);
  uint8_t* pc = take(slots * m.E * 4);
  uint8_t* pz = take(slots * 4);
  uint8_t* pn = take(slots * 4);
  uint8_t* sl = take(static_cast<size_t>(m.S) * 8);
  if (a) {
    a->counter = reinterpret_cast<int32_t*>(counter);
    a->part_p = reinterpret_cast<float*>(pp);
    a->part_c = reinterpret_cast<int32_t*>(pc);
    a->part_z = reinterpret_cast<float*>(pz);
    a->part_n = reinterpret_cast<int32_t*>(pn);
    a->seq_loss = reinterpret_cast<float*>(sl);
  }
  return at;
}

static BalanceArgs balance_args(const moe_balance_dims& m) {
  BalanceArgs a{};
  a.T = m.T; a.E = m.E; a.k = m.k; a.S = m.S; a.coef = m.coef; a.z_coef = m.z_coef;
  return a;
}

template <int PL>
static void launch_fwd(const BalanceArgs& a, bool sigmoid, int grid, cudaStream_t s) {
  if (sigmoid) balance_fwd_kernel<PL, true><<<grid, BAL_WARPS * 32, 0, s>>>(a);
  else balance_fwd_kernel<PL, false><<<grid, BAL_WARPS * 32, 0, s>>>(a);
}
template <int PL>
static void launch_bwd(const BalanceArgs& a, bool sigmoid, int grid, int run, cudaStream_t s) {
  if (sigmoid) balance_bwd_kernel<PL, true><<<grid, 256, 0, s>>>(a, run);
  else balance_bwd_kernel<PL, false><<<grid, 256, 0, s>>>(a, run);
}

static cudaError_t launch_balance_fwd(const BalanceArgs& a, bool sigmoid, cudaStream_t s) {
  cudaError_t err = cudaMemsetAsync(a.counter, 0, 4, s);
  if (err != cudaSuccess) return err;
  if (a.T > 0) {
    const int grid = (a.T + BAL_CHUNK - 1) / BAL_CHUNK;
    if (a.E <= 32) launch_fwd<1>(a, sigmoid, grid, s);
    else if (a.E <= 64) launch_fwd<2>(a, sigmoid, grid, s);
    else if (a.E <= 128) launch_fwd<4>(a, sigmoid, grid, s);
    else if (a.E <= 256) launch_fwd<8>(a, sigmoid, grid, s);
    else if (a.E <= 512) launch_fwd<16>(a, sigmoid, grid, s);
    else launch_fwd<32>(a, sigmoid, grid, s);
    count_launch();
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  balance_join_kernel<<<a.S, 256, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

static cudaError_t launch_balance_bwd(const BalanceArgs& a, bool sigmoid, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const long long warps = static_cast<long long>(num_sms()) * 32;
  const int run = static_cast<int>((a.T + warps - 1) / warps);
  const int grid = static_cast<int>((a.T + 8ll * run - 1) / (8ll * run));
  if (a.E <= 32) launch_bwd<1>(a, sigmoid, grid, run, s);
  else if (a.E <= 64) launch_bwd<2>(a, sigmoid, grid, run, s);
  else if (a.E <= 128) launch_bwd<4>(a, sigmoid, grid, run, s);
  else if (a.E <= 256) launch_bwd<8>(a, sigmoid, grid, run, s);
  else if (a.E <= 512) launch_bwd<16>(a, sigmoid, grid, run, s);
  else launch_bwd<32>(a, sigmoid, grid, run, s);
  count_launch();
  return cudaGetLastError();
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_balance_check_dims(const moe_balance_dims* dims) {
  if (!dims) return MOE_ERR_INVALID_ARG;
  const moe_balance_dims& m = *dims;
  if (m.T < 0 || m.E <= 0 || m.k <= 0 || m.k > m.E || m.k > 32 || m.S <= 0) return MOE_ERR_INVALID_ARG;
  if (m.score != MOE_SCORE_SOFTMAX && m.score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!isfinite(m.coef) || !isfinite(m.z_coef)) return MOE_ERR_INVALID_ARG;
  if (m.E > BAL_MAX_E || m.S > BAL_MAX_S) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t moe_balance_workspace_size(const moe_balance_dims* dims) {
  if (moe_balance_check_dims(dims) != MOE_OK) return 0;
  return balance_carve(*dims, nullptr, nullptr);
}

moe_status moe_balance_fwd(const moe_balance_dims* dims, const float* logits, const int32_t* topk_idx,
                           const int32_t* seq_offsets, const uint8_t* mask, float* losses, int32_t* counts,
                           float* prob_mean, int32_t* seq_tokens, void* workspace, int32_t* dev_status,
                           void* stream) {
  const moe_status st = moe_balance_check_dims(dims);
  if (st != MOE_OK) return st;
  if (!losses || !counts || !prob_mean || !seq_tokens || !dev_status) return MOE_ERR_INVALID_ARG;
  if (dims->T > 0 && (!logits || !topk_idx)) return MOE_ERR_INVALID_ARG;
  if (dims->S > 1 && !seq_offsets) return MOE_ERR_INVALID_ARG;
  if (!workspace) return MOE_ERR_WORKSPACE;
  const void* every[] = {logits, topk_idx, losses, counts, prob_mean, seq_tokens, workspace};
  for (const void* p : every)
    if (!ptr_aligned16(p)) return MOE_ERR_ALIGNMENT;
  BalanceArgs a = balance_args(*dims);
  balance_carve(*dims, workspace, &a);
  a.logits = logits; a.topk_idx = topk_idx; a.seq_offsets = seq_offsets; a.mask = mask; a.losses = losses;
  a.counts = counts; a.prob_mean = prob_mean; a.seq_tokens = seq_tokens; a.status = dev_status;
  return status_of(launch_balance_fwd(a, dims->score == MOE_SCORE_SIGMOID, static_cast<cudaStream_t>(stream)));
}

moe_status moe_balance_bwd(const moe_balance_dims* dims, const float* logits, const int32_t* seq_offsets,
                           const uint8_t* mask, const int32_t* counts, const int32_t* seq_tokens,
                           const float* grad_losses, int32_t accumulate, float* d_logits, void* stream) {
  const moe_status st = moe_balance_check_dims(dims);
  if (st != MOE_OK) return st;
  if (!counts || !seq_tokens || (dims->T > 0 && (!logits || !d_logits))) return MOE_ERR_INVALID_ARG;
  if (dims->S > 1 && !seq_offsets) return MOE_ERR_INVALID_ARG;
  if (!ptr_aligned16(logits) || !ptr_aligned16(counts) || !ptr_aligned16(seq_tokens) || !ptr_aligned16(d_logits))
    return MOE_ERR_ALIGNMENT;
  BalanceArgs a = balance_args(*dims);
  a.logits = logits; a.seq_offsets = seq_offsets; a.mask = mask; a.counts_in = counts; a.tokens_in = seq_tokens;
  a.grad_losses = grad_losses; a.accumulate = accumulate; a.d_logits = d_logits;
  return status_of(launch_balance_bwd(a, dims->score == MOE_SCORE_SIGMOID, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
