// Balance loss of the router over ragged sequences, per-expert counts, the z-loss, and
// their gradient by the logits.
//
// A token's E logits lie over the G lanes of a group, PLV vectors of VEC a lane (16 logits a
// lane up to 512 experts: a token's sums then take few shuffles a logit, and a warp has
// several tokens under way; 30001 x 131 over all 32 lanes: 29 us, over 16: 16 us).
// Exponentials are 2^x of the scaled argument; its difference, its product and log2(e) are each
// rounded, so their relative error is at most |l - c| 2^-22.8 + 2^-22.  Softmax: c is the row's
// maximum, and the arguments lie at or below 0.  Sigmoid scores: e^(c - l) with c the smaller
// of the maximum and 0; in a row without a positive logit the arguments lie at or above 0, and
// one that overflows makes the share 0.
//
// Measured (GB300, in a graph): losses of 393215 x 128, 43 us (5.0 TB/s), with sigmoid scores and
// the z-loss 49 us (three special functions a logit), of 16384 x 256 13 us (bound by the chain
// of dependent reads through two kernels); gradients 10.5 us for the latter, 96 us for 393216 x
// 128 softmax (6.28 TB/s, the rate of memory), 100 us with sigmoid scores.
#include "around.cuh"

namespace moe {

constexpr int BAL_MAX_E = 1024;
constexpr int BAL_MAX_S = 65535;
constexpr int BAL_MAX_T = 1 << 30;
constexpr int BAL_THREADS = 256;
constexpr int JOIN_COLS = 32;  // experts of a join block

struct BalanceArgs {
  int T, E, k, S;
  float coef, z_coef;
  const float* logits;
  const int32_t* topk_idx;
  const int32_t* seq_offsets;  // NULL: one sequence of T tokens
  const uint8_t* mask;
  // forward
  int chunk;           // tokens of a block
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
  float* seq_loss;     // [S][join blocks a sequence] sums f P
  float* seq_z;        // [S] sums of logsumexp^2
  int32_t* counter;
  // backward
  int run;             // tokens of a group
  const int32_t* counts_in;
  const int32_t* tokens_in;
  const float* grad_losses;
  int accumulate;
  float* d_logits;
};

// Starts of the sequences, whatever the array holds inside [0, T]; up to SEQ_TABLE of them
// are read into shared memory at once, so that a search does not wait for memory at each step.
constexpr int SEQ_TABLE = 512;
struct Sequences {
  const int32_t* offsets;
  int T, S;
  const int* table;
  // The caller synchronises the block before the first use.
  __device__ __forceinline__ Sequences(const BalanceArgs& a, int* shared)
      : offsets(a.seq_offsets), T(a.T), S(a.S), table(a.seq_offsets && a.S <= SEQ_TABLE ? shared : nullptr) {
    if (table)
      for (int i = threadIdx.x; i <= S; i += blockDim.x) shared[i] = min(max(offsets[i], 0), T);
  }
  __device__ __forceinline__ int at(int s) const {
    if (table) return table[s];
    if (!offsets) return s == 0 ? 0 : T;
    return min(max(offsets[s], 0), T);
  }
  // The last sequence that starts at or before token t (0 if none does).
  __device__ __forceinline__ int of(int t) const {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (at(mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A lane's logits (or other [T][E] values) of one token, in pairs; `fill` where the row ends,
// and everywhere where `there` is false.
template <int VEC, int G, int PLV>
__device__ __forceinline__ void load_row(const float* row, int E, int gl, bool there, float fill, f32x2 (&l)[VEC * PLV / 2]) {
  if (VEC == 4) {
#pragma unroll
    for (int i = 0; i < PLV; ++i) {
      const int e = (gl + G * i) * VEC;
      float4 q = make_float4(fill, fill, fill, fill);
      if (there && e < E) q = *reinterpret_cast<const float4*>(row + e);
      l[VEC / 2 * i] = pair(q.x, q.y);
      l[VEC / 2 * i + VEC / 4] = pair(q.z, q.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PLV; i += 2) {
      const int e = gl + G * i;
      l[i / 2] = pair(there && e < E ? row[e] : fill, there && e + G < E ? row[e + G] : fill);
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The row's largest logit.
template <int G, int M>
__device__ __forceinline__ float row_top(const f32x2 (&l)[M]) {
  const float2 f = unpair(l[0]);
  float top = fmaxf(f.x, f.y);
#pragma unroll
  for (int c = 1; c < M; ++c) {
    const float2 v = unpair(l[c]);
    top = max3(top, v.x, v.y);
  }
  return group_max<G>(top);
}

// Softmax of the row, not yet divided by its sum, the sum's inverse and the logsumexp; all 0
// for a row of -inf.  (A NaN reaches the sum through its own exponential.)
template <int G, int M>
__device__ __forceinline__ void row_softmax(const f32x2 (&l)[M], float top, bool with_lse, f32x2 (&p)[M], float& inv, float& lse) {
  if (top == -INFINITY) top = 0.0f;
  f32x2 sums = pair(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < M; ++c) {
    // the difference first: logits near fp32's lowest
    const float2 x = unpair(mul2(add2(l[c], pair(-top, -top)), pair(LOG2E, LOG2E)));
    p[c] = pair(exp2_fast(x.x), exp2_fast(x.y));
    sums = add2(sums, p[c]);
  }
  const float sum = group_sum<G>(sum_pair(sums));
  inv = sum == 0.0f ? 0.0f : rcp_fast(sum);
  lse = with_lse && sum != 0.0f ? top + logf(sum) : 0.0f;
}

// p = sigmoid(l), each taken times e^-c with c = min(top, 0): 1 / (e^c + e^(c - l)), and the
// inverse of their sum.  The largest is then at least 1/2, so that a row of far negative
// logits, whose sigmoids fp32 cannot hold, keeps its shares; the inverse is 0 for a row of
// -inf.  rest = 1 - sigmoid(l) = e^(c - l) p, without the cancellation of the difference.
template <int G, int M>
__device__ __forceinline__ void row_sigmoid(const f32x2 (&l)[M], float top, f32x2 (&p)[M], float& inv, f32x2 (*rest)[M]) {
  const float c0 = top == -INFINITY ? 0.0f : fminf(top, 0.0f);
  const float ec = exp2_fast(c0 * LOG2E);
  f32x2 sums = pair(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < M; ++c) {
    const float2 x = unpair(mul2(fma2(l[c], pair(-1.0f, -1.0f), pair(c0, c0)), pair(LOG2E, LOG2E)));
    const f32x2 e = pair(exp2_fast(x.x), exp2_fast(x.y));
    const float2 den = unpair(add2(e, pair(ec, ec)));
    p[c] = pair(rcp_fast(den.x), rcp_fast(den.y));
    sums = add2(sums, p[c]);
    if (rest) {
      const float2 q = unpair(mul2(e, p[c]));
      (*rest)[c] = pair(fminf(q.x, 1.0f), fminf(q.y, 1.0f));  // inf * 0 where l is far below the top: 1
    }
  }
  const float sum = group_sum<G>(sum_pair(sums));
  inv = sum == 0.0f ? 0.0f : rcp_fast(sum);
}

// Blocks of the forward that an SM holds, by their registers (393215 x 128 with two: 55 us, with
// three 41 us).
constexpr int balance_fwd_blocks(int vec, int lanes, int E) { return E > 512 ? 1 : vec == 4 && lanes >= 8 ? 3 : 2; }

// A block takes a chunk of tokens, sequence by sequence: its groups take the tokens in turn
// and keep the sums of p in registers; the counts are integer sums in shared memory.  A
// single block with a single sequence writes the results itself.
template <int VEC, int G, int PLV, bool SIGMOID>
__global__ void __launch_bounds__(BAL_THREADS, balance_fwd_blocks(VEC, G, VEC * PLV * G)) balance_fwd_kernel(const BalanceArgs a) {
  constexpr int N = VEC * PLV, M = N / 2, GROUPS = BAL_THREADS / G, WARP_COLS = N * G;
  constexpr int C = G < 8 ? 8 / G : 1;  // choices of a lane that are read ahead
  __shared__ float s_p[BAL_THREADS / 32][WARP_COLS];
  __shared__ int s_c[WARP_COLS];
  __shared__ float s_z[BAL_THREADS / 32];
  __shared__ int s_n[BAL_THREADS / 32];
  __shared__ float buf[32];
  __shared__ int s_off[SEQ_TABLE + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % G, group = threadIdx.x / G;
  const int c0 = blockIdx.x * a.chunk, c1 = min(a.T, c0 + a.chunk);
  wait_for_previous();
  launch_dependents();
  // The chunk's first tokens are on their way before their sequences are known.  A token's
  // mask is read two tokens ahead, its logits and its first C choices a lane one ahead (one
  // choice a lane: 11.5 us for 88517 x 16, 7 choices; so 8.7 us).
  auto kept = [&](int t, int e) { return t < e && (!a.mask || a.mask[t]); };
  auto choices = [&](int t, bool there, int (&x)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = there && gl + G * i < a.k ? a.topk_idx[static_cast<long long>(t) * a.k + gl + G * i] : -1;
  };
  auto count = [&](int x) {
    if (x >= 0 && x < a.E) atomicAdd(&s_c[x], 1);
    else set_status(a.status, MOE_ERR_INVARIANT);
  };
  int t = c0 + group, x[C];
  bool keep = kept(t, c1), keep_next = kept(t + GROUPS, c1);
  f32x2 l[M];
  load_row<VEC, G, PLV>(a.logits + static_cast<long long>(t) * a.E, a.E, gl, t < c1, -INFINITY, l);
  choices(t, t < c1, x);
  const Sequences seqs(a, s_off);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0;  // of the join's blocks
  __syncthreads();
  bool fresh = true;
  for (int s = seqs.of(c0); s < a.S; ++s) {
    const int start = seqs.at(s);
    if (start >= c1) break;
    const int b = max(c0, start), e = min(c1, seqs.at(s + 1));
    if (b >= e) continue;
    for (int i = threadIdx.x; i < WARP_COLS; i += BAL_THREADS) s_c[i] = 0;
    if (fresh && b == c0) {  // what was read above is this part's, as far as that goes
      keep = keep && t < e;
      keep_next = keep_next && t + GROUPS < e;
    } else {
      t = b + group;
      keep = kept(t, e);
      keep_next = kept(t + GROUPS, e);
      load_row<VEC, G, PLV>(a.logits + static_cast<long long>(t) * a.E, a.E, gl, keep, -INFINITY, l);
      choices(t, keep, x);
    }
    fresh = false;
    if (!keep) {
#pragma unroll
      for (int c = 0; c < M; ++c) l[c] = pair(-INFINITY, -INFINITY);
    }
    f32x2 acc2[M];
    float z = 0.0f;
    int n = 0;
#pragma unroll
    for (int c = 0; c < M; ++c) acc2[c] = pair(0.0f, 0.0f);
    __syncthreads();
    for (int done = b; done < e; done += GROUPS) {  // a token of every group
      const int tn = t + GROUPS;
      const bool keep_after = kept(tn + GROUPS, e);
      f32x2 next[M];
      load_row<VEC, G, PLV>(a.logits + static_cast<long long>(tn) * a.E, a.E, gl, keep_next, -INFINITY, next);
      int x_next[C];
      choices(tn, keep_next, x_next);
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (keep && gl + G * i < a.k) count(x[i]);
      for (int j = gl + G * C; keep && j < a.k; j += G) count(a.topk_idx[static_cast<long long>(t) * a.k + j]);
      __syncwarp();
      f32x2 p[M];
      float inv, lse = 0.0f;
      const float top = row_top<G>(l);
      if (!SIGMOID || a.z_coef != 0.0f) row_softmax<G>(l, top, a.z_coef != 0.0f, p, inv, lse);
      if (SIGMOID) row_sigmoid<G>(l, top, p, inv, static_cast<f32x2 (*)[M]>(nullptr));
      z = fmaf(lse, lse, z);
      n += keep;
#pragma unroll
      for (int c = 0; c < M; ++c) {
        acc2[c] = fma2(p[c], pair(inv, inv), acc2[c]);
        l[c] = next[c];
      }
#pragma unroll
      for (int i = 0; i < C; ++i) x[i] = x_next[i];
      t = tn;
      keep = keep_next;
      keep_next = keep_after;
    }
    float acc[N];
#pragma unroll
    for (int c = 0; c < M; ++c) {
      const float2 f = unpair(acc2[c]);
      acc[2 * c] = f.x;
      acc[2 * c + 1] = f.y;
    }
    // the warp's groups, then the block's warps, in order
#pragma unroll
    for (int off = G; off < 32; off <<= 1) {
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], off);
      z += __shfl_xor_sync(0xffffffffu, z, off);
      n += __shfl_xor_sync(0xffffffffu, n, off);
    }
    if (lane < G) {
#pragma unroll
      for (int c = 0; c < N; ++c) s_p[warp][(gl + G * (c / VEC)) * VEC + c % VEC] = acc[c];
    }
    if (lane == 0) {
      s_z[warp] = z;
      s_n[warp] = n;
    }
    __syncthreads();
    float zs = 0.0f;
    int ns = 0;
#pragma unroll
    for (int w = 0; w < BAL_THREADS / 32; ++w) {
      zs += s_z[w];
      ns += s_n[w];
    }
    const bool whole = gridDim.x == 1 && a.S == 1;
    const float inv_n = ns > 0 ? 1.0f / static_cast<float>(ns) : 0.0f;
    const float fs = inv_n * static_cast<float>(a.E) / static_cast<float>(a.k);
    const long long slot = blockIdx.x + s;
    float sum[1] = {0.0f};
    for (int i = threadIdx.x; i < a.E; i += BAL_THREADS) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < BAL_THREADS / 32; ++w) v += s_p[w][i];
      if (whole) {
        a.counts[i] = s_c[i];
        a.prob_mean[i] = v * inv_n;
        sum[0] = fmaf(static_cast<float>(s_c[i]) * fs, v * inv_n, sum[0]);
      } else {
        a.part_p[slot * a.E + i] = v;
        a.part_c[slot * a.E + i] = s_c[i];
      }
    }
    if (whole) row_sums<false, 1>(sum, buf);
    if (threadIdx.x == 0) {
      if (whole) {
        a.seq_tokens[0] = ns;
        a.losses[0] = a.coef * sum[0];
        a.losses[1] = a.z_coef * zs * inv_n;
      } else {
        a.part_z[slot] = zs;
        a.part_n[slot] = ns;
      }
    }
    __syncthreads();
  }
  if (gridDim.x == 1 && a.S == 1 && a.seq_offsets && threadIdx.x == 0 && (a.seq_offsets[0] != 0 || a.seq_offsets[1] != a.T))
    set_status(a.status, MOE_ERR_INVARIANT);
}

// Block (x, s) adds the parts of sequence s for 32 experts: 32 threads an expert's four,
// each every 32nd part in token order, then the 32 in order.  The last block to finish turns
// the sums into the losses.
__global__ void __launch_bounds__(256) balance_join_kernel(const BalanceArgs a) {
  __shared__ float4 s_p[32][8];
  __shared__ int4 s_c[32][8];
  __shared__ float buf[32 * 2];
  __shared__ float buf4[32 * 4];
  __shared__ int s_last;
  const int s = blockIdx.y;
  const int b = a.seq_offsets ? min(max(a.seq_offsets[s], 0), a.T) : 0;
  const int e = a.seq_offsets ? min(max(a.seq_offsets[s + 1], 0), a.T) : a.T;
  if (threadIdx.x == 0 && blockIdx.x == 0 && a.seq_offsets) {
    const int x = a.seq_offsets[s], y = a.seq_offsets[s + 1];
    if (x > y || (s == 0 && x != 0) || (s == a.S - 1 && y != a.T)) set_status(a.status, MOE_ERR_INVARIANT);
  }
  int first = 0, last = -1;  // slots
  if (b < e) {
    first = b / a.chunk + s;
    last = (e - 1) / a.chunk + s;
  }
  wait_for_previous();
  launch_dependents();
  // n in two parts, whose sums over at most 450 chunks fp32 holds exactly
  float nz[3] = {0.0f, 0.0f, 0.0f};
  for (int i = first + static_cast<int>(threadIdx.x); i <= last; i += 256) {
    const int c = a.part_n[i];
    nz[0] += static_cast<float>(c & 0xFFF);
    nz[1] += static_cast<float>(c >> 12);
    nz[2] += a.part_z[i];
  }
  const int col = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int x = blockIdx.x * JOIN_COLS + col * 4;
  float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  int4 c = make_int4(0, 0, 0, 0);
  const bool vec = a.E % 4 == 0;
  constexpr int AHEAD = 4;  // parts that are read together: the 300 of one sequence are ten a thread
                            // (16385 x 256 one by one: 15.6 us, so 12.6 us)
  for (int j0 = first + grp; j0 <= last; j0 += 32 * AHEAD) {
    float4 q[AHEAD];
    int4 d[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const long long at = static_cast<long long>(j0 + 32 * i) * a.E + x;
      const int left = j0 + 32 * i <= last ? a.E - x : 0;
      q[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      d[i] = make_int4(0, 0, 0, 0);
      if (vec) {
        if (left > 0) {
          q[i] = *reinterpret_cast<const float4*>(a.part_p + at);
          d[i] = *reinterpret_cast<const int4*>(a.part_c + at);
        }
      } else {
        if (left > 0) { q[i].x = a.part_p[at]; d[i].x = a.part_c[at]; }
        if (left > 1) { q[i].y = a.part_p[at + 1]; d[i].y = a.part_c[at + 1]; }
        if (left > 2) { q[i].z = a.part_p[at + 2]; d[i].z = a.part_c[at + 2]; }
        if (left > 3) { q[i].w = a.part_p[at + 3]; d[i].w = a.part_c[at + 3]; }
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      p.x += q[i].x; p.y += q[i].y; p.z += q[i].z; p.w += q[i].w;
      c.x += d[i].x; c.y += d[i].y; c.z += d[i].z; c.w += d[i].w;
    }
  }
  s_p[grp][col] = p;
  s_c[grp][col] = c;
  __shared__ float buf3[32 * 3];
  row_sums<false, 3>(nz, buf3);  // and the parts are in shared memory
  const int n = static_cast<int>(nz[0]) + (static_cast<int>(nz[1]) << 12);
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  const float fs = inv_n * static_cast<float>(a.E) / static_cast<float>(a.k);
  float sum[1] = {0.0f};
  if (threadIdx.x < JOIN_COLS) {
    const int i = blockIdx.x * JOIN_COLS + threadIdx.x;
    float v = 0.0f;
    int k = 0;
#pragma unroll
    for (int g = 0; g < 32; ++g) {
      v += reinterpret_cast<const float*>(s_p[g])[threadIdx.x];
      k += reinterpret_cast<const int*>(s_c[g])[threadIdx.x];
    }
    if (i < a.E) {
      a.counts[static_cast<long long>(s) * a.E + i] = k;
      a.prob_mean[static_cast<long long>(s) * a.E + i] = v * inv_n;
      sum[0] = static_cast<float>(k) * fs * (v * inv_n);
    }
    row_sums<true, 1>(sum, buf);
    if (gridDim.x * gridDim.y == 1) {  // all there is
      if (threadIdx.x == 0) {
        a.seq_tokens[0] = n;
        a.losses[0] = a.coef * sum[0];
        a.losses[1] = a.z_coef != 0.0f ? a.z_coef * nz[2] * inv_n : 0.0f;
        s_last = 0;
      }
    } else if (threadIdx.x == 0) {
      a.seq_loss[static_cast<long long>(s) * gridDim.x + blockIdx.x] = sum[0];
      if (blockIdx.x == 0) {
        a.seq_tokens[s] = n;
        a.seq_z[s] = nz[2];
      }
      __threadfence();
      s_last = atomicAdd(a.counter, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // losses, sequences and tokens that count
  for (int i = threadIdx.x; i < a.S; i += 256) {
    const int k = __ldcg(&a.seq_tokens[i]);
    t[1] += __ldcg(&a.seq_z[i]);
    t[2] += k > 0 ? 1.0f : 0.0f;
    t[3] += static_cast<float>(k);
  }
  for (long long i = threadIdx.x; i < static_cast<long long>(a.S) * gridDim.x; i += 256) t[0] += __ldcg(&a.seq_loss[i]);
  row_sums<false, 4>(t, buf4);
  if (threadIdx.x == 0) {
    a.losses[0] = t[2] > 0.0f ? a.coef * t[0] / t[2] : 0.0f;
    a.losses[1] = t[3] > 0.0f && a.z_coef != 0.0f ? a.z_coef * t[1] / t[3] : 0.0f;
  }
}

// A group takes a run of consecutive tokens.  dl_j = g0 coef / (S' n_s) p_j (f_j - sum f p)
// [(1 - sigmoid(l_j)) for sigmoid scores] + g1 z_coef 2 / N lse softmax(l)_j.
template <int VEC, int G, int PLV, bool SIGMOID>
__global__ void __launch_bounds__(BAL_THREADS, VEC * PLV <= 16 ? 2 : 1) balance_bwd_kernel(const BalanceArgs a) {
  constexpr int N = VEC * PLV, M = N / 2;
  __shared__ float buf[32 * 2];
  __shared__ int s_off[SEQ_TABLE + 1];
  const int gl = threadIdx.x % G;
  const long long t0 = (static_cast<long long>(blockIdx.x) * (BAL_THREADS / G) + threadIdx.x / G) * a.run;
  const int t1 = static_cast<int>(min(static_cast<long long>(a.T), t0 + a.run));
  auto kept = [&](long long t) { return t < t1 && (!a.mask || a.mask[t]); };
  wait_for_previous();
  launch_dependents();
  // the first token's values are on their way while the totals are added up
  f32x2 l[M], old[M];
  bool keep = kept(t0), keep_next = a.run > 1 && kept(t0 + 1);
  load_row<VEC, G, PLV>(a.logits + t0 * a.E, a.E, gl, keep, -INFINITY, l);
  load_row<VEC, G, PLV>(a.d_logits + t0 * a.E, a.E, gl, keep && a.accumulate, 0.0f, old);
  const Sequences seqs(a, s_off);  // the sum's barrier is its
  float tot[2] = {0.0f, 0.0f};     // sequences and tokens that count
  for (int i = threadIdx.x; i < a.S; i += BAL_THREADS) {
    const int c = a.tokens_in[i];
    tot[0] += c > 0 ? 1.0f : 0.0f;
    tot[1] += static_cast<float>(c);
  }
  row_sums<false, 2>(tot, buf);
  const float g0 = (a.grad_losses ? a.grad_losses[0] : 1.0f) * a.coef / fmaxf(tot[0], 1.0f);
  const float g1 = (a.grad_losses ? a.grad_losses[1] : 1.0f) * a.z_coef * 2.0f / fmaxf(tot[1], 1.0f);
  int s = t0 < a.T ? seqs.of(static_cast<int>(t0)) : 0;
  int end = -1;
  f32x2 f[M];
  float gs = 0.0f;
#pragma unroll
  for (int c = 0; c < M; ++c) f[c] = pair(0.0f, 0.0f);
  for (int step = 0; step < a.run; ++step) {
    const long long t = t0 + step;
    if (t < t1 && t >= end) {  // first token of the run, or of a sequence
      while (s + 1 < a.S && seqs.at(s + 1) <= t) ++s;
      end = s + 1 < a.S ? seqs.at(s + 1) : a.T;
      const int n = a.tokens_in[s];
      const float inv = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
      gs = g0 * inv;
      const float fs = inv * static_cast<float>(a.E) / static_cast<float>(a.k);
      const int32_t* counts = a.counts_in + static_cast<long long>(s) * a.E;
      auto at = [&](int c) {
        const int i = (gl + G * (c / VEC)) * VEC + c % VEC;
        return i < a.E ? static_cast<float>(counts[i]) * fs : 0.0f;
      };
#pragma unroll
      for (int c = 0; c < M; ++c) f[c] = pair(at(2 * c), at(2 * c + 1));
    }
    __syncwarp();
    const bool keep_after = step + 2 < a.run && kept(t + 2);
    f32x2 l_next[M], old_next[M];
    load_row<VEC, G, PLV>(a.logits + (t + 1) * a.E, a.E, gl, keep_next, -INFINITY, l_next);
    load_row<VEC, G, PLV>(a.d_logits + (t + 1) * a.E, a.E, gl, keep_next && a.accumulate, 0.0f, old_next);
    const float top = row_top<G>(l);
    f32x2 p[M], d[M], m2 = pair(0.0f, 0.0f);
    float inv, lse, q_inv;
    if (!SIGMOID) {
      row_softmax<G>(l, top, a.z_coef != 0.0f, p, inv, lse);
#pragma unroll
      for (int c = 0; c < M; ++c) m2 = fma2(f[c], p[c], m2);
      const float m = group_sum<G>(sum_pair(m2)) * inv, gp = gs * inv, gz = g1 * lse * inv;
#pragma unroll
      for (int c = 0; c < M; ++c) d[c] = mul2(p[c], fma2(pair(gp, gp), add2(f[c], pair(-m, -m)), pair(gz, gz)));
    } else {
      f32x2 rest[M];
      row_sigmoid<G>(l, top, p, inv, &rest);
#pragma unroll
      for (int c = 0; c < M; ++c) m2 = fma2(f[c], p[c], m2);
      const float m = group_sum<G>(sum_pair(m2)) * inv, gp = gs * inv;
#pragma unroll
      for (int c = 0; c < M; ++c) d[c] = mul2(mul2(mul2(p[c], pair(gp, gp)), add2(f[c], pair(-m, -m))), rest[c]);
      if (a.z_coef != 0.0f) {
        row_softmax<G>(l, top, true, p, q_inv, lse);
        const float gz = g1 * lse * q_inv;
#pragma unroll
        for (int c = 0; c < M; ++c) d[c] = fma2(pair(gz, gz), p[c], d[c]);
      }
    }
    if (t < t1 && (keep || !a.accumulate)) {
      float* out = a.d_logits + t * a.E;
#pragma unroll
      for (int c = 0; c < M; ++c) d[c] = keep ? add2(old[c], d[c]) : pair(0.0f, 0.0f);
      if (VEC == 4) {
#pragma unroll
        for (int i = 0; i < PLV; ++i) {
          const int e = (gl + G * i) * VEC;
          if (e < a.E) *reinterpret_cast<ulonglong2*>(out + e) = make_ulonglong2(d[VEC / 2 * i], d[VEC / 2 * i + VEC / 4]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < PLV; i += 2) {
          const int e = gl + G * i;
          const float2 v = unpair(d[i / 2]);
          if (e < a.E) out[e] = v.x;
          if (e + G < a.E) out[e + G] = v.y;
        }
      }
    }
    keep = keep_next;
    keep_next = keep_after;
#pragma unroll
    for (int c = 0; c < M; ++c) {
      l[c] = l_next[c];
      old[c] = old_next[c];
    }
  }
}

// ------------------------------------------------------------------ launchers

static size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// Lanes of a token's group.
static int balance_lanes(int E) {
  int g = 1;
  while (g < 32 && g * 16 < E) g *= 2;
  return g;
}

// Tokens of a forward block: the blocks that 150 SMs hold (whatever the GPU, as the
// workspace's size goes by it: one wave), each group with at least one token; up to four a group
// stay in one block, whose results then need no join.
static int balance_chunk(const moe_balance_dims& m) {
  const int groups = BAL_THREADS / balance_lanes(m.E);
  if (m.T <= 4 * groups) return 4 * groups;
  const int blocks = 150 * balance_fwd_blocks(m.E % 4 == 0 ? 4 : 1, balance_lanes(m.E), m.E);
  const long long per = (static_cast<long long>(m.T) + blocks - 1) / blocks;
  return static_cast<int>((per + groups - 1) / groups * groups);
}
static long long balance_chunks(const moe_balance_dims& m) {
  const int chunk = balance_chunk(m);
  return (static_cast<long long>(m.T) + chunk - 1) / chunk;
}

static size_t balance_carve(const moe_balance_dims& m, void* ws, BalanceArgs* a) {
  const size_t slots = balance_chunks(m) + m.S, joins = (m.E + JOIN_COLS - 1) / JOIN_COLS;
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
  uint8_t* sl = take(static_cast<size_t>(m.S) * joins * 4);
  uint8_t* sz = take(static_cast<size_t>(m.S) * 4);
  if (a) {
    a->counter = reinterpret_cast<int32_t*>(counter);
    a->part_p = reinterpret_cast<float*>(pp);
    a->part_c = reinterpret_cast<int32_t*>(pc);
    a->part_z = reinterpret_cast<float*>(pz);
    a->part_n = reinterpret_cast<int32_t*>(pn);
    a->seq_loss = reinterpret_cast<float*>(sl);
    a->seq_z = reinterpret_cast<float*>(sz);
  }
  return at;
}

static BalanceArgs balance_args(const moe_balance_dims& m) {
  BalanceArgs a{};
  a.T = m.T; a.E = m.E; a.k = m.k; a.S = m.S; a.coef = m.coef; a.z_coef = m.z_coef;
  return a;
}

using BalanceKernel = void (*)(BalanceArgs);

template <int VEC, bool SIGMOID>
static BalanceKernel pick_fwd(int E) {
  constexpr int PLV = 16 / VEC;
  switch (balance_lanes(E)) {
    case 1: return balance_fwd_kernel<VEC, 1, PLV, SIGMOID>;
    case 2: return balance_fwd_kernel<VEC, 2, PLV, SIGMOID>;
    case 4: return balance_fwd_kernel<VEC, 4, PLV, SIGMOID>;
    case 8: return balance_fwd_kernel<VEC, 8, PLV, SIGMOID>;
    case 16: return balance_fwd_kernel<VEC, 16, PLV, SIGMOID>;
    default: return E <= 512 ? balance_fwd_kernel<VEC, 32, PLV, SIGMOID> : balance_fwd_kernel<VEC, 32, 2 * PLV, SIGMOID>;
  }
}
static BalanceKernel pick_fwd(int E, bool sigmoid) {
  if (E % 4 != 0) return sigmoid ? pick_fwd<1, true>(E) : pick_fwd<1, false>(E);
  return sigmoid ? pick_fwd<4, true>(E) : pick_fwd<4, false>(E);
}
template <int VEC, bool SIGMOID>
static BalanceKernel pick_bwd(int E) {
  constexpr int PLV = 16 / VEC;
  switch (balance_lanes(E)) {
    case 1: return balance_bwd_kernel<VEC, 1, PLV, SIGMOID>;
    case 2: return balance_bwd_kernel<VEC, 2, PLV, SIGMOID>;
    case 4: return balance_bwd_kernel<VEC, 4, PLV, SIGMOID>;
    case 8: return balance_bwd_kernel<VEC, 8, PLV, SIGMOID>;
    case 16: return balance_bwd_kernel<VEC, 16, PLV, SIGMOID>;
    default: return E <= 512 ? balance_bwd_kernel<VEC, 32, PLV, SIGMOID> : balance_bwd_kernel<VEC, 32, 2 * PLV, SIGMOID>;
  }
}
static BalanceKernel pick_bwd(int E, bool sigmoid) {
  if (E % 4 != 0) return sigmoid ? pick_bwd<1, true>(E) : pick_bwd<1, false>(E);
  return sigmoid ? pick_bwd<4, true>(E) : pick_bwd<4, false>(E);
}

static cudaError_t launch_balance_fwd(BalanceArgs a, const moe_balance_dims& m, cudaStream_t s) {
  cudaError_t err;
  a.chunk = balance_chunk(m);
  const long long chunks = balance_chunks(m);
  if (chunks > 0) {
    const BalanceKernel kern = pick_fwd(a.E, m.score == MOE_SCORE_SIGMOID);
    err = launch_early(kern, dim3(static_cast<unsigned>(chunks)), dim3(BAL_THREADS), 0, s, a);
    if (err != cudaSuccess) return err;
    if (chunks == 1 && a.S == 1) return cudaSuccess;
  } else if ((err = cudaMemsetAsync(a.counter, 0, 4, s)) != cudaSuccess) {
    return err;
  }
  return launch_early(balance_join_kernel, dim3((a.E + JOIN_COLS - 1) / JOIN_COLS, a.S), dim3(256), 0, s, a);
}

static cudaError_t launch_balance_bwd(BalanceArgs a, const moe_balance_dims& m, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int groups = BAL_THREADS / balance_lanes(a.E);
  // one wave of the two blocks that an SM holds
  const long long most = static_cast<long long>(num_sms()) * 2 * groups;
  a.run = static_cast<int>((a.T + most - 1) / most);
  const long long grid = (a.T + static_cast<long long>(groups) * a.run - 1) / (static_cast<long long>(groups) * a.run);
  const BalanceKernel kern = pick_bwd(a.E, m.score == MOE_SCORE_SIGMOID);
  return launch_early(kern, dim3(static_cast<unsigned>(grid)), dim3(BAL_THREADS), 0, s, a);
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
  if (m.E > BAL_MAX_E || m.S > BAL_MAX_S || m.T > BAL_MAX_T) return MOE_ERR_UNSUPPORTED;
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
  return status_of(launch_balance_fwd(a, *dims, static_cast<cudaStream_t>(stream)));
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
  return status_of(launch_balance_bwd(a, *dims, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
