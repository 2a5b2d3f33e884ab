// AdamW over a list of tensors, with the moments in fp32 or in 8-bit codes that share a
// scale in blocks of 128 elements.
#include "around.cuh"

#include <cmath>

namespace moe {

constexpr int ADAM_BLOCK = 128;         // elements that share a scale: a warp's step, 4 a lane
constexpr int ADAM_CHUNK = 4096;        // elements of a unit of work
constexpr int ADAM_TENSORS = 96;        // tensors of one launch (their descriptors are its arguments)
constexpr int ADAM_THREADS = 256;

struct AdamTensor {
  float* w;
  moe_bf16* w16;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long n;
  float weight_decay;
  int grad_bf16;
  long long first;  // units of work before this tensor
};

struct AdamArgs {
  int count;
  int base;         // number of tensors[0] in the caller's list
  long long units;
  float lr, beta1, beta2, keep1, keep2, eps;  // keep = 1 - beta
  float inv_bc1, inv_bc2;                     // 1 / (1 - beta^t)
  float log_beta1, log_beta2;
  uint32_t seed;
  int step;
  const moe_adamw_control* control;
  AdamTensor t[ADAM_TENSORS];
};

__device__ __forceinline__ uint32_t adam_mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Codes <-> values.  m = s sign(c) (c / 127)^2, v = s (c / 255)^4.
__device__ __forceinline__ float decode_m(int c, float s) {
  const float f = static_cast<float>(c);
  return s * (f * fabsf(f) * (1.0f / 16129.0f));
}
__device__ __forceinline__ float decode_v(uint32_t c, float s) {
  const float f = static_cast<float>(c);
  const float q = f * f * (1.0f / 65025.0f);
  return s * (q * q);
}

// The code of x = |m| / s (0..1): the largest k with (k / 127)^2 <= x, or k + 1 with the
// chance that makes the mean x.  A root that rounds across k changes nothing: the chance
// is then 0 or 1.
__device__ __forceinline__ int encode_m(float x, uint32_t bits) {
  const float y = x * 16129.0f;
  const float k = floorf(sqrtf(y));
  const float u = (static_cast<float>(bits) + 0.5f) * (1.0f / 65536.0f);
  const float up = u * (2.0f * k + 1.0f) < y - k * k ? 1.0f : 0.0f;
  return static_cast<int>(fminf(k + up, 127.0f));
}
__device__ __forceinline__ uint32_t encode_v(float x, uint32_t bits) {
  const float y = x * 4228250625.0f;
  const float k = floorf(sqrtf(sqrtf(y)));
  const float k2 = k * k, n2 = (k + 1.0f) * (k + 1.0f);
  const float lo = k2 * k2, hi = n2 * n2;
  const float u = (static_cast<float>(bits) + 0.5f) * (1.0f / 65536.0f);
  const float c = fminf(k + (u * (hi - lo) < y - lo ? 1.0f : 0.0f), 255.0f);
  return x > 0.0f ? static_cast<uint32_t>(fmaxf(c, 1.0f)) : 0u;
}

struct AdamScalars {
  float gs, lr, inv_bc1, inv_bc2;
};

// The step's moments and weight for one element.  The moments' operations are rounded one
// by one (no contraction): the codes then do not depend on how a compiler joins them.
__device__ __forceinline__ void adam_element(const AdamArgs& a, const AdamScalars& c, float wd, float g, float& w,
                                             float& m, float& v) {
  g = __fmul_rn(g, c.gs);
  m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.keep1));
  v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.keep2));
  const float update = (m * c.inv_bc1) / (sqrtf(v * c.inv_bc2) + a.eps);
  w = w - c.lr * (update + wd * w);
}

template <bool EIGHT>
__global__ void __launch_bounds__(ADAM_THREADS) adamw_kernel(const __grid_constant__ AdamArgs a) {
  AdamScalars sc{1.0f, a.lr, a.inv_bc1, a.inv_bc2};
  int step = a.step;
  if (a.control) {
    if (a.control->skip) return;
    sc.gs = a.control->grad_scale;
    sc.lr = a.lr * a.control->lr_scale;
    step = a.control->step;
    // 1 - beta^t without cancellation
    sc.inv_bc1 = -1.0f / expm1f(static_cast<float>(step) * a.log_beta1);
    sc.inv_bc2 = -1.0f / expm1f(static_cast<float>(step) * a.log_beta2);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (long long unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    int lo = 0, hi = a.count - 1;  // the last tensor that starts at or before the unit
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.t[mid].first <= unit) lo = mid;
      else hi = mid - 1;
    }
    const AdamTensor& t = a.t[lo];
    const long long start = (unit - t.first) * ADAM_CHUNK;
    const long long stop = min(t.n, start + ADAM_CHUNK);
    uint32_t key = 0;
    if (EIGHT) {  // a unit does not cross a multiple of 2^32
      key = adam_mix(adam_mix(a.seed) + static_cast<uint32_t>(step));
      key = adam_mix(key + static_cast<uint32_t>(a.base + lo) * 0x6A09E667u + static_cast<uint32_t>(start >> 32) * 0xBB67AE85u);
    }
    for (long long b = start + warp * ADAM_BLOCK; b < stop; b += ADAM_BLOCK * (ADAM_THREADS / 32)) {
      const long long i = b + lane * 4;
      float w[4] = {}, g[4] = {}, m[4] = {}, v[4] = {};
      const bool full = i + 4 <= stop;
      float ms = 0.0f, vs = 0.0f;
      if (EIGHT) {
        ms = t.m_scale[b / ADAM_BLOCK];
        vs = t.v_scale[b / ADAM_BLOCK];
      }
      if (full) {
        const float4 x = *reinterpret_cast<const float4*>(t.w + i);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        if (t.grad_bf16) {
          const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const moe_bf16*>(t.grad) + i);
          g[0] = bf16_lo(q.x); g[1] = bf16_hi(q.x); g[2] = bf16_lo(q.y); g[3] = bf16_hi(q.y);
        } else {
          const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(t.grad) + i);
          g[0] = q.x; g[1] = q.y; g[2] = q.z; g[3] = q.w;
        }
        if (EIGHT) {
          const char4 cm = *reinterpret_cast<const char4*>(static_cast<const int8_t*>(t.m) + i);
          const uchar4 cv = *reinterpret_cast<const uchar4*>(static_cast<const uint8_t*>(t.v) + i);
          m[0] = decode_m(static_cast<signed char>(cm.x), ms); m[1] = decode_m(static_cast<signed char>(cm.y), ms);
          m[2] = decode_m(static_cast<signed char>(cm.z), ms); m[3] = decode_m(static_cast<signed char>(cm.w), ms);
          v[0] = decode_v(cv.x, vs); v[1] = decode_v(cv.y, vs); v[2] = decode_v(cv.z, vs); v[3] = decode_v(cv.w, vs);
        } else {
          const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + i);
          const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + i);
          m[0] = q.x; m[1] = q.y; m[2] = q.z; m[3] = q.w;
          v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        }
      } else {
        for (int j = 0; j < 4; ++j) {
          if (i + j >= stop) break;
          w[j] = t.w[i + j];
          g[j] = t.grad_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const moe_bf16*>(t.grad)[i + j]) << 16)
                             : static_cast<const float*>(t.grad)[i + j];
          m[j] = EIGHT ? decode_m(static_cast<const int8_t*>(t.m)[i + j], ms) : static_cast<const float*>(t.m)[i + j];
          v[j] = EIGHT ? decode_v(static_cast<const uint8_t*>(t.v)[i + j], vs) : static_cast<const float*>(t.v)[i + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) adam_element(a, sc, t.weight_decay, g[j], w[j], m[j], v[j]);
      int cm[4] = {};
      uint32_t cv[4] = {};
      if (EIGHT) {
        // elements past the end hold 0: they do not raise a maximum (bits of non-negative
        // floats order as the numbers do; a NaN is the largest)
        uint32_t bm = 0, bv = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bm = max(bm, __float_as_uint(fabsf(m[j])));
          bv = max(bv, __float_as_uint(v[j]));
        }
        ms = __uint_as_float(__reduce_max_sync(0xffffffffu, bm));
        vs = __uint_as_float(__reduce_max_sync(0xffffffffu, bv));
        if (ms < 1.17549435e-38f) ms = 0.0f;
        if (vs < 1.17549435e-38f) vs = 0.0f;
        const float im = ms > 0.0f ? 1.0f / ms : 0.0f, iv = vs > 0.0f ? 1.0f / vs : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t u = adam_mix(static_cast<uint32_t>(i + j) * 0x9E3779B9u + key);
          const int c = encode_m(fabsf(m[j]) * im, u & 0xFFFFu);
          cm[j] = m[j] < 0.0f ? -c : c;
          cv[j] = encode_v(v[j] * iv, u >> 16);
        }
        if (lane == 0) {
          t.m_scale[b / ADAM_BLOCK] = ms;
          t.v_scale[b / ADAM_BLOCK] = vs;
        }
      }
      if (full) {
        *reinterpret_cast<float4*>(t.w + i) = make_float4(w[0], w[1], w[2], w[3]);
        if (t.w16) *reinterpret_cast<uint2*>(t.w16 + i) = make_uint2(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]));
        if (EIGHT) {
          *reinterpret_cast<char4*>(static_cast<int8_t*>(t.m) + i) =
              make_char4(static_cast<signed char>(cm[0]), static_cast<signed char>(cm[1]),
                         static_cast<signed char>(cm[2]), static_cast<signed char>(cm[3]));
          *reinterpret_cast<uchar4*>(static_cast<uint8_t*>(t.v) + i) = make_uchar4(cv[0], cv[1], cv[2], cv[3]);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(t.m) + i) = make_float4(m[0], m[1], m[2], m[3]);
          *reinterpret_cast<float4*>(static_cast<float*>(t.v) + i) = make_float4(v[0], v[1], v[2], v[3]);
        }
      } else {
        for (int j = 0; j < 4; ++j) {
          if (i + j >= stop) break;
          t.w[i + j] = w[j];
          if (t.w16) t.w16[i + j] = static_cast<moe_bf16>(pack_bf16(w[j], 0.0f) & 0xFFFFu);
          if (EIGHT) {
            static_cast<int8_t*>(t.m)[i + j] = static_cast<int8_t>(cm[j]);
            static_cast<uint8_t*>(t.v)[i + j] = static_cast<uint8_t>(cv[j]);
          } else {
            static_cast<float*>(t.m)[i + j] = m[j];
            static_cast<float*>(t.v)[i + j] = v[j];
          }
        }
      }
    }
  }
}

struct AdamValue {
  const int8_t* m;
  const uint8_t* v;
  const float* m_scale;
  const float* v_scale;
  void* m_out;
  void* v_out;
  long long n;
  long long first;
};
struct AdamValueArgs {
  int count;
  long long units;
  AdamValue t[ADAM_TENSORS];
};

// The values of 8-bit states.
template <typename OT>
__global__ void __launch_bounds__(ADAM_THREADS) adamw_values_kernel(const __grid_constant__ AdamValueArgs a) {
  for (long long unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.t[mid].first <= unit) lo = mid;
      else hi = mid - 1;
    }
    const AdamValue& t = a.t[lo];
    const long long start = (unit - t.first) * ADAM_CHUNK;
    const long long stop = min(t.n, start + ADAM_CHUNK);
    for (long long i = start + threadIdx.x * 8; i < stop; i += ADAM_THREADS * 8) {
      const float ms = t.m_scale[i / ADAM_BLOCK], vs = t.v_scale[i / ADAM_BLOCK];
      float m[8], v[8];
      if (i + 8 <= stop) {
        const uint2 cm = *reinterpret_cast<const uint2*>(t.m + i), cv = *reinterpret_cast<const uint2*>(t.v + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[j] = decode_m(static_cast<int8_t>((j < 4 ? cm.x : cm.y) >> (8 * (j & 3))), ms);
          v[j] = decode_v(((j < 4 ? cv.x : cv.y) >> (8 * (j & 3))) & 0xFFu, vs);
        }
        store8(static_cast<OT*>(t.m_out) + i, m);
        store8(static_cast<OT*>(t.v_out) + i, v);
      } else {
        for (int j = 0; i + j < stop; ++j) {
          const float x = decode_m(t.m[i + j], ms), y = decode_v(t.v[i + j], vs);
          if (sizeof(OT) == 4) {
            static_cast<float*>(t.m_out)[i + j] = x;
            static_cast<float*>(t.v_out)[i + j] = y;
          } else {
            static_cast<moe_bf16*>(t.m_out)[i + j] = static_cast<moe_bf16>(pack_bf16(x, 0.0f) & 0xFFFFu);
            static_cast<moe_bf16*>(t.v_out)[i + j] = static_cast<moe_bf16>(pack_bf16(y, 0.0f) & 0xFFFFu);
          }
        }
      }
    }
  }
}

static long long adam_units(long long n) { return (n + ADAM_CHUNK - 1) / ADAM_CHUNK; }
static int adam_grid(long long units) {
  const long long most = static_cast<long long>(num_sms()) * 8;
  return static_cast<int>(units < most ? units : most);
}

}  // namespace moe

using namespace moe;

extern "C" {

static moe_status adam_check_tensor(const moe_adamw_tensor& t, bool eight, bool step) {
  if (t.n < 0) return MOE_ERR_INVALID_ARG;
  if (t.n == 0) return MOE_OK;
  if (!t.m || !t.v || (step && (!t.w || !t.grad))) return MOE_ERR_INVALID_ARG;
  if (eight != (t.m_scale != nullptr) || eight != (t.v_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (step && t.grad_type != MOE_TYPE_BF16 && t.grad_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (step && !std::isfinite(t.weight_decay)) return MOE_ERR_INVALID_ARG;
  if (!ptr_aligned16(t.m) || !ptr_aligned16(t.v)) return MOE_ERR_ALIGNMENT;
  if (step && (!ptr_aligned16(t.w) || !ptr_aligned16(t.w16) || !ptr_aligned16(t.grad))) return MOE_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(t.m_scale) % 4 || reinterpret_cast<uintptr_t>(t.v_scale) % 4)
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

moe_status moe_adamw_step(const moe_adamw_hyper* hyper, const moe_adamw_tensor* tensors, int32_t count,
                          const moe_adamw_control* control, void* stream) {
  if (!hyper || count < 0 || (count > 0 && !tensors)) return MOE_ERR_INVALID_ARG;
  const moe_adamw_hyper& h = *hyper;
  if (h.bits != 32 && h.bits != 8) return MOE_ERR_INVALID_ARG;
  if (!(h.lr >= 0.0) || !std::isfinite(h.lr) || !(h.beta1 >= 0.0 && h.beta1 < 1.0) ||
      !(h.beta2 >= 0.0 && h.beta2 < 1.0) || !(h.eps > 0.0) || !std::isfinite(h.eps))
    return MOE_ERR_INVALID_ARG;
  if (!control && h.step < 1) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(control) % 4) return MOE_ERR_ALIGNMENT;
  const bool eight = h.bits == 8;
  for (int i = 0; i < count; ++i) {
    const moe_status st = adam_check_tensor(tensors[i], eight, true);
    if (st != MOE_OK) return st;
  }
  AdamArgs a{};
  a.lr = static_cast<float>(h.lr);
  a.beta1 = static_cast<float>(h.beta1);
  a.beta2 = static_cast<float>(h.beta2);
  a.keep1 = static_cast<float>(1.0 - h.beta1);
  a.keep2 = static_cast<float>(1.0 - h.beta2);
  a.eps = static_cast<float>(h.eps);
  a.log_beta1 = static_cast<float>(std::log(h.beta1));
  a.log_beta2 = static_cast<float>(std::log(h.beta2));
  if (!control) {
    a.inv_bc1 = static_cast<float>(1.0 / (1.0 - std::pow(h.beta1, h.step)));
    a.inv_bc2 = static_cast<float>(1.0 / (1.0 - std::pow(h.beta2, h.step)));
  }
  a.seed = h.seed;
  a.step = h.step;
  a.control = control;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int i = 0; i < count;) {
    a.base = i;
    a.count = 0;
    a.units = 0;
    for (; i < count && a.count < ADAM_TENSORS; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      AdamTensor& o = a.t[a.count++];
      o = AdamTensor{t.w, t.w16, t.grad, t.m, t.v, t.m_scale, t.v_scale, static_cast<long long>(t.n),
                     t.weight_decay, t.grad_type == MOE_TYPE_BF16, a.units};
      a.units += adam_units(t.n);
    }
    if (a.units == 0) continue;
    if (eight) adamw_kernel<true><<<adam_grid(a.units), ADAM_THREADS, 0, s>>>(a);
    else adamw_kernel<false><<<adam_grid(a.units), ADAM_THREADS, 0, s>>>(a);
    count_launch();
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

moe_status moe_adamw_values(const moe_adamw_tensor* tensors, int32_t count, int32_t out_type, void* const* m_out,
                            void* const* v_out, void* stream) {
  if (count < 0 || (count > 0 && (!tensors || !m_out || !v_out))) return MOE_ERR_INVALID_ARG;
  if (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const moe_status st = adam_check_tensor(tensors[i], true, false);
    if (st != MOE_OK) return st;
    if (tensors[i].n > 0 && (!m_out[i] || !v_out[i])) return MOE_ERR_INVALID_ARG;
    if (!ptr_aligned16(m_out[i]) || !ptr_aligned16(v_out[i])) return MOE_ERR_ALIGNMENT;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  AdamValueArgs a{};
  for (int i = 0; i < count;) {
    a.count = 0;
    a.units = 0;
    for (; i < count && a.count < ADAM_TENSORS; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      a.t[a.count++] = AdamValue{static_cast<const int8_t*>(t.m), static_cast<const uint8_t*>(t.v), t.m_scale,
                                 t.v_scale, m_out[i], v_out[i], static_cast<long long>(t.n), a.units};
      a.units += adam_units(t.n);
    }
    if (a.units == 0) continue;
    if (out_type == MOE_TYPE_BF16) adamw_values_kernel<moe_bf16><<<adam_grid(a.units), ADAM_THREADS, 0, s>>>(a);
    else adamw_values_kernel<float><<<adam_grid(a.units), ADAM_THREADS, 0, s>>>(a);
    count_launch();
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
