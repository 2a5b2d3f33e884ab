// AdamW over a list of tensors, with the moments in fp32 or in 8-bit codes that share a
// scale in blocks of 128 elements.  One pass over every array; a launch takes up to 96
// tensors, whose descriptors are its arguments, in units of elements that the blocks deal
// out.  604M elements (GB300, bf16 gradients and copy): fp32 states 2.55 ms (6.63 TB/s, the
// rate of a copy), 8-bit states 1.93 ms (5.05 TB/s).
#include "around.cuh"

#include <cfloat>
#include <cmath>

namespace moe {

constexpr int ADAM_BLOCK = 128;         // elements that share a scale: a warp's step, 4 a lane
// The least eps with 8-bit states: they hold no v below fp32's smallest normal number, 2^-126,
// but an m down to that, so an update may lack its root, which eps has to stand in for.
constexpr float ADAM_MIN_EPS8 = 0x1p-63f;
constexpr int ADAM_TENSORS = 96;        // tensors of one launch (their descriptors are its arguments)
constexpr int ADAM_THREADS = 256;
constexpr int BLOCKS_32 = 5, BLOCKS_8 = 2, BLOCKS_VALUES = 8;  // of a kernel on an SM

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
  int chunk;        // elements of a unit of work: 2048 << n
  int base;         // number of tensors[0] in the caller's list
  long long units;
  float lr, beta1, beta2, keep1, keep2, eps;  // keep = 1 - beta
  float one;                                  // 1
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

// Codes <-> values.  m = s sign(c) (c / 127)^2, v = s (c / 255)^4.  A byte becomes a float as
// the low byte of 2^23's mantissa (one permute and an exact difference; a conversion
// instruction runs at a quarter of the rate), and a code becomes a byte the same way.
constexpr float TWO23 = 8388608.0f;
__device__ __forceinline__ float byte_at_two23(uint32_t word, int j) {
  return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440u | j));
}
// Four codes from one word: m's (two's complement bytes) or v's.
__device__ __forceinline__ void decode4_m(uint32_t word, float s, f32x2 (&v)[2]) {
  constexpr float SCALE = 1.0f / 16129.0f;
  word ^= 0x80808080u;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x2 c = add2(pair(byte_at_two23(word, 2 * j), byte_at_two23(word, 2 * j + 1)), pair(-TWO23 - 128.0f, -TWO23 - 128.0f));
    const float2 f = unpair(c);
    v[j] = mul2(mul2(pair(f.x * fabsf(f.x), f.y * fabsf(f.y)), pair(SCALE, SCALE)), pair(s, s));
  }
}
__device__ __forceinline__ void decode4_v(uint32_t word, float s, f32x2 (&v)[2]) {
  constexpr float SCALE = 1.0f / 65025.0f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x2 c = add2(pair(byte_at_two23(word, 2 * j), byte_at_two23(word, 2 * j + 1)), pair(-TWO23, -TWO23));
    const f32x2 q = mul2(mul2(c, c), pair(SCALE, SCALE));
    v[j] = mul2(mul2(q, q), pair(s, s));
  }
}
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
// b + 1/2 for the low or high 16 bits b of two hashes.
__device__ __forceinline__ f32x2 draws(uint32_t h0, uint32_t h1, bool high) {
  const uint32_t sel = high ? 0x7432u : 0x7410u;
  return add2(pair(__uint_as_float(__byte_perm(h0, 0x4B000000u, sel)), __uint_as_float(__byte_perm(h1, 0x4B000000u, sel))),
              pair(-TWO23 + 0.5f, -TWO23 + 0.5f));
}
__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 0xFF in the bytes of the four that are negative.
__device__ __forceinline__ uint32_t sign_bytes(float a, float b, float c, float d) {
  uint32_t lo, hi;
  asm("prmt.b32 %0, %1, %2, 0xFB;" : "=r"(lo) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
  asm("prmt.b32 %0, %1, %2, 0xFB;" : "=r"(hi) : "r"(__float_as_uint(c)), "r"(__float_as_uint(d)));
  return __byte_perm(lo, hi, 0x5410);
}
// max |a|, |b|, |c|; NaN if one of them is.
__device__ __forceinline__ float absmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 1 / s times `top` as a sum of two floats, for products that are exact to some 2^-40.
struct Inverse {
  float hi, lo;
};
__device__ __forceinline__ Inverse inverse(float s, float r, float top) {  // r = about 1 / s
  const float hi = top * r;
  return {hi, fmaf(-hi, s, top) * r};
}

// Codes of two |m| of a block with the scale s: with y = 127^2 |m| / s, k = the largest with
// k^2 <= y, in the low byte of t, or k + 1 where e < 0, with the chance that makes the mean
// right: y lies between k^2 and k^2 + 2 k + 1, and e = u (2 k + 1) + k^2 - y.  An approximate
// root that falls on the other side of a k changes nothing: the draw then decides for k in
// either case.  k^2 - y is a difference of near numbers: y comes as |m| (hi + lo), whose
// rounding against k^2 is less than a 2^-24th of the codes' distance; with y rounded once a
// code in 10^5 was another.
__device__ __forceinline__ void encode2_m(f32x2 m, f32x2 root, Inverse inv, f32x2 u, float2& t, float2& e) {
  const f32x2 t2 = fma2_down(root, pair(127.0f, 127.0f), pair(TWO23, TWO23));
  const f32x2 k = add2(t2, pair(-TWO23, -TWO23));
  const f32x2 d = fma2(m, pair(-inv.lo, -inv.lo), fma2(m, pair(-inv.hi, -inv.hi), mul2(k, k)));
  const f32x2 n = fma2(k, pair(0x1p-15f, 0x1p-15f), pair(0x1p-16f, 0x1p-16f));  // u comes times 2^16
  t = unpair(t2);
  e = unpair(fma2(u, n, d));
}
// The same for v, y = 255^4 v / s and fourth powers, k^4 .. (k + 1)^4 = k^4 + (2 k + 1) ((k + 1)^2
// + k^2); y^(1/4) = root * scale, from a root that the step has already.  k^4 takes 32 bits, so
// the product v hi is split into its rounding and the rest.
__device__ __forceinline__ void encode2_v(f32x2 v, f32x2 root, float scale, Inverse inv, f32x2 u, float2& t, float2& e) {
  const f32x2 t2 = fma2_down(root, pair(scale, scale), pair(TWO23, TWO23));
  const f32x2 k = add2(t2, pair(-TWO23, -TWO23)), k1 = add2(k, pair(1.0f, 1.0f));
  const f32x2 k2 = mul2(k, k), ny = mul2(v, pair(-inv.hi, -inv.hi));
  const f32x2 rest = fma2(v, pair(inv.lo, inv.lo), fma2(v, pair(inv.hi, inv.hi), ny));
  const f32x2 d = fma2(rest, pair(-1.0f, -1.0f), fma2(k2, k2, ny));
  const f32x2 n = mul2(fma2(k, pair(0x1p-15f, 0x1p-15f), pair(0x1p-16f, 0x1p-16f)), fma2(k1, k1, k2));
  t = unpair(t2);
  e = unpair(fma2(u, n, d));
}

struct AdamScalars {
  float gs, lr, inv_bc1, inv_bc2;
};

// The values a step takes from the device, if it does; false: nothing is to be changed.
__device__ __forceinline__ bool adam_scalars(const AdamArgs& a, AdamScalars& sc, int& step) {
  sc = AdamScalars{1.0f, a.lr, a.inv_bc1, a.inv_bc2};
  step = a.step;
  if (!a.control) return true;
  if (a.control->skip) return false;
  sc.gs = a.control->grad_scale;
  sc.lr = a.lr * a.control->lr_scale;
  step = a.control->step;
  // 1 - beta^t without cancellation
  sc.inv_bc1 = -1.0f / expm1f(static_cast<float>(step) * a.log_beta1);
  sc.inv_bc2 = -1.0f / expm1f(static_cast<float>(step) * a.log_beta2);
  return true;
}

// The last of the tensors that starts at or before a unit of work.
template <typename A>
__device__ __forceinline__ int tensor_of(const A& a, long long unit) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].first <= unit) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// fp32 states.  A unit of elements a block, four consecutive ones a thread: wide loads of
// all arrays before the first use, and enough threads (five blocks an SM) to cover them.
__global__ void __launch_bounds__(ADAM_THREADS, BLOCKS_32) adamw_kernel(const __grid_constant__ AdamArgs a) {
  wait_for_previous();  // (the next kernel's blocks among the last of these: 2562 us for 604M elements, 2545 without)
  AdamScalars sc;
  int step;
  if (!adam_scalars(a, sc, step)) return;
  for (long long unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const AdamTensor& t = a.t[tensor_of(a, unit)];
    const long long start = (unit - t.first) * a.chunk;
    const long long stop = min(t.n, start + a.chunk);
    float* const tm = static_cast<float*>(t.m);
    float* const tv = static_cast<float*>(t.v);
    for (long long i = start + threadIdx.x * 4; i < stop; i += ADAM_THREADS * 4) {
      float w[4] = {}, g[4] = {}, m[4] = {}, v[4] = {};
      const bool full = i + 4 <= stop;
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
        const float4 q = *reinterpret_cast<const float4*>(tm + i);
        const float4 r = *reinterpret_cast<const float4*>(tv + i);
        m[0] = q.x; m[1] = q.y; m[2] = q.z; m[3] = q.w;
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
      } else {
        for (int j = 0; j < 4; ++j) {
          if (i + j >= stop) break;
          w[j] = t.w[i + j];
          g[j] = t.grad_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const moe_bf16*>(t.grad)[i + j]) << 16)
                             : static_cast<const float*>(t.grad)[i + j];
          m[j] = tm[i + j];
          v[j] = tv[i + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = g[j] * sc.gs;
        m[j] = fmaf(m[j], a.beta1, x * a.keep1);
        v[j] = fmaf(v[j], a.beta2, x * x * a.keep2);
        const float update = (m[j] * sc.inv_bc1) / (sqrtf(v[j] * sc.inv_bc2) + a.eps);
        w[j] = w[j] - sc.lr * (update + t.weight_decay * w[j]);
      }
      if (full) {
        *reinterpret_cast<float4*>(t.w + i) = make_float4(w[0], w[1], w[2], w[3]);
        if (t.w16) *reinterpret_cast<uint2*>(t.w16 + i) = make_uint2(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]));
        *reinterpret_cast<float4*>(tm + i) = make_float4(m[0], m[1], m[2], m[3]);
        *reinterpret_cast<float4*>(tv + i) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        for (int j = 0; j < 4; ++j) {
          if (i + j >= stop) break;
          t.w[i + j] = w[j];
          if (t.w16) t.w16[i + j] = static_cast<moe_bf16>(pack_bf16(w[j], 0.0f) & 0xFFFFu);
          tm[i + j] = m[j];
          tv[i + j] = v[j];
        }
      }
    }
  }
}

// 8-bit states.  A warp takes pairs of blocks of 128 elements, four consecutive ones a lane of
// each, with the next pairs on their way to shared memory meanwhile.  HBM would allow an
// element about 88 issued instructions (at 16 bytes an element); one at a time with exact
// roots and conversions it took 158 (3.1 ms for 604M elements), with arithmetic on pairs,
// approximate roots and quotients of the update (within 2^-22; a v below fp32's normal numbers
// has the root 0), bytes and floats by permutes 79 (1.93 ms), two thirds of the issue slots:
// four warps a scheduler, as many as two blocks in registers allow, wait for results of the
// same few pipes.
struct Block8 {
  float4 w;
  uint2 g16;
  float4 g32;
  uint32_t m, v;
  float ms, vs;
};
__device__ __forceinline__ uint32_t word_of(const uint8_t* p, int n) {  // n < 4 bytes, zeros above
  uint32_t r = 0;
  for (int j = 0; j < n; ++j) r |= static_cast<uint32_t>(p[j]) << (8 * j);
  return r;
}
// Four elements from i on, of which the tensor may end before the last.
template <bool G16>
__device__ __forceinline__ Block8 fetch8(const AdamTensor& t, long long i) {
  const uint8_t* m = static_cast<const uint8_t*>(t.m) + i;
  const uint8_t* v = static_cast<const uint8_t*>(t.v) + i;
  const moe_bf16* g = static_cast<const moe_bf16*>(t.grad) + i;
  const float* f = static_cast<const float*>(t.grad) + i;
  Block8 x;
  x.ms = t.m_scale[i / ADAM_BLOCK];
  x.vs = t.v_scale[i / ADAM_BLOCK];
  const long long left = t.n - i;
  if (left >= 4) {
    x.w = *reinterpret_cast<const float4*>(t.w + i);
    if (G16) x.g16 = *reinterpret_cast<const uint2*>(g);
    else x.g32 = *reinterpret_cast<const float4*>(f);
    x.m = *reinterpret_cast<const uint32_t*>(m);
    x.v = *reinterpret_cast<const uint32_t*>(v);
    return x;
  }
  const int n = left > 0 ? static_cast<int>(left) : 0;
  x.w = make_float4(n > 0 ? t.w[i] : 0.0f, n > 1 ? t.w[i + 1] : 0.0f, n > 2 ? t.w[i + 2] : 0.0f, 0.0f);
  if (G16) x.g16 = make_uint2((n > 0 ? g[0] : 0u) | (n > 1 ? static_cast<uint32_t>(g[1]) << 16 : 0u), n > 2 ? g[2] : 0u);
  else x.g32 = make_float4(n > 0 ? f[0] : 0.0f, n > 1 ? f[1] : 0.0f, n > 2 ? f[2] : 0.0f, 0.0f);
  x.m = word_of(m, n);
  x.v = word_of(v, n);
  return x;
}

// What is the same for a unit's elements.
struct Unit8 {
  float gs, b1, b2, c1, c2;    // m = b1 m + c1 g, v = b2 v + c2 g^2
  float one, root_bc2, eps;
  float rate, decay;           // w += rate m / (root_bc2 sqrt(v) + eps) + decay w
  uint32_t key;
};

// The step of four elements in each of H blocks of 128 that follow each other, and its
// stores.  Two blocks go through each stage together: their chains of roots and sums over
// the warp fill each other's waits.
template <bool G16, bool TAIL, int H>
__device__ __forceinline__ void step8(const Unit8& c, const AdamTensor& t, long long i, const Block8 (&x)[H]) {
  f32x2 m[H][2], v[H][2], w[H][2], root[H][2];  // root = v^(1/4)
  float ms[H], vs[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    f32x2 g[2];
    w[h][0] = pair(x[h].w.x, x[h].w.y);
    w[h][1] = pair(x[h].w.z, x[h].w.w);
    if (G16) {
      g[0] = pair(bf16_lo(x[h].g16.x), bf16_hi(x[h].g16.x));
      g[1] = pair(bf16_lo(x[h].g16.y), bf16_hi(x[h].g16.y));
    } else {
      g[0] = pair(x[h].g32.x, x[h].g32.y);
      g[1] = pair(x[h].g32.z, x[h].g32.w);
    }
    decode4_m(x[h].m, x[h].ms, m[h]);
    decode4_v(x[h].v, x[h].vs, v[h]);
    float2 am[2], av[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // Each operation rounded: the codes then do not depend on how a compiler joins them.  (A
      // packed product and sum are joined for all their .rn; a product by 1 is not, where 1 is
      // an argument.)
      const f32x2 one = pair(c.one, c.one);
      g[j] = mul2(g[j], pair(c.gs, c.gs));
      m[h][j] = fma2(mul2(m[h][j], pair(c.b1, c.b1)), one, mul2(g[j], pair(c.c1, c.c1)));
      v[h][j] = fma2(mul2(v[h][j], pair(c.b2, c.b2)), one, mul2(mul2(g[j], g[j]), pair(c.c2, c.c2)));
      am[j] = unpair(m[h][j]);
      av[j] = unpair(v[h][j]);
      const float2 r = make_float2(sqrt_fast(av[j].x), sqrt_fast(av[j].y));
      const float2 den = unpair(fma2(pair(r.x, r.y), pair(c.root_bc2, c.root_bc2), pair(c.eps, c.eps)));
      const f32x2 update = mul2(m[h][j], pair(rcp_fast(den.x), rcp_fast(den.y)));
      // the change first: a factor 1 - lr weight_decay keeps of a small decay what 1 + 2^-24 shows of it
      w[h][j] = add2(w[h][j], fma2(update, pair(c.rate, c.rate), mul2(w[h][j], pair(c.decay, c.decay))));
      root[h][j] = pair(sqrt_fast(r.x), sqrt_fast(r.y));
    }
    ms[h] = absmax3_nan(absmax3_nan(am[0].x, am[0].y, am[1].x), am[1].y, am[1].y);
    vs[h] = absmax3_nan(absmax3_nan(av[0].x, av[0].y, av[1].x), av[1].y, av[1].y);
  }
  // elements past the end hold 0: they do not raise a maximum (bits of non-negative floats
  // order as the numbers do; a NaN is the largest)
#pragma unroll
  for (int h = 0; h < H; ++h) {
    ms[h] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ms[h])));
    vs[h] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vs[h])));
  }
  uint32_t wm[H], wv[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (ms[h] < 1.17549435e-38f) ms[h] = 0.0f;
    if (vs[h] < 1.17549435e-38f) vs[h] = 0.0f;
    // what the codes are made of; scales whose inverses would leave fp32's normal numbers at
    // either end, and their moments, times 2^60 or 2^-60
    float sm = ms[h], sv = vs[h];
    if (fminf(sm, sv) < 0x1p-60f || fmaxf(sm, sv) > 0x1p100f) {
      auto nearer = [](float x) { return x < 0x1p-60f ? 0x1p60f : x > 0x1p100f ? 0x1p-60f : 1.0f; };
      const float fm = nearer(sm), fv = nearer(sv);
      sm *= fm;
      sv *= fv;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[h][j] = mul2(m[h][j], pair(fm, fm));
        v[h][j] = mul2(v[h][j], pair(fv, fv));
        const float2 f = unpair(v[h][j]);
        root[h][j] = pair(sqrt_fast(sqrt_fast(f.x)), sqrt_fast(sqrt_fast(f.y)));
      }
    }
    const float im = sm > 0.0f ? rcp_fast(sm) : 0.0f, iv = sv > 0.0f ? rcp_fast(sv) : 0.0f;
    const Inverse em2 = sm > 0.0f ? inverse(sm, im, 16129.0f) : Inverse{0.0f, 0.0f};
    const Inverse ev4 = sv > 0.0f ? inverse(sv, iv, 4228250625.0f) : Inverse{0.0f, 0.0f};
    const float rs = 255.0f * sqrt_fast(sqrt_fast(iv));  // 255 (v / s)^(1/4) = root * rs
    float2 am[2], tm[2], em[2], tv[2], ev[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t at = static_cast<uint32_t>(i) + h * ADAM_BLOCK + 2 * j;
      const uint32_t h0 = adam_mix(at * 0x9E3779B9u + c.key), h1 = adam_mix((at + 1) * 0x9E3779B9u + c.key);
      am[j] = unpair(m[h][j]);
      const float2 ab = make_float2(fabsf(am[j].x), fabsf(am[j].y));
      const f32x2 root_m = pair(sqrt_fast(ab.x * im), sqrt_fast(ab.y * im));
      encode2_m(pair(ab.x, ab.y), root_m, em2, draws(h0, h1, false), tm[j], em[j]);
      encode2_v(v[h][j], root[h][j], rs, ev4, draws(h0, h1, true), tv[j], ev[j]);
    }
    // four codes at a time as bytes: k or k + 1 (at most 127 and 255), then m's sign, whose
    // two's complement is added without a carry between bytes
    wm[h] = low_bytes(tm[0].x, tm[0].y, tm[1].x, tm[1].y) + (sign_bytes(em[0].x, em[0].y, em[1].x, em[1].y) & 0x01010101u);
    wv[h] = low_bytes(tv[0].x, tv[0].y, tv[1].x, tv[1].y) + (sign_bytes(ev[0].x, ev[0].y, ev[1].x, ev[1].y) & 0x01010101u);
    const uint32_t neg = sign_bytes(am[0].x, am[0].y, am[1].x, am[1].y);
    wm[h] ^= neg;
    wm[h] = ((wm[h] & 0x7F7F7F7Fu) + (neg & 0x01010101u)) ^ (wm[h] & 0x80808080u);
  }
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if ((wv[h] - 0x01010101u) & ~wv[h] & 0x80808080u) {  // a code 0, seldom: no v > 0 becomes 0
      const float2 v0 = unpair(v[h][0]), v1 = unpair(v[h][1]);
      const float vs4[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (vs4[j] > 0.0f && vs[h] > 0.0f && !((wv[h] >> (8 * j)) & 0xFFu)) wv[h] |= 1u << (8 * j);
    }
    const long long k = i + h * ADAM_BLOCK;
    const float2 w0 = unpair(w[h][0]), w1 = unpair(w[h][1]);
    const uint2 w16 = make_uint2(pack_bf16(w0.x, w0.y), pack_bf16(w1.x, w1.y));
    if ((threadIdx.x & 31) == 0) {
      t.m_scale[k / ADAM_BLOCK] = ms[h];
      t.v_scale[k / ADAM_BLOCK] = vs[h];
    }
    uint8_t* const pm = static_cast<uint8_t*>(t.m) + k;
    uint8_t* const pv = static_cast<uint8_t*>(t.v) + k;
    if (!TAIL || k + 4 <= t.n) {
      *reinterpret_cast<float4*>(t.w + k) = make_float4(w0.x, w0.y, w1.x, w1.y);
      if (t.w16) *reinterpret_cast<uint2*>(t.w16 + k) = w16;
      *reinterpret_cast<uint32_t*>(pm) = wm[h];
      *reinterpret_cast<uint32_t*>(pv) = wv[h];
    } else {
      const float ws[3] = {w0.x, w0.y, w1.x};
      const uint32_t hs[3] = {w16.x, w16.x >> 16, w16.y};
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        if (k + j >= t.n) continue;
        t.w[k + j] = ws[j];
        if (t.w16) t.w16[k + j] = static_cast<moe_bf16>(hs[j]);
        pm[j] = static_cast<uint8_t>(wm[h] >> (8 * j));
        pv[j] = static_cast<uint8_t>(wv[h] >> (8 * j));
      }
    }
  }
}

// Two blocks of 128 elements in the warp's ring in shared memory: weights, gradients, codes,
// scales.  Lanes copy and read their own elements; the scales are the first lanes'.  (A pair
// shares the addresses, constants and loop of its elements.)
struct Slot8 {
  float4 w[2][32];
  float4 g[2][32];
  uint32_t m[2][32];
  uint32_t v[2][32];
  float scale[2][2];  // [m, v][block]
};
constexpr int RING8 = 4;  // pairs on their way
constexpr int RING8_BYTES = ADAM_THREADS / 32 * RING8 * sizeof(Slot8);

template <bool G16>
__device__ __forceinline__ void fetch8_async(const AdamTensor& t, long long i, Slot8& slot, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    copy_async<16>(smem_u32(&slot.w[h][lane]), t.w + i + h * ADAM_BLOCK);
    if (G16) copy_async<8>(smem_u32(&slot.g[h][lane]), static_cast<const moe_bf16*>(t.grad) + i + h * ADAM_BLOCK);
    else copy_async<16>(smem_u32(&slot.g[h][lane]), static_cast<const float*>(t.grad) + i + h * ADAM_BLOCK);
    copy_async<4>(smem_u32(&slot.m[h][lane]), static_cast<const uint8_t*>(t.m) + i + h * ADAM_BLOCK);
    copy_async<4>(smem_u32(&slot.v[h][lane]), static_cast<const uint8_t*>(t.v) + i + h * ADAM_BLOCK);
  }
  if (lane < 4) copy_async<4>(smem_u32(&slot.scale[lane >> 1][lane & 1]), (lane >> 1 ? t.v_scale : t.m_scale) + i / ADAM_BLOCK + (lane & 1));
}

// Elements start .. stop of a tensor: pairs of whole blocks, then what is left of the tensor,
// by one warp.
template <bool G16>
__device__ __forceinline__ void adam8_unit(const Unit8& c, const AdamTensor& t, long long start, long long stop, Slot8* ring) {
  constexpr int WARPS = ADAM_THREADS / 32, PAIR = 2 * ADAM_BLOCK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = static_cast<int>((stop - start) / PAIR);
  const long long i0 = start + lane * 4;
  auto fetch = [&](int b, int slot) {
    if (b < pairs) fetch8_async<G16>(t, i0 + static_cast<long long>(b) * PAIR, ring[slot], lane);
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < RING8; ++k) fetch(warp + k * WARPS, k);
  int slot = 0;
  for (int b = warp; b < pairs; b += WARPS) {
    copy_wait<RING8 - 1>();
    __syncwarp();
    const long long i = i0 + static_cast<long long>(b) * PAIR;
    const Slot8& s = ring[slot];
    Block8 x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[h].w = s.w[h][lane];
      if (G16) x[h].g16 = *reinterpret_cast<const uint2*>(&s.g[h][lane]);
      else x[h].g32 = s.g[h][lane];
      x[h].m = s.m[h][lane];
      x[h].v = s.v[h][lane];
      x[h].ms = s.scale[0][h];
      x[h].vs = s.scale[1][h];
    }
    step8<G16, false, 2>(c, t, i, x);
    __syncwarp();  // every lane has used the slot
    fetch(b + RING8 * WARPS, slot);
    slot = (slot + 1) % RING8;
  }
  copy_wait<0>();
  for (long long i = start + static_cast<long long>(pairs) * PAIR; warp == pairs % WARPS && i < stop; i += ADAM_BLOCK) {
    const Block8 x[1] = {fetch8<G16>(t, i + lane * 4)};
    step8<G16, true, 1>(c, t, i + lane * 4, x);
  }
}

__global__ void __launch_bounds__(ADAM_THREADS, BLOCKS_8) adamw8_kernel(const __grid_constant__ AdamArgs a) {
  extern __shared__ Slot8 rings[];
  Slot8* const ring = rings + (threadIdx.x >> 5) * RING8;
  wait_for_previous();
  launch_dependents();
  AdamScalars sc;
  int step;
  if (!adam_scalars(a, sc, step)) return;
  Unit8 c;
  c.one = a.one;
  c.gs = sc.gs;
  c.c1 = a.keep1;
  c.c2 = a.keep2;
  c.b1 = a.beta1;
  c.b2 = a.beta2;
  c.root_bc2 = sqrtf(sc.inv_bc2);
  c.eps = a.eps;
  c.rate = -sc.lr * sc.inv_bc1;
  const uint32_t base = adam_mix(adam_mix(a.seed) + static_cast<uint32_t>(step));
  for (long long unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int at = tensor_of(a, unit);
    const AdamTensor t = a.t[at];  // in registers: read from the arguments, 22 more loads a pair
    const long long start = (unit - t.first) * a.chunk;
    const long long stop = min(t.n, start + a.chunk);
    c.decay = -sc.lr * t.weight_decay;
    // a unit does not cross a multiple of 2^32
    c.key = adam_mix(base + static_cast<uint32_t>(a.base + at) * 0x6A09E667u + static_cast<uint32_t>(start >> 32) * 0xBB67AE85u);
    if (t.grad_bf16) adam8_unit<true>(c, t, start, stop, ring);
    else adam8_unit<false>(c, t, start, stop, ring);
  }
}

struct AdamValue {
  const uint8_t* m;
  const uint8_t* v;
  const float* m_scale;
  const float* v_scale;
  void* m_out;
  void* v_out;
  long long n;
  long long first;
};
struct AdamValueArgs {
  int count, chunk;
  long long units;
  AdamValue t[ADAM_TENSORS];
};

// The values of 8-bit states.
template <typename OT>
__global__ void __launch_bounds__(ADAM_THREADS, BLOCKS_VALUES) adamw_values_kernel(const __grid_constant__ AdamValueArgs a) {
  wait_for_previous();
  launch_dependents();
  for (long long unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const AdamValue& t = a.t[tensor_of(a, unit)];
    const long long start = (unit - t.first) * a.chunk;
    const long long stop = min(t.n, start + a.chunk);
    for (long long i = start + threadIdx.x * 8; i < stop; i += ADAM_THREADS * 8) {
      const float ms = t.m_scale[i / ADAM_BLOCK], vs = t.v_scale[i / ADAM_BLOCK];
      const bool full = i + 8 <= stop;
      const int n = full ? 8 : static_cast<int>(stop - i);
      uint2 cm, cv;
      if (full) {
        cm = *reinterpret_cast<const uint2*>(t.m + i);
        cv = *reinterpret_cast<const uint2*>(t.v + i);
      } else {
        cm = make_uint2(word_of(t.m + i, min(n, 4)), n > 4 ? word_of(t.m + i + 4, n - 4) : 0u);
        cv = make_uint2(word_of(t.v + i, min(n, 4)), n > 4 ? word_of(t.v + i + 4, n - 4) : 0u);
      }
      f32x2 pm[4], pv[4];
      decode4_m(cm.x, ms, *reinterpret_cast<f32x2(*)[2]>(pm));
      decode4_m(cm.y, ms, *reinterpret_cast<f32x2(*)[2]>(pm + 2));
      decode4_v(cv.x, vs, *reinterpret_cast<f32x2(*)[2]>(pv));
      decode4_v(cv.y, vs, *reinterpret_cast<f32x2(*)[2]>(pv + 2));
      float m[8], v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = unpair(pm[j]), y = unpair(pv[j]);
        m[2 * j] = x.x; m[2 * j + 1] = x.y;
        v[2 * j] = y.x; v[2 * j + 1] = y.y;
      }
      if (full) {
        store8(static_cast<OT*>(t.m_out) + i, m);
        store8(static_cast<OT*>(t.v_out) + i, v);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j) {
          if (j >= n) continue;
          if (sizeof(OT) == 4) {
            static_cast<float*>(t.m_out)[i + j] = m[j];
            static_cast<float*>(t.v_out)[i + j] = v[j];
          } else {
            static_cast<moe_bf16*>(t.m_out)[i + j] = static_cast<moe_bf16>(pack_bf16(m[j], 0.0f) & 0xFFFFu);
            static_cast<moe_bf16*>(t.v_out)[i + j] = static_cast<moe_bf16>(pack_bf16(v[j], 0.0f) & 0xFFFFu);
          }
        }
      }
    }
  }
}

static long long adam_units(long long n, int chunk) { return (n + chunk - 1) / chunk; }
// Units of 16384 elements, or, where those would leave the SMs less than eight blocks each,
// smaller ones (2.2M elements of 95 tensors: 2048; 16.4 us with 8192, 12.7 us with 4096).
static int adam_chunk(long long total) {
  int chunk = 16384;
  while (chunk > 2048 && total < static_cast<long long>(chunk) * num_sms() * 8) chunk /= 2;
  return chunk;
}
// The blocks that the SMs hold at once (the kernels' launch bounds): a second, partial wave
// would leave SMs idle at its end.
static int adam_grid(long long units, int per_sm) {
  const long long most = static_cast<long long>(num_sms()) * per_sm;
  return static_cast<int>(units < most ? units : most);
}
template <auto KERN, int SMEM = 0, typename A>
static cudaError_t launch_adam(int grid, const A& a, cudaStream_t s) {
  if (SMEM > 0) {
    const cudaError_t err = allow_smem<KERN>(SMEM);
    if (err != cudaSuccess) return err;
  }
  return launch_early(KERN, dim3(grid), dim3(ADAM_THREADS), SMEM, s, a);
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
  // lr and eps as the kernels have them, in fp32
  const float lr = static_cast<float>(h.lr), eps = static_cast<float>(h.eps);
  if (!(lr >= 0.0f) || !std::isfinite(lr) || !(h.beta1 >= 0.0 && h.beta1 < 1.0) ||
      !(h.beta2 >= 0.0 && h.beta2 < 1.0) || !(eps >= (h.bits == 8 ? ADAM_MIN_EPS8 : FLT_TRUE_MIN)) || !std::isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  if (!control && h.step < 1) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(control) % 4) return MOE_ERR_ALIGNMENT;
  const bool eight = h.bits == 8;
  for (int i = 0; i < count; ++i) {
    const moe_status st = adam_check_tensor(tensors[i], eight, true);
    if (st != MOE_OK) return st;
  }
  AdamArgs a{};
  a.lr = lr;
  a.beta1 = static_cast<float>(h.beta1);
  a.beta2 = static_cast<float>(h.beta2);
  a.keep1 = static_cast<float>(1.0 - h.beta1);
  a.keep2 = static_cast<float>(1.0 - h.beta2);
  a.eps = eps;
  a.one = 1.0f;
  a.log_beta1 = static_cast<float>(std::log(h.beta1));
  a.log_beta2 = static_cast<float>(std::log(h.beta2));
  if (!control) {
    a.inv_bc1 = static_cast<float>(1.0 / (1.0 - std::pow(h.beta1, h.step)));
    a.inv_bc2 = static_cast<float>(1.0 / (1.0 - std::pow(h.beta2, h.step)));
  }
  a.seed = h.seed;
  a.step = h.step;
  a.control = control;
  long long total = 0;
  for (int i = 0; i < count; ++i) total += tensors[i].n;
  a.chunk = adam_chunk(total);
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
      a.units += adam_units(t.n, a.chunk);
    }
    if (a.units == 0) continue;
    const cudaError_t err = eight ? launch_adam<adamw8_kernel, RING8_BYTES>(adam_grid(a.units, BLOCKS_8), a, s)
                                  : launch_adam<adamw_kernel>(adam_grid(a.units, BLOCKS_32), a, s);
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
  long long total = 0;
  for (int i = 0; i < count; ++i) total += tensors[i].n;
  a.chunk = adam_chunk(total);
  for (int i = 0; i < count;) {
    a.count = 0;
    a.units = 0;
    for (; i < count && a.count < ADAM_TENSORS; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      a.t[a.count++] = AdamValue{static_cast<const uint8_t*>(t.m), static_cast<const uint8_t*>(t.v), t.m_scale,
                                 t.v_scale, m_out[i], v_out[i], static_cast<long long>(t.n), a.units};
      a.units += adam_units(t.n, a.chunk);
    }
    if (a.units == 0) continue;
    const cudaError_t err = out_type == MOE_TYPE_BF16
                                ? launch_adam<adamw_values_kernel<moe_bf16>>(adam_grid(a.units, BLOCKS_VALUES), a, s)
                                : launch_adam<adamw_values_kernel<float>>(adam_grid(a.units, BLOCKS_VALUES), a, s);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
