// adamw.cu -- one AdamW step over many tensors in one launch, moments in fp32 or in 8 bits:
//   g = grad_scale clip grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//   clip = min(1, max_norm / (||grad_scale grad|| + 1e-6)) over all tensors; a norm that is not
//   finite as an fp32 number leaves parameters, moments and the step count as they are.
//
// 8-bit moments, in blocks of 256 elements with one fp32 scale, the block's largest magnitude:
//   m: a sign and a float of 4 exponent and 3 mantissa bits of |m| / scale;
//   v: a float of 4 exponent and 4 mantissa bits of sqrt(v) / scale (the root is what the step
//      divides by, and halves the range); a v above 0 never becomes 0.
// Both grids are the leading bits of the fp32 number, from 1 down to 2^-16, so encoding is a
// shift of its bits.  Rounding is stochastic: a step of v changes it by 1 - b2 = 0.1 %, far less
// than half a step of any 8-bit grid, and rounding to nearest would leave it where it is for
// good.  The random bits are a hash of (seed, step, element), so a step is reproducible.  Without
// an fp32 master copy a bf16 parameter is rounded the same way, for the same reason.
// The fp32 operations that lead to a code (moments, root, scale, quotient) are kept unfused and
// correctly rounded, so that codes do not depend on how the compiler contracts them.
//
// Bound by memory; with 8-bit moments by instruction issue (18 bytes an element with a master copy
// and fp32 gradients, and about 85 instructions for them).  A warp takes one block of 256 at a time,
// 8 consecutive elements a lane, so every access is 16 or 32 bytes a lane (8 for codes) and a block's
// scale is one warp reduction.  Codes are decoded through tables in shared memory; codes below the
// grid's least value are rare and made by a second pass over the warp's block.
// Measured: 54.5 M fp32 elements and moments, no norm (28 bytes an element) 232 us, 6.6 TB/s; 42 M bf16
// ones in 448 tensors with masters, 8-bit moments and the clip 180 us, with the moments read as bf16
// after it 220; 1.3 M in 14 tensors, 32 bits and the clip, 13.9 us.  42 M bf16 without masters, 32 bits
// and the clip: 235 us.
#include <cuda_bf16.h>

#include <cstdint>
#include <cstring>

#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace qlora {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;

// A 32-bit integer hash, multiplications by odd numbers between shifted exclusive ors, with the shifts
// and the two factors of C. Wellons, "Prospecting for Hash Functions" (2018).
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t element_bits(uint32_t word, int64_t e) {
  const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(e) >> 32);
  return mix32((static_cast<uint32_t>(e) ^ (hi * 0x9E3779B1u)) + word);
}

constexpr uint32_t kMBase = 889, kVBase = 1777;  // fp32 bits of 1.0 >> 20 less 127, >> 19 less 255
constexpr float kMLeast = 1.25f / 65536.f, kVLeast = 1.125f / 65536.f;  // the values of code 1

// The values of the 256 codes, over the scale (of v: of its root).
struct CodeTables {
  float m[256], v[256];
};
__device__ __forceinline__ void fill_tables(CodeTables& t) {
  for (int c = threadIdx.x; c < 256; c += blockDim.x) {
    const uint32_t mag = c & 127u;
    const float x = mag ? __uint_as_float((mag + kMBase) << 20) : 0.f;
    t.m[c] = (c & 128) ? -x : x;
    t.v[c] = c ? __uint_as_float((static_cast<uint32_t>(c) + kVBase) << 19) : 0.f;
  }
}
// Two consecutive elements' values from byte `k` and `k + 1` of a word of codes.
__device__ __forceinline__ f2 decode2(const float* table, uint32_t word, int k, f2 scale) {
  const uint32_t a = (word >> (8 * k)) & 255u, b = (word >> (8 * k + 8)) & 255u;
  return mul2(pair(table[a], table[b]), scale);
}
// Codes, in the top byte, of a magnitude x = |m| / scale or sqrt(v) / scale in [0, 1] that is not
// below the least value; r: 32 random bits, m's 16 the low ones.  The fp32 bits with the code in
// their top byte, less the grid's base, plus the random bits below the code: a byte permutation
// places these and the base's byte.  (A little past 1 the carry still stays within the top code;
// what a NaN or infinity gives does not matter, its block's scale is not finite.)
static_assert((kMBase + 0x87u) % 256 == 0 && (kVBase + 0x0Fu) % 256 == 0, "the bases' bytes");
__device__ __forceinline__ uint32_t encode_m(float x, uint32_t r) {
  return (__float_as_uint(x) << 4) + __byte_perm(r, 0x87u, 0x4105);
}
__device__ __forceinline__ uint32_t encode_v(float x, uint32_t r) {
  return (__float_as_uint(x) << 5) + __byte_perm(r, 0x0Fu, 0x4325);
}
// ... and of any x.
__device__ __forceinline__ uint32_t encode_m_any(float x, uint32_t r) {
  if (x < kMLeast)
    return __fmul_rn(static_cast<float>(r & 0xFFFFu), kMLeast / 65536.f) < x ? 1u << 24 : 0u;
  return encode_m(x, r);
}
__device__ __forceinline__ uint32_t encode_v_any(float x, uint32_t r) {
  if (x < kVLeast) return x > 0.f ? 1u << 24 : 0u;
  return encode_v(x, r);
}
// The top bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(const uint32_t (&u)[8], int k) {
  return __byte_perm(__byte_perm(u[k], u[k + 1], 0x0073), __byte_perm(u[k + 2], u[k + 3], 0x0073),
                     0x5410);
}
// The larger magnitude, NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// a + b, where a and b may be products: a packed multiplication and addition are contracted into a
// fused one in spite of their rounding modifiers, the scalar intrinsic is not.
__device__ __forceinline__ f2 add2_unfused(f2 a, f2 b) {
  const float2 x = split(a), y = split(b);
  return pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// Square roots of two numbers in [kRootLow, kRootHigh], correctly rounded: the approximate
// reciprocal root r, s = v r, and Markstein's correction s + (v - s^2) r / 2 with a fused residual
// ("IA-64 and Elementary Functions", square root), which leaves a relative 2^-45 before the last
// rounding.  That this is the nearest for every mantissa and both parities of the exponent was
// tested exhaustively (qlora_selftest_root); scaling by a power of 4 changes nothing.
constexpr float kRootLow = 1e-30f, kRootHigh = 1e30f;
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 root2(f2 v) {
  const float2 x = split(v);
  const f2 r = pair(rsqrt_approx(x.x), rsqrt_approx(x.y));
  const f2 s = mul2(v, r);
  const f2 e = fma2(mul2(s, both(-1.f)), s, v);
  return fma2(e, mul2(r, both(0.5f)), s);
}

// The tensor that block `b` of the launch belongs to.
template <int N>
__device__ __forceinline__ int tensor_of(const AdamTable<N>& t, int n, uint32_t b) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.t[mid].block0 <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// 8 elements at i of a tensor of n (bf16 or fp32); elements past the end read 0.
__device__ __forceinline__ void load8(const void* p, bool f32, int64_t i, int64_t n,
                                      float (&f)[8]) {
  if (i + 8 <= n) {
    load_either<8>(p, f32, i, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < n ? load_either1(p, f32, i + k) : 0.f;
  }
}

// This CTA's blocks of the norm: a contiguous share of the launch's, its warps taking turns.
__device__ __forceinline__ uint32_t share(uint32_t blocks, uint32_t cta) {
  return static_cast<uint32_t>(static_cast<uint64_t>(blocks) * cta / gridDim.x);
}

__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// The factors of the bias corrections of step t.
__device__ __forceinline__ void corrections(const AdamArgs& a, int64_t t, float* c1, float* c2) {
  *c1 = static_cast<float>(1.0 / (1.0 - power(a.b1d, t)));
  *c2 = static_cast<float>(1.0 / sqrt(1.0 - power(a.b2d, t)));
}

// Sums of squares of the gradients, in 64 bits (no overflow for finite gradients), one a CTA.  Each
// CTA of the step adds them up, in the same order, instead of a last CTA here: that one would wait
// for a fence, a ticket and the other sums, and the step for it.
template <int N>
__global__ void __launch_bounds__(kAdamThreads)
    adam_norm_kernel(const __grid_constant__ AdamTable<N> table, const AdamArgs a) {
  __shared__ double s[kAdamWarps];
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t end = share(a.blocks, blockIdx.x + 1);
  uint32_t b = share(a.blocks, blockIdx.x) + warp;
  double sum = 0.0;
  if (b < end) {
    int ti = tensor_of(table, a.tensors, b);
    for (; b < end; b += kAdamWarps) {
      while (ti + 1 < a.tensors && table.t[ti + 1].block0 <= b) ++ti;
      const AdamTensor& t = table.t[ti];
      float g[8];
      load8(t.g, t.flags & 2u, static_cast<int64_t>(b - t.block0) * kAdamBlock + lane * 8, t.n, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double d = static_cast<double>(g[k]);
        sum += d * d;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) s[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < kAdamWarps; ++i) t += s[i];
    a.part[a.part_first + blockIdx.x] = t;
  }
}

// What a lane holds of a block: 8 elements' parameters, gradients and moments.
template <bool BITS8>
struct Held {
  float p[8], g[8];
  f2 m[BITS8 ? 1 : 4], v[BITS8 ? 1 : 4];  // 32 bits
  uint2 cm, cv;
  float sm, sv;
};

// The parameter that the step is taken on: the master copy, or p itself.
__device__ __forceinline__ bool lead_f32(const AdamTensor& t) { return t.master || (t.flags & 1u); }
__device__ __forceinline__ void* lead(const AdamTensor& t) { return t.master ? t.master : t.p; }

template <bool BITS8>
__device__ __forceinline__ void load_block(const AdamTensor& t, const AdamArgs& a, uint32_t b,
                                           int lane, Held<BITS8>& h) {
  const int64_t i = static_cast<int64_t>(b - t.block0) * kAdamBlock + lane * 8;
  const int64_t gb = a.first_block + b, e0 = gb * kAdamBlock + lane * 8;
  load8(t.g, t.flags & 2u, i, t.n, h.g);
  load8(lead(t), lead_f32(t), i, t.n, h.p);
  if constexpr (BITS8) {
    h.cm = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + e0);
    h.cv = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + e0);
    h.sm = a.m_scale[gb];
    h.sv = a.v_scale[gb];
  } else {
    float m[8], v[8];
    load_vec<8>(static_cast<const float*>(a.m) + e0, m);
    load_vec<8>(static_cast<const float*>(a.v) + e0, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h.m[k] = pair(m[2 * k], m[2 * k + 1]);
      h.v[k] = pair(v[2 * k], v[2 * k + 1]);
    }
  }
}

template <bool BITS8, int N>
__global__ void __launch_bounds__(kAdamThreads, 3)
    adam_step_kernel(const __grid_constant__ AdamTable<N> table,
                     const __grid_constant__ AdamArgs a) {
  __shared__ float sc[2];
  __shared__ double parts[kAdamWarps];
  __shared__ int64_t step_s;
  __shared__ uint32_t ahead[2];  // the next chunk, by turns, and the tensor of its first block
  __shared__ int ahead_ti[2];
  __shared__ CodeTables codes;
  if constexpr (BITS8) fill_tables(codes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The CTA's chunks of blocks: two by its place, the others by tickets.  The chunk after the
  // current one is known, so that its first blocks can be on their way.
  const int size_bits = 3 + a.round_bits;
  static_assert(kAdamWarps == 8, "size_bits");
  const uint32_t chunks = (a.blocks + (1u << size_bits) - 1) >> size_bits;
  const bool tickets = chunks > 2 * gridDim.x;
  uint32_t chunk = blockIdx.x, drawn = 0;
  uint32_t b = (chunk << size_bits) + warp;
  int round = 0, parity = 0, ti = 0;
  if (b < a.blocks) ti = tensor_of(table, a.tensors, b);
  if (threadIdx.x == 0) {
    ahead[0] = chunk + gridDim.x;
    ahead_ti[0] = ahead[0] < chunks ? tensor_of(table, a.tensors, ahead[0] << size_bits) : 0;
    ahead[1] = chunks;
  }
  // What earlier kernels wrote is promised after this grid's own wait only, so nothing is read before
  // it, though the norm's kernel in front has waited for them.  (With the first loads ahead of it: one
  // block's adapters 12.5 us instead of 13.9, the 8B ones in 8 bits 217 instead of 220.)
  pdl_wait();
  AdamState* st = static_cast<AdamState*>(a.state);
  Held<BITS8> h;
  if (b < a.blocks)  // the first block is on its way while the corrections are worked out
    load_block(table.t[ti], a, b, lane, h);
  if (threadIdx.x == 0) {
    step_s = st->step + 1;
    corrections(a, step_s, &sc[0], &sc[1]);
  }
  float factor = static_cast<float>(a.grad_scale);
  if (a.use_norm) {
    double t = 0.0;
    for (int i = threadIdx.x; i < a.part_count; i += kAdamThreads) t += a.part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if (lane == 0) parts[warp] = t;
  }
  __syncthreads();
  pdl_trigger();
  if (a.use_norm) {
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < kAdamWarps; ++i) t += parts[i];
    const double norm = sqrt(t) * fabs(a.grad_scale);
    if (a.max_norm > 0.0)
      factor = static_cast<float>(a.grad_scale * fmin(1.0, a.max_norm / (norm + 1e-6)));
    const float reported = static_cast<float>(norm);
    const bool ok = isfinite(reported);  // what the caller sees decides
    if (a.last && blockIdx.x == 0 && threadIdx.x == 0) {
      st->norm = reported;
      st->skipped += !ok;
    }
    if (!ok) return;  // the whole step is left out
  }
  const float c1 = sc[0];
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const uint32_t word = mix32(mix32(a.seed) + static_cast<uint32_t>(step_s));
  const f2 c2 = both(sc[1]), eps = both(a.eps), fac = both(factor);

  while (chunk < chunks) {
    if (tickets && round == 0 && threadIdx.x == 0)
      drawn = 2 * gridDim.x + atomicAdd(&st->next, 1u);
    const bool more = (++round >> a.round_bits) == 0;
    const uint32_t next = more ? b + kAdamWarps : (ahead[parity] << size_bits) + warp;
    if (b < a.blocks) {
      const AdamTensor& t = table.t[ti];
      const int64_t i = static_cast<int64_t>(b - t.block0) * kAdamBlock + lane * 8;
      const int64_t gb = a.first_block + b;           // block of the list
      const int64_t e0 = gb * kAdamBlock + lane * 8;  // element of the list
      const float rate = lr * t.lr_scale;
      const f2 decay = both(-rate * t.weight_decay), move = both(-rate * c1);
      f2 m2[4], v2[4];
      float vmax = 0.f, vmin = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f2 g = mul2(pair(h.g[2 * k], h.g[2 * k + 1]), fac);
        f2 mk, vk;
        if constexpr (BITS8) {
          mk = decode2(codes.m, k < 2 ? h.cm.x : h.cm.y, 2 * (k & 1), both(h.sm));
          vk = decode2(codes.v, k < 2 ? h.cv.x : h.cv.y, 2 * (k & 1), both(h.sv));
          vk = mul2(vk, vk);
        } else {
          mk = h.m[k];
          vk = h.v[k];
        }
        m2[k] = add2_unfused(mul2(mk, both(a.b1)), mul2(g, both(a.one_b1)));
        v2[k] = add2_unfused(mul2(vk, both(a.b2)), mul2(mul2(g, g), both(a.one_b2)));
        const float2 v = split(v2[k]);
        vmax = k == 0 ? max_nan(v.x, v.y) : max_nan(vmax, max_nan(v.x, v.y));
        vmin = k == 0 ? fminf(v.x, v.y) : fminf(vmin, fminf(v.x, v.y));
      }
      f2 root[4];
      if (__all_sync(0xFFFFFFFFu, vmin >= kRootLow && vmax <= kRootHigh)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) root[k] = root2(v2[k]);
      } else {  // zeros and other extremes
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = split(v2[k]);
          root[k] = pair(sqrtf(v.x), sqrtf(v.y));
        }
      }
      float p[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 d = split(fma2(root[k], c2, eps)), mm = split(m2[k]);
        const f2 u = pair(__fdividef(mm.x, d.x), __fdividef(mm.y, d.y));
        // (p + (decay + move), not p (1 - lr wd) + move: 1 - lr wd would round lr wd to 2^-24.)
        const f2 ph = pair(h.p[2 * k], h.p[2 * k + 1]);
        const float2 q = split(add2(ph, fma2(u, move, mul2(ph, decay))));
        p[2 * k] = q.x;
        p[2 * k + 1] = q.y;
      }
      // Parameters.
      const bool whole = i + 8 <= t.n;
      if (lead_f32(t)) {
        float* pf = static_cast<float*>(lead(t));
        if (whole) {
          store_vec<8>(pf + i, p);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < t.n) pf[i + k] = p[k];
        }
      } else {
        const uint32_t word2 =
            mix32(mix32(a.seed ^ 0x55555555u) + static_cast<uint32_t>(step_s));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // 16 random bits added below the bf16 ones; a NaN or infinity keeps its bits.
          const uint32_t w = __float_as_uint(p[k]);
          if ((w & 0x7F800000u) != 0x7F800000u)
            p[k] = __uint_as_float((w + (element_bits(word2, e0 + k) & 0xFFFFu)) & 0xFFFF0000u);
        }
      }
      if (!(t.flags & 1u)) {
        __nv_bfloat16* pb = static_cast<__nv_bfloat16*>(t.p);
        if (whole) {
          store_vec<8>(pb + i, p);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < t.n) pb[i + k] = __float2bfloat16_rn(p[k]);
        }
      }
      if constexpr (!BITS8) {
        float f[8];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = split(s == 0 ? m2[k] : v2[k]);
            f[2 * k] = x.x;
            f[2 * k + 1] = x.y;
          }
          store_vec<8>(static_cast<float*>(s == 0 ? a.m : a.v) + e0, f);
        }
      }
      // The next block's loads go out before this one's codes are made.
      if (next < a.blocks) {
        if (!more) ti = ahead_ti[parity];
        while (ti + 1 < a.tensors && table.t[ti + 1].block0 <= next) ++ti;
        load_block(table.t[ti], a, next, lane, h);
      }
      if constexpr (BITS8) {
        // The largest |m| and v of the block, as bits, of which a NaN is the largest of all.
        float tm = 0.f, lm = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = split(m2[k]);
          const float hi2 = max_nan(fabsf(x.x), fabsf(x.y)), lo2 = fminf(fabsf(x.x), fabsf(x.y));
          tm = k == 0 ? hi2 : max_nan(tm, hi2);
          lm = k == 0 ? lo2 : fminf(lm, lo2);
        }
        uint32_t am = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tm));
        // (The root rounds monotonically: the largest root is the largest v's.)
        uint32_t ar = __float_as_uint(
            sqrtf(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vmax)))));
        if (am < 0x00800000u) am = 0;  // below the normal numbers: a block of zeros
        if (ar < 0x00800000u) ar = 0;
        const float sm = __uint_as_float(am), sv = __uint_as_float(ar);
        const f2 im = both(am ? __fdiv_rn(1.f, sm) : 0.f), iv = both(ar ? __fdiv_rn(1.f, sv) : 0.f);
        const uint32_t lo = static_cast<uint32_t>(e0);
        const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(e0) >> 32) * 0x9E3779B1u;
        uint32_t um[8], uv[8];
        auto make = [&](auto em, auto ev) {
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float2 s = split(m2[k / 2]);
            const float2 x = split(mul2(pair(fabsf(s.x), fabsf(s.y)), im));
            const float2 y = split(mul2(root[k / 2], iv));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t r = mix32(((lo + k + q) ^ hi) + word);
              const uint32_t c = em(q ? x.y : x.x, r);
              um[k + q] =
                  (c & 0x7FFFFFFFu) | (__float_as_uint(q ? s.y : s.x) & 0x80000000u);
              uv[k + q] = ev(q ? y.y : y.x, r);
            }
          }
        };
        // (A little above, for the rounding of the quotients.)
        if (__any_sync(0xFFFFFFFFu, !(lm > 1.001f * kMLeast * sm &&
                                        vmin > 1.002f * (kVLeast * sv) * (kVLeast * sv))))
          make(encode_m_any, encode_v_any);
        else
          make(encode_m, encode_v);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + e0) = make_uint2(top_bytes(um, 0), top_bytes(um, 4));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + e0) = make_uint2(top_bytes(uv, 0), top_bytes(uv, 4));
        if (lane == 0) {
          a.m_scale[gb] = sm;
          a.v_scale[gb] = sv;
        }
      }
    }
    b = next;
    if (more) continue;
    round = 0;
    chunk = ahead[parity];
    parity ^= 1;
    if (tickets) {  // (what was read is written again only after the next chunk's barrier)
      if (threadIdx.x == 0) {
        ahead[parity] = drawn;
        ahead_ti[parity] = drawn < chunks ? tensor_of(table, a.tensors, drawn << size_bits) : 0;
      }
      __syncthreads();
    }
  }
  // The last CTA closes the launch: no ticket is drawn, and the step count not read, any more.
  __syncthreads();
  if ((tickets || a.last) && threadIdx.x == 0 &&
      atomicAdd(&st->ticket, 1u) == gridDim.x - 1) {
    if (a.last) st->step = step_s;
    st->next = 0;
    st->ticket = 0;
  }
}

// Counts the numbers first, first + 1, ... (as bits) whose root2 is not sqrtf's.
__global__ void __launch_bounds__(kAdamThreads)
    root_selftest_kernel(uint32_t first, uint32_t count, uint32_t* wrong) {
  uint32_t bad = 0;
  for (uint32_t i = blockIdx.x * kAdamThreads + threadIdx.x; i < count;
       i += gridDim.x * kAdamThreads) {
    const float x = __uint_as_float(first + i);
    const float2 r = split(root2(both(x)));
    bad += r.x != sqrtf(x) || r.y != r.x;
  }
  if (bad) atomicAdd(wrong, bad);
}

// The values that 8-bit moments stand for.
template <typename T>
__global__ void __launch_bounds__(kAdamThreads)
    adam_moments_kernel(const uint8_t* mc, const uint8_t* vc, const float* ms, const float* vs,
                        int64_t vectors, T* m_out, T* v_out) {
  __shared__ CodeTables codes;
  fill_tables(codes);
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kAdamThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAdamThreads + threadIdx.x; i < vectors;
       i += stride) {
    const uint2 cm = reinterpret_cast<const uint2*>(mc)[i];
    const uint2 cv = reinterpret_cast<const uint2*>(vc)[i];
    const float sm = ms[i / (kAdamBlock / 8)], sv = vs[i / (kAdamBlock / 8)];
    float m[8], v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = split(decode2(codes.m, k < 2 ? cm.x : cm.y, 2 * (k & 1), both(sm)));
      const f2 r = decode2(codes.v, k < 2 ? cv.x : cv.y, 2 * (k & 1), both(sv));
      const float2 y = split(mul2(r, r));
      m[2 * k] = x.x;
      m[2 * k + 1] = x.y;
      v[2 * k] = y.x;
      v[2 * k + 1] = y.y;
    }
    store_vec<8>(m_out + i * 8, m);
    store_vec<8>(v_out + i * 8, v);
  }
}

int adam_ctas(uint32_t blocks, int cap) {
  const int64_t want = (static_cast<int64_t>(blocks) + kAdamWarps - 1) / kAdamWarps;
  return static_cast<int>(want < 1 ? 1 : (want < cap ? want : cap));
}
// CTAs of the step that the SMs hold at a time.  Three an SM with 80 registers, not four with 64 that
// spill: 233 us against 247 (54.5 M elements, 32 bits) and 221 against 225 (8 bits, with norm and the moments read).
// They draw chunks of blocks as they finish: with equal shares the SMs ended up to 15 % apart, 284 us.
// A warp's two blocks a chunk: 221 us, with one 232, with four 235.
constexpr int kStepCtas = 148 * 3, kRoundBits = 1;

}  // namespace

int adam_norm_ctas(uint32_t blocks) { return adam_ctas(blocks, kAdamNormCtas); }

namespace {
template <int N>
AdamTable<N> table_of(const AdamTensor* t, int n) {
  AdamTable<N> table;
  std::memcpy(table.t, t, n * sizeof(AdamTensor));
  return table;
}
template <int N>
cudaError_t launch_norm(const AdamTensor* t, const AdamArgs& a, cudaStream_t stream) {
  return launch_pdl(adam_norm_kernel<N>, dim3(adam_norm_ctas(a.blocks)), dim3(kAdamThreads), 0,
                    stream, 1, table_of<N>(t, a.tensors), a);
}
template <int N>
cudaError_t launch_step(const AdamTensor* t, const AdamArgs& args, cudaStream_t stream) {
  const dim3 grid(adam_ctas(args.blocks, kStepCtas));
  AdamArgs a = args;
  a.round_bits = args.blocks > 8 * kAdamWarps * kStepCtas ? kRoundBits : 0;
  if (a.bits8)
    return launch_pdl(adam_step_kernel<true, N>, grid, dim3(kAdamThreads), 0, stream, 1,
                      table_of<N>(t, a.tensors), a);
  return launch_pdl(adam_step_kernel<false, N>, grid, dim3(kAdamThreads), 0, stream, 1,
                    table_of<N>(t, a.tensors), a);
}
}  // namespace

cudaError_t launch_adam_norm(const AdamTensor* t, const AdamArgs& a, cudaStream_t stream) {
  return a.tensors <= kAdamFew ? launch_norm<kAdamFew>(t, a, stream)
                               : launch_norm<kAdamTensors>(t, a, stream);
}

cudaError_t launch_adam_step(const AdamTensor* t, const AdamArgs& a, cudaStream_t stream) {
  return a.tensors <= kAdamFew ? launch_step<kAdamFew>(t, a, stream)
                               : launch_step<kAdamTensors>(t, a, stream);
}

cudaError_t launch_adam_moments(const AdamArgs& a, int64_t blocks, void* m_out, void* v_out,
                                bool out_f32, cudaStream_t stream) {
  const int64_t vectors = blocks * (kAdamBlock / 8);
  const int64_t want = (vectors + kAdamThreads - 1) / kAdamThreads;
  const dim3 grid(static_cast<unsigned>(want < 148 * 32 ? want : 148 * 32));
  const uint8_t* m = static_cast<const uint8_t*>(a.m);
  const uint8_t* v = static_cast<const uint8_t*>(a.v);
  if (out_f32)
    return launch_pdl(adam_moments_kernel<float>, grid, dim3(kAdamThreads), 0, stream, 1, m, v,
                      a.m_scale, a.v_scale, vectors, static_cast<float*>(m_out),
                      static_cast<float*>(v_out));
  return launch_pdl(adam_moments_kernel<__nv_bfloat16>, grid, dim3(kAdamThreads), 0, stream, 1, m,
                    v, a.m_scale, a.v_scale, vectors, static_cast<__nv_bfloat16*>(m_out),
                    static_cast<__nv_bfloat16*>(v_out));
}

cudaError_t launch_root_selftest(uint32_t first, uint32_t count, uint32_t* wrong,
                                 cudaStream_t stream) {
  root_selftest_kernel<<<148 * 8, kAdamThreads, 0, stream>>>(first, count, wrong);
  return cudaGetLastError();
}

}  // namespace qlora
