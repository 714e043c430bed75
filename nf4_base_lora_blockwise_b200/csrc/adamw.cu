// adamw.cu -- one AdamW step over many tensors in one launch, moments in fp32 or in 8 bits:
//   g = grad_scale clip grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//   clip = min(1, max_norm / (||grad_scale grad|| + 1e-6)) over all tensors; a norm that is not
//   finite leaves parameters, moments and the step count as they are.
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
// Bound by memory.  A warp takes one block of 256 at a time, 8 consecutive elements a lane, so
// every access is 16 or 32 bytes a lane (8 for codes) and a block's scale is one warp reduction.
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace qlora {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;

// A 32-bit integer hash: multiplications by odd numbers between shifted exclusive ors.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t element_bits(uint32_t word, int64_t e) {
  const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(e) >> 32);
  return mix32((static_cast<uint32_t>(e) ^ (hi * 0x9E3779B1u)) + word);
}

constexpr int kMBase = 889, kVBase = 1777;  // fp32 bits >> 20 of 1.0 less 127, >> 19 less 255
constexpr float kMLeast = 1.25f / 65536.f;  // the value of m's code 1

__device__ __forceinline__ float decode_m(uint32_t c, float scale) {
  const uint32_t mag = c & 127u;
  const float x = mag ? __uint_as_float((mag + kMBase) << 20) : 0.f;
  return __fmul_rn((c & 128u) ? -x : x, scale);
}
__device__ __forceinline__ float decode_v(uint32_t c, float scale) {
  const float root = __fmul_rn(c ? __uint_as_float((c + kVBase) << 19) : 0.f, scale);
  return __fmul_rn(root, root);
}
// Codes for a magnitude x = |m| / scale or sqrt(v) / scale in [0, 1]; r: 16 random bits.
__device__ __forceinline__ uint32_t encode_m(float x, uint32_t r) {
  if (x < kMLeast) return __fmul_rn(static_cast<float>(r), kMLeast / 65536.f) < x ? 1u : 0u;
  const uint32_t c = ((__float_as_uint(x) + (r << 4)) >> 20) - kMBase;
  return c > 127u ? 127u : c;
}
__device__ __forceinline__ uint32_t encode_v(float x, uint32_t r) {
  if (!(x > 0.f)) return 0u;
  const int c = static_cast<int>((__float_as_uint(x) + (r << 3)) >> 19) - kVBase;
  return c < 1 ? 1u : (c > 255 ? 255u : static_cast<uint32_t>(c));
}

// The tensor that block `b` of the launch belongs to.
__device__ __forceinline__ int tensor_of(const AdamTable& t, int n, uint32_t b) {
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

// This CTA's blocks: a contiguous share of the launch's, its warps taking turns.
__device__ __forceinline__ uint32_t share(uint32_t blocks, uint32_t cta) {
  return static_cast<uint32_t>(static_cast<uint64_t>(blocks) * cta / gridDim.x);
}

__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// Sums of squares of the scaled gradients, in 64 bits (no overflow for finite gradients), one a
// CTA; the last CTA of the list adds them in order and leaves norm and factor in the state.
__global__ void __launch_bounds__(kAdamThreads)
    adam_norm_kernel(const __grid_constant__ AdamTable table, const AdamArgs a) {
  __shared__ double s[kAdamWarps];
  __shared__ bool last;
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
  AdamState* st = static_cast<AdamState*>(a.state);
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < kAdamWarps; ++i) t += s[i];
    a.part[a.part_first + blockIdx.x] = t;
    last = false;
    if (a.last) {
      __threadfence();
      last = atomicAdd(&st->ticket, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0.0;
  for (int i = threadIdx.x; i < a.part_count; i += kAdamThreads) t += __ldcg(a.part + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  if (lane == 0) s[warp] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = 0.0;
    for (int i = 0; i < kAdamWarps; ++i) t += s[i];
    const double norm = sqrt(t) * fabs(static_cast<double>(a.grad_scale));
    double clip = 1.0;
    if (a.max_norm > 0.f) clip = fmin(1.0, static_cast<double>(a.max_norm) / (norm + 1e-6));
    st->norm = static_cast<float>(norm);
    st->factor = static_cast<float>(static_cast<double>(a.grad_scale) * clip);
    const int ok = isfinite(norm);
    st->finite = ok;
    if (!ok) st->skipped += 1;
    st->ticket = 0;
  }
}

template <bool BITS8>
__global__ void __launch_bounds__(kAdamThreads)
    adam_step_kernel(const __grid_constant__ AdamTable table, const AdamArgs a) {
  __shared__ float sc[2];
  __shared__ int64_t step_s;
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  AdamState* st = static_cast<AdamState*>(a.state);
  if (a.use_norm && !st->finite) return;  // the whole step is left out
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    const int64_t t = st->step + 1;
    step_s = t;
    sc[0] = static_cast<float>(1.0 / (1.0 - power(a.b1d, t)));
    sc[1] = static_cast<float>(1.0 / sqrt(1.0 - power(a.b2d, t)));
  }
  __syncthreads();
  const float c1 = sc[0], c2 = sc[1];
  const float factor = a.use_norm ? st->factor : a.grad_scale;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const uint32_t word = mix32(mix32(a.seed) + static_cast<uint32_t>(step_s));
  const uint32_t word2 = mix32(mix32(a.seed ^ 0x55555555u) + static_cast<uint32_t>(step_s));

  const uint32_t end = share(a.blocks, blockIdx.x + 1);
  uint32_t b = share(a.blocks, blockIdx.x) + warp;
  if (b < end) {
    int ti = tensor_of(table, a.tensors, b);
    for (; b < end; b += kAdamWarps) {
      while (ti + 1 < a.tensors && table.t[ti + 1].block0 <= b) ++ti;
      const AdamTensor& t = table.t[ti];
      const int64_t i = static_cast<int64_t>(b - t.block0) * kAdamBlock + lane * 8;
      const int64_t gb = a.first_block + b;          // block of the list
      const int64_t e0 = gb * kAdamBlock + lane * 8;  // element of the list
      float g[8], p[8], m[8], v[8];
      load8(t.g, t.flags & 2u, i, t.n, g);
      const bool p32 = t.master || (t.flags & 1u);
      float* pf = t.master ? t.master : static_cast<float*>(t.p);
      load8(p32 ? static_cast<const void*>(pf) : t.p, p32, i, t.n, p);
      if constexpr (BITS8) {
        const uint2 cm = reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + e0)[0];
        const uint2 cv = reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + e0)[0];
        const float sm = a.m_scale[gb], sv = a.v_scale[gb];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m[k] = decode_m(((k < 4 ? cm.x : cm.y) >> (8 * (k & 3))) & 255u, sm);
          v[k] = decode_v(((k < 4 ? cv.x : cv.y) >> (8 * (k & 3))) & 255u, sv);
        }
      } else {
        load_vec<8>(static_cast<const float*>(a.m) + e0, m);
        load_vec<8>(static_cast<const float*>(a.v) + e0, v);
      }
      const float rate = lr * t.lr_scale;
      const float keep = 1.f - rate * t.weight_decay, move = rate * c1;
      float root[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float gk = __fmul_rn(g[k], factor);
        m[k] = __fadd_rn(__fmul_rn(m[k], a.b1), __fmul_rn(gk, a.one_b1));
        v[k] = __fadd_rn(__fmul_rn(v[k], a.b2), __fmul_rn(__fmul_rn(gk, gk), a.one_b2));
        root[k] = sqrtf(v[k]);
        p[k] = p[k] * keep - move * __fdividef(m[k], root[k] * c2 + a.eps);
      }
      // Parameters.
      const bool whole = i + 8 <= t.n;
      if (p32) {
        if (whole) {
          store_vec<8>(pf + i, p);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < t.n) pf[i + k] = p[k];
        }
      } else {
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
      // Moments.
      if constexpr (BITS8) {
        uint32_t am = 0, ar = 0;  // as bits: a NaN is the largest, and the block's scale
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          am = max(am, __float_as_uint(m[k]) & 0x7FFFFFFFu);
          ar = max(ar, __float_as_uint(root[k]) & 0x7FFFFFFFu);
        }
        am = __reduce_max_sync(0xFFFFFFFFu, am);
        ar = __reduce_max_sync(0xFFFFFFFFu, ar);
        if (am < 0x00800000u) am = 0;  // below the normal numbers: a block of zeros
        if (ar < 0x00800000u) ar = 0;
        const float sm = __uint_as_float(am), sv = __uint_as_float(ar);
        const float im = am ? __fdiv_rn(1.f, sm) : 0.f, iv = ar ? __fdiv_rn(1.f, sv) : 0.f;
        uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t r = element_bits(word, e0 + k);
          const uint32_t c = encode_m(__fmul_rn(fabsf(m[k]), im), r & 0xFFFFu) |
                             (m[k] < 0.f ? 128u : 0u);
          cm[k >> 2] |= c << (8 * (k & 3));
          cv[k >> 2] |= encode_v(__fmul_rn(root[k], iv), r >> 16) << (8 * (k & 3));
        }
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + e0)[0] = make_uint2(cm[0], cm[1]);
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + e0)[0] = make_uint2(cv[0], cv[1]);
        if (lane == 0) {
          a.m_scale[gb] = sm;
          a.v_scale[gb] = sv;
        }
      } else {
        store_vec<8>(static_cast<float*>(a.m) + e0, m);
        store_vec<8>(static_cast<float*>(a.v) + e0, v);
      }
    }
  }
  if (a.last) {  // every CTA has read the step count before it takes its ticket
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(&st->ticket, 1u) == gridDim.x - 1) {
      st->step = step_s;
      st->ticket = 0;
    }
  }
}

// The values that 8-bit moments stand for.
template <typename T>
__global__ void __launch_bounds__(kAdamThreads)
    adam_moments_kernel(const uint8_t* mc, const uint8_t* vc, const float* ms, const float* vs,
                        int64_t vectors, T* m_out, T* v_out) {
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
    for (int k = 0; k < 8; ++k) {
      m[k] = decode_m(((k < 4 ? cm.x : cm.y) >> (8 * (k & 3))) & 255u, sm);
      v[k] = decode_v(((k < 4 ? cv.x : cv.y) >> (8 * (k & 3))) & 255u, sv);
    }
    store_vec<8>(m_out + i * 8, m);
    store_vec<8>(v_out + i * 8, v);
  }
}

int adam_ctas(uint32_t blocks, int cap) {
  const int64_t want = (static_cast<int64_t>(blocks) + kAdamWarps - 1) / kAdamWarps;
  return static_cast<int>(want < 1 ? 1 : (want < cap ? want : cap));
}
constexpr int kStepCtas = 148 * 4;

}  // namespace

int adam_norm_ctas(uint32_t blocks) { return adam_ctas(blocks, kAdamNormCtas); }

cudaError_t launch_adam_norm(const AdamTable& table, const AdamArgs& a, cudaStream_t stream) {
  return launch_pdl(adam_norm_kernel, dim3(adam_norm_ctas(a.blocks)), dim3(kAdamThreads), 0,
                    stream, 1, table, a);
}

cudaError_t launch_adam_step(const AdamTable& table, const AdamArgs& a, cudaStream_t stream) {
  if (a.bits8)
    return launch_pdl(adam_step_kernel<true>, dim3(adam_ctas(a.blocks, kStepCtas)), dim3(kAdamThreads), 0,
                      stream, 1, table, a);
  return launch_pdl(adam_step_kernel<false>, dim3(adam_ctas(a.blocks, kStepCtas)), dim3(kAdamThreads), 0,
                    stream, 1, table, a);
}

cudaError_t launch_adam_moments(const AdamArgs& a, int64_t blocks, void* m_out, void* v_out,
                                bool out_f32, cudaStream_t stream) {
  const int64_t vectors = blocks * (kAdamBlock / 8);
  const int64_t want = (vectors + kAdamThreads - 1) / kAdamThreads;
  const dim3 grid(static_cast<unsigned>(want < 148 * 8 ? want : 148 * 8));
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

}  // namespace qlora
