// rope.cu -- rotary positions on heads of queries and keys, forward or inverse (the backward pass:
// the rotation's transpose).  Pair i of a head at position p turns by p f_i:
//   (a, b) -> s (a cos - b sin, b cos + a sin),
// the pair being (i, i + rd/2) of the head's first rd elements, or (2i, 2i + 1) when interleaved.
//
// Angles: f_i is held as turns per position times 2^64, so p f_i modulo 2^64 is the exact
// fraction of a turn at any position, by one 64-bit integer product; its top 32 bits become the
// fp32 argument (in half turns, [-1, 1)) of sincospif.  An fp32 product p f_i would be off by
// p 2^-24 radians: 0.06 at position 10^6.
//
// Bound by memory: each rotated head is read and written once.  A CTA takes a few tokens, works
// out their cosines and sines once for all heads into shared memory, then turns 16-byte vectors.
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace qlora {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 1024;  // cosines (and sines) a CTA holds

// Work of one token, in items of VEC elements (interleaved) or VEC pairs (halves), heads of both
// tensors one after the other; after them the items of VEC elements that are copied.
struct RopeShape {
  int tokens;       // of one CTA
  int groups;       // turned items of a head
  int turned;       // of a token
  int copies;       // copied items of a head
  int items;        // of a token, copied ones included
};

template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, RopeShape s) {
  __shared__ float cs[kRopeAngles], sn[kRopeAngles];
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const int half = a.rotary_dim / 2;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * s.tokens;
  const int tokens = a.M - m0 < s.tokens ? static_cast<int>(a.M - m0) : s.tokens;
  for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
    const int tok = i / half, pair = i - tok * half;
    const int64_t m = m0 + tok;
    const int64_t p = !a.positions ? a.start + m % a.S
                      : a.pos64    ? static_cast<const int64_t*>(a.positions)[m]
                                   : static_cast<const int32_t*>(a.positions)[m];
    const uint64_t turn = static_cast<uint64_t>(p) * a.phase[pair];
    const int32_t top = static_cast<int32_t>(turn >> 32);
    float c, n;
    sincospif(static_cast<float>(top) * (1.f / 2147483648.f), &n, &c);
    cs[i] = c * a.scale;
    sn[i] = (a.inverse ? -n : n) * a.scale;
  }
  __syncthreads();
  // Items of the CTA's tokens, this CTA's share (blockIdx.y) of each token's.
  const int stride = kRopeThreads * gridDim.y;
  for (int tok = 0; tok < tokens; ++tok) {
    const int64_t m = m0 + tok;
    const int64_t b = m / a.S, t = m - b * a.S;
    const float* ct = cs + tok * half;
    const float* st = sn + tok * half;
    for (int i = blockIdx.y * kRopeThreads + threadIdx.x; i < s.items; i += stride) {
      const bool turn = i < s.turned;
      const int per = turn ? s.groups : s.copies;
      const int j = turn ? i : i - s.turned;
      int head = j / per;
      const int g = j - head * per;
      const int which = head >= a.t[0].heads;
      head -= which ? a.t[0].heads : 0;
      const RopeHeads& h = a.t[which];
      const T* x = static_cast<const T*>(h.x) + b * h.x_batch + t * h.x_token + head * h.x_head;
      T* o = static_cast<T*>(h.out) + b * h.out_batch + t * h.out_token + head * h.out_head;
      if (!turn) {
        float v[VEC];
        load_vec<VEC>(x + a.rotary_dim + g * VEC, v);
        store_vec<VEC>(o + a.rotary_dim + g * VEC, v);
      } else if constexpr (INTERLEAVED) {
        constexpr int W = VEC < 2 ? 2 : VEC;
        float v[W];
        if constexpr (VEC >= 2) {
          load_vec<VEC>(x + g * W, v);
        } else {
          v[0] = load_either1(x, sizeof(T) == 4, g * 2);
          v[1] = load_either1(x, sizeof(T) == 4, g * 2 + 1);
        }
#pragma unroll
        for (int k = 0; k < W; k += 2) {
          const float c = ct[(g * W + k) / 2], n = st[(g * W + k) / 2];
          const float v0 = v[k] * c - v[k + 1] * n;
          v[k + 1] = v[k + 1] * c + v[k] * n;
          v[k] = v0;
        }
        if constexpr (VEC >= 2) {
          store_vec<VEC>(o + g * W, v);
        } else {
          float e[1] = {v[0]};
          store_vec<1>(o + g * 2, e);
          e[0] = v[1];
          store_vec<1>(o + g * 2 + 1, e);
        }
      } else {
        float lo[VEC], hi[VEC];
        load_vec<VEC>(x + g * VEC, lo);
        load_vec<VEC>(x + half + g * VEC, hi);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float c = ct[g * VEC + k], n = st[g * VEC + k];
          const float v0 = lo[k] * c - hi[k] * n;
          hi[k] = hi[k] * c + lo[k] * n;
          lo[k] = v0;
        }
        store_vec<VEC>(o + g * VEC, lo);
        store_vec<VEC>(o + half + g * VEC, hi);
      }
    }
  }
}

template <typename T, int VEC>
cudaError_t launch(const RopeArgs& a, const RopeShape& s, dim3 grid, cudaStream_t stream) {
  if (a.interleaved)
    return launch_pdl(rope_kernel<T, VEC, true>, grid, dim3(kRopeThreads), 0, stream, 1, a, s);
  return launch_pdl(rope_kernel<T, VEC, false>, grid, dim3(kRopeThreads), 0, stream, 1, a, s);
}

// The widest access that every vector of every head is aligned to: 8 elements, 2 or 1.
int rope_vec(const RopeArgs& a) {
  const int e = a.f32 ? 4 : 2;
  const int half = a.rotary_dim / 2;
  const int run = a.interleaved ? a.rotary_dim : half;
  for (int vec : {8, 2}) {
    const uintptr_t bytes = static_cast<uintptr_t>(vec) * e > 16 ? 16 : vec * e;
    bool ok = run % vec == 0 && (!a.copy || (a.head_dim - a.rotary_dim) % vec == 0);
    if (!a.interleaved && a.copy) ok = ok && a.rotary_dim % vec == 0;
    for (const RopeHeads& h : a.t) {
      if (!h.heads) continue;
      ok = ok && reinterpret_cast<uintptr_t>(h.x) % bytes == 0 &&
           reinterpret_cast<uintptr_t>(h.out) % bytes == 0;
      for (int64_t st : {h.x_batch, h.x_token, h.x_head, h.out_batch, h.out_token, h.out_head})
        ok = ok && (st * e) % static_cast<int64_t>(bytes) == 0;
    }
    if (ok) return vec;
  }
  return 1;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const int vec = rope_vec(a);
  const int half = a.rotary_dim / 2;
  const int heads = a.t[0].heads + a.t[1].heads;
  RopeShape s;
  s.groups = a.interleaved ? a.rotary_dim / (vec < 2 ? 2 : vec) : half / vec;
  s.copies = a.copy ? (a.head_dim - a.rotary_dim) / vec : 0;
  s.turned = heads * s.groups;
  s.items = heads * (s.groups + s.copies);
  s.tokens = kRopeAngles / half < 4 ? kRopeAngles / half : 4;
  // Few tokens: one a CTA, and its items over several.
  int split = 1;
  if (a.M < 4 * 148) {
    s.tokens = 1;
    split = (s.items + kRopeThreads - 1) / kRopeThreads;
    if (split > 8) split = 8;
  }
  const int64_t ctas = (a.M + s.tokens - 1) / s.tokens;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(split));
  if (a.f32) {
    if (vec == 8) return launch<float, 8>(a, s, grid, stream);
    if (vec == 2) return launch<float, 2>(a, s, grid, stream);
    return launch<float, 1>(a, s, grid, stream);
  }
  if (vec == 8) return launch<__nv_bfloat16, 8>(a, s, grid, stream);
  if (vec == 2) return launch<__nv_bfloat16, 2>(a, s, grid, stream);
  return launch<__nv_bfloat16, 1>(a, s, grid, stream);
}

}  // namespace qlora
