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
// Bound by memory: each rotated head is read and written once.  A CTA takes a few tokens; every
// thread has four 16-byte vectors on their way while the tokens' cosines and
// sines, once for all heads, go to shared memory.
// Measured, bf16: 4096 tokens of 40 of 48 heads of 128 in place 16.8 us, 5.0 TB/s; 16384 tokens of
// two tensors of 40 heads of 80, half of each interleaved, to others 76 us, 5.5 TB/s; 16 tokens 1.8 us.
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "divide.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace qlora {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 1024;  // cosines (and sines) a CTA holds
constexpr int kRopeTokens = 8;     // tokens of a CTA at most
// Items of a thread in flight: 32 bytes each in two vectors, 16 in one.  (4 of two vectors measured
// 10 % slower: fewer CTAs fit.)
constexpr int kRopePairs = 2, kRopeSingles = 4;
constexpr int kRopeCtas = 4 * 148;  // that the SMs hold at a time

// Work of one token: items of VEC elements (interleaved) or VEC pairs (halves), `groups` a head and
// the heads of both tensors one after the other; then `copies` a head of VEC elements that pass.
struct RopeShape {
  int tokens;       // of one CTA
  int turned;       // items of a token
  int items;        // ... copied ones included
  Divide by_items, by_groups, by_copies, by_half;
};

// A vector of VEC elements as it lies in memory.
template <typename T, int VEC>
struct Raw {
  static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
  using Word = std::conditional_t<kBytes >= 16, uint4,
                                  std::conditional_t<kBytes == 8, uint2,
                                                     std::conditional_t<kBytes == 4, uint32_t,
                                                                        uint16_t>>>;
  static constexpr int kWords = kBytes / static_cast<int>(sizeof(Word));
  Word w[kWords];
};
template <typename T, int VEC>
__device__ __forceinline__ void get(const T* p, Raw<T, VEC>& r) {
#pragma unroll
  for (int i = 0; i < Raw<T, VEC>::kWords; ++i)
    r.w[i] = reinterpret_cast<const typename Raw<T, VEC>::Word*>(p)[i];
}
template <typename T, int VEC>
__device__ __forceinline__ void floats(const Raw<T, VEC>& r, float (&f)[VEC]) {
  const T* p = reinterpret_cast<const T*>(&r);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = p[k];
  } else if constexpr (VEC == 1) {
    f[0] = __bfloat162float(p[0]);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      const float2 x = bf16x2_floats(w[k]);
      f[2 * k] = x.x;
      f[2 * k + 1] = x.y;
    }
  }
}

template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 4)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeShape s) {
  // Items in flight; vectors of an item (two neighbours where a vector is one element), and how
  // far the second lies from the first.
  constexpr int V = INTERLEAVED && VEC > 1 ? 1 : 2;
  constexpr int U = V == 1 && sizeof(T) == 2 ? kRopeSingles : kRopePairs;
  __shared__ __align__(16) float cs[kRopeAngles], sn[kRopeAngles];
  __shared__ int64_t at[kRopeTokens][4];  // x and out of q and of k: the tokens' offsets
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const int half = a.rotary_dim / 2;
  const int apart = INTERLEAVED ? 1 : half;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * s.tokens;
  const int tokens = a.M - m0 < s.tokens ? static_cast<int>(a.M - m0) : s.tokens;
  const int total = tokens * s.items;
  if (threadIdx.x < tokens) {
    const int64_t m = m0 + threadIdx.x;
    const int64_t b = a.S == a.M ? 0 : m / a.S, t = m - b * a.S;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      at[threadIdx.x][2 * i] = b * a.t[i].x_batch + t * a.t[i].x_token;
      at[threadIdx.x][2 * i + 1] = b * a.t[i].out_batch + t * a.t[i].out_token;
    }
  }
  __syncthreads();

  // Where item n's vectors lie, and its angles: the first in the CTA's tables, or -1 (copied).
  auto place = [&](int n, const T*& x, T*& o, int& angle) {
    const int tok = s.tokens == 1 ? 0 : quotient(n, s.by_items);
    int j = n - tok * s.items;
    const bool turn = j < s.turned;
    j -= turn ? 0 : s.turned;
    const Divide d = turn ? s.by_groups : s.by_copies;
    int head = quotient(j, d);
    const int g = j - head * d.d;
    const bool second = head >= a.t[0].heads;
    head -= second ? a.t[0].heads : 0;
    const RopeHeads& h = second ? a.t[1] : a.t[0];
    const int e = !turn ? a.rotary_dim + g * VEC : (INTERLEAVED && VEC == 1 ? g * 2 : g * VEC);
    x = static_cast<const T*>(h.x) + at[tok][second ? 2 : 0] + head * h.x_head + e;
    o = static_cast<T*>(h.out) + at[tok][second ? 3 : 1] + head * h.out_head + e;
    angle = !turn ? -1 : tok * half + (INTERLEAVED && VEC > 1 ? g * (VEC / 2) : g * VEC);
  };

  bool angles = false;
  const int stride = kRopeThreads * gridDim.y;
  for (int n0 = blockIdx.y * kRopeThreads; n0 < total; n0 += U * stride) {
    T* out[U];
    int angle[U];
    Raw<T, VEC> r[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + threadIdx.x + u * stride;
      if (n >= total) continue;
      const T* x;
      place(n, x, out[u], angle[u]);
      get(x, r[u][0]);
      if (V == 2 && angle[u] >= 0) get(x + apart, r[u][V - 1]);
    }
    if (!angles) {  // while the first loads are on their way
      angles = true;
      for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
        const int tok = quotient(i, s.by_half), pair = i - tok * half;
        const int64_t m = m0 + tok;
        const int64_t pos = !a.positions ? a.start + (a.S == a.M ? m : m % a.S)
                            : a.pos64    ? static_cast<const int64_t*>(a.positions)[m]
                                         : static_cast<const int32_t*>(a.positions)[m];
        const uint64_t turn = static_cast<uint64_t>(pos) * a.phase[pair];
        const int32_t top = static_cast<int32_t>(turn >> 32);
        float c, n;
        sincospif(static_cast<float>(top) * (1.f / 2147483648.f), &n, &c);
        cs[i] = c * a.scale;
        sn[i] = (a.inverse ? -n : n) * a.scale;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + threadIdx.x + u * stride;
      if (n >= total) continue;
      float lo[VEC];
      floats<T, VEC>(r[u][0], lo);
      if (angle[u] < 0) {
        store_vec<VEC>(out[u], lo);
      } else if constexpr (V == 1) {
        float c[VEC / 2], q[VEC / 2];
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          c[k] = cs[angle[u] + k];
          q[k] = sn[angle[u] + k];
        }
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
          const float x = lo[k], y = lo[k + 1];
          lo[k] = x * c[k / 2] - y * q[k / 2];
          lo[k + 1] = y * c[k / 2] + x * q[k / 2];
        }
        store_vec<VEC>(out[u], lo);
      } else {
        float hi[VEC], c[VEC], q[VEC];
        floats<T, VEC>(r[u][V - 1], hi);
        load_vec<VEC>(cs + angle[u], c);
        load_vec<VEC>(sn + angle[u], q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float x = lo[k], y = hi[k];
          lo[k] = x * c[k] - y * q[k];
          hi[k] = y * c[k] + x * q[k];
        }
        store_vec<VEC>(out[u], lo);
        store_vec<VEC>(out[u] + apart, hi);
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

// The widest access that every vector of every head is aligned to: 8 elements, 4, 2 or 1.
int rope_vec(const RopeArgs& a) {
  const int e = a.f32 ? 4 : 2;
  const int half = a.rotary_dim / 2;
  const int run = a.interleaved ? a.rotary_dim : half;
  for (int vec : {8, 4, 2}) {
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

// Items of a head that are turned, and copied ones, in vectors of vec.
int turned_items(const RopeArgs& a, int vec) {
  return a.interleaved ? a.rotary_dim / (vec < 2 ? 2 : vec) : a.rotary_dim / 2 / vec;
}
int copied_items(const RopeArgs& a, int vec) {
  return a.copy ? (a.head_dim - a.rotary_dim) / vec : 0;
}

// One launch, of no more heads than its divisions are exact for.
cudaError_t launch_heads(const RopeArgs& a, int vec, cudaStream_t stream) {
  const int half = a.rotary_dim / 2;
  const int heads = a.t[0].heads + a.t[1].heads;
  const int groups = turned_items(a, vec), copies = copied_items(a, vec);
  RopeShape s;
  s.turned = heads * groups;
  s.items = heads * (groups + copies);
  s.by_groups = divide_by(groups);
  s.by_copies = divide_by(copies > 0 ? copies : 1);
  s.by_half = divide_by(half);
  s.by_items = divide_by(s.items);
  // Tokens of a CTA: as many as fill its threads' items best, of those its tables hold and its
  // divisions take, and that leave the SMs full.
  const bool singles = a.interleaved && vec > 1 && !a.f32;
  const int round = kRopeThreads * (singles ? kRopeSingles : kRopePairs);
  s.tokens = 1;
  double best = 0.0;
  for (int t = 1; t <= kRopeTokens; ++t) {
    if (t * half > kRopeAngles || (t > 1 && a.M < 2ll * kRopeCtas * t)) break;
    const int64_t n = static_cast<int64_t>(t) * s.items;
    if (t > 1 && n * s.items >= 0x100000000ll) break;
    const double fill = static_cast<double>(n) / ((n + round - 1) / round * round);
    if (fill > best + 0.02) {
      best = fill;
      s.tokens = t;
    }
  }
  // Few tokens: the items of one over several CTAs.
  int split = 1;
  if (a.M < kRopeCtas) {
    split = (s.items + kRopeThreads - 1) / kRopeThreads;
    const int room = static_cast<int>((kRopeCtas + a.M - 1) / a.M);
    if (split > room) split = room;
    if (split > 8) split = 8;
  }
  const int64_t ctas = (a.M + s.tokens - 1) / s.tokens;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(split));
  if (a.f32) {
    if (vec == 8) return launch<float, 8>(a, s, grid, stream);
    if (vec == 4) return launch<float, 4>(a, s, grid, stream);
    if (vec == 2) return launch<float, 2>(a, s, grid, stream);
    return launch<float, 1>(a, s, grid, stream);
  }
  if (vec == 8) return launch<__nv_bfloat16, 8>(a, s, grid, stream);
  if (vec == 4) return launch<__nv_bfloat16, 4>(a, s, grid, stream);
  if (vec == 2) return launch<__nv_bfloat16, 2>(a, s, grid, stream);
  return launch<__nv_bfloat16, 1>(a, s, grid, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream, int* launches) {
  const int vec = rope_vec(a);
  const int copied = exact_heads(copied_items(a, vec)), turned = exact_heads(turned_items(a, vec));
  const int most = copied < turned ? copied : turned;
  if (a.t[0].heads + a.t[1].heads <= most) {
    *launches = 1;
    return launch_heads(a, vec, stream);
  }
  // Out of place, over 1000 heads that copy over 1000 elements each, one by one: some heads a launch.
  for (const RopeHeads& h : a.t)
    for (int first = 0; first < h.heads; first += most) {
      RopeArgs some = a;
      RopeHeads& t = some.t[0];
      t = h;
      t.heads = h.heads - first < most ? h.heads - first : most;
      t.x = static_cast<const char*>(h.x) + first * h.x_head * (a.f32 ? 4 : 2);
      t.out = static_cast<char*>(h.out) + first * h.out_head * (a.f32 ? 4 : 2);
      some.t[1] = RopeHeads{};
      const cudaError_t e = launch_heads(some, vec, stream);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
  return cudaSuccess;
}

}  // namespace qlora
