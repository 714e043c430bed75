// residual_norm.cuh -- what the forward and the backward of the residual norm share: pairs of fp32,
// row streams through shared memory, combined weights, row sums and launch shapes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace qlora {

namespace {

// ---------------------------------------------------------------------------------------------
// Row streams: [M, D] tensors read row by row.  Every thread has `slots` 16-byte slots in shared
// memory, [slot][T threads] (a copy whose lanes do not write one contiguous piece of shared memory
// measured a third slower); a stream's, and the T that a CTA has room for, are given at compile
// time, so that an access is one register and a constant.  Rows that start inside a
// granule need the granule after a warp's last: `extra`, one for each stream, vector and warp.
// ---------------------------------------------------------------------------------------------
struct Ring {
  int slots;       // of a thread
  int extra;       // byte of the extra granules, [stream][nv][warp]
  int weights;     // byte of the combined weights' [2][weights_ld] fp32
  int weights_ld;  // D rounded up to 8, and 8 zeros
  int gate_f32;    // a whole gate's type
  int gate_direct; // a whole gate that does not fit: read from global memory where it is used
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Thread geometry of one row.
struct RowAt {
  int64_t at;     // first element of the row
  int64_t total;  // M D
  int D;
  bool row;       // whether there is a row
};

// The granule of 16 bytes that starts at element e (a multiple of 16 / ESIZE; zeros from the
// tensor's end on), straight from global memory.
// (Tails are functions of their own: they are rare, and their code would be in every copy.)
template <int ESIZE>
__device__ __noinline__ uint4 ldg16_tail(const char* q, int64_t left) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 16 / ESIZE; ++k) {
    if (k >= left) break;
    if constexpr (ESIZE == 4)
      w[k] = reinterpret_cast<const uint32_t*>(q)[k];
    else
      w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(q)[k]) << (16 * (k & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int ESIZE>
__device__ __forceinline__ uint4 ldg16(const void* p, int64_t e, int64_t total) {
  const char* q = static_cast<const char*>(p) + e * ESIZE;
  if (e + 16 / ESIZE <= total) return *reinterpret_cast<const uint4*>(q);
  return ldg16_tail<ESIZE>(q, total - e);
}

template <int NV>
struct Lane {
  uint32_t slots;  // shared address of the thread's first slot
  uint32_t extra;  // of its warp's first extra granule
  uint32_t w[NV];  // of the combined weights of its columns
  int c[NV];       // first column of its vectors
};
template <int NV, int T>
__device__ __forceinline__ Lane<NV> lane_of(const Ring& ring, uint32_t smem, int D) {
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  Lane<NV> l;
  l.slots = smem + tid * 16;
  l.extra = smem + ring.extra + (tid >> 5) * 16;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    l.c[j] = (j * blockDim.x + threadIdx.x) * 8;
    // Past the row's end: the zeros behind the weights.
    const int at = l.c[j] < D ? l.c[j] : ring.weights_ld - 8;
    l.w[j] = smem + ring.weights + at * 4;
  }
  return l;
}

// Slots of threads past the end of a row of whole granules, and of groups without a row: nothing is
// copied there, they read 0.
template <int NV, int T>
__device__ __forceinline__ void clear_slots(const Ring& ring, const Lane<NV>& l, const RowAt& r) {
  if (r.row && l.c[NV - 1] < r.D) return;
  for (int i = 0; i < ring.slots; ++i)
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(l.slots + i * T * 16), "r"(0)
                 : "memory");
}

// Starts the copies of row r's granules of one stream (its number and first slot: STREAM, SLOT).
template <int ESIZE, int NV, int T, bool ALIGNED, int STREAM, int SLOT>
__device__ __forceinline__ void issue(const void* p, const Lane<NV>& l, const RowAt& r) {
  if (!r.row) return;
  constexpr int N = 16 / ESIZE;  // elements of a granule
  constexpr int G = 8 / N;       // granules of 8 columns
  if constexpr (ALIGNED) {
    const char* q = static_cast<const char*>(p) + r.at * ESIZE;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (l.c[j] < r.D) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          copy16(l.slots + (SLOT + j * G + g) * (T * 16), q + l.c[j] * ESIZE + g * 16, 16);
      }
    }
  } else {
    const int shift = static_cast<int>(r.at & (N - 1));
    const int64_t a = r.at - shift;
    const char* base = static_cast<const char*>(p);
    auto start = [&](uint32_t dst, int first) {  // the granule `first` elements after the row's
      if (first >= r.D + shift) return;
      const int64_t e = a + first;
      const int bytes = e + N > r.total ? static_cast<int>(r.total - e) * ESIZE : 16;
      copy16(dst, base + e * ESIZE, bytes);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int g = 0; g < G; ++g) start(l.slots + (SLOT + j * G + g) * (T * 16), l.c[j] + g * N);
      if ((threadIdx.x & 31) == 31) start(l.extra + (STREAM * NV + j) * (T / 32 * 16), l.c[j] + 8);
    }
  }
}

// 8 columns of row r, j-th vector of the thread, as fp32 pairs; columns outside the row read 0.
// DIRECT: from global memory.
template <int ESIZE, int NV, int T, bool ALIGNED, int STREAM, int SLOT, bool DIRECT = false>
__device__ __forceinline__ void fetch(const void* p, const Lane<NV>& l, const RowAt& r, int j,
                                      f2 (&f)[4]) {
  constexpr int N = 16 / ESIZE;
  constexpr int G = 8 / N;
  const int c = l.c[j];
  const int shift = ALIGNED ? 0 : static_cast<int>(r.at & (N - 1));
  auto granule = [&](uint32_t src, int first) {
    if constexpr (!DIRECT) return lds16(src);
    return r.row && first < r.D + shift ? ldg16<ESIZE>(p, r.at - shift + first, r.total)
                                        : make_uint4(0, 0, 0, 0);
  };
  uint32_t w[4 * G + 4];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint4 q = granule(l.slots + (SLOT + j * G + g) * (T * 16), c + g * N);
    w[4 * g] = q.x;
    w[4 * g + 1] = q.y;
    w[4 * g + 2] = q.z;
    w[4 * g + 3] = q.w;
  }
  if constexpr (!ALIGNED) {
    // The next thread's first granule, then the window moves `shift` elements up.
    uint32_t n[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = __shfl_down_sync(0xFFFFFFFFu, w[k], 1);
    if ((threadIdx.x & 31) == 31) {
      const uint4 q = granule(l.extra + (STREAM * NV + j) * (T / 32 * 16), c + 8);
      n[0] = q.x;
      n[1] = q.y;
      n[2] = q.z;
      n[3] = q.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[4 * G + k] = n[k];
    const int words = ESIZE == 4 ? shift : shift >> 1;
    if (words & 2) {
#pragma unroll
      for (int k = 0; k + 2 < 4 * G + 4; ++k) w[k] = w[k + 2];
    }
    if (words & 1) {
#pragma unroll
      for (int k = 0; k + 1 < 4 * G + 4; ++k) w[k] = w[k + 1];
    }
    if (ESIZE == 2 && (shift & 1)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
    }
    // What lies past the row's end is the next row's, or left from another row.
    const int left = r.row ? r.D - c : 0;
    if (left < 8) {
#pragma unroll
      for (int k = 0; k < 4 * G; ++k) {
        if constexpr (ESIZE == 4) {
          if (k >= left) w[k] = 0;
        } else {
          if (2 * k >= left) w[k] = 0;
          if (2 * k + 1 == left) w[k] &= 0xFFFFu;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (ESIZE == 4)
      f[k] = pair_bits(w[2 * k], w[2 * k + 1]);
    else
      f[k] = unpack_bf16(w[k]);
  }
}

// A whole gate, of a type known at run time.
template <int NV, int T, bool ALIGNED, int STREAM, int SLOT>
__device__ __forceinline__ void issue_gate(const void* p, const Ring& ring, const Lane<NV>& l,
                                           const RowAt& r) {
  if (ring.gate_direct) return;
  if (ring.gate_f32)
    issue<4, NV, T, ALIGNED, STREAM, SLOT>(p, l, r);
  else
    issue<2, NV, T, ALIGNED, STREAM, SLOT>(p, l, r);
}
template <int NV, int T, bool ALIGNED, int STREAM, int SLOT>
__device__ __forceinline__ void fetch_gate(const void* p, const Ring& ring, const Lane<NV>& l,
                                           const RowAt& r, int j, f2 (&f)[4]) {
  if (ring.gate_direct) {
    if (ring.gate_f32)
      fetch<4, NV, T, ALIGNED, STREAM, SLOT, true>(p, l, r, j, f);
    else
      fetch<2, NV, T, ALIGNED, STREAM, SLOT, true>(p, l, r, j, f);
  } else if (ring.gate_f32) {
    fetch<4, NV, T, ALIGNED, STREAM, SLOT>(p, l, r, j, f);
  } else {
    fetch<2, NV, T, ALIGNED, STREAM, SLOT>(p, l, r, j, f);
  }
}

// Stores 8 columns of row r (columns outside the row are left alone).  All threads of the warp
// call it together.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void put(T* p, const RowAt& r, int c, const f2 (&f2s)[4]) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = split(f2s[k]);
    f[2 * k] = t.x;
    f[2 * k + 1] = t.y;
  }
  if constexpr (ALIGNED) {
    if (r.row && c < r.D) store_vec<8>(p + r.at + c, f);
  } else {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    const int shift = static_cast<int>(r.at & (N - 1));
    const int lane = threadIdx.x & 31;
    // e[k]: the element at a + 8 v + k, a the row's first granule; its column is c - shift + k.
    float e[8];
    if constexpr (sizeof(T) == 4) {
      float w[11];
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k] = __shfl_up_sync(0xFFFFFFFFu, f[5 + k], 1);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[3 + k] = f[k];
      // window from 3 - shift on
      const int t = 3 - shift;
      if (t & 2) {
#pragma unroll
        for (int k = 0; k + 2 < 11; ++k) w[k] = w[k + 2];
      }
      if (t & 1) {
#pragma unroll
        for (int k = 0; k + 1 < 11; ++k) w[k] = w[k + 1];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = w[k];
    } else {
      // halfwords: the previous thread's 8, then this one's; window from 8 - shift on
      uint32_t w[9];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 + k] = floats_bf16x2(f[2 * k], f[2 * k + 1]);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __shfl_up_sync(0xFFFFFFFFu, w[4 + k], 1);
      w[8] = 0;
      const int t = 8 - shift, h = t >> 1;
      if (h & 4) {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 4];
      }
      if (h & 2) {
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
      }
      if (h & 1) {
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 1];
      }
      if (t & 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 q = bf16x2_floats(w[k]);
        e[2 * k] = q.x;
        e[2 * k + 1] = q.y;
      }
    }
    if (!r.row) return;
    T* q = p + (r.at - shift) + c;
    const int c0 = c - shift;
    if ((lane > 0 || shift == 0) && c0 >= 0 && c0 + 8 <= r.D) {
      store_vec<8>(q, e);
    } else {
      // The row's ends, and the first lane's granule, of which the warp before has the start.
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = c0 + k;
        if (col >= 0 && col < r.D && (lane > 0 || k >= shift)) {
          const float one[1] = {e[k]};
          store_vec<1>(q + k, one);
        }
      }
    }
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // the last `shift` columns of f start the next granule
        if (k >= 8 - shift && c + k < r.D) {
          const float one[1] = {f[k]};
          store_vec<1>(q + shift + k, one);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Weights of 8 columns: 0: w_pre + o; 1: (w_post + o) gate, without what is not there.
// ---------------------------------------------------------------------------------------------
struct Weights {
  const void* w_pre;
  const void* w_post;
  const void* gate;  // of a channel gate
  int weight_f32, gate_f32;
  float offset;
  int D;
};
__device__ __noinline__ void columns_tail(const void* p, bool f32, int c, int D, float* f) {
  for (int k = 0; k < 8; ++k) f[k] = c + k < D ? load_either1(p, f32, c + k) : 0.f;
}
template <bool ALIGNED>
__device__ __forceinline__ void columns8(const void* p, bool f32, int c, int D, float (&f)[8]) {
  if (ALIGNED || c + 8 <= D) {
    load_either<8>(p, f32, c, f);
  } else {
    float t[8];
    columns_tail(p, f32, c, D, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = t[k];
  }
}
template <int WHICH, bool ALIGNED>
__device__ __forceinline__ void combine8(const Weights& w, int c, float (&f)[8]) {
  const void* p = WHICH == 0 ? w.w_pre : w.w_post;
  if (p) {
    columns8<ALIGNED>(p, w.weight_f32, c, w.D, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += w.offset;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 1.f;
  }
  if (WHICH == 1) {
    if (w.gate) {
      float g[8];
      columns8<ALIGNED>(w.gate, w.gate_f32, c, w.D, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= g[k];
    }
  }
}
// Fills the CTA's shared copy (a barrier follows before the first use).
template <bool ALIGNED>
__device__ __forceinline__ void stage_weights(const Weights& w, const Ring& ring,
                                              unsigned char* smem, bool second) {
  float* d = reinterpret_cast<float*>(smem + ring.weights);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  for (int c = tid * 8; c < ring.weights_ld; c += threads * 8) {
    float f[8] = {};
    if (w.w_pre) {
      if (c < w.D) combine8<0, ALIGNED>(w, c, f);
      store_vec<8>(d + c, f);
    }
    if (second) {
      if (c < w.D) combine8<1, ALIGNED>(w, c, f);
      store_vec<8>(d + ring.weights_ld + c, f);
    }
  }
}
template <int WHICH, bool WS, bool ALIGNED, int NV>
__device__ __forceinline__ void weights8(const Weights& w, const Ring& ring, const Lane<NV>& l,
                                         int j, f2 (&f)[4]) {
  if constexpr (WS) {
    const uint32_t p = l.w[j] + WHICH * ring.weights_ld * 4;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];"
                   : "=l"(f[2 * k]), "=l"(f[2 * k + 1])
                   : "r"(p + k * 16)
                   : "memory");
  } else {
    float t[8] = {};
    if (l.c[j] < w.D) combine8<WHICH, ALIGNED>(w, l.c[j], t);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = pair(t[2 * k], t[2 * k + 1]);
  }
}

// Sums of NS values over the row's threads (blockDim.x of them, row group threadIdx.y of the
// CTA); the result in every thread.  Past one warp the warps' sums go through `buf`, which the
// group's next call with the same buf may overwrite only after another barrier: callers
// alternate.  Each group has its own barrier (1 + its number; past one warp there are at most 8).
template <int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float* buf) {
  const int tpr = blockDim.x;
  if (tpr >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int s = 0; s < NS; ++s) v[s] += __shfl_xor_sync(0xFFFFFFFFu, v[s], o);
  } else {
    for (int o = tpr / 2; o > 0; o >>= 1)
#pragma unroll
      for (int s = 0; s < NS; ++s) v[s] += __shfl_xor_sync(0xFFFFFFFFu, v[s], o);
  }
  if (tpr > 32) {
    // [group][NS][warps rounded up to 4], the padding zero from the kernel's start.
    const int warps = tpr >> 5, ld = (warps + 3) & ~3;
    float* mine = buf + threadIdx.y * NS * ld;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s) mine[s * ld + (threadIdx.x >> 5)] = v[s];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.y) + 1), "r"(tpr) : "memory");
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float t = 0.f;
      for (int i = 0; i < ld; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(mine + s * ld + i);
        t += (q.x + q.y) + (q.z + q.w);
      }
      v[s] = t;
    }
  }
}
constexpr int kSumBuf = 2 * 48;  // floats of one buffer: 2 values, 32 warps padded to 4 a group
__device__ __forceinline__ void clear_sums(float (*buf)[kSumBuf], int n) {
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int i = tid; i < n * kSumBuf; i += blockDim.x * blockDim.y) (&buf[0][0])[i] = 0.f;
}

__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int PENDING>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}


__device__ __forceinline__ void advance(RowAt& r, int64_t m, int64_t M) {
  r.row = m < M;
  r.at = m * r.D;
}

// ---------------------------------------------------------------------------------------------
// Launch shapes.
// ---------------------------------------------------------------------------------------------
// How rows of D columns are spread: two vectors of 8 a thread, tpr threads a row, rpc rows a CTA, one
// CTA an SM.  Whole granules (D % 8 == 0) let narrow rows share a warp; other rows exchange
// granules between lanes and take whole warps.
struct RowShape {
  bool aligned;
  int tpr, rpc;
  int threads;  // that a CTA has room for
  int64_t ctas;
};
constexpr int kSms = 148;
constexpr int kSmemPerCta = 222 * 1024;
inline int least_groups(const RowShape& s) { return s.tpr >= 32 ? 1 : 32 / s.tpr; }  // whole warps
inline RowShape row_shape(int64_t M, int D, int threads) {
  RowShape s;
  s.aligned = D % 8 == 0;
  s.threads = threads;
  const int need = (D + 15) / 16;
  if (s.aligned && need <= 32) {
    s.tpr = 1;
    while (s.tpr < need) s.tpr *= 2;
  } else {
    s.tpr = (need + 31) / 32 * 32;
  }
  // A CTA's groups share the weights: as many as its threads hold (8 past one warp, for their
  // barriers), no more than spreads the rows over every SM.
  s.rpc = threads / s.tpr;
  if (s.tpr > 32 && s.rpc > 8) s.rpc = 8;
  const int64_t spread = (M + kSms - 1) / kSms;
  const int least = least_groups(s);
  if (s.rpc > spread) s.rpc = static_cast<int>((spread + least - 1) / least * least);
  const int64_t want = (M + s.rpc - 1) / s.rpc;
  s.ctas = want < kSms ? want : kSms;
  return s;
}

// Lays `streams` streams of `slots` slots a thread (without the gate's) and the weights out in
// shared memory.  The weights are staged where a group has several rows to use them for and the
// widest rows leave room; a whole gate of the widest rows may not fit either.  Bytes.
inline int plan_ring(int64_t M, int D, int streams, int slots, bool gate, bool gate_f32,
                     bool weights, const RowShape& s, Ring* ring, bool* staged_weights) {
  ring->weights_ld = (D + 7) / 8 * 8 + 8;
  ring->gate_f32 = gate_f32;
  const int wb = 2 * ring->weights_ld * 4;
  const int extra = s.aligned ? 0 : streams * 2 * (s.threads / 32) * 16;
  auto bytes = [&](int n) { return s.threads * n * 16 + extra; };
  const int gate_slots = gate ? (gate_f32 ? 4 : 2) : 0;
  ring->gate_direct = bytes(slots + gate_slots) > kSmemPerCta;
  ring->slots = slots + (ring->gate_direct ? 0 : gate_slots);
  ring->extra = s.threads * ring->slots * 16;
  int used = bytes(ring->slots);
  *staged_weights = weights && M > 2 * s.ctas * s.rpc && used + wb <= kSmemPerCta;
  if (*staged_weights) {
    ring->weights = used;
    used += wb;
  }
  return used;
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const RowShape& s, const A& a, const Ring& ring, int smem,
                        cudaStream_t stream) {
  if (smem > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(s.ctas)), dim3(s.tpr, s.rpc),
                    static_cast<size_t>(smem), stream, 1, a, ring);
}

}  // namespace

}  // namespace qlora
