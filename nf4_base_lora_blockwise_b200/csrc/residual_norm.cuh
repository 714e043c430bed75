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
// Groups and pairs.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void st_peer(float* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_peer(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}
template <bool PAIR>
__device__ __forceinline__ void all_sync() {
  if constexpr (PAIR)
    cluster_sync_all();
  else
    __syncthreads();
}

// The group's threads, whole warps or slices of one.
__device__ __forceinline__ void group_sync() {
  if (blockDim.x > 32)
    asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.y) + 1), "r"(blockDim.x)
                 : "memory");
  else
    __syncwarp();
}

// ---------------------------------------------------------------------------------------------
// Row streams: [M, D] tensors read row by row.  Every thread has `slots` 16-byte slots in shared
// memory, [slot][T threads] (a copy whose lanes do not write one contiguous piece of shared memory
// measured a third slower); a stream's, and the T that a CTA has room for, are given at compile
// time, so that an access is one register and a constant.
//
// ALIGNED: D % 8 == 0, a vector is columns 8 v .. 8 v + 7.  Otherwise a row starts `shift` elements
// inside a granule of 8, and vector v is the granule that starts 8 v elements after the row's
// first one: columns 8 v - shift .. 8 v - shift + 7, where there are such columns.  All streams
// and outputs share that, so whole granules are read and stored as they lie, but for a row's
// ends; only what belongs to columns (weights, column sums) is addressed by column.
//
// PAIR (backward): rows wider than 8192 columns are shared by a cluster of two CTAs, half the
// vectors each, where 1024 threads of one CTA would leave too few registers or too little shared
// memory for column sums or weights; a row's sums cross through each other's shared memory with
// a barrier of the cluster.  (1024 x 16384 with column sums 91 -> 70 us; without them, and
// forward, one CTA a row measured 45 and 31 us against a pair's 62 and 47.)
// ---------------------------------------------------------------------------------------------
struct Ring {
  int slots;       // of a thread
  int weights;     // byte of the combined weights' [2][weights_ld] fp32
  int width;       // of the CTA's part of a row: D rounded up to 8, or 16 columns a thread
  int weights_ld;  // width and 8 zeros; or skewed_size(width)
  int sums;        // byte of the column sums' [group][2][weights_ld] fp32, or -1: in `part`
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

// Rows that are not ALIGNED address fp32 arrays over columns -8 .. (D up to 8) + 15 in shared memory,
// with a gap after every 8: neighbouring vectors lie 9 words apart and meet different banks.
__host__ __device__ constexpr int skewed_size(int D) { return ((D + 7) / 8 + 3) * 9; }
__device__ __forceinline__ int skewed(int c) { return (c + 8) + ((c + 8) >> 3); }

template <int NV>
struct Lane {
  uint32_t slots;  // shared address of the thread's first slot
  uint32_t w[NV];  // ALIGNED: of the combined weights of its columns; else vector v's skewed index
  int c[NV];       // 8 v
};
// First column (or 8 v) of the CTA's part of a row.
template <bool PAIR>
__device__ __forceinline__ int part_first(const Ring& ring) {
  return PAIR ? static_cast<int>(cluster_ctarank()) * ring.width : 0;
}
template <int NV, int T, bool ALIGNED, bool PAIR>
__device__ __forceinline__ Lane<NV> lane_of(const Ring& ring, uint32_t smem, int D) {
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  Lane<NV> l;
  l.slots = smem + tid * 16;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int here = (j * blockDim.x + threadIdx.x) * 8;
    l.c[j] = part_first<PAIR>(ring) + here;
    if constexpr (ALIGNED) {
      // Past the row's end: the zeros behind the weights.
      const int at = l.c[j] < D ? here : ring.width;
      l.w[j] = smem + ring.weights + at * 4;
    } else {
      const int last = ring.width + 8;  // its columns are past the end for every shift
      l.w[j] = (here < last ? here : last) / 8 * 9 + 9;
    }
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

// Starts the copies of row r's granules of one stream, whose first slot is SLOT.
template <int ESIZE, int NV, int T, bool ALIGNED, int SLOT>
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
    const int shift = static_cast<int>(r.at & 7);
    const int64_t a = r.at - shift;
    const char* base = static_cast<const char*>(p);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int first = l.c[j] + g * N;
        if (first >= r.D + shift) continue;
        const int64_t e = a + first;
        const int bytes = e + N > r.total ? static_cast<int>(r.total - e) * ESIZE : 16;
        copy16(l.slots + (SLOT + j * G + g) * (T * 16), base + e * ESIZE, bytes);
      }
    }
  }
}

// The j-th vector of the thread as fp32 pairs; what lies outside the row reads 0.
// DIRECT: from global memory.
template <int ESIZE, int NV, int T, bool ALIGNED, int SLOT, bool DIRECT = false>
__device__ __forceinline__ void fetch(const void* p, const Lane<NV>& l, const RowAt& r, int j,
                                      f2 (&f)[4]) {
  constexpr int N = 16 / ESIZE;
  constexpr int G = 8 / N;
  const int c = l.c[j];
  const int shift = ALIGNED ? 0 : static_cast<int>(r.at & 7);
  uint32_t w[4 * G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint4 q;
    if constexpr (DIRECT)
      q = r.row && c + g * N < r.D + shift ? ldg16<ESIZE>(p, r.at - shift + c + g * N, r.total)
                                           : make_uint4(0, 0, 0, 0);
    else
      q = lds16(l.slots + (SLOT + j * G + g) * (T * 16));
    w[4 * g] = q.x;
    w[4 * g + 1] = q.y;
    w[4 * g + 2] = q.z;
    w[4 * g + 3] = q.w;
  }
  if constexpr (!ALIGNED) {
    // Before the row's start, past its end or without a row lies another row's, or nothing.
    const int first = shift - c, end = r.row ? r.D + shift - c : 0;
    if (first > 0 || end < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= first && k < end) continue;
        if constexpr (ESIZE == 4)
          w[k] = 0;
        else
          w[k / 2] &= k % 2 ? 0xFFFFu : 0xFFFF0000u;
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
template <int NV, int T, bool ALIGNED, int SLOT>
__device__ __forceinline__ void issue_gate(const void* p, const Ring& ring, const Lane<NV>& l,
                                           const RowAt& r) {
  if (ring.gate_direct) return;
  if (ring.gate_f32)
    issue<4, NV, T, ALIGNED, SLOT>(p, l, r);
  else
    issue<2, NV, T, ALIGNED, SLOT>(p, l, r);
}
template <int NV, int T, bool ALIGNED, int SLOT>
__device__ __forceinline__ void fetch_gate(const void* p, const Ring& ring, const Lane<NV>& l,
                                           const RowAt& r, int j, f2 (&f)[4]) {
  if (ring.gate_direct) {
    if (ring.gate_f32)
      fetch<4, NV, T, ALIGNED, SLOT, true>(p, l, r, j, f);
    else
      fetch<2, NV, T, ALIGNED, SLOT, true>(p, l, r, j, f);
  } else if (ring.gate_f32) {
    fetch<4, NV, T, ALIGNED, SLOT>(p, l, r, j, f);
  } else {
    fetch<2, NV, T, ALIGNED, SLOT>(p, l, r, j, f);
  }
}

// Stores the vector whose l.c[j] is c; what lies outside the row is left alone.
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
    if (!r.row) return;
    const int shift = static_cast<int>(r.at & 7);
    T* q = p + (r.at - shift) + c;
    const int first = shift - c, end = r.D + shift - c;
    if (first <= 0 && end >= 8) {
      store_vec<8>(q, f);
    } else if (end > 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k < first || k >= end) continue;
        const float one[1] = {f[k]};
        store_vec<1>(q + k, one);
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
template <int WHICH>
__device__ __forceinline__ float combine1(const Weights& w, int c) {
  const void* p = WHICH == 0 ? w.w_pre : w.w_post;
  float f = p ? load_either1(p, w.weight_f32, c) + w.offset : 1.f;
  if (WHICH == 1 && w.gate) f *= load_either1(w.gate, w.gate_f32, c);
  return f;
}
template <int WHICH>
__device__ __forceinline__ void combine8(const Weights& w, int c, float (&f)[8]) {
  const void* p = WHICH == 0 ? w.w_pre : w.w_post;
  if (p) {
    load_either<8>(p, w.weight_f32, c, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += w.offset;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 1.f;
  }
  if (WHICH == 1 && w.gate) {
    float g[8];
    load_either<8>(w.gate, w.gate_f32, c, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= g[k];
  }
}
// Fills the CTA's shared copy (a barrier follows before the first use).
template <bool ALIGNED, bool PAIR>
__device__ __forceinline__ void stage_weights(const Weights& w, const Ring& ring,
                                              unsigned char* smem, bool second) {
  const int first = part_first<PAIR>(ring);
  float* d = reinterpret_cast<float*>(smem + ring.weights);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  if constexpr (ALIGNED) {
    for (int c = tid * 8; c < ring.weights_ld; c += threads * 8) {
      float f[8] = {};
      const bool in = c < ring.width && first + c < w.D;
      if (w.w_pre) {
        if (in) combine8<0>(w, first + c, f);
        store_vec<8>(d + c, f);
      }
      if (second) {
        if (in) combine8<1>(w, first + c, f);
        store_vec<8>(d + ring.weights_ld + c, f);
      }
    }
  } else {
    // Four columns' loads at a time: a CTA of few rows has few threads, which would wait for each.
    constexpr int U = 4;
    for (int c0 = tid - 8; c0 < ring.width + 16; c0 += threads * U) {
      float f[U], g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * threads;
        const bool in = first + c >= 0 && first + c < w.D;
        f[u] = in && w.w_pre ? combine1<0>(w, first + c) : 0.f;
        g[u] = in && second ? combine1<1>(w, first + c) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * threads;
        if (c >= ring.width + 16) break;
        if (w.w_pre) d[skewed(c)] = f[u];
        if (second) d[ring.weights_ld + skewed(c)] = g[u];
      }
    }
  }
}
// The weights of the thread's j-th vector; 0 where it lies outside the row.
template <int WHICH>
__device__ __noinline__ void weights_outside(const Weights& w, int c0, float* f) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = c0 + k;
    f[k] = c >= 0 && c < w.D ? combine1<WHICH>(w, c) : 0.f;
  }
}
template <int WHICH, bool WS, bool ALIGNED, int NV>
__device__ __forceinline__ void weights8(const Weights& w, const Ring& ring, const Lane<NV>& l,
                                         const unsigned char* smem, const RowAt& r, int j,
                                         f2 (&f)[4]) {
  if constexpr (ALIGNED && WS) {
    const uint32_t p = l.w[j] + WHICH * ring.weights_ld * 4;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];"
                   : "=l"(f[2 * k]), "=l"(f[2 * k + 1])
                   : "r"(p + k * 16)
                   : "memory");
  } else {
    float t[8] = {};
    if constexpr (ALIGNED) {
      if (l.c[j] < w.D) combine8<WHICH>(w, l.c[j], t);
    } else {
      const int shift = static_cast<int>(r.at & 7);
      if constexpr (WS) {
        const float* p = reinterpret_cast<const float*>(smem + ring.weights) +
                         WHICH * ring.weights_ld + l.w[j] - shift;
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = (k < shift ? p - 1 : p)[k];
      } else {
        float u[8];
        weights_outside<WHICH>(w, l.c[j] - shift, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = u[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = pair(t[2 * k], t[2 * k + 1]);
  }
}

// The sum of v over the row's threads (row group threadIdx.y of the CTA, or of both CTAs of a PAIR);
// the result in every thread.  Past one warp the warps' sums go through `buf`, which the group's
// next call with the same buf may overwrite only after another barrier: callers alternate.
template <bool PAIR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  const int tpr = blockDim.x;
  if (tpr >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  } else {
    for (int o = tpr / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  if (!PAIR && tpr <= 32) return v;
  // [group][CTA of the pair][warps rounded up to 4], the padding zero from the kernel's start.
  const int warps = tpr >> 5, ld = (warps + 3) & ~3, all = PAIR ? 2 * ld : ld;
  float* mine = buf + threadIdx.y * all;
  if ((threadIdx.x & 31) == 0) {
    float* at = mine + (PAIR ? cluster_ctarank() * ld : 0) + (threadIdx.x >> 5);
    *at = v;
    if constexpr (PAIR) st_peer(at, cluster_ctarank() ^ 1u, v);
  }
  if constexpr (PAIR)
    cluster_sync_all();
  else
    group_sync();
  v = 0.f;
  for (int i = 0; i < all; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(mine + i);
    v += (q.x + q.y) + (q.z + q.w);
  }
  return v;
}
constexpr int kSumBuf = 96;  // floats of one buffer
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
// CTA an SM.  Whole granules (D % 8 == 0) let narrow rows share a warp.
struct RowShape {
  bool aligned, pair;
  int tpr, rpc;     // tpr: of one CTA
  int threads;      // that a CTA has room for
  int64_t walkers;  // CTAs, or pairs, that walk the rows
};
constexpr int kSms = 148;
constexpr int kSmemPerCta = 222 * 1024;
inline int least_groups(const RowShape& s) { return s.tpr >= 32 ? 1 : 32 / s.tpr; }  // whole warps
inline RowShape row_shape(int64_t M, int D, int threads, bool pair) {
  RowShape s;
  s.aligned = D % 8 == 0;
  s.threads = threads;
  // (A row that starts inside a granule may touch one more.)
  const int vectors = s.aligned ? D / 8 : (D + 14) / 8;
  s.pair = pair;
  const int need = (vectors + (s.pair ? 3 : 1)) / (s.pair ? 4 : 2);
  if (need <= 32) {
    s.tpr = s.aligned ? 1 : 8;  // (every group of the latter has column sums of its own)
    while (s.tpr < need) s.tpr *= 2;
  } else {
    s.tpr = (need + 31) / 32 * 32;
  }
  // A CTA's groups share the weights: as many as its threads hold (8 past one warp, for their
  // barriers), no more than spreads the rows over every SM.
  s.rpc = threads / s.tpr;
  if (s.tpr > 32 && s.rpc > 8) s.rpc = 8;
  const int sms = s.pair ? kSms / 2 : kSms;
  const int64_t spread = (M + sms - 1) / sms;
  const int least = least_groups(s);
  if (s.rpc > spread) s.rpc = static_cast<int>((spread + least - 1) / least * least);
  const int64_t want = (M + s.rpc - 1) / s.rpc;
  s.walkers = want < sms ? want : sms;
  return s;
}

// Lays streams of `slots` slots a thread (without a whole gate's), the weights and, for rows that
// are not of whole granules, the groups' column sums out in shared memory.  Of the widest rows a
// whole gate, the sums and then the weights may not fit; weights are not staged either for rows
// of whole granules that a group has few of.  Bytes.
inline int plan_ring(int64_t M, int D, int slots, bool gate, bool gate_f32, bool weights,
                     bool sums, RowShape& s, Ring* ring, bool* staged_weights) {
  ring->width = s.pair ? 16 * s.tpr : (D + 7) / 8 * 8;
  ring->weights_ld = s.aligned ? ring->width + 8 : skewed_size(ring->width);
  ring->gate_f32 = gate_f32;
  const int gate_slots = gate ? (gate_f32 ? 4 : 2) : 0;
  auto bytes = [&](int n) { return s.threads * n * 16; };
  ring->gate_direct = bytes(slots + gate_slots) > kSmemPerCta;
  ring->slots = slots + (ring->gate_direct ? 0 : gate_slots);
  int used = bytes(ring->slots);
  const int array = (2 * ring->weights_ld * 4 + 15) / 16 * 16;
  ring->sums = -1;
  // Only one group may add to `part`: fewer groups where their sums would not fit.
  while (sums && !s.aligned && s.rpc > least_groups(s) && used + s.rpc * array > kSmemPerCta)
    s.rpc = (s.rpc / least_groups(s) + 1) / 2 * least_groups(s);
  if (sums && !s.aligned && used + s.rpc * array <= kSmemPerCta) {
    ring->sums = used;
    used += s.rpc * array;
  }
  *staged_weights =
      weights && (!s.aligned || M > 2 * s.walkers * s.rpc) && used + array <= kSmemPerCta;
  if (*staged_weights) {
    ring->weights = used;
    used += array;
  }
  return used;
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const RowShape& s, const A& a, const Ring& ring, int smem,
                        cudaStream_t stream) {
  if (smem > 40 * 1024) {
    // Always the same: a call of another host thread must not lower what this launch takes.
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerCta);
    if (e != cudaSuccess) return e;
  }
  const int cluster = s.pair ? 2 : 1;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(s.walkers * cluster)), dim3(s.tpr, s.rpc),
                    static_cast<size_t>(smem), stream, cluster, a, ring);
}

}  // namespace

}  // namespace qlora
