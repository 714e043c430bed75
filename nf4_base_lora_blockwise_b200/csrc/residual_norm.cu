// residual_norm.cu -- the residual update around a block with its RMS norms, forward and
// backward.  Forward, per token row:
//   a  = y r_y (w_post + o),  r_y = rsqrt(mean(y^2) + eps)     (a = y without w_post)
//   h' = res h + br gate a                                      (stored in the residual's type)
//   n  = h' r_h (w_pre + o),  r_h = rsqrt(mean(h'^2) + eps)     (of h' as stored)
// Backward, with x = h' r_h, z = y r_y, u = dn (w_pre + o):
//   G  = dh' + r_h (u - x mean(u x)),      dh = res G,          dw_pre  = sum_m dn x
//   E  = br G,  dgate = E a (summed along what the gate is broadcast over),  E := gate E
//   t  = E (w_post + o),  dy = r_y (t - z mean(t z)),           dw_post = sum_m E z
// (dy = E without w_post.)  fp32 throughout, one rounding at each stored output.
//
// Bound by memory: a row is read once into registers, its sums cross the row's threads through
// shuffles (and shared memory past one warp), and the outputs are written from the registers.
// Rows of up to 32 vectors take a power-of-two slice of a warp, so narrow rows share a CTA.
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace qlora {

namespace {

constexpr int kMaxRowWarps = 32;

// Sums of NS values over the row's threads (blockDim.x of them, row threadIdx.y of the CTA); the
// result in every thread.  Past one warp the warps' sums go through `buf`, which the next call
// with the same buf may overwrite only after another barrier: callers alternate two buffers.
template <int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float (*buf)[kMaxRowWarps]) {
  const int tpr = blockDim.x;
  const int width = tpr < 32 ? tpr : 32;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    for (int o = width / 2; o > 0; o >>= 1) v[s] += __shfl_xor_sync(0xFFFFFFFFu, v[s], o);
  if (tpr > 32) {
    const int warps = tpr >> 5, w = threadIdx.x >> 5;
    const int first = threadIdx.y * warps;  // rows of one CTA share the buffer
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s) buf[s][first + w] = v[s];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float t = 0.f;
      for (int i = 0; i < warps; ++i) t += buf[s][first + i];
      v[s] = t;
    }
  }
}

template <typename R, int VEC, int NV>
__global__ void __launch_bounds__(1024) residual_norm_fwd_kernel(ResidualNormFwd a) {
  __shared__ float buf[2][1][kMaxRowWarps];
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const int D = a.D;
  const float inv_d = 1.f / static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  // The loop's bound is the same for every thread of the CTA, so all meet its barriers.
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * blockDim.y; base < a.M; base += step) {
    const int64_t m = base + threadIdx.y;
    const bool row = m < a.M;
    const int64_t at = m * D;
    float h[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) h[j][k] = 0.f;
      if (row && c < D) load_vec<VEC>(static_cast<const R*>(a.h) + at + c, h[j]);
    }
    if (a.y) {
      float y[NV][VEC];
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[j][k] = 0.f;
        if (row && c < D) load_vec<VEC>(a.y + at + c, y[j]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss[0] += y[j][k] * y[j][k];
      }
      float r = 1.f;
      if (a.w_post) {
        row_sum<1>(ss, buf[0]);
        r = rsqrtf(ss[0] * inv_d + a.eps);
        if (row && threadIdx.x == 0 && a.rstd_post) a.rstd_post[m] = r;
      }
      float scale = a.branch_scale;
      if (row && a.gate_kind == kGateToken) scale *= load_either1(a.gate, a.gate_f32, m);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        if (!row || c >= D) continue;
        float v[VEC];
        if (a.w_post) {
          float w[VEC];
          load_either<VEC>(a.w_post, a.weight_f32, c, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[k] = y[j][k] * r * (w[k] + a.weight_offset);
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[k] = y[j][k];
        }
        if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
          float g[VEC];
          load_either<VEC>(a.gate, a.gate_f32, a.gate_kind == kGateFull ? at + c : c, g);
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[k] *= g[k];
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          h[j][k] = stored<R>(h[j][k] * a.res_scale + v[k] * scale);
        store_vec<VEC>(static_cast<R*>(a.h_out) + at + c, h[j]);
      }
    }
    if (a.w_pre) {
      float ss[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss[0] += h[j][k] * h[j][k];
      row_sum<1>(ss, buf[1]);
      const float r = rsqrtf(ss[0] * inv_d + a.eps);
      if (row && threadIdx.x == 0 && a.rstd_pre) a.rstd_pre[m] = r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        if (!row || c >= D) continue;
        float w[VEC];
        load_either<VEC>(a.w_pre, a.weight_f32, c, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) h[j][k] = h[j][k] * r * (w[k] + a.weight_offset);
        store_vec<VEC>(a.n + at + c, h[j]);
      }
    }
    if (blockDim.x > 32) __syncthreads();  // buf is free again
  }
}

// DW: with the weights' and the channel gate's gradients.  A CTA walks rows, each thread sums
// its own columns over them in registers, and the CTA's rows of sums go to `part` for
// column_sum_kernel, which adds them in a fixed order: the results do not depend on timing.
template <typename R, int VEC, int NV, bool DW>
__global__ void __launch_bounds__(1024) residual_norm_bwd_kernel(ResidualNormBwd a) {
  __shared__ float buf[2][2][kMaxRowWarps];
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const int D = a.D;
  const float inv_d = 1.f / static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  float s_pre[DW ? NV : 1][VEC], s_post[DW ? NV : 1][VEC], s_gate[DW ? NV : 1][VEC];
  if constexpr (DW) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) s_pre[j][k] = s_post[j][k] = s_gate[j][k] = 0.f;
  }
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * blockDim.y; base < a.M; base += step) {
    const int64_t m = base + threadIdx.y;
    const bool row = m < a.M;
    const int64_t at = m * D;
    float G[NV][VEC];  // dh', then G
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) G[j][k] = 0.f;
      if (a.dh_out && row && c < D) load_vec<VEC>(static_cast<const R*>(a.dh_out) + at + c, G[j]);
    }
    if (a.w_pre) {
      float x[NV][VEC], u[NV][VEC];
      float s[1] = {0.f};
      const float r = row ? a.rstd_pre[m] : 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[j][k] = u[j][k] = 0.f;
        if (!row || c >= D) continue;
        load_vec<VEC>(static_cast<const R*>(a.h_out) + at + c, x[j]);
        load_vec<VEC>(a.dn + at + c, u[j]);
        float w[VEC];
        load_either<VEC>(a.w_pre, a.weight_f32, c, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          x[j][k] *= r;
          if constexpr (DW) s_pre[j][k] += u[j][k] * x[j][k];
          u[j][k] *= w[k] + a.weight_offset;
          s[0] += u[j][k] * x[j][k];
        }
      }
      row_sum<1>(s, buf[0]);
      const float mean = s[0] * inv_d;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) G[j][k] += r * (u[j][k] - x[j][k] * mean);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (!row || c >= D) continue;
      float o[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = G[j][k] * a.res_scale;
      store_vec<VEC>(static_cast<R*>(a.dh) + at + c, o);
    }
    if (a.dy) {
      const bool post = a.w_post != nullptr;
      const bool need_y = post || a.dgate != nullptr;
      float z[NV][VEC];
      float s[2] = {0.f, 0.f};  // t z; dgate of the token
      const float r = (row && post) ? a.rstd_post[m] : 0.f;
      const float token =
          (row && a.gate_kind == kGateToken) ? load_either1(a.gate, a.gate_f32, m) : 1.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) z[j][k] = 0.f;
        if (!row || c >= D) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) G[j][k] = 0.f;
          continue;
        }
        if (need_y) load_vec<VEC>(a.y + at + c, z[j]);
        float w[VEC], g[VEC];
        if (post) {
          load_either<VEC>(a.w_post, a.weight_f32, c, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            z[j][k] *= r;
            w[k] += a.weight_offset;
          }
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) w[k] = 1.f;
        }
        const bool wide = a.gate_kind == kGateChannel || a.gate_kind == kGateFull;
        if (wide) {
          load_either<VEC>(a.gate, a.gate_f32, a.gate_kind == kGateFull ? at + c : c, g);
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) g[k] = token;
        }
        float dg[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float e = G[j][k] * a.branch_scale;
          dg[k] = e * z[j][k] * w[k];
          s[1] += dg[k];
          const float eg = e * g[k];
          if constexpr (DW) {
            s_gate[j][k] += dg[k];
            s_post[j][k] += eg * z[j][k];
          }
          G[j][k] = eg * w[k];  // t (E without w_post)
          s[0] += G[j][k] * z[j][k];
        }
        if (a.dgate && a.gate_kind == kGateFull) {
          if (a.gate_f32)
            store_vec<VEC>(static_cast<float*>(a.dgate) + at + c, dg);
          else
            store_vec<VEC>(static_cast<__nv_bfloat16*>(a.dgate) + at + c, dg);
        }
      }
      if (post || (a.dgate && a.gate_kind == kGateToken)) {
        row_sum<2>(s, buf[1]);
        if (row && threadIdx.x == 0 && a.dgate && a.gate_kind == kGateToken)
          static_cast<float*>(a.dgate)[m] = s[1];
      }
      const float mean = s[0] * inv_d;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        if (!row || c >= D) continue;
        if (post) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) G[j][k] = r * (G[j][k] - z[j][k] * mean);
        }
        store_vec<VEC>(a.dy + at + c, G[j]);
      }
    }
    if (blockDim.x > 32) __syncthreads();  // buf is free again
  }
  if constexpr (DW) {
    const int64_t p = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t rows = static_cast<int64_t>(gridDim.x) * blockDim.y;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c >= D) continue;
      // Gradient q (0 dw_pre, 1 dw_post, 2 dgate) has its rows at part[q].
      if (a.dw_pre) store_vec<VEC>(a.part + p * a.part_ld + c, s_pre[j]);
      if (a.dw_post) store_vec<VEC>(a.part + (rows + p) * a.part_ld + c, s_post[j]);
      if (a.dgate && a.gate_kind == kGateChannel)
        store_vec<VEC>(a.part + (2 * rows + p) * a.part_ld + c, s_gate[j]);
    }
  }
}

// out[q][c] = sum over `rows` partial rows of part[q][.][c], in order of the rows.  32 columns a
// CTA; 16 threads a column take every 16th row and are added in order.
constexpr int kSumLanes = 16;
__global__ void __launch_bounds__(32 * kSumLanes)
    column_sum_kernel(const float* __restrict__ part, int64_t ld, int rows, int D, float* o0,
                      float* o1, float* o2) {
  __shared__ float s[kSumLanes][33];
  pdl_wait();
  pdl_trigger();
  float* out = blockIdx.y == 0 ? o0 : (blockIdx.y == 1 ? o1 : o2);
  if (!out) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * rows * ld;
  float t = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < rows; i += kSumLanes) t += p[i * ld + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kSumLanes; ++i) sum += s[i][threadIdx.x];
    out[c] = sum;
  }
}

// How a row of D elements is spread: VEC elements an access, NV accesses a thread, tpr threads a
// row (a power of two up to 32, else whole warps), rpc rows a CTA.
struct RowShape {
  int vec, nv, tpr, rpc;
};
RowShape row_shape(int D) {
  RowShape s;
  // 16-byte accesses where every row starts on one; rows of even length start on 4 bytes.
  s.vec = D % 8 == 0 ? 8 : (D % 2 == 0 ? 2 : 1);
  const int nc = D / s.vec;
  if (s.vec == 8)
    s.nv = nc <= 256 ? 1 : 2;
  else
    s.nv = s.vec == 2 ? 8 : 16;
  const int need = (nc + s.nv - 1) / s.nv;
  if (need <= 32) {
    s.tpr = 1;
    while (s.tpr < need) s.tpr *= 2;
  } else {
    s.tpr = (need + 31) / 32 * 32;
  }
  s.rpc = s.tpr >= 256 ? 1 : 256 / s.tpr;
  return s;
}

template <typename F>
cudaError_t with_shape(const RowShape& s, F f) {
  if (s.vec == 8) return s.nv == 1 ? f.template operator()<8, 1>() : f.template operator()<8, 2>();
  if (s.vec == 2) return f.template operator()<2, 8>();
  return f.template operator()<1, 16>();
}

// CTAs that walk the rows: up to 8 of 256 threads an SM.
int64_t fwd_ctas(const RowShape& s, int64_t M) {
  const int64_t want = (M + s.rpc - 1) / s.rpc;
  const int64_t cap = 148ll * (2048 / (s.tpr * s.rpc));
  return want < cap ? want : cap;
}

// The backward with weight gradients keeps 48 sums a thread, so fewer CTAs fit an SM, and each
// leaves rpc rows of sums.
int64_t bwd_ctas(const RowShape& s, int64_t M) {
  const int64_t want = (M + s.rpc - 1) / s.rpc;
  const int per_sm = s.tpr * s.rpc > 512 ? 1 : 512 / (s.tpr * s.rpc);
  const int64_t cap = 148ll * per_sm;
  return want < cap ? want : cap;
}

template <typename R>
struct FwdLaunch {
  const ResidualNormFwd& a;
  const RowShape& s;
  cudaStream_t stream;
  template <int VEC, int NV>
  cudaError_t operator()() const {
    return launch_pdl(residual_norm_fwd_kernel<R, VEC, NV>,
                      dim3(static_cast<unsigned>(fwd_ctas(s, a.M))),
                      dim3(s.tpr, s.rpc), 0, stream, 1, a);
  }
};

template <typename R, bool DW>
struct BwdLaunch {
  const ResidualNormBwd& a;
  const RowShape& s;
  cudaStream_t stream;
  template <int VEC, int NV>
  cudaError_t operator()() const {
    return launch_pdl(residual_norm_bwd_kernel<R, VEC, NV, DW>,
                      dim3(static_cast<unsigned>(bwd_ctas(s, a.M))), dim3(s.tpr, s.rpc), 0,
                      stream, 1, a);
  }
};

}  // namespace

cudaError_t launch_residual_norm_fwd(const ResidualNormFwd& a, cudaStream_t stream) {
  const RowShape s = row_shape(a.D);
  if (a.resid_f32) return with_shape(s, FwdLaunch<float>{a, s, stream});
  return with_shape(s, FwdLaunch<__nv_bfloat16>{a, s, stream});
}

size_t residual_norm_part_bytes(int64_t M, int D) {
  const RowShape s = row_shape(D);
  return static_cast<size_t>(3 * bwd_ctas(s, M) * s.rpc) * ((D + 7) / 8 * 8) * sizeof(float);
}

cudaError_t launch_residual_norm_bwd(const ResidualNormBwd& args, cudaStream_t stream, int* n) {
  const RowShape s = row_shape(args.D);
  ResidualNormBwd a = args;
  a.part_ld = (a.D + 7) / 8 * 8;
  float* dgate_c = a.gate_kind == kGateChannel ? static_cast<float*>(a.dgate) : nullptr;
  const bool dw = a.dw_pre || a.dw_post || dgate_c;
  cudaError_t e;
  if (a.resid_f32)
    e = dw ? with_shape(s, BwdLaunch<float, true>{a, s, stream})
           : with_shape(s, BwdLaunch<float, false>{a, s, stream});
  else
    e = dw ? with_shape(s, BwdLaunch<__nv_bfloat16, true>{a, s, stream})
           : with_shape(s, BwdLaunch<__nv_bfloat16, false>{a, s, stream});
  *n = 1;
  if (e != cudaSuccess || !dw) return e;
  *n = 2;
  return launch_pdl(column_sum_kernel, dim3((a.D + 31) / 32, 3), dim3(32, kSumLanes), 0, stream, 1,
                    a.part, static_cast<int64_t>(a.part_ld),
                    static_cast<int>(bwd_ctas(s, a.M) * s.rpc), a.D, a.dw_pre, a.dw_post, dgate_c);
}

}  // namespace qlora
