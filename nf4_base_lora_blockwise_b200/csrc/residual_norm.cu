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
// Bound by memory, and nearly by instruction issue: 4 bytes an element leave about 25 instructions
// for each at full rate.  So: 16 columns a thread, packed fp32 pairs (two lanes an instruction),
// the weights combined once a CTA into fp32 in shared memory.  A CTA of up to 1024 threads walks
// rows in groups of tpr threads with a barrier of their own.  A thread copies what it reads
// itself into its own slots by cp.async and starts the next row's copy as soon as it has read a
// slot for the last time, so a row is on its way while the one before is worked on, without a
// barrier or a second stage.  (Slots laid out by thread instead of by granule: 36 us against 26 at
// 4096 x 4096; scalar fp32 instead of pairs: 27.5 against 26.2.)
// Measured, bf16 with both norms and a channel gate: 4096 x 4096 24 us, 5.6 TB/s; without the gate
// 16384 x 8192 164 us, 6.5 TB/s.  1 x 4096: 2.3 us.
//
// Rows of D % 8 != 0 start anywhere in a 16-byte granule: threads copy and store the granules as
// they lie, and address what belongs to columns by the row's offset (residual_norm.cuh).  1531 x 2051
// with an fp32 residual and a whole gate: 14.9 us, 3.0 TB/s, bound by the instructions of that
// (rows joined from two granules by shuffles: 20.7 us).
#include "residual_norm.cuh"

namespace qlora {

namespace {

// Streams of the forward: y, h, then a whole gate.
template <typename R, int NV>
struct FwdSlots {
  static constexpr int GR = sizeof(R) == 4 ? 2 : 1;
  static constexpr int Y = 0, H = NV, GATE = NV + NV * GR;
};

constexpr int kFwdThreads = 1024;

// WS: with the weights staged; GF: with a whole gate.
template <typename R, bool ALIGNED, bool WS, bool GF>
__global__ void __launch_bounds__(kFwdThreads, 1)
    residual_norm_fwd_kernel(const __grid_constant__ ResidualNormFwd a,
                             const __grid_constant__ Ring ring) {
  constexpr int RB = sizeof(R), NV = 2, T = kFwdThreads;
  using S = FwdSlots<R, NV>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ __align__(16) float buf[4][kSumBuf];
  const uint32_t smem = smem_u32(smem_raw);
  const Lane<NV> l = lane_of<NV, T, ALIGNED, false>(ring, smem, a.D);
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const float inv_d = 1.f / static_cast<float>(a.D);
  const bool wide = a.w_post || a.gate_kind == kGateChannel;  // the branch has weights
  Weights w;
  w.w_pre = a.w_pre;
  w.w_post = a.w_post;
  w.gate = a.gate_kind == kGateChannel ? a.gate : nullptr;
  w.weight_f32 = a.weight_f32;
  w.gate_f32 = a.gate_f32;
  w.offset = a.weight_offset;
  w.D = a.D;

  const int64_t walker = blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  RowAt r, next;
  r.total = next.total = a.M * a.D;
  r.D = next.D = a.D;
  int64_t m = walker * blockDim.y + threadIdx.y;
  advance(r, m, a.M);
  if constexpr (ALIGNED) clear_slots<NV, T>(ring, l, r);
  // Two copy groups a row: y, then h and a whole gate.
  auto start_y = [&](const RowAt& q) {
    if (a.y) issue<2, NV, T, ALIGNED, S::Y>(a.y, l, q);
    commit_copies();
  };
  auto start_h = [&](const RowAt& q) {
    issue<RB, NV, T, ALIGNED, S::H>(a.h, l, q);
    if constexpr (GF) issue_gate<NV, T, ALIGNED, S::GATE>(a.gate, ring, l, q);
    commit_copies();
  };
  start_y(r);
  start_h(r);
  if constexpr (WS) stage_weights<ALIGNED, false>(w, ring, smem_raw, wide);
  clear_sums(buf, 4);
  __syncthreads();

  // A token's gate, read a round ahead.
  auto token_of = [&](const RowAt& q, int64_t at) {
    return q.row && a.gate_kind == kGateToken ? load_either1(a.gate, a.gate_f32, at) : 1.f;
  };
  float token = token_of(r, m);

  // The same number of rounds for every group, so that a warp's slices stay together.
  int parity = 0;
  for (int64_t base = walker * blockDim.y; base < a.M; base += step) {
    advance(next, m + step, a.M);
    const float then = token_of(next, m + step);
    f2 h[NV][4];
    wait_copies<1>();
    if (a.y) {
      f2 y[NV][4];
      f2 ss = both(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        fetch<2, NV, T, ALIGNED, S::Y>(a.y, l, r, j, y[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fma2(y[j][k], y[j][k], ss);
      }
      start_y(next);
      float scale = a.branch_scale * token;
      if (a.w_post) {
        const float rs = rsqrtf(row_sum<false>(sum2(ss), buf[parity * 2]) * inv_d + a.eps);
        if (r.row && l.c[0] == 0 && a.rstd_post) a.rstd_post[m] = rs;
        scale *= rs;
      }
      wait_copies<1>();
      const f2 sc = both(scale), res = both(a.res_scale);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (wide) {
          f2 v[4];
          weights8<1, WS, ALIGNED>(w, ring, l, smem_raw, r, j, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) y[j][k] = mul2(y[j][k], v[k]);
        }
        if constexpr (GF) {
          f2 g[4];
          fetch_gate<NV, T, ALIGNED, S::GATE>(a.gate, ring, l, r, j, g);
#pragma unroll
          for (int k = 0; k < 4; ++k) y[j][k] = mul2(y[j][k], g[k]);
        }
        fetch<RB, NV, T, ALIGNED, S::H>(a.h, l, r, j, h[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[j][k] = fma2(y[j][k], sc, mul2(h[j][k], res));
          if constexpr (RB == 2) h[j][k] = unpack_bf16(pack_bf16(h[j][k]));  // as stored
        }
        put<R, ALIGNED>(static_cast<R*>(a.h_out), r, l.c[j], h[j]);
      }
    } else {
      start_y(next);
      wait_copies<1>();
#pragma unroll
      for (int j = 0; j < NV; ++j) fetch<RB, NV, T, ALIGNED, S::H>(a.h, l, r, j, h[j]);
    }
    start_h(next);
    if (a.w_pre) {
      f2 ss = both(0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fma2(h[j][k], h[j][k], ss);
      const float rs = rsqrtf(row_sum<false>(sum2(ss), buf[parity * 2 + 1]) * inv_d + a.eps);
      if (r.row && l.c[0] == 0 && a.rstd_pre) a.rstd_pre[m] = rs;
      const f2 rr = both(rs);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        f2 v[4];
        weights8<0, WS, ALIGNED>(w, ring, l, smem_raw, r, j, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[j][k] = mul2(mul2(h[j][k], rr), v[k]);
        put<__nv_bfloat16, ALIGNED>(a.n, r, l.c[j], h[j]);
      }
    }
    r = next;
    token = then;
    m += step;
    parity ^= 1;
  }
}

template <typename R, bool ALIGNED, bool GF>
cudaError_t launch_fwd(const ResidualNormFwd& a, RowShape s, cudaStream_t st) {
  Ring ring = {};
  bool ws;
  const bool weights = a.w_pre || a.w_post || a.gate_kind == kGateChannel;
  const int smem = plan_ring(a.M, a.D, FwdSlots<R, 2>::GATE, GF, a.gate_f32, weights, false, s,
                             &ring, &ws);
  return ws ? launch_rows(residual_norm_fwd_kernel<R, ALIGNED, true, GF>, s, a, ring, smem, st)
            : launch_rows(residual_norm_fwd_kernel<R, ALIGNED, false, GF>, s, a, ring, smem, st);
}
template <typename R>
cudaError_t launch_fwd(const ResidualNormFwd& a, cudaStream_t st) {
  const RowShape s = row_shape(a.M, a.D, kFwdThreads, false);
  if (a.gate_kind == kGateFull)
    return s.aligned ? launch_fwd<R, true, true>(a, s, st) : launch_fwd<R, false, true>(a, s, st);
  return s.aligned ? launch_fwd<R, true, false>(a, s, st) : launch_fwd<R, false, false>(a, s, st);
}

}  // namespace

cudaError_t launch_residual_norm_fwd(const ResidualNormFwd& a, cudaStream_t stream) {
  return a.resid_f32 ? launch_fwd<float>(a, stream) : launch_fwd<__nv_bfloat16>(a, stream);
}

}  // namespace qlora
