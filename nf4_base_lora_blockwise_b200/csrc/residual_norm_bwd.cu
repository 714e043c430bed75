// residual_norm_bwd.cu -- the backward of the residual norm; the formulas and the way rows are read
// are described in residual_norm.cu.  With everything constant over a row taken out of its sums
// (h, y as stored; v the combined weights of the branch; k a token's gate or 1):
//   q = sum_c dn w_pre h,   G = dh' + r_h dn w_pre - h (r_h^3 q / D)
//   p = sum_c (G y) v g,    dy = (br k r_y) G v g - y (br k r_y^3 p / D)
//   dw_pre += (dn h) r_h,   S += (G y) (r_y k g),   a token's dgate = br r_y p,
// v without the gate for a whole gate g, whose dgate is (G y) v br r_y.
//
// Bound by memory without the branch's norm: 16384 x 8192 bf16, weights frozen, 201 us, 6.7 TB/s.
// With it the two sums that every row waits for, and 16 warps an SM (128 registers a thread), bound
// it: 4096 x 4096 with all gradients 44.3 us, 4.5 TB/s, some 5 of them for the sums of columns.
// (1 / rms read with the row instead of a round ahead: 60 us.)
#include "residual_norm.cuh"

namespace qlora {

namespace {

// Streams of the backward: dn, h', dh', y, then a whole gate.
template <typename R, int NV>
struct BwdSlots {
  static constexpr int GR = sizeof(R) == 4 ? 2 : 1;
  static constexpr int DN = 0, H = NV, DH = H + NV * GR, Y = DH + NV * GR, GATE = Y + NV;
};

// Adds a vector to one group's sums of columns (skewed), in rows that are not ALIGNED.
__device__ __forceinline__ void add_columns(float* sums, int at, int shift, const f2 (&q)[4]) {
  float* p = sums + at - shift;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = split(q[k]);
    (2 * k < shift ? p - 1 : p)[2 * k] += t.x;
    (2 * k + 1 < shift ? p - 1 : p)[2 * k + 1] += t.y;
  }
}

// DW: with the weights' and the channel gate's gradients.  Each thread sums its own columns over
// its group's rows in registers: dw_pre, and S, from which dw_post = br gate S and dgate =
// br (w_post + o) S for a channel gate, both constant over m.  The CTA's sums go to `part` for
// column_sum_kernel, which adds them in a fixed order: the results do not depend on timing.  In rows
// that start inside a granule a thread's columns change from row to row: there each group adds to
// sums in shared memory, its rows kept apart by its barrier.
// T = 512 threads leave the 128 registers that the sums and a row's data take.  WS: with the weights
// staged; GF: with a whole gate; AHEAD: rows that are on their way beside the current one.
template <typename R, int T, bool PAIR, bool ALIGNED, bool DW, bool WS, bool GF, int AHEAD>
__global__ void __launch_bounds__(T, 1)
    residual_norm_bwd_kernel(const __grid_constant__ ResidualNormBwd a,
                             const __grid_constant__ Ring ring) {
  constexpr int RB = sizeof(R), NV = 2;
  using S = BwdSlots<R, NV>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ __align__(16) float buf[4][kSumBuf];
  const uint32_t smem = smem_u32(smem_raw);
  Lane<NV> l = lane_of<NV, T, ALIGNED, PAIR>(ring, smem, a.D);
  pdl_wait();  // the previous kernel's outputs are complete
  pdl_trigger();
  const float inv_d = 1.f / static_cast<float>(a.D);
  const bool gate_c = a.gate_kind == kGateChannel;
  const bool post = a.w_post != nullptr;
  const bool wide = post || gate_c;
  const bool need_y = a.dy && (post || a.dgate);
  const bool token_sum = a.dgate && a.gate_kind == kGateToken;
  Weights w;
  w.w_pre = a.w_pre;
  w.w_post = a.w_post;
  w.gate = gate_c ? a.gate : nullptr;
  w.weight_f32 = a.weight_f32;
  w.gate_f32 = a.gate_f32;
  w.offset = a.weight_offset;
  w.D = a.D;
  constexpr int NS = DW && ALIGNED ? NV : 1;
  f2 s_pre[NS][4], s_post[NS][4];
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) s_pre[j][k] = s_post[j][k] = both(0.f);

  const int64_t walker = PAIR ? blockIdx.x / 2 : blockIdx.x, walkers = PAIR ? gridDim.x / 2 : gridDim.x;
  const int64_t step = walkers * blockDim.y;
  RowAt r, next;
  r.total = next.total = a.M * a.D;
  r.D = next.D = a.D;
  int64_t m = walker * blockDim.y + threadIdx.y;
  advance(r, m, a.M);
  constexpr int MORE = 4 * (AHEAD - 1);  // copy groups in flight of the row after the next
  const uint32_t turn = AHEAD == 2 ? l.slots ^ (l.slots + T * ring.slots * 16) : 0;
  auto other = [&] { l.slots ^= turn; };  // two sets of slots take turns
  if constexpr (ALIGNED) clear_slots<NV, T>(ring, l, r);
  // Four copy groups a row, in the order of their use: dn, h', dh', then y and a whole gate.
  auto start_dn = [&](const RowAt& q) {
    if (a.w_pre) issue<2, NV, T, ALIGNED, S::DN>(a.dn, l, q);
    commit_copies();
  };
  auto start_h = [&](const RowAt& q) {
    if (a.w_pre) issue<RB, NV, T, ALIGNED, S::H>(a.h_out, l, q);
    commit_copies();
  };
  auto start_dh = [&](const RowAt& q) {
    if (a.dh_out) issue<RB, NV, T, ALIGNED, S::DH>(a.dh_out, l, q);
    commit_copies();
  };
  auto start_y = [&](const RowAt& q) {
    if (need_y) issue<2, NV, T, ALIGNED, S::Y>(a.y, l, q);
    if constexpr (GF) issue_gate<NV, T, ALIGNED, S::GATE>(a.gate, ring, l, q);
    commit_copies();
  };
  start_dn(r);
  start_h(r);
  start_dh(r);
  start_y(r);
  if constexpr (AHEAD == 2) {
    other();
    advance(next, m + step, a.M);
    clear_slots<NV, T>(ring, l, next);
    start_dn(next);
    start_h(next);
    start_dh(next);
    start_y(next);
    other();
  }
  float* sums = reinterpret_cast<float*>(smem_raw + ring.sums) + threadIdx.y * 2 * ring.weights_ld;
  if constexpr (DW && !ALIGNED)
    for (int i = threadIdx.x; i < 2 * ring.weights_ld; i += blockDim.x) sums[i] = 0.f;
  if constexpr (WS) stage_weights<ALIGNED, PAIR>(w, ring, smem_raw, wide);
  clear_sums(buf, 4);
  all_sync<PAIR>();

  // A row's scalars, read a round ahead: 1 / rms of h' and of y (1 without w_post; 0 without a
  // row), a token's gate or 1.
  struct Scalars {
    float rh, ry, token;
  };
  auto scalars = [&](const RowAt& q, int64_t at) {
    Scalars s = {0.f, 0.f, 1.f};
    if (q.row) {
      if (a.w_pre) s.rh = a.rstd_pre[at];
      s.ry = post ? a.rstd_post[at] : 1.f;
      if (a.gate_kind == kGateToken) s.token = load_either1(a.gate, a.gate_f32, at);
    }
    return s;
  };
  Scalars now = scalars(r, m);

  // The same number of rounds for every group, so that a warp's slices stay together.  A round
  // without a row finds zeros, and zero factors.
  int parity = 0;
  for (int64_t base = walker * blockDim.y; base < a.M; base += step) {
    advance(next, m + step, a.M);
    const Scalars then = scalars(next, m + step);
    if constexpr (AHEAD == 2) advance(next, m + 2 * step, a.M);
    f2 G[NV][4];
    if (a.w_pre) {
      const float rh = now.rh;
      const f2 rh2 = both(rh);
      f2 ss = both(0.f);
      wait_copies<2 + MORE>();  // dn and h'
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        f2 h[4], v[4];
        fetch<2, NV, T, ALIGNED, S::DN>(a.dn, l, r, j, G[j]);
        fetch<RB, NV, T, ALIGNED, S::H>(a.h_out, l, r, j, h);
        weights8<0, WS, ALIGNED>(w, ring, l, smem_raw, r, j, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f2 p = mul2(G[j][k], h[k]);
          if constexpr (DW && ALIGNED) s_pre[j][k] = fma2(p, rh2, s_pre[j][k]);
          ss = fma2(p, v[k], ss);
          G[j][k] = mul2(G[j][k], v[k]);
          if constexpr (DW && !ALIGNED) h[k] = mul2(p, rh2);
        }
        if constexpr (DW && !ALIGNED) {
          if (a.dw_pre) add_columns(sums, l.w[j], static_cast<int>(r.at & 7), h);
        }
      }
      start_dn(next);
      const float s = row_sum<PAIR>(sum2(ss), buf[parity * 2]);
      const f2 c2 = both(-s * inv_d * rh * rh * rh);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        f2 h[4];
        fetch<RB, NV, T, ALIGNED, S::H>(a.h_out, l, r, j, h);
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = fma2(h[k], c2, mul2(G[j][k], rh2));
      }
      start_h(next);
    } else {
      start_dn(next);
      start_h(next);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = both(0.f);
    }
    wait_copies<3 + MORE>();  // dh'
    const f2 res = both(a.res_scale);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 d[4];
      if (a.dh_out) {
        fetch<RB, NV, T, ALIGNED, S::DH>(a.dh_out, l, r, j, d);
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = add2(G[j][k], d[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = mul2(G[j][k], res);
      put<R, ALIGNED>(static_cast<R*>(a.dh), r, l.c[j], d);
    }
    start_dh(next);
    if (a.dy) {
      wait_copies<3 + MORE>();  // y and the gate
      f2 ss = both(0.f);
      const float ry = now.ry, token = now.token;
      const f2 ryk = both(ry * token), bry = both(a.branch_scale * ry);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        f2 y[4], v[4], t[4], g[4];
        if (need_y) fetch<2, NV, T, ALIGNED, S::Y>(a.y, l, r, j, y);
        if (wide) {
          weights8<1, WS, ALIGNED>(w, ring, l, smem_raw, r, j, v);
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = mul2(G[j][k], v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = G[j][k];
        }
        if constexpr (GF) {
          fetch_gate<NV, T, ALIGNED, S::GATE>(a.gate, ring, l, r, j, g);
          if (a.dgate) {
            f2 dg[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) dg[k] = mul2(mul2(t[k], y[k]), bry);
            if (a.gate_f32)
              put<float, ALIGNED>(static_cast<float*>(a.dgate), r, l.c[j], dg);
            else
              put<__nv_bfloat16, ALIGNED>(static_cast<__nv_bfloat16*>(a.dgate), r, l.c[j], dg);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = mul2(t[k], g[k]);
        }
        if (need_y) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ss = fma2(t[k], y[k], ss);
            if constexpr (DW) {
              f2 p = mul2(G[j][k], y[k]);
              if constexpr (GF) p = mul2(p, g[k]);
              if constexpr (ALIGNED)
                s_post[j][k] = fma2(p, ryk, s_post[j][k]);
              else
                y[k] = mul2(p, ryk);
            }
          }
          if constexpr (DW && !ALIGNED) {
            if (a.dw_post || (a.dgate && gate_c))
              add_columns(sums + ring.weights_ld, l.w[j], static_cast<int>(r.at & 7), y);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = t[k];
      }
      float s = 0.f;
      if (post || token_sum) {
        s = row_sum<PAIR>(sum2(ss), buf[parity * 2 + 1]);
        if (token_sum && r.row && l.c[0] == 0)
          static_cast<float*>(a.dgate)[m] = a.branch_scale * ry * s;
      }
      const float brk = a.branch_scale * token;
      // (The sum holds y once: its product with r_y first, a cube of r_y leaves fp32 sooner.)
      const f2 ct = both(post ? brk * ry : brk), cy = both(-(brk * ry) * (ry * s * inv_d * ry));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) G[j][k] = mul2(G[j][k], ct);
        if (post) {
          f2 y[4];
          fetch<2, NV, T, ALIGNED, S::Y>(a.y, l, r, j, y);
#pragma unroll
          for (int k = 0; k < 4; ++k) G[j][k] = fma2(y[k], cy, G[j][k]);
        }
        put<__nv_bfloat16, ALIGNED>(a.dy, r, l.c[j], G[j]);
      }
    }
    start_y(next);
    if constexpr (AHEAD == 2) advance(next, m + step, a.M);  // again: it was the row after it
    const bool end = r.row && !next.row;
    r = next;
    now = then;
    m += step;
    parity ^= 1;
    other();
    if constexpr (ALIGNED) {
      // A last round without a row: the zero factors would make NaN of an infinity left here.
      if (end) {
        wait_copies<0>();
        clear_slots<NV, T>(ring, l, r);
      }
    }
    if constexpr (DW && !ALIGNED) group_sync();  // the next row's sums follow this one's
  }

  if constexpr (DW && !ALIGNED) {
    all_sync<PAIR>();
    const float* all = reinterpret_cast<const float*>(smem_raw + ring.sums);
    const int first = part_first<PAIR>(ring);
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    // The second CTA of a pair also met the first one's last columns.
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const int end = PAIR && rank == 0 ? ring.width : a.D - first;
    for (int c = tid; c < end; c += threads) {
      float s[2] = {0.f, 0.f};
      for (int y = 0; y < static_cast<int>(blockDim.y); ++y)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          s[q] += all[(y * 2 + q) * ring.weights_ld + skewed(c)];
          if (PAIR && rank == 0 && c >= end - 8)
            s[q] += ld_peer(all + (y * 2 + q) * ring.weights_ld + skewed(c - end), 1);
        }
      a.part[walker * a.part_ld + first + c] = s[0];
      a.part[(walkers + walker) * a.part_ld + first + c] = s[1];
    }
    if constexpr (PAIR) cluster_sync_all();  // the peer has read
  }
  if constexpr (DW && ALIGNED) {
    // The CTA's row groups are added in order through the streams' memory (no copy is in flight: a
    // row past the last starts none), then one row of sums is left for each gradient.
    const int rpc = blockDim.y;
    float* groups = reinterpret_cast<float*>(smem_raw);  // [rpc][2][ld]
    const int ld = a.part_ld;
    auto spill = [&](float* d, const f2 (&s)[4]) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 t = split(s[k]);
        f[2 * k] = t.x;
        f[2 * k + 1] = t.y;
      }
      store_vec<8>(d, f);
    };
    if (rpc > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = l.c[j];
        if (c >= a.D) continue;
        spill(groups + (threadIdx.y * 2) * ld + c, s_pre[j]);  // (several groups: no pair)
        spill(groups + (threadIdx.y * 2 + 1) * ld + c, s_post[j]);
      }
      __syncthreads();
      if (threadIdx.y != 0) return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = l.c[j];
      if (c >= a.D) continue;
      for (int y = 1; y < rpc; ++y) {
        float t[8];
        load_vec<8>(groups + (y * 2) * ld + c, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) s_pre[j][k] = add2(s_pre[j][k], pair(t[2 * k], t[2 * k + 1]));
        load_vec<8>(groups + (y * 2 + 1) * ld + c, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) s_post[j][k] = add2(s_post[j][k], pair(t[2 * k], t[2 * k + 1]));
      }
      if (a.dw_pre) spill(a.part + walker * ld + c, s_pre[j]);
      if (a.dw_post || (a.dgate && gate_c)) spill(a.part + (walkers + walker) * ld + c, s_post[j]);
    }
  }
}

// Sums over `rows` partial rows in order, 32 columns a CTA: blockDim.y threads a column take every
// blockDim.y-th row and are added in order.  y = 0: dw_pre; y = 1: S, from which dw_post and a
// channel gate's dgate.
constexpr int kSumLanes = 16;
__global__ void __launch_bounds__(32 * kSumLanes)
    column_sum_kernel(const float* __restrict__ part, int rows,
                      const __grid_constant__ ResidualNormBwd a) {
  __shared__ float s[kSumLanes][33];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + threadIdx.x;
  const bool second = blockIdx.y == 1;
  const float* p = part + (second ? static_cast<int64_t>(rows) * a.part_ld : 0) + c;
  float t = 0.f;
  if (c < a.D) {
    // Eight loads at a time: the rows are summed in order, whatever their number.
    int i = threadIdx.y;
    for (; i + 7 * static_cast<int>(blockDim.y) < rows; i += 8 * blockDim.y) {
      float q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = p[static_cast<int64_t>(i + k * blockDim.y) * a.part_ld];
#pragma unroll
      for (int k = 0; k < 8; ++k) t += q[k];
    }
    for (; i < rows; i += blockDim.y) t += p[static_cast<int64_t>(i) * a.part_ld];
  }
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.D) return;
  float sum = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.y); ++i) sum += s[i][threadIdx.x];
  if (!second) {
    if (a.dw_pre) a.dw_pre[c] = sum;
    return;
  }
  const bool gate_c = a.gate_kind == kGateChannel;
  sum *= a.branch_scale;
  if (a.dw_post)
    a.dw_post[c] = gate_c ? sum * load_either1(a.gate, a.gate_f32, c) : sum;
  if (a.dgate && gate_c)
    static_cast<float*>(a.dgate)[c] =
        a.w_post ? sum * (load_either1(a.w_post, a.weight_f32, c) + a.weight_offset) : sum;
}

template <typename R, int T, bool PAIR, bool ALIGNED, bool DW, bool GF>
cudaError_t launch_bwd(const ResidualNormBwd& a, RowShape s, cudaStream_t st) {
  Ring ring = {};
  bool ws;
  const bool weights = a.w_pre || a.w_post || a.gate_kind == kGateChannel;
  int smem = plan_ring(a.M, a.D, BwdSlots<R, 2>::GATE, GF, a.gate_f32, weights, DW, s, &ring, &ws);
  if (DW && !ALIGNED && ring.sums < 0) return cudaErrorInvalidConfiguration;
  if (DW && ALIGNED && s.rpc > 1) {  // the row groups' sums go through the same memory
    const int sums = s.rpc * 2 * a.part_ld * static_cast<int>(sizeof(float));
    if (sums > smem) smem = sums;
  }
  // Two rows ahead where y is not read and a group has more than 6: 4096 x 8192 (without sums of
  // columns) 59.3 -> 53.4 us, 2048 x 4096 17.2 -> 16.5; with fewer the copies before the first row
  // cost more than they save (600 x 4096 8.8 -> 9.7), and with y the two sums of a row bound the
  // loop, not its loads (4096 x 8192 73.5 -> 75.1).
  if constexpr (ALIGNED && !PAIR && T == 512 && !GF) {
    const int more = T * ring.slots * 16;
    const bool reads_y = a.dy && (a.w_post || a.dgate);
    if (ws && !reads_y && a.M > 6 * s.walkers * s.rpc && smem + more <= kSmemPerCta) {
      ring.weights += more;
      return launch_rows(residual_norm_bwd_kernel<R, T, PAIR, ALIGNED, DW, true, GF, 2>, s, a, ring,
                         smem + more, st);
    }
  }
  return ws ? launch_rows(residual_norm_bwd_kernel<R, T, PAIR, ALIGNED, DW, true, GF, 1>, s, a, ring,
                          smem, st)
            : launch_rows(residual_norm_bwd_kernel<R, T, PAIR, ALIGNED, DW, false, GF, 1>, s, a, ring,
                          smem, st);
}
template <typename R, int T, bool PAIR, bool ALIGNED, bool DW>
cudaError_t launch_bwd(const ResidualNormBwd& a, const RowShape& s, cudaStream_t st) {
  return a.gate_kind == kGateFull ? launch_bwd<R, T, PAIR, ALIGNED, DW, true>(a, s, st)
                                  : launch_bwd<R, T, PAIR, ALIGNED, DW, false>(a, s, st);
}
template <typename R>
cudaError_t launch_bwd(const ResidualNormBwd& a, const RowShape& s, bool dw, cudaStream_t st) {
  if (s.threads == 1024) return launch_bwd<R, 1024, false, true, false>(a, s, st);
  if (s.pair) {
    if (!s.aligned)
      return dw ? launch_bwd<R, 512, true, false, true>(a, s, st)
                : launch_bwd<R, 512, true, false, false>(a, s, st);
    return launch_bwd<R, 512, true, true, true>(a, s, st);
  }
  if (s.aligned)
    return dw ? launch_bwd<R, 512, false, true, true>(a, s, st)
              : launch_bwd<R, 512, false, true, false>(a, s, st);
  return dw ? launch_bwd<R, 512, false, false, true>(a, s, st)
            : launch_bwd<R, 512, false, false, false>(a, s, st);
}

// Up to 8192 columns (or the granules of as many) 512 threads take a row; then 1024 without column
// sums in rows of whole granules, else a pair of 512.
RowShape bwd_shape(int64_t M, int D, bool dw) {
  const bool wide = D + (D % 8 ? 7 : 0) > 8192;
  const bool one = wide && D % 8 == 0 && !dw;
  return row_shape(M, D, one ? 1024 : 512, wide && !one);
}

}  // namespace

size_t residual_norm_part_bytes(int64_t M, int D) {
  return static_cast<size_t>(2 * bwd_shape(M, D, true).walkers) * ((D + 7) / 8 * 8) * sizeof(float);
}

cudaError_t launch_residual_norm_bwd(const ResidualNormBwd& args, cudaStream_t stream, int* n) {
  ResidualNormBwd a = args;
  a.part_ld = (a.D + 7) / 8 * 8;
  const bool second = a.dw_post || (a.dgate && a.gate_kind == kGateChannel);
  const bool dw = a.dw_pre || second;
  const RowShape s = bwd_shape(a.M, a.D, dw);
  const cudaError_t e = a.resid_f32 ? launch_bwd<float>(a, s, dw, stream)
                                    : launch_bwd<__nv_bfloat16>(a, s, dw, stream);
  *n = 1;
  if (e != cudaSuccess || !dw) return e;
  *n = 2;
  int lanes = 1;
  while (lanes < kSumLanes && lanes * 8 < s.walkers) lanes *= 2;
  return launch_pdl(column_sum_kernel, dim3((a.D + 31) / 32, second ? 2 : 1), dim3(32, lanes), 0,
                    stream, 1, a.part, static_cast<int>(s.walkers), a);
}

}  // namespace qlora
