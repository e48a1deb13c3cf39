// Backward of the block norms: see block_norm.cu for the formulas.
#include "block_norm.cuh"

namespace e4b {
namespace {

// Rows of any width, stride and base.
template <class XT, class YT, int VPT, int T>
__global__ void __launch_bounds__(T, VPT == 1 ? 768 / T : 1)
    block_norm_backward_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  // Buffers alternate by row: a row may have one sum only, and so no other
  // barrier before the next row's.
  __shared__ float red[2][2][64];
  const Cols<VPT, T> c{static_cast<int>(threadIdx.x), a.H};
  pdl_wait();
  pdl_launch_dependents();
  Rows<XT, YT, VPT, T, true> rows(a, c, ring);
  const bool has_y = a.y.p != nullptr, next = a.w_next != nullptr, post = a.w_post != nullptr;
  const int kind = a.gate_kind;
  const F2 offset = f2(a.offset);
  F8 s_post[VPT], s_next[VPT], s_gate[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) s_post[v] = s_next[v] = s_gate[v] = zero8();
  int odd = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, odd ^= 1) {
    rows.next();
    F2 t0 = f2(0.0f), t1 = t0, t2 = t0;  // r^2, h * r, y^2
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (has_y) {
        const F8 y = rows.template load<YT>(a.y, m, v);
        t2 = dot8(y, y, t2);
      }
      if (next) {
        const F8 r = rows.template load<XT>(a.x, m, v);
        const F8 h = rows.load(a.dn, m, a.n_f32, v) * (c.load(a.w_next, a.w_f32, v) + offset);
        t0 = dot8(r, r, t0);
        t1 = dot8(h, r, t1);
      }
    }
    float s1[3] = {lo(t0) + hi(t0), lo(t1) + hi(t1), lo(t2) + hi(t2)};
    row_sum<3>(s1, T, red[odd][0]);
    const float rstd_r = rsqrtf(s1[0] * a.inv_h + a.eps), rstd_y = post ? rsqrtf(s1[2] * a.inv_h + a.eps) : 1.0f;
    const float mean_r = s1[1] * rstd_r * a.inv_h;  // mean(h * rhat)
    F8 k[VPT];
    F2 u0 = f2(0.0f), u1 = u0;  // k * yhat, d * z * slope
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      F8 d = a.dr.p ? rows.template load<XT>(a.dr, m, v) : zero8();
      if (next) {
        const F8 hat = rows.template load<XT>(a.x, m, v) * f2(rstd_r);
        const F8 dn = rows.load(a.dn, m, a.n_f32, v);
        const F8 h = dn * (c.load(a.w_next, a.w_f32, v) + offset);
        s_next[v] = fma8(dn, hat, s_next[v]);
        d = fma8(fma8(hat, f2(-mean_r), h), f2(rstd_r), d);
      }
      if (a.dx.p) c.store(reinterpret_cast<XT*>(static_cast<unsigned char*>(a.dx.p) + m * a.dx.row), v, d);
      if (!has_y) continue;
      const F8 hat = rows.template load<YT>(a.y, m, v) * f2(rstd_y);
      const F8 w = post ? c.load(a.w_post, a.w_f32, v) + offset : fill8(1.0f);
      F8 dz = d * f2(a.scale);
      if (kind != E4B_GATE_NONE) {
        F8 f = rows.gate(m, v);
        F8 dg = dz * (hat * w);
        if (a.sigmoid) {
          f = sigmoid8(f);
          dg = dg * (f * (fma8(f, f2(-1.0f), fill8(1.0f))));
        }
        dz = dz * f;
        if (kind == E4B_GATE_CHANNEL)
#pragma unroll
          for (int j = 0; j < 4; ++j) s_gate[v].p[j] = s_gate[v].p[j] + dg.p[j];
        else if (kind == E4B_GATE_TOKEN)
#pragma unroll
          for (int j = 0; j < 4; ++j) u1 = u1 + dg.p[j];
        else if (a.dgate)
          c.store(a.dgate, m * a.H, a.gate_f32, v, dg);
      }
      s_post[v] = fma8(dz, hat, s_post[v]);
      k[v] = dz * w;
      u0 = dot8(k[v], hat, u0);
    }
    if (!has_y) continue;
    float s2[2] = {lo(u0) + hi(u0), lo(u1) + hi(u1)};
    if (post || kind == E4B_GATE_TOKEN) row_sum<2>(s2, T, red[odd][1]);
    if (kind == E4B_GATE_TOKEN && a.dgate && threadIdx.x == 0) store1(a.dgate, m, a.gate_f32, s2[1]);
    if (!a.dy.p) continue;
    const float mean_y = post ? s2[0] * a.inv_h * rstd_y : 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      F8 dy = k[v];  // without its norm dy does not depend on y, which may be infinite
      if (post) dy = fma8(rows.template load<YT>(a.y, m, v), f2(-mean_y), dy) * f2(rstd_y);
      c.store(reinterpret_cast<YT*>(static_cast<unsigned char*>(a.dy.p) + m * a.dy.row), v, dy);
    }
  }
  const int64_t plane = static_cast<int64_t>(a.parts) * a.H;
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.H;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (post) c.store(part, v, s_post[v]);
    if (next) c.store(part + plane, v, s_next[v]);
    if (kind == E4B_GATE_CHANNEL) c.store(part + 2 * plane, v, s_gate[v]);
  }
}

// Rows moved as vectors, aligned or shifted (COLS).  ALL: y, both weights, dr, dx and dy are there, the step
// between two blocks in training; what each row would ask of them at run time
// costs about a third of the kernel's instructions.
template <class XT, class YT, int VPT, class COLS, bool ALL>
__global__ void __launch_bounds__(norm_threads(VPT), VPT == 1 ? 2 : 1)
    block_norm_backward_vec_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float red[2][128];  // by turns, a row's sums
  const int T = blockDim.x;
  const COLS c(T, threadIdx.x, a.H);
  const bool has_y = ALL || a.y.p, next = ALL || a.w_next, post = ALL || a.w_post;
  const bool has_dr = ALL || a.dr.p, has_dx = ALL || a.dx.p, has_dy = ALL || a.dy.p;
  const int kind = a.gate_kind, stages = a.stages;
  const int step = static_cast<int>(gridDim.x);
  auto row_of = [&](const RowSrc& t) { return static_cast<const unsigned char*>(t.p) + blockIdx.x * t.row; };
  const unsigned char *r_p = row_of(a.x), *dr_p = row_of(a.dr), *y_p = row_of(a.y), *dn_p = row_of(a.dn), *g_p = row_of(a.gate);
  const uint32_t ring_u = smem_addr(ring) + c.place();
  const unsigned char* ring_p = ring + c.place();
  int64_t put_row = blockIdx.x;
  int put_stage = 0, stage = 0;
  // Aligned: a thread reads its own places only, so that filling the last row's stage
  // needs no barrier.  Shifted: see below.
  auto put = [&]() {
    if (put_row < a.M) {
      const int64_t last = a.M - 1 - put_row;
      const uint32_t to = ring_u + put_stage * a.stage_bytes;
      if (next) {
        c.template fetch<XT>(to + a.x.off, r_p, a.x, last);
        if (a.n_f32)
          c.template fetch<float>(to + a.dn.off, dn_p, a.dn, last);
        else
          c.template fetch<uint16_t>(to + a.dn.off, dn_p, a.dn, last);
        r_p += a.x.step;
        dn_p += a.dn.step;
      }
      if (has_y) {
        c.template fetch<YT>(to + a.y.off, y_p, a.y, last);
        y_p += a.y.step;
      }
      if (has_dr) {
        c.template fetch<XT>(to + a.dr.off, dr_p, a.dr, last);
        dr_p += a.dr.step;
      }
      if (kind == E4B_GATE_FULL) {
        if (a.gate_f32)
          c.template fetch<float>(to + a.gate.off, g_p, a.gate, last);
        else
          c.template fetch<uint16_t>(to + a.gate.off, g_p, a.gate, last);
        g_p += a.gate.step;
      }
      put_row += step;
    }
    cp_commit();
    put_stage = put_stage + 1 == stages ? 0 : put_stage + 1;
  };
  pdl_wait();
  pdl_launch_dependents();
  for (int i = 0; i + 1 < stages; ++i) put();
  const F2 offset = f2(a.offset);
  // Sums over rows of dn * rhat, and of d * yhat times a row's or an element's f: dw_post
  // and a channel gate's gradient are that times what is the same in every row.
  F8 s_next[VPT], s_post[VPT];
  auto channel = [&](int v) {  // f of a channel gate
    const F8 f = kind == E4B_GATE_CHANNEL ? c.vector(a.vec_gate, a.gate_f32, v) : fill8(1.0f);
    return a.sigmoid && kind == E4B_GATE_CHANNEL ? sigmoid8(f) : f;
  };
  auto w_post = [&](int v) { return post ? c.vector(a.w_post, a.w_f32, v) + offset : fill8(1.0f); };
  auto w_next = [&](int v) { return c.vector(a.w_next, a.w_f32, v) + offset; };
  // w_post and the channel's f, and w_next: in registers where a thread has one group.
  constexpr bool kHeld = VPT == 1;
  F8 held_y = fill8(1.0f), held_n = zero8();
  if constexpr (kHeld) {
    held_y = w_post(0) * channel(0);
    if (next) held_n = w_next(0);
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) s_post[v] = s_next[v] = zero8();
  auto flush = [&](int set, int64_t m, unsigned char* dx_row, unsigned char* dy_row) {
    if constexpr (COLS::kShared) {
      const unsigned char* out = ring + a.out_off + set * a.out_bytes;
      if (has_dx) c.template flush<XT>(dx_row, out + a.out_slot[0]);
      if (has_y && has_dy) c.template flush<YT>(dy_row, out + a.out_slot[1]);
      if (kind == E4B_GATE_FULL && a.dgate) {
        unsigned char* row = static_cast<unsigned char*>(a.dgate) + m * a.gate.row;
        if (a.gate_f32)
          c.template flush<float>(row, out + a.out_slot[2]);
        else
          c.template flush<uint16_t>(row, out + a.out_slot[2]);
      }
    }
  };
  int odd = 0;
  int64_t m_last = -1;
  unsigned char* dx_p = static_cast<unsigned char*>(a.dx.p) + blockIdx.x * a.dx.row;
  unsigned char* dy_p = static_cast<unsigned char*>(a.dy.p) + blockIdx.x * a.dy.row;
  for (int64_t m = blockIdx.x; m < a.M; m += step, odd ^= 1, dx_p += a.dx.step, dy_p += a.dy.step) {
    m_last = m;
    cp_wait(stages);
    unsigned char *dx_s = nullptr, *dy_s = nullptr, *dg_s = nullptr;
    if constexpr (COLS::kShared) {
      // The copies are in and the last row is done with: its stage and its outputs' rows.
      // Two sets of output rows: one is written while the other is put together.
      __syncthreads();
      unsigned char* out = ring + a.out_off + odd * a.out_bytes;
      dx_s = out + a.out_slot[0], dy_s = out + a.out_slot[1], dg_s = out + a.out_slot[2];
      if (m != blockIdx.x) flush(odd ^ 1, m - step, dx_p - a.dx.step, dy_p - a.dy.step);
    }
    put();
    const unsigned char* cur = ring_p + stage * a.stage_bytes;
    stage = stage + 1 == stages ? 0 : stage + 1;
    auto load_dn = [&](int v) {
      return a.n_f32 ? c.template staged<float>(cur, a.dn, m, v) : c.template staged<uint16_t>(cur, a.dn, m, v);
    };
    auto full = [&](int v) {  // f of a gate that has one for every element
      const F8 f = a.gate_f32 ? c.template staged<float>(cur, a.gate, m, v) : c.template staged<uint16_t>(cur, a.gate, m, v);
      return a.sigmoid ? sigmoid8(f) : f;
    };
    auto weight = [&](int v) { return kHeld ? held_y : w_post(v) * channel(v); };
    // The sum of d * e, e = f * (w_post + offset) * y, which the post norm's and a token's
    // gradient need, is taken term by term of d, so that one round of sums does for a row.
    const bool along = has_y && (post || kind == E4B_GATE_TOKEN);
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};  // of r^2, h * r, y^2; e * dr, e * h, e * r
    auto add = [&](float& to, F2 q, int v) { to += c.in[v] ? lo(q) + hi(q) : 0.0f; };
    F8 h[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const F2 z = f2(0.0f);
      F8 e = zero8();
      if (has_y) {
        const F8 y = c.template staged<YT>(cur, a.y, m, v);
        add(s[2], dot8(y, y, z), v);
        if (along) {
          e = y * weight(v);
          if (kind == E4B_GATE_FULL) e = e * full(v);
          if (has_dr) add(s[3], dot8(e, c.template staged<XT>(cur, a.dr, m, v), z), v);
        }
      }
      if (next) {
        const F8 r = c.template staged<XT>(cur, a.x, m, v);
        h[v] = load_dn(v) * (kHeld ? held_n : w_next(v));
        add(s[0], dot8(r, r, z), v);
        add(s[1], dot8(h[v], r, z), v);
        if (along) {
          add(s[4], dot8(e, h[v], z), v);
          add(s[5], dot8(e, r, z), v);
        }
      }
    }
    row_sum<6>(s, T, red[odd]);
    const float rstd_r = rsqrtf(s[0] * a.inv_h + a.eps), rstd_y = post ? rsqrtf(s[2] * a.inv_h + a.eps) : 1.0f;
    const float mean_r = s[1] * rstd_r * a.inv_h;  // mean(h * rhat)
    // scale * sum of d * e / f * rstd_y, f of a token's gate
    const float de = a.scale * rstd_y * (next ? s[3] + rstd_r * (s[4] - rstd_r * mean_r * s[5]) : s[3]);
    float f_token = 1.0f;
    if (kind == E4B_GATE_TOKEN) {
      f_token = load1(a.vec_gate, m, a.gate_f32);
      float slope = 1.0f;
      if (a.sigmoid) {
        f_token = sigmoid_f32(f_token);
        slope = f_token * (1.0f - f_token);
      }
      if (a.dgate && threadIdx.x == 0) store1(a.dgate, m, a.gate_f32, de * slope);
    }
    const float mean_y = post ? de * f_token * a.inv_h : 0.0f;  // mean(k * yhat)
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      F8 d = has_dr ? c.template staged<XT>(cur, a.dr, m, v) : zero8();
      if (next) {
        const F8 hat = c.template staged<XT>(cur, a.x, m, v) * f2(rstd_r);
        s_next[v] = fma8(load_dn(v), hat, s_next[v]);
        d = fma8(fma8(hat, f2(-mean_r), h[v]), f2(rstd_r), d);
      }
      if (has_dx) c.template store<XT>(dx_p, dx_s, v, d);
      if (!has_y) continue;
      const F8 hat = c.template staged<YT>(cur, a.y, m, v) * f2(rstd_y);
      const F8 w = weight(v);
      F8 df = d;  // times a row's or an element's f
      if (kind == E4B_GATE_TOKEN) df = d * f2(f_token);
      if (kind == E4B_GATE_FULL) {
        const F8 f = full(v);
        df = d * f;
        if (a.dgate) {
          F8 dg = d * (hat * w) * f2(a.scale);
          if (a.sigmoid) dg = dg * (f * fma8(f, f2(-1.0f), fill8(1.0f)));
          unsigned char* row = static_cast<unsigned char*>(a.dgate) + m * a.gate.row;
          if (a.gate_f32)
            c.template store<float>(row, dg_s, v, dg);
          else
            c.template store<uint16_t>(row, dg_s, v, dg);
        }
      }
      s_post[v] = fma8(df, hat, s_post[v]);
      if (has_dy) {
        F8 dy = df * w * f2(a.scale);
        if (post) dy = fma8(hat, f2(-mean_y), dy) * f2(rstd_y);  // without its norm dy does not depend on y, which may be infinite
        c.template store<YT>(dy_p, dy_s, v, dy);
      }
    }
  }
  if constexpr (COLS::kShared) {
    __syncthreads();
    flush(odd ^ 1, m_last, dx_p - a.dx.step, dy_p - a.dy.step);
  }
  const int64_t plane = static_cast<int64_t>(a.parts) * a.H;
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.H;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const F8 f = channel(v), all = s_post[v] * f2(a.scale);
    if (post) c.sums(part, v, all * f);
    if (next) c.sums(part + plane, v, s_next[v]);
    if (kind == E4B_GATE_CHANNEL)
      c.sums(part + 2 * plane, v, all * w_post(v) * (a.sigmoid ? f * fma8(f, f2(-1.0f), fill8(1.0f)) : fill8(1.0f)));
  }
}

template <class K>
cudaError_t launch_kernel(K kernel, const NormArgs& a, const NormShape& s, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(a.stages) * a.stage_bytes + 2 * a.out_bytes;
  if (cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem); err != cudaSuccess) return err;
  return launch_overlapped(kernel, s.grid, s.T, smem, 1, stream, a);
}

template <class XT, class YT, int VPT, class COLS>
cudaError_t launch_cols(const NormArgs& a, const NormShape& s, cudaStream_t stream) {
  const bool all = a.y.p && a.w_next && a.w_post && a.dr.p && a.dx.p && a.dy.p;
  return all ? launch_kernel(block_norm_backward_vec_kernel<XT, YT, VPT, COLS, true>, a, s, stream)
             : launch_kernel(block_norm_backward_vec_kernel<XT, YT, VPT, COLS, false>, a, s, stream);
}

template <class XT, class YT, int VPT>
cudaError_t launch_vec(const NormArgs& a, const NormShape& s, Moved moved, cudaStream_t stream) {
  return moved == kVector ? launch_cols<XT, YT, VPT, VecCols<VPT>>(a, s, stream)
                          : launch_cols<XT, YT, VPT, ShiftCols<VPT>>(a, s, stream);
}

template <class XT, class YT>
cudaError_t launch_typed(const NormArgs& a, const NormShape& s, Moved moved, cudaStream_t stream) {
  if (moved != kElements)
    return s.vpt == 1   ? launch_vec<XT, YT, 1>(a, s, moved, stream)
           : s.vpt == 2 ? launch_vec<XT, YT, 2>(a, s, moved, stream)
                        : launch_vec<XT, YT, 4>(a, s, moved, stream);
  // norm_shape() rounds these rows' threads to one of the sizes below.
  if (s.vpt == 4) return launch_kernel(block_norm_backward_kernel<XT, YT, 4, 512>, a, s, stream);
  if (s.vpt == 2) return launch_kernel(block_norm_backward_kernel<XT, YT, 2, 384>, a, s, stream);
  if (s.T == 64) return launch_kernel(block_norm_backward_kernel<XT, YT, 1, 64>, a, s, stream);
  if (s.T == 128) return launch_kernel(block_norm_backward_kernel<XT, YT, 1, 128>, a, s, stream);
  if (s.T == 256) return launch_kernel(block_norm_backward_kernel<XT, YT, 1, 256>, a, s, stream);
  return launch_kernel(block_norm_backward_kernel<XT, YT, 1, 384>, a, s, stream);
}

}  // namespace

cudaError_t launch_block_norm_backward(const NormArgs& a, bool x_f32, bool y_f32, const NormShape& s, Moved moved,
                                       cudaStream_t stream) {
  if (x_f32) return y_f32 ? launch_typed<float, float>(a, s, moved, stream) : launch_typed<float, uint16_t>(a, s, moved, stream);
  return y_f32 ? launch_typed<uint16_t, float>(a, s, moved, stream) : launch_typed<uint16_t, uint16_t>(a, s, moved, stream);
}

}  // namespace e4b
