// The norms after and before a block, fused with the block's gate, its
// residual scale and the residual sum; forward and backward.
//
//   z = N(y; w_post)                       (or z = y without w_post)
//   r = x + s * f(gate) * z                f(g) = g or sigmoid(g)
//   n = N(r; w_next)
//   N(v; w) = v * rstd(v) * (w + offset),  rstd(v) = 1 / sqrt(mean(v^2) + eps)
//
// Bound: HBM.  CTAs are persistent and take a row at a time; T threads share
// it, each with VPT groups of 8 columns.  The rows ahead come through a ring of
// cp.async stages in shared memory, so that loads stay in flight while a row's
// sums meet (a warp shuffle and a block barrier per sum).  Where rows can be
// moved as vectors, a thread copies and reads its own columns only; other rows
// (odd widths, strides) are copied as the 16-byte units that they touch and
// read by element.  Both norms are taken on 32-bit values in registers (n from the
// unrounded r), and every output is rounded once.
//
// Backward, with d = dr + (dn through the next norm):
//   h = dn * (w_next + offset):  d += rstd_r * (h - rhat * mean(h * rhat))
//   dx = d,  dz = s * f * d,  df = s * d * z  (summed over a gate's broadcast axis)
//   k = dz * (w_post + offset):  dy = rstd_y * (k - yhat * mean(k * yhat))
//   dw_next = sum_m dn * rhat,  dw_post = sum_m dz * yhat
// Both rstd are taken again from r and y, which the gradients need anyway, so
// the forward saves nothing.  A CTA keeps its columns' sums over rows in
// registers; a second kernel adds the CTAs' partial sums in CTA order, so every
// sum has a fixed order.
#include <algorithm>
#include <string>

#include "common.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr int kMaxNormH = 16384;
constexpr int kMaxNormThreads = 512;

// A tensor of rows that a kernel reads: leading dimension in elements, place in a
// ring stage.
struct RowSrc {
  const void* p;
  int64_t ld;
  uint32_t off;
};

struct NormArgs {
  RowSrc x, y, gate;                 // x: also r of the backward; gate: E4B_GATE_FULL's rows
  RowSrc dr, dn;                     // backward
  const void *vec_gate, *w_post, *w_next;  // vec_gate: channel or token gate
  void *r, *n;                       // forward
  void *dx, *dy, *dgate;             // backward
  float* partial;                    // backward: [3][parts][H] column sums (w_post, w_next, channel gate)
  int64_t ldr, ldn, lddx, lddy;      // of the outputs
  int64_t M;
  int H, parts;
  int stages;                        // of the ring; 0: rows are read from memory directly
  uint32_t stage_bytes;
  int gate_kind, gate_f32, sigmoid, w_f32, n_f32;
  float scale, offset, eps, inv_h;
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = float_to_bf16_bits(v); }

__device__ __forceinline__ void load8(const float* p, float v[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float v[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// One 32-byte store: two of 16 bytes would each write half of every sector.
__device__ __forceinline__ void store8(float* p, const float v[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
// Through L1: the two halves of a 32-byte sector are asked for by two instructions.
__device__ __forceinline__ void cp16_l1(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the newest stages - 2 groups are in (stages is 2 to 4).
__device__ __forceinline__ void cp_wait(int stages) {
  if (stages == 4)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (stages == 3)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// One thread's share of a row: VPT groups of 8 columns.  VEC: a group is 8
// adjacent columns, moved as vectors; otherwise its columns lie T apart, so
// that a warp's accesses stay adjacent.
template <bool VEC>
struct Cols {
  int T, t, H;
  __device__ __forceinline__ int col(int v, int j) const { return VEC ? (v * T + t) * 8 + j : (v * 8 + j) * T + t; }
  template <class E>
  __device__ __forceinline__ void load(const E* row, int v, float out[8]) const {
    if constexpr (VEC) {
      if (col(v, 0) < H) {
        load8(row + col(v, 0), out);
        return;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = col(v, j) < H ? load1(row + col(v, j)) : 0.0f;
    }
  }
  template <class E>
  __device__ __forceinline__ void store(E* row, int v, const float in[8]) const {
    if constexpr (VEC) {
      if (col(v, 0) < H) store8(row + col(v, 0), in);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col(v, j) < H) store1(row + col(v, j), in[j]);
    }
  }
  // The element type known at run time only (uniform over the launch).
  __device__ __forceinline__ void load(const void* base, int64_t off, int f32, int v, float out[8]) const {
    if (f32)
      load(static_cast<const float*>(base) + off, v, out);
    else
      load(static_cast<const uint16_t*>(base) + off, v, out);
  }
  __device__ __forceinline__ void store(void* base, int64_t off, int f32, int v, const float in[8]) const {
    if (f32)
      store(static_cast<float*>(base) + off, v, in);
    else
      store(static_cast<uint16_t*>(base) + off, v, in);
  }

  // Row m of `s` into its place in `stage`.
  template <class E>
  __device__ __forceinline__ void fetch(unsigned char* stage, const RowSrc& s, int64_t m, int64_t M, int VPT) const {
    const E* row = static_cast<const E*>(s.p) + m * s.ld;
    unsigned char* dst = stage + s.off;
    if constexpr (VEC) {
      // 8 bf16: one unit per thread; 8 floats: two, in two planes
      for (int v = 0; v < VPT; ++v) {
        if (col(v, 0) >= H) break;
        if constexpr (sizeof(E) == 2) {
          cp16(dst + (v * T + t) * 16, row + col(v, 0), 16);
        } else {
          cp16_l1(dst + (v * T + t) * 16, row + col(v, 0));
          cp16_l1(dst + ((VPT + v) * T + t) * 16, row + col(v, 0) + 4);
        }
      }
    } else {
      // the 16-byte units that the row touches: its neighbours' ends come along,
      // but nothing past the last row's end
      const uintptr_t at = reinterpret_cast<uintptr_t>(row), lead = at & 15;
      const uintptr_t end = at + ((M - 1 - m) * s.ld + H) * sizeof(E);
      const int bytes = static_cast<int>(lead) + H * static_cast<int>(sizeof(E));
      for (int u = t; u * 16 < bytes; u += T) {
        const uintptr_t from = at - lead + u * 16;
        cp16(dst + u * 16, reinterpret_cast<const void*>(from), end - from < 16 ? static_cast<int>(end - from) : 16);
      }
    }
  }
  // Group v of row m, from the stage that fetch() filled.
  template <class E>
  __device__ __forceinline__ void staged(const unsigned char* stage, const RowSrc& s, int64_t m, int v, int VPT,
                                         float out[8]) const {
    const unsigned char* src = stage + s.off;
    if constexpr (VEC) {
      if (col(v, 0) >= H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = 0.0f;
        return;
      }
      if constexpr (sizeof(E) == 2) {
        load8(reinterpret_cast<const uint16_t*>(src + (v * T + t) * 16), out);
      } else {
        const float4 lo = *reinterpret_cast<const float4*>(src + (v * T + t) * 16);
        const float4 hi = *reinterpret_cast<const float4*>(src + ((VPT + v) * T + t) * 16);
        out[0] = lo.x, out[1] = lo.y, out[2] = lo.z, out[3] = lo.w, out[4] = hi.x, out[5] = hi.y, out[6] = hi.z, out[7] = hi.w;
      }
    } else {
      const uintptr_t lead = reinterpret_cast<uintptr_t>(static_cast<const E*>(s.p) + m * s.ld) & 15;
      load(reinterpret_cast<const E*>(src + lead), v, out);
    }
  }
};

__device__ __forceinline__ float sigmoid_f32(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// The rows of a CTA, one after another.
template <class XT, class YT, int VPT, bool VEC, bool BWD>
struct Rows {
  const NormArgs& a;
  const Cols<VEC>& c;
  unsigned char* ring;
  int put_stage = 0, stage = 0;
  int64_t put_row, step;

  __device__ __forceinline__ Rows(const NormArgs& a_, const Cols<VEC>& c_, unsigned char* ring_)
      : a(a_), c(c_), ring(ring_), put_row(blockIdx.x), step(gridDim.x) {
    for (int i = 0; i + 1 < a.stages; ++i) put();
  }
  __device__ __forceinline__ void put() {
    if (put_row < a.M) {
      unsigned char* to = ring + put_stage * a.stage_bytes;
      if constexpr (BWD) {
        if (a.dr.p) c.template fetch<XT>(to, a.dr, put_row, a.M, VPT);
        if (a.w_next) {
          c.template fetch<XT>(to, a.x, put_row, a.M, VPT);
          a.n_f32 ? c.template fetch<float>(to, a.dn, put_row, a.M, VPT) : c.template fetch<uint16_t>(to, a.dn, put_row, a.M, VPT);
        }
      } else {
        c.template fetch<XT>(to, a.x, put_row, a.M, VPT);
      }
      if (a.y.p) c.template fetch<YT>(to, a.y, put_row, a.M, VPT);
      if (a.gate.p)
        a.gate_f32 ? c.template fetch<float>(to, a.gate, put_row, a.M, VPT) : c.template fetch<uint16_t>(to, a.gate, put_row, a.M, VPT);
      put_row += step;
    }
    cp_commit();
    put_stage = put_stage + 1 == a.stages ? 0 : put_stage + 1;
  }
  // Makes the next row readable and sets the row `stages - 1` further off.  The
  // stage that it fills is the last row's: this thread's own part of it, or,
  // read across threads, behind a barrier that they all reach after it.
  __device__ __forceinline__ void next() {
    if (!a.stages) return;
    cp_wait(a.stages);
    if constexpr (!VEC) __syncthreads();
    put();
  }
  __device__ __forceinline__ void done() {
    if (a.stages) stage = stage + 1 == a.stages ? 0 : stage + 1;
  }
  template <class E>
  __device__ __forceinline__ void load(const RowSrc& s, int64_t m, int v, float out[8]) const {
    if (a.stages)
      c.template staged<E>(ring + stage * a.stage_bytes, s, m, v, VPT, out);
    else
      c.load(static_cast<const E*>(s.p) + m * s.ld, v, out);
  }
  __device__ __forceinline__ void load(const RowSrc& s, int64_t m, int f32, int v, float out[8]) const {
    if (f32)
      load<float>(s, m, v, out);
    else
      load<uint16_t>(s, m, v, out);
  }
  // Factor f of the gate for a group of columns; with `slope`, also df/dgate.
  __device__ __forceinline__ void factor(int64_t m, int v, float f[8], float* slope) const {
    if (a.gate_kind == E4B_GATE_NONE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 1.0f;
      return;
    }
    if (a.gate_kind == E4B_GATE_TOKEN) {
      const float g = a.gate_f32 ? load1(static_cast<const float*>(a.vec_gate) + m)
                                 : load1(static_cast<const uint16_t*>(a.vec_gate) + m);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = g;
    } else if (a.gate_kind == E4B_GATE_CHANNEL) {
      c.load(a.vec_gate, 0, a.gate_f32, v, f);
    } else {
      load(a.gate, m, a.gate_f32, v, f);
    }
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = sigmoid_f32(f[j]);
    }
    if (slope) {
#pragma unroll
      for (int j = 0; j < 8; ++j) slope[j] = a.sigmoid ? f[j] * (1.0f - f[j]) : 1.0f;
    }
  }
};


// Sums of up to three values over the CTA's T threads (a multiple of 32).  One
// barrier above one warp: a caller that sums again passes another buffer.
template <int NV>
__device__ __forceinline__ void row_sum(float v[NV], int T, float4* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (T == 32) return;
  if ((threadIdx.x & 31) == 0)
    red[threadIdx.x >> 5] = make_float4(v[0], NV > 1 ? v[NV > 1 ? 1 : 0] : 0.0f, NV > 2 ? v[NV > 2 ? 2 : 0] : 0.0f, 0.0f);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.0f;
  for (int w = 0; w < T >> 5; ++w) {
    const float4 q = red[w];
    v[0] += q.x;
    if (NV > 1) v[NV > 1 ? 1 : 0] += q.y;
    if (NV > 2) v[NV > 2 ? 2 : 0] += q.z;
  }
}

// Most threads of a CTA, and CTAs an SM should hold, by the groups of a thread.
constexpr int norm_threads(int vpt) { return vpt == 4 ? 512 : 384; }

template <class XT, class YT, int VPT, bool VEC>
__global__ void __launch_bounds__(norm_threads(VPT), VPT == 1 ? 3 : VPT == 2 ? 2 : 1) block_norm_forward_kernel(NormArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  // Buffers alternate by row: a row may have one sum only, and so no other
  // barrier before the next row's.
  __shared__ float4 red[2][2][kMaxNormThreads / 32];
  const int T = blockDim.x;
  const Cols<VEC> c{T, static_cast<int>(threadIdx.x), a.H};
  Rows<XT, YT, VPT, VEC, false> rows(a, c, ring);
  int odd = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, odd ^= 1, rows.done()) {
    rows.next();
    float r[VPT][8], z[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v) rows.template load<XT>(a.x, m, v, r[v]);
    if (a.y.p) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        rows.template load<YT>(a.y, m, v, z[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] += z[v][j] * z[v][j];
      }
      float rstd = 1.0f;
      if (a.w_post) {
        row_sum<1>(ss, T, red[odd][0]);
        rstd = rsqrtf(ss[0] * a.inv_h + a.eps);
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float f[8];
        rows.factor(m, v, f, nullptr);
        if (a.w_post) {
          float w[8];
          c.load(a.w_post, 0, a.w_f32, v, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[v][j] *= rstd * (w[j] + a.offset);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[v][j] = fmaf(a.scale * f[j], z[v][j], r[v][j]);
        c.store(static_cast<XT*>(a.r) + m * a.ldr, v, r[v]);
      }
    }
    if (!a.w_next) continue;
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += c.col(v, j) < c.H ? r[v][j] * r[v][j] : 0.0f;
    row_sum<1>(ss, T, red[odd][1]);
    const float rstd = rsqrtf(ss[0] * a.inv_h + a.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float w[8];
      c.load(a.w_next, 0, a.w_f32, v, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = r[v][j] * rstd * (w[j] + a.offset);
      c.store(a.n, m * a.ldn, a.n_f32, v, w);
    }
  }
}

template <class XT, class YT, int VPT, bool VEC>
__global__ void __launch_bounds__(norm_threads(VPT), VPT == 1 ? 2 : 1) block_norm_backward_kernel(NormArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float4 red[2][2][kMaxNormThreads / 32];  // as in the forward
  const int T = blockDim.x;
  const Cols<VEC> c{T, static_cast<int>(threadIdx.x), a.H};
  Rows<XT, YT, VPT, VEC, true> rows(a, c, ring);
  float s_post[VPT][8] = {}, s_next[VPT][8] = {}, s_gate[VPT][8] = {};
  int odd = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, odd ^= 1, rows.done()) {
    rows.next();
    float s1[3] = {0.0f, 0.0f, 0.0f};  // sum r^2, sum h * r, sum y^2
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float p[8], q[8], w[8];
      if (a.y.p) {
        rows.template load<YT>(a.y, m, v, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) s1[2] += p[j] * p[j];
      }
      if (a.w_next) {
        rows.template load<XT>(a.x, m, v, p);
        rows.load(a.dn, m, a.n_f32, v, q);
        c.load(a.w_next, 0, a.w_f32, v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s1[0] += p[j] * p[j];
          s1[1] += q[j] * (w[j] + a.offset) * p[j];
        }
      }
    }
    row_sum<3>(s1, T, red[odd][0]);
    const float rstd_r = rsqrtf(s1[0] * a.inv_h + a.eps), rstd_y = a.w_post ? rsqrtf(s1[2] * a.inv_h + a.eps) : 1.0f;
    const float mean_r = s1[1] * rstd_r * a.inv_h;  // mean(h * rhat)
    float k[VPT][8];
    float s2[2] = {0.0f, 0.0f};  // sum k * yhat, sum d * z * slope
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float* d = k[v];
      if (a.dr.p) {
        rows.template load<XT>(a.dr, m, v, d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.0f;
      }
      if (a.w_next) {
        float p[8], q[8], w[8];
        rows.template load<XT>(a.x, m, v, p);
        rows.load(a.dn, m, a.n_f32, v, q);
        c.load(a.w_next, 0, a.w_f32, v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hat = p[j] * rstd_r;
          s_next[v][j] += q[j] * hat;
          d[j] += rstd_r * (q[j] * (w[j] + a.offset) - hat * mean_r);
        }
      }
      if (a.dx) c.store(static_cast<XT*>(a.dx) + m * a.lddx, v, d);
      if (!a.y.p) continue;
      float y[8], f[8], slope[8], w[8];
      rows.template load<YT>(a.y, m, v, y);
      rows.factor(m, v, f, slope);
      if (a.w_post) {
        c.load(a.w_post, 0, a.w_f32, v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += a.offset;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.0f;
      }
      float dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hat = y[j] * rstd_y, ds = a.scale * d[j];
        const float dz = ds * f[j];
        if (a.gate_kind != E4B_GATE_NONE) dg[j] = ds * hat * w[j] * slope[j];
        if (a.gate_kind == E4B_GATE_CHANNEL) s_gate[v][j] += dg[j];
        if (a.gate_kind == E4B_GATE_TOKEN) s2[1] += dg[j];
        s_post[v][j] += dz * hat;
        d[j] = dz * w[j];
        s2[0] += d[j] * hat;
      }
      if (a.gate_kind == E4B_GATE_FULL && a.dgate) c.store(a.dgate, m * a.H, a.gate_f32, v, dg);
    }
    if (!a.y.p) continue;
    if (a.w_post || a.gate_kind == E4B_GATE_TOKEN) row_sum<2>(s2, T, red[odd][1]);
    if (a.gate_kind == E4B_GATE_TOKEN && a.dgate && threadIdx.x == 0) {
      if (a.gate_f32)
        store1(static_cast<float*>(a.dgate) + m, s2[1]);
      else
        store1(static_cast<uint16_t*>(a.dgate) + m, s2[1]);
    }
    if (!a.dy) continue;
    const float mean_y = a.w_post ? s2[0] * a.inv_h : 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float y[8];
      rows.template load<YT>(a.y, m, v, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = rstd_y * (k[v][j] - y[j] * rstd_y * mean_y);
      c.store(static_cast<YT*>(a.dy) + m * a.lddy, v, y);
    }
  }
  const int64_t plane = static_cast<int64_t>(a.parts) * a.H;
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.H;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (a.w_post) c.store(part, v, s_post[v]);
    if (a.w_next) c.store(part + plane, v, s_next[v]);
    if (a.gate_kind == E4B_GATE_CHANNEL) c.store(part + 2 * plane, v, s_gate[v]);
  }
}

// out[q][col] = sum over parts of partial[q][part][col], in a fixed order: 16
// threads of a column take every 16th part, then are added in order.
struct ReduceArgs {
  const float* partial;
  float* out[3];
  int parts, H;
};
constexpr int kRedCols = 32, kRedLanes = 16;

__global__ void __launch_bounds__(kRedCols * kRedLanes) block_norm_reduce_kernel(ReduceArgs a) {
  float* out = a.out[blockIdx.y];
  if (!out) return;
  __shared__ float s[kRedLanes][kRedCols];
  const int col = blockIdx.x * kRedCols + threadIdx.x;
  float sum = 0.0f;
  if (col < a.H) {
    const float* p = a.partial + static_cast<int64_t>(blockIdx.y) * a.parts * a.H + col;
#pragma unroll 4
    for (int i = threadIdx.y; i < a.parts; i += kRedLanes) sum += p[static_cast<int64_t>(i) * a.H];
  }
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && col < a.H) {
    for (int i = 1; i < kRedLanes; ++i) sum += s[i][threadIdx.x];
    out[col] = sum;
  }
}

struct NormShape {
  int T, vpt, grid;
};

constexpr int kSms = 148;

// Threads of a row, their groups, and the persistent CTAs.  The workspace query
// and the launch agree because both go by M and H alone.
NormShape norm_shape(int64_t M, int H, int threads_per_sm) {
  const int nvec = (H + 7) / 8;
  NormShape s{};
  s.vpt = nvec <= norm_threads(1) ? 1 : nvec <= 2 * norm_threads(2) ? 2 : 4;
  s.T = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  const int per_sm = std::min(16, std::max(1, threads_per_sm / s.T));
  s.grid = static_cast<int>(std::min<int64_t>(M, kSms * per_sm));
  return s;
}
constexpr int kForwardThreads = 1152, kBackwardThreads = 768;  // per SM

// The ring: as many stages (2 to 4) as leave room for the SM's other CTAs, or, of
// rows too long for that, none.
void plan_ring(NormArgs* a, const NormShape& s, bool vec, bool x_f32, bool y_f32, int threads_per_sm, bool may_stage) {
  uint32_t off = 0;
  auto place = [&](RowSrc* r, bool f32) {
    if (!r->p) return;
    r->off = off;
    off += vec ? static_cast<uint32_t>(s.T * s.vpt * 8 * (f32 ? 4 : 2))
               : static_cast<uint32_t>(align_up(static_cast<size_t>(a->H) * (f32 ? 4 : 2), 16) + 16);
  };
  place(&a->dr, x_f32);
  place(&a->x, x_f32);
  place(&a->dn, a->n_f32);
  place(&a->y, y_f32);
  place(&a->gate, a->gate_f32);
  a->stage_bytes = off;
  const int ctas = std::min(16, std::max(1, threads_per_sm / s.T));
  const uint32_t room = 216 * 1024 / ctas;
  a->stages = may_stage ? static_cast<int>(std::min(4u, room / std::max(1u, off))) : 0;
  if (a->stages < 2) a->stages = may_stage && 2 * off <= 216 * 1024 ? 2 : 0;
}

template <class K>
cudaError_t launch_kernel(K kernel, const NormArgs& a, const NormShape& s, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(a.stages) * a.stage_bytes;
  if (cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem); err != cudaSuccess) return err;
  kernel<<<s.grid, s.T, smem, stream>>>(a);
  return cudaGetLastError();
}

template <bool BWD, class XT, class YT, int VPT>
cudaError_t launch_groups(const NormArgs& a, const NormShape& s, bool vec, cudaStream_t stream) {
  if constexpr (BWD)
    return vec ? launch_kernel(block_norm_backward_kernel<XT, YT, VPT, true>, a, s, stream)
               : launch_kernel(block_norm_backward_kernel<XT, YT, VPT, false>, a, s, stream);
  else
    return vec ? launch_kernel(block_norm_forward_kernel<XT, YT, VPT, true>, a, s, stream)
               : launch_kernel(block_norm_forward_kernel<XT, YT, VPT, false>, a, s, stream);
}

template <bool BWD, class XT, class YT>
cudaError_t launch_typed(const NormArgs& a, const NormShape& s, bool vec, cudaStream_t stream) {
  if (s.vpt == 1) return launch_groups<BWD, XT, YT, 1>(a, s, vec, stream);
  if (s.vpt == 2) return launch_groups<BWD, XT, YT, 2>(a, s, vec, stream);
  return launch_groups<BWD, XT, YT, 4>(a, s, vec, stream);
}

template <bool BWD>
cudaError_t launch(const NormArgs& a, bool x_f32, bool y_f32, const NormShape& s, bool vec, cudaStream_t stream) {
  if (x_f32)
    return y_f32 ? launch_typed<BWD, float, float>(a, s, vec, stream) : launch_typed<BWD, float, uint16_t>(a, s, vec, stream);
  return y_f32 ? launch_typed<BWD, uint16_t, float>(a, s, vec, stream)
               : launch_typed<BWD, uint16_t, uint16_t>(a, s, vec, stream);
}

bool is_dtype(int d) { return d == E4B_F32 || d == E4B_BF16; }
bool on_element(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == E4B_F32 ? 3u : 1u)) == 0;
}

// 8 elements of a base like this are one 16-byte (bf16) or 32-byte (fp32) vector.
bool vec_base(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == E4B_F32 ? 31u : 15u)) == 0; }

// What the two calls check alike.
e4b_status check_norm(const e4b_block_norm* p, int64_t M, const void* y, const void* gate, e4b_gate_kind kind,
                      e4b_dtype gate_dtype) {
  if (!p) return fail(E4B_ERR_INVALID_ARGUMENT, "null block norm");
  if (p->H < 1 || p->H > kMaxNormH)
    return fail(E4B_ERR_UNSUPPORTED, "H must be in [1, " + std::to_string(kMaxNormH) + "]");
  if (M < 0 || M > INT32_MAX) return fail(E4B_ERR_INVALID_ARGUMENT, "M must be in [0, 2^31)");
  if (!is_dtype(p->w_dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, "w_dtype must be F32 or BF16");
  if (!(p->eps > 0.0f)) return fail(E4B_ERR_INVALID_ARGUMENT, "eps must be positive");
  if (!on_element(p->w_post, p->w_dtype) || !on_element(p->w_next, p->w_dtype))
    return fail(E4B_ERR_INVALID_ARGUMENT, "w_post and w_next must be aligned to their elements");
  if (kind < E4B_GATE_NONE || kind > E4B_GATE_FULL) return fail(E4B_ERR_INVALID_ARGUMENT, "unknown gate kind");
  if ((kind != E4B_GATE_NONE) != (gate != nullptr) && M > 0)
    return fail(E4B_ERR_INVALID_ARGUMENT, "gate and gate_kind must be both set or both none");
  if (kind != E4B_GATE_NONE && (!is_dtype(gate_dtype) || !on_element(gate, gate_dtype)))
    return fail(E4B_ERR_INVALID_ARGUMENT, "gate_dtype must be F32 or BF16 and gate aligned to its elements");
  if (!y && M > 0 && (kind != E4B_GATE_NONE || p->w_post))
    return fail(E4B_ERR_INVALID_ARGUMENT, "a gate or w_post needs the block's output y");
  if (!y && !p->w_next) return fail(E4B_ERR_INVALID_ARGUMENT, "nothing to compute: neither y nor w_next");
  return E4B_OK;
}

// How a call's rows can be moved: as vectors of 8 columns, or else in units of 16 bytes.
struct Moves {
  bool vec, units;
};

// One tensor of rows: its type, stride and alignment.
e4b_status check_rows(const char* name, const void* p, int dtype, int64_t ld, int64_t H, Moves* moves) {
  if (!p) return E4B_OK;
  if (!is_dtype(dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + "'s type must be F32 or BF16");
  if (ld < H) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + "'s leading dimension must be >= H");
  if (!on_element(p, dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + " must be aligned to its elements");
  moves->vec = moves->vec && vec_base(p, dtype) && ld % 8 == 0;
  moves->units = moves->units && aligned16(p);
  return E4B_OK;
}

NormArgs norm_args(const e4b_block_norm* p, int64_t M, const void* y, int64_t ldy, const void* gate, e4b_gate_kind kind,
                   e4b_dtype gate_dtype, e4b_dtype n_dtype) {
  NormArgs a{};
  a.y = {y, ldy, 0};
  (kind == E4B_GATE_FULL ? a.gate.p : a.vec_gate) = gate;
  a.gate.ld = p->H;
  a.w_post = p->w_post;
  a.w_next = p->w_next;
  a.M = M;
  a.H = static_cast<int>(p->H);
  a.gate_kind = kind;
  a.gate_f32 = gate_dtype == E4B_F32;
  a.sigmoid = p->gate_sigmoid != 0;
  a.w_f32 = p->w_dtype == E4B_F32;
  a.n_f32 = n_dtype == E4B_F32;
  a.scale = p->residual_scale;
  a.offset = p->weight_offset;
  a.eps = p->eps;
  a.inv_h = 1.0f / static_cast<float>(p->H);
  return a;
}

// Whether weights, gate and (backward) its gradient allow vectors and units.
Moves moves_of(const e4b_block_norm* p, const void* gate, e4b_gate_kind kind, e4b_dtype gate_dtype, const void* dgate) {
  Moves m{p->H % 8 == 0 && vec_base(p->w_post, p->w_dtype) && vec_base(p->w_next, p->w_dtype), true};
  if (kind == E4B_GATE_CHANNEL || kind == E4B_GATE_FULL) m.vec = m.vec && vec_base(gate, gate_dtype);
  if (kind == E4B_GATE_FULL) {
    m.vec = m.vec && vec_base(dgate, gate_dtype);
    m.units = aligned16(gate);
  }
  return m;
}

}  // namespace
}  // namespace e4b

using namespace e4b;

extern "C" {

e4b_status e4b_block_norm_forward(const void* x, e4b_dtype x_dtype, int64_t ldx, const void* y, e4b_dtype y_dtype,
                                  int64_t ldy, const void* gate, e4b_gate_kind gate_kind, e4b_dtype gate_dtype,
                                  int64_t M, const e4b_block_norm* norm, void* r, int64_t ldr, void* n,
                                  e4b_dtype n_dtype, int64_t ldn, e4b_stream stream) {
  begin_call();
  if (e4b_status s = check_norm(norm, M, y, gate, gate_kind, gate_dtype); s != E4B_OK) return s;
  if (M > 0 && !x) return fail(E4B_ERR_INVALID_ARGUMENT, "null x");
  if (M > 0 && (y != nullptr) != (r != nullptr)) return fail(E4B_ERR_INVALID_ARGUMENT, "r is written exactly when y is given");
  if (M > 0 && (norm->w_next != nullptr) != (n != nullptr))
    return fail(E4B_ERR_INVALID_ARGUMENT, "n is written exactly when w_next is given");
  Moves moves = moves_of(norm, gate, gate_kind, gate_dtype, nullptr);
  if (e4b_status s = check_rows("x", x, x_dtype, ldx, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("y", y, y_dtype, ldy, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("r", r, x_dtype, ldr, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("n", n, n_dtype, ldn, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  if (M == 0) {
    set_path("block_norm.empty");
    return E4B_OK;
  }
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormArgs a = norm_args(norm, M, y, ldy, gate, gate_kind, gate_dtype, n_dtype);
  a.x = {x, ldx, 0};
  a.r = r;
  a.n = n;
  a.ldr = ldr;
  a.ldn = ldn;
  const NormShape s = norm_shape(M, a.H, kForwardThreads);
  const bool x_f32 = x_dtype == E4B_F32, y_f32 = y && y_dtype == E4B_F32;
  plan_ring(&a, s, moves.vec, x_f32, y_f32, kForwardThreads, moves.vec || moves.units);
  LaunchScope ls("block_norm.forward", st);
  if (cudaError_t err = launch<false>(a, x_f32, y_f32, s, moves.vec, st); err != cudaSuccess)
    return cuda_fail(err, "block norm forward launch");
  set_path(moves.vec ? "block_norm.forward" : "block_norm.forward.scalar");
  return E4B_OK;
}

size_t e4b_block_norm_backward_workspace_size(int64_t M, const e4b_block_norm* norm) {
  if (!norm || M < 1 || norm->H < 1 || norm->H > kMaxNormH) return 0;
  const NormShape s = norm_shape(M, static_cast<int>(norm->H), kBackwardThreads);
  return static_cast<size_t>(3) * s.grid * norm->H * sizeof(float);
}

e4b_status e4b_block_norm_backward(const void* dr, int64_t lddr, const void* dn, e4b_dtype n_dtype, int64_t lddn,
                                   const void* r, e4b_dtype x_dtype, int64_t ldr, const void* y, e4b_dtype y_dtype,
                                   int64_t ldy, const void* gate, e4b_gate_kind gate_kind, e4b_dtype gate_dtype,
                                   int64_t M, const e4b_block_norm* norm, void* dx, int64_t lddx, void* dy,
                                   int64_t lddy, void* dgate, float* dw_post, float* dw_next, void* workspace,
                                   size_t workspace_bytes, e4b_stream stream) {
  begin_call();
  if (e4b_status s = check_norm(norm, M, y, gate, gate_kind, gate_dtype); s != E4B_OK) return s;
  if (M > 0 && (norm->w_next != nullptr) != (dn != nullptr))
    return fail(E4B_ERR_INVALID_ARGUMENT, "dn is read exactly when w_next is given");
  if (M > 0 && norm->w_next && !r) return fail(E4B_ERR_INVALID_ARGUMENT, "null r");
  if (M > 0 && !dr && !dn) return fail(E4B_ERR_INVALID_ARGUMENT, "neither dr nor dn is given");
  if ((dy && !y && M > 0) || (dgate && gate_kind == E4B_GATE_NONE) || (dw_post && !norm->w_post) ||
      (dw_next && !norm->w_next))
    return fail(E4B_ERR_INVALID_ARGUMENT, "a gradient is asked for of an input that the block does not have");
  Moves moves = moves_of(norm, gate, gate_kind, gate_dtype, dgate);
  if (e4b_status s = check_rows("dr", dr, x_dtype, lddr, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("dn", dn, n_dtype, lddn, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("r", r, x_dtype, ldr, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("y", y, y_dtype, ldy, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("dx", dx, x_dtype, lddx, norm->H, &moves); s != E4B_OK) return s;
  if (e4b_status s = check_rows("dy", dy, y_dtype, lddy, norm->H, &moves); s != E4B_OK) return s;
  if (!on_element(dgate, gate_kind == E4B_GATE_CHANNEL ? E4B_F32 : gate_dtype) || !on_element(dw_post, E4B_F32) ||
      !on_element(dw_next, E4B_F32))
    return fail(E4B_ERR_INVALID_ARGUMENT, "dgate, dw_post and dw_next must be aligned to their elements");
  if (e4b_status s = check_workspace("block norm backward", e4b_block_norm_backward_workspace_size(M, norm), workspace,
                                     workspace_bytes);
      s != E4B_OK)
    return s;
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormArgs a = norm_args(norm, M, y, ldy, gate, gate_kind, gate_dtype, n_dtype);
  a.dr = {dr, lddr, 0};
  a.dn = {dn, lddn, 0};
  if (norm->w_next) a.x = {r, ldr, 0};
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.partial = static_cast<float*>(workspace);
  a.lddx = lddx;
  a.lddy = lddy;
  if (M > 0) {
    const NormShape s = norm_shape(M, a.H, kBackwardThreads);
    a.parts = s.grid;
    const bool x_f32 = x_dtype == E4B_F32, y_f32 = y && y_dtype == E4B_F32;
    // the partial sums' rows are vectors of 32 bytes
    const bool vec = moves.vec && vec_base(workspace, E4B_F32);
    plan_ring(&a, s, vec, x_f32, y_f32, kBackwardThreads, vec || moves.units);
    LaunchScope ls("block_norm.backward", st);
    if (cudaError_t err = launch<true>(a, x_f32, y_f32, s, vec, st); err != cudaSuccess)
      return cuda_fail(err, "block norm backward launch");
  }
  float* dchannel = gate_kind == E4B_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  if (dw_post || dw_next || dchannel) {
    ReduceArgs ra{a.partial, {dw_post, dw_next, dchannel}, a.parts, a.H};
    LaunchScope ls("block_norm.reduce", st);
    block_norm_reduce_kernel<<<dim3((a.H + kRedCols - 1) / kRedCols, 3), dim3(kRedCols, kRedLanes), 0, st>>>(ra);
  }
  if (cudaError_t err = cudaGetLastError(); err != cudaSuccess) return cuda_fail(err, "block norm reduce launch");
  set_path(M == 0 ? "block_norm.backward.empty" : moves.vec ? "block_norm.backward" : "block_norm.backward.scalar");
  return E4B_OK;
}

}  // extern "C"
