// The norms after and before a block, fused with the block's gate, its
// residual scale and the residual sum; forward and backward.
//
//   z = N(y; w_post)                       (or z = y without w_post)
//   r = x + s * f(gate) * z                f(g) = g or sigmoid(g)
//   n = N(r; w_next)
//   N(v; w) = v * rstd(v) * (w + offset),  rstd(v) = 1 / sqrt(mean(v^2) + eps)
//
// Bound: HBM.  A row is read once into registers, both norms are taken on the
// 32-bit values there (n from the unrounded r), and every output is rounded
// once.  T threads share a row, each with VPT vectors of 8 columns: a row's
// sum of squares is a warp shuffle and, above one warp, one block barrier.
//
// Backward, with d = dr + (dn through the next norm):
//   h = dn * (w_next + offset):  d += rstd_r * (h - rhat * mean(h * rhat))
//   dx = d,  dz = s * f * d,  df = s * d * z  (summed over a gate's broadcast axis)
//   k = dz * (w_post + offset):  dy = rstd_y * (k - yhat * mean(k * yhat))
//   dw_next = sum_m dn * rhat,  dw_post = sum_m dz * yhat
// Both rstd are taken again from r and y, which the gradients need anyway, so
// the forward saves nothing.  The CTAs are persistent and keep their columns'
// sums over rows in registers; a second kernel adds the CTAs' partial sums in
// CTA order, so every sum has a fixed order.
#include <algorithm>
#include <string>

#include "common.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

constexpr int kMaxNormH = 16384;
constexpr int kMaxNormThreads = 512;

struct NormArgs {
  const void *x, *y, *gate, *w_post, *w_next;
  const void *dr, *dn;               // backward
  void *r, *n;                       // forward
  void *dx, *dy, *dgate;             // backward
  float* partial;                    // backward: [3][parts][H] column sums (w_post, w_next, channel gate)
  int64_t ldx, ldy, ldr, ldn;        // ldx also of dr and dx, ldy of dy, ldn of dn
  int64_t lddr, lddx, lddy;
  int64_t M;
  int H, parts;
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
__device__ __forceinline__ void store8(float* p, const float v[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// One thread's share of a row: VPT groups of 8 columns.  VEC: a group is 8
// adjacent columns, moved as 16-byte vectors; otherwise (odd widths, strides
// or bases) its columns lie T apart, so that a warp's accesses stay adjacent.
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
};

__device__ __forceinline__ float sigmoid_f32(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// Sums of NV values over the T threads of a row (T a multiple of 32; every
// thread of the block calls this).  `red` holds NV floats per warp of the
// block.  One barrier: a caller that sums again passes another buffer.
template <int NV>
__device__ __forceinline__ void row_sum(float v[NV], int T, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (T == 32) return;
  const int warps = T >> 5;
  float* mine = red + threadIdx.y * warps * NV;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[(threadIdx.x >> 5) * NV + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += mine[w * NV + i];
}

// Factor f of the gate for one group of columns; with `slope`, also df/dgate.
template <bool VEC>
__device__ __forceinline__ void gate_factor(const NormArgs& a, const Cols<VEC>& c, int64_t m, int v, float f[8],
                                            float* slope) {
  if (a.gate_kind == E4B_GATE_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.0f;
    return;
  }
  if (a.gate_kind == E4B_GATE_TOKEN) {
    float g = 0.0f;
    if (c.H > 0)  // a row past the last one reads nothing
      g = a.gate_f32 ? load1(static_cast<const float*>(a.gate) + m) : load1(static_cast<const uint16_t*>(a.gate) + m);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = g;
  } else {
    c.load(a.gate, a.gate_kind == E4B_GATE_FULL ? m * a.H : 0, a.gate_f32, v, f);
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

template <class XT, class YT, int VPT, bool VEC>
__global__ void __launch_bounds__(kMaxNormThreads) block_norm_forward_kernel(NormArgs a) {
  __shared__ float red[2][kMaxNormThreads / 32];
  const int T = blockDim.x;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = m < a.M;
  const Cols<VEC> c{T, static_cast<int>(threadIdx.x), live ? a.H : 0};
  float r[VPT][8], z[VPT][8];
  const XT* x = static_cast<const XT*>(a.x) + m * a.ldx;
#pragma unroll
  for (int v = 0; v < VPT; ++v) c.load(x, v, r[v]);
  if (a.y) {
    const YT* y = static_cast<const YT*>(a.y) + m * a.ldy;
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      c.load(y, v, z[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += z[v][j] * z[v][j];
    }
    float rstd = 1.0f;
    if (a.w_post) {
      row_sum<1>(ss, T, red[0]);
      rstd = rsqrtf(ss[0] * a.inv_h + a.eps);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float f[8];
      gate_factor(a, c, m, v, f, nullptr);
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
  if (!a.w_next) return;
  float ss[1] = {0.0f};
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.col(v, j) < c.H) ss[0] += r[v][j] * r[v][j];
  row_sum<1>(ss, T, red[1]);
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

template <class XT, class YT, int VPT, bool VEC>
__global__ void __launch_bounds__(kMaxNormThreads) block_norm_backward_kernel(NormArgs a) {
  // The first sum of a row alternates between two buffers: there may be no
  // second sum, and so no other barrier, before the next row's.
  __shared__ float red[3][3 * kMaxNormThreads / 32];
  int odd = 0;
  const int T = blockDim.x;
  const Cols<VEC> all{T, static_cast<int>(threadIdx.x), a.H};
  float s_post[VPT][8] = {}, s_next[VPT][8] = {}, s_gate[VPT][8] = {};
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  // All rows of a block go through the loop together (row_sum has a barrier).
  for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * blockDim.y; m0 < a.M; m0 += step) {
    const int64_t m = m0 + threadIdx.y;
    const bool live = m < a.M;
    const Cols<VEC> c{T, static_cast<int>(threadIdx.x), live ? a.H : 0};
    float d[VPT][8], r[VPT][8], h[VPT][8], y[VPT][8];
    float s1[3] = {0.0f, 0.0f, 0.0f};  // sum r^2, sum h * r, sum y^2
    const XT* dr = static_cast<const XT*>(a.dr) + m * a.lddr;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (a.dr) {
        c.load(dr, v, d[v]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[v][j] = 0.0f;
      }
      if (a.y) c.load(static_cast<const YT*>(a.y) + m * a.ldy, v, y[v]);
      if (a.w_next) {
        c.load(static_cast<const XT*>(a.r) + m * a.ldr, v, r[v]);
        c.load(a.dn, m * a.ldn, a.n_f32, v, h[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (a.y) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s1[2] += y[v][j] * y[v][j];
      }
      if (a.w_next) {
        float w[8];
        c.load(a.w_next, 0, a.w_f32, v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s1[0] += r[v][j] * r[v][j];
          s1[1] += h[v][j] * (w[j] + a.offset) * r[v][j];
        }
      }
    }
    row_sum<3>(s1, T, red[odd]);
    odd ^= 1;
    if (a.w_next) {
      const float rstd = rsqrtf(s1[0] * a.inv_h + a.eps);
      const float mean = s1[1] * rstd * a.inv_h;  // mean(h * rhat)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float w[8];
        c.load(a.w_next, 0, a.w_f32, v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hat = r[v][j] * rstd;
          s_next[v][j] += h[v][j] * hat;
          d[v][j] += rstd * (h[v][j] * (w[j] + a.offset) - hat * mean);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (a.dx) c.store(static_cast<XT*>(a.dx) + m * a.lddx, v, d[v]);
    if (!a.y) continue;
    const float rstd = a.w_post ? rsqrtf(s1[2] * a.inv_h + a.eps) : 1.0f;
    float s2[2] = {0.0f, 0.0f};  // sum k * yhat, sum d * z * slope
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float f[8], slope[8], w[8];
      gate_factor(a, c, m, v, f, slope);
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
        const float hat = y[v][j] * rstd, ds = a.scale * d[v][j];
        const float dz = ds * f[j];
        if (a.gate_kind != E4B_GATE_NONE) dg[j] = ds * hat * w[j] * slope[j];
        if (a.gate_kind == E4B_GATE_CHANNEL) s_gate[v][j] += dg[j];
        if (a.gate_kind == E4B_GATE_TOKEN) s2[1] += dg[j];
        s_post[v][j] += dz * hat;
        d[v][j] = dz * w[j];  // k
        s2[0] += d[v][j] * hat;
      }
      if (a.gate_kind == E4B_GATE_FULL && a.dgate) c.store(a.dgate, m * a.H, a.gate_f32, v, dg);
    }
    if (a.w_post || a.gate_kind == E4B_GATE_TOKEN) row_sum<2>(s2, T, red[2]);
    if (a.gate_kind == E4B_GATE_TOKEN && a.dgate && threadIdx.x == 0 && live) {
      if (a.gate_f32)
        store1(static_cast<float*>(a.dgate) + m, s2[1]);
      else
        store1(static_cast<uint16_t*>(a.dgate) + m, s2[1]);
    }
    const float mean = a.w_post ? s2[0] * a.inv_h : 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (d[v][j] - y[v][j] * rstd * mean);
      if (a.dy) c.store(static_cast<YT*>(a.dy) + m * a.lddy, v, o);
    }
  }
  const int64_t part = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y, plane = static_cast<int64_t>(a.parts) * a.H;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (a.w_post) all.store(a.partial + part * a.H, v, s_post[v]);
    if (a.w_next) all.store(a.partial + plane + part * a.H, v, s_next[v]);
    if (a.gate_kind == E4B_GATE_CHANNEL) all.store(a.partial + 2 * plane + part * a.H, v, s_gate[v]);
  }
}

// out[q][col] = sum over parts of partial[q][part][col], in a fixed order: 8
// threads of a column take every 8th part, then are added in order.
struct ReduceArgs {
  const float* partial;
  float* out[3];
  int parts, H;
};
constexpr int kRedCols = 32, kRedLanes = 8;

__global__ void __launch_bounds__(kRedCols * kRedLanes) block_norm_reduce_kernel(ReduceArgs a) {
  float* out = a.out[blockIdx.y];
  if (!out) return;
  __shared__ float s[kRedLanes][kRedCols];
  const int col = blockIdx.x * kRedCols + threadIdx.x;
  float sum = 0.0f;
  if (col < a.H) {
    const float* p = a.partial + static_cast<int64_t>(blockIdx.y) * a.parts * a.H + col;
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
  int T, rows, vpt;
};

NormShape norm_shape(int H, int vpt_max) {
  const int nvec = (H + 7) / 8;
  NormShape s{};
  s.vpt = 1;
  while (s.vpt < 4 && (s.vpt < vpt_max ? nvec > 32 * s.vpt : nvec > kMaxNormThreads * s.vpt)) s.vpt *= 2;
  s.T = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  s.rows = s.T >= 128 ? 1 : 128 / s.T;
  return s;
}

// Persistent CTAs of the backward, 768 threads on each of the B200's 148 SMs,
// and the partial sums they leave: one for each row slot of a CTA.
int backward_parts(int64_t M, const NormShape& s, int* grid) {
  const int64_t blocks = (M + s.rows - 1) / s.rows;
  const int per_sm = std::max(1, 768 / (s.T * s.rows));
  *grid = static_cast<int>(std::min<int64_t>(blocks, 148 * per_sm));
  return *grid * s.rows;
}

template <bool BWD, class XT, class YT>
void launch_typed(const NormArgs& a, const NormShape& s, int grid, bool vec, cudaStream_t stream) {
  const dim3 block(s.T, s.rows);
  auto go = [&](auto vpt) {
    constexpr int V = decltype(vpt)::value;
    if constexpr (BWD) {
      if (vec)
        block_norm_backward_kernel<XT, YT, V, true><<<grid, block, 0, stream>>>(a);
      else
        block_norm_backward_kernel<XT, YT, V, false><<<grid, block, 0, stream>>>(a);
    } else {
      if (vec)
        block_norm_forward_kernel<XT, YT, V, true><<<grid, block, 0, stream>>>(a);
      else
        block_norm_forward_kernel<XT, YT, V, false><<<grid, block, 0, stream>>>(a);
    }
  };
  if (s.vpt == 1)
    go(std::integral_constant<int, 1>());
  else if (s.vpt == 2)
    go(std::integral_constant<int, 2>());
  else
    go(std::integral_constant<int, 4>());
}

template <bool BWD>
void launch(const NormArgs& a, bool x_f32, bool y_f32, const NormShape& s, int grid, bool vec, cudaStream_t stream) {
  if (x_f32)
    y_f32 ? launch_typed<BWD, float, float>(a, s, grid, vec, stream)
          : launch_typed<BWD, float, uint16_t>(a, s, grid, vec, stream);
  else
    y_f32 ? launch_typed<BWD, uint16_t, float>(a, s, grid, vec, stream)
          : launch_typed<BWD, uint16_t, uint16_t>(a, s, grid, vec, stream);
}

bool is_dtype(int d) { return d == E4B_F32 || d == E4B_BF16; }
bool on_element(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == E4B_F32 ? 3u : 1u)) == 0;
}

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

// One tensor of rows: its type, stride and alignment.  `vec` stays true while
// 8 columns of every row can be moved as 16-byte vectors.
e4b_status check_rows(const char* name, const void* p, int dtype, int64_t ld, int64_t H, bool* vec) {
  if (!p) return E4B_OK;
  if (!is_dtype(dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + "'s type must be F32 or BF16");
  if (ld < H) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + "'s leading dimension must be >= H");
  if (!on_element(p, dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + " must be aligned to its elements");
  *vec = *vec && aligned16(p) && ld % 8 == 0;
  return E4B_OK;
}

NormArgs norm_args(const e4b_block_norm* p, int64_t M, const void* y, const void* gate, e4b_gate_kind kind,
                   e4b_dtype gate_dtype, e4b_dtype n_dtype) {
  NormArgs a{};
  a.y = y;
  a.gate = gate;
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
  bool vec = norm->H % 8 == 0 && aligned16(norm->w_post) && aligned16(norm->w_next) &&
             (gate_kind < E4B_GATE_CHANNEL || gate_kind == E4B_GATE_TOKEN || aligned16(gate));
  if (e4b_status s = check_rows("x", x, x_dtype, ldx, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("y", y, y_dtype, ldy, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("r", r, x_dtype, ldr, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("n", n, n_dtype, ldn, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  if (M == 0) {
    set_path("block_norm.empty");
    return E4B_OK;
  }
  NormArgs a = norm_args(norm, M, y, gate, gate_kind, gate_dtype, n_dtype);
  a.x = x;
  a.r = r;
  a.n = n;
  a.ldx = ldx;
  a.ldy = ldy;
  a.ldr = ldr;
  a.ldn = ldn;
  // A few rows leave most SMs idle: the widest split of a row is the shortest.
  const NormShape s = norm_shape(a.H, M < 296 ? 1 : 4);
  {
    LaunchScope ls("block_norm.forward", reinterpret_cast<cudaStream_t>(stream));
    launch<false>(a, x_dtype == E4B_F32, y && y_dtype == E4B_F32, s, static_cast<int>((M + s.rows - 1) / s.rows), vec,
                  reinterpret_cast<cudaStream_t>(stream));
  }
  if (cudaError_t err = cudaGetLastError(); err != cudaSuccess) return cuda_fail(err, "block norm forward launch");
  set_path(vec ? "block_norm.forward" : "block_norm.forward.scalar");
  return E4B_OK;
}

size_t e4b_block_norm_backward_workspace_size(int64_t M, const e4b_block_norm* norm) {
  if (!norm || M < 1 || norm->H < 1 || norm->H > kMaxNormH) return 0;
  int grid = 0;
  const int parts = backward_parts(M, norm_shape(static_cast<int>(norm->H), 1), &grid);
  return static_cast<size_t>(3) * parts * norm->H * sizeof(float);
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
  bool vec = norm->H % 8 == 0 && aligned16(norm->w_post) && aligned16(norm->w_next) &&
             (gate_kind == E4B_GATE_NONE || gate_kind == E4B_GATE_TOKEN || aligned16(gate)) &&
             (gate_kind != E4B_GATE_FULL || aligned16(dgate));
  if (e4b_status s = check_rows("dr", dr, x_dtype, lddr, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("dn", dn, n_dtype, lddn, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("r", r, x_dtype, ldr, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("y", y, y_dtype, ldy, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("dx", dx, x_dtype, lddx, norm->H, &vec); s != E4B_OK) return s;
  if (e4b_status s = check_rows("dy", dy, y_dtype, lddy, norm->H, &vec); s != E4B_OK) return s;
  if (!on_element(dgate, gate_kind == E4B_GATE_CHANNEL ? E4B_F32 : gate_dtype) || !on_element(dw_post, E4B_F32) ||
      !on_element(dw_next, E4B_F32))
    return fail(E4B_ERR_INVALID_ARGUMENT, "dgate, dw_post and dw_next must be aligned to their elements");
  if (e4b_status s = check_workspace("block norm backward", e4b_block_norm_backward_workspace_size(M, norm), workspace,
                                     workspace_bytes);
      s != E4B_OK)
    return s;
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormArgs a = norm_args(norm, M, y, gate, gate_kind, gate_dtype, n_dtype);
  a.dr = dr;
  a.dn = dn;
  a.x = nullptr;
  a.r = const_cast<void*>(r);
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.partial = static_cast<float*>(workspace);
  a.lddr = lddr;
  a.ldn = lddn;
  a.ldr = ldr;
  a.ldy = ldy;
  a.lddx = lddx;
  a.lddy = lddy;
  if (M > 0) {
    const NormShape s = norm_shape(a.H, 1);
    int grid = 0;
    a.parts = backward_parts(M, s, &grid);
    LaunchScope ls("block_norm.backward", st);
    launch<true>(a, x_dtype == E4B_F32, y && y_dtype == E4B_F32, s, grid, vec, st);
  }
  if (cudaError_t err = cudaGetLastError(); err != cudaSuccess) return cuda_fail(err, "block norm backward launch");
  float* dchannel = gate_kind == E4B_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  if (dw_post || dw_next || dchannel) {
    ReduceArgs ra{a.partial, {dw_post, dw_next, dchannel}, a.parts, a.H};
    LaunchScope ls("block_norm.reduce", st);
    block_norm_reduce_kernel<<<dim3((a.H + kRedCols - 1) / kRedCols, 3), dim3(kRedCols, kRedLanes), 0, st>>>(ra);
  }
  if (cudaError_t err = cudaGetLastError(); err != cudaSuccess) return cuda_fail(err, "block norm reduce launch");
  set_path(M == 0 ? "block_norm.backward.empty" : vec ? "block_norm.backward" : "block_norm.backward.scalar");
  return E4B_OK;
}

}  // extern "C"
