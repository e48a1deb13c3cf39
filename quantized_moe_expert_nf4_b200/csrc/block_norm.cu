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
// sums meet (a warp shuffle and a block barrier per sum).  Where 8 columns of every row
// are aligned vectors, a thread copies and reads its own columns only.  Rows that start
// anywhere within 16 bytes (odd widths, odd strides) are copied as the 16-byte units
// that they touch and read as shifted vectors.  Tensors that are not 16-byte aligned, and
// rows too long for a ring of vectors (see plan()), are read by element.  Both norms
// are taken on 32-bit values in registers (n from the unrounded r), and every output is
// rounded once.
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
//
// Measured (bandwidth of the bytes that a call cannot do without):
//   forward, 8192 x 2880, bf16 y, fp32 stream, bf16 n   45-50 us, 5.7 TB/s
//   forward, 8192 x 2880, all bf16, channel gate        35 us, 5.3 TB/s
//   forward, 8192 x 4096, all bf16, channel gate        64 us, 4.2 TB/s
//   forward, 8192 x 2049, all bf16, no gate (shifted)   54 us, 2.5 TB/s
//   backward, 8192 x 2880, bf16, fp32 dgate and dw      61.5 us, 4.6 TB/s
//   backward, 8192 x 4096, the same                     144 us, 2.8 TB/s (see norm_shape())
//   backward, 4096 x 8192, the same                     209 us, 1.9 TB/s
//   backward, 2048 x 2049, full gate (shifted)          45 us, 1.5 TB/s
//   forward of one row                                  2.6 us on the device, 9.5 with the call
// The forward is bound by HBM.  The backward of one group of columns a thread is full
// neither in issue (65%) nor in HBM (67%) at 24 warps an SM: registers (a thread's columns
// of the weights and their gradients) allow no more, and shared memory is read twice a row.  What
// carried it: rows ahead in a ring 265 -> 132 us, packed fp32 -> 104, kernels with the usual
// inputs and outputs known at compile time -> 85, weights in registers and what is the same
// in every row taken out of the sums over rows -> 61.  A row's sums meet once: the sum
// of k * yhat is taken term by term of d.  A row's weights in registers took the forward from 61 us to
// 45; two or four groups of columns a thread where one is enough measured slower in both.
#include <algorithm>
#include <string>

#include "block_norm.cuh"

namespace e4b {
namespace {

constexpr int kMaxNormH = 16384;

// Rows of any width, stride and base.
template <class XT, class YT, int VPT, int T>
__global__ void __launch_bounds__(T, VPT == 1 ? 768 / T : 1)
    block_norm_forward_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  // Buffers alternate by row: a row may have one sum only, and so no other
  // barrier before the next row's.
  __shared__ float red[2][2][64];
  const Cols<VPT, T> c{static_cast<int>(threadIdx.x), a.H};
  pdl_wait();
  pdl_launch_dependents();
  Rows<XT, YT, VPT, T, false> rows(a, c, ring);
  const F2 offset = f2(a.offset);
  int odd = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, odd ^= 1) {
    rows.next();
    F8 r[VPT];
    if (a.y.p) {
      F8 z[VPT];
      F2 sq = f2(0.0f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        z[v] = rows.template load<YT>(a.y, m, v);
        sq = dot8(z[v], z[v], sq);
      }
      float factor = a.scale;  // residual scale and the row's 1 / rms
      if (a.w_post) {
        float ss[1] = {lo(sq) + hi(sq)};
        row_sum<1>(ss, T, red[odd][0]);
        factor *= rsqrtf(ss[0] * a.inv_h + a.eps);
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        z[v] = z[v] * f2(factor);
        if (a.w_post) z[v] = z[v] * (c.load(a.w_post, a.w_f32, v) + offset);
        r[v] = rows.template load<XT>(a.x, m, v);
        if (a.gate_kind != E4B_GATE_NONE) {
          F8 f = rows.gate(m, v);
          if (a.sigmoid) f = sigmoid8(f);
          r[v] = fma8(z[v], f, r[v]);
        } else {
          r[v] = fma8(z[v], f2(1.0f), r[v]);
        }
        c.store(reinterpret_cast<XT*>(static_cast<unsigned char*>(a.r.p) + m * a.r.row), v, r[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < VPT; ++v) r[v] = rows.template load<XT>(a.x, m, v);
    }
    if (!a.w_next) continue;
    F2 sq = f2(0.0f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) sq = dot8(r[v], r[v], sq);
    float ss[1] = {lo(sq) + hi(sq)};
    row_sum<1>(ss, T, red[odd][1]);
    const F2 rstd = f2(rsqrtf(ss[0] * a.inv_h + a.eps));
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      c.store(static_cast<unsigned char*>(a.n.p) + m * a.n.row, 0, a.n_f32, v, r[v] * rstd * (c.load(a.w_next, a.w_f32, v) + offset));
  }
}

// Rows moved as vectors, aligned or shifted (COLS).  ALL: y and both weights are there, the step between two
// blocks.
template <class XT, class YT, int VPT, class COLS, bool ALL>
__global__ void __launch_bounds__(norm_threads(VPT), VPT < 4 ? 2 : 1)
    block_norm_forward_vec_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float red[2][2][64];  // as above
  const int T = blockDim.x;
  const COLS c(T, threadIdx.x, a.H);
  const bool has_y = ALL || a.y.p, next = ALL || a.w_next, post = ALL || a.w_post;
  const int kind = a.gate_kind, stages = a.stages;
  const int step = static_cast<int>(gridDim.x);
  auto row_of = [&](const RowSrc& t) { return static_cast<const unsigned char*>(t.p) + blockIdx.x * t.row; };
  const unsigned char *x_p = row_of(a.x), *y_p = row_of(a.y), *g_p = row_of(a.gate);
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
      c.template fetch<XT>(to + a.x.off, x_p, a.x, last);
      x_p += a.x.step;
      if (has_y) {
        c.template fetch<YT>(to + a.y.off, y_p, a.y, last);
        y_p += a.y.step;
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
  // One group per thread: its weights and channel gate stay in registers.
  constexpr bool kHold = VPT == 1;
  F8 hold_post, hold_next, hold_gate;
  if constexpr (kHold) {
    if (post) hold_post = c.vector(a.w_post, a.w_f32, 0) + offset;
    if (next) hold_next = c.vector(a.w_next, a.w_f32, 0) + offset;
    if (kind == E4B_GATE_CHANNEL) hold_gate = c.vector(a.vec_gate, a.gate_f32, 0);
  }
  auto w_post = [&](int v) { return kHold ? hold_post : c.vector(a.w_post, a.w_f32, v) + offset; };
  auto w_next = [&](int v) { return kHold ? hold_next : c.vector(a.w_next, a.w_f32, v) + offset; };
  unsigned char* r_p = static_cast<unsigned char*>(a.r.p) + blockIdx.x * a.r.row;
  unsigned char* n_p = static_cast<unsigned char*>(a.n.p) + blockIdx.x * a.n.row;
  auto flush = [&](int set, unsigned char* r_row, unsigned char* n_row) {
    if constexpr (COLS::kShared) {
      const unsigned char* out = ring + a.out_off + set * a.out_bytes;
      if (has_y) c.template flush<XT>(r_row, out + a.out_slot[0]);
      if (next) {
        if (a.n_f32)
          c.template flush<float>(n_row, out + a.out_slot[1]);
        else
          c.template flush<uint16_t>(n_row, out + a.out_slot[1]);
      }
    }
  };
  int odd = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += step, odd ^= 1, r_p += a.r.step, n_p += a.n.step) {
    cp_wait(stages);
    unsigned char *r_s = nullptr, *n_s = nullptr;
    if constexpr (COLS::kShared) {
      // The copies are in and the last row is done with: its stage and its outputs' rows.
      // Two sets of output rows: one is written while the other is put together.
      __syncthreads();
      unsigned char* out = ring + a.out_off + odd * a.out_bytes;
      r_s = out + a.out_slot[0], n_s = out + a.out_slot[1];
      if (m != blockIdx.x) flush(odd ^ 1, r_p - a.r.step, n_p - a.n.step);
    }
    put();
    const unsigned char* cur = ring_p + stage * a.stage_bytes;
    stage = stage + 1 == stages ? 0 : stage + 1;
    F8 r[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) r[v] = c.template staged<XT>(cur, a.x, m, v);
    if (has_y) {
      float factor = a.scale;  // residual scale and the row's 1 / rms
      if (post) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const F8 y = c.template staged<YT>(cur, a.y, m, v);
          const F2 q = dot8(y, y, f2(0.0f));
          ss[0] += c.in[v] ? lo(q) + hi(q) : 0.0f;
        }
        row_sum<1>(ss, T, red[odd][0]);
        factor *= rsqrtf(ss[0] * a.inv_h + a.eps);
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        F8 z = c.template staged<YT>(cur, a.y, m, v) * f2(factor);
        if (post) z = z * w_post(v);
        if (kind != E4B_GATE_NONE) {
          F8 f = kind == E4B_GATE_CHANNEL ? (kHold ? hold_gate : c.vector(a.vec_gate, a.gate_f32, v))
                 : kind == E4B_GATE_TOKEN ? fill8(load1(a.vec_gate, m, a.gate_f32))
                 : a.gate_f32             ? c.template staged<float>(cur, a.gate, m, v)
                                          : c.template staged<uint16_t>(cur, a.gate, m, v);
          if (a.sigmoid) f = sigmoid8(f);
          r[v] = fma8(z, f, r[v]);
        } else {
          r[v] = fma8(z, f2(1.0f), r[v]);
        }
        c.template store<XT>(r_p, r_s, v, r[v]);
      }
    }
    if (!next) continue;
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const F2 q = dot8(r[v], r[v], f2(0.0f));
      ss[0] += c.in[v] ? lo(q) + hi(q) : 0.0f;
    }
    row_sum<1>(ss, T, red[odd][1]);
    const F2 rstd = f2(rsqrtf(ss[0] * a.inv_h + a.eps));
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const F8 n = r[v] * rstd * w_next(v);
      if (a.n_f32)
        c.template store<float>(n_p, n_s, v, n);
      else
        c.template store<uint16_t>(n_p, n_s, v, n);
    }
  }
  if constexpr (COLS::kShared) {
    __syncthreads();
    flush(odd ^ 1, r_p - a.r.step, n_p - a.n.step);
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
  const bool all = a.y.p && a.w_next && a.w_post;
  return all ? launch_kernel(block_norm_forward_vec_kernel<XT, YT, VPT, COLS, true>, a, s, stream)
             : launch_kernel(block_norm_forward_vec_kernel<XT, YT, VPT, COLS, false>, a, s, stream);
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
  if (s.vpt == 4) return launch_kernel(block_norm_forward_kernel<XT, YT, 4, 512>, a, s, stream);
  if (s.vpt == 2) return launch_kernel(block_norm_forward_kernel<XT, YT, 2, 384>, a, s, stream);
  if (s.T == 64) return launch_kernel(block_norm_forward_kernel<XT, YT, 1, 64>, a, s, stream);
  if (s.T == 128) return launch_kernel(block_norm_forward_kernel<XT, YT, 1, 128>, a, s, stream);
  if (s.T == 256) return launch_kernel(block_norm_forward_kernel<XT, YT, 1, 256>, a, s, stream);
  return launch_kernel(block_norm_forward_kernel<XT, YT, 1, 384>, a, s, stream);
}

// out[q][col] = sum over parts of partial[q][part][col], in a fixed order: 32
// threads of a column take every 32nd part, then are added in order.
struct ReduceArgs {
  const float* partial;
  float* out[3];
  int parts, H;
};
constexpr int kRedCols = 32, kRedLanes = 32;

__global__ void __launch_bounds__(kRedCols * kRedLanes) block_norm_reduce_kernel(ReduceArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % kRedCols, row = threadIdx.x / kRedCols;
  const int blocks = (a.H + kRedCols - 1) / kRedCols, which = blockIdx.x / blocks, block = blockIdx.x % blocks;
  float* out = a.out[which];
  if (!out) return;
  __shared__ float s[kRedLanes][kRedCols];
  const int col = block * kRedCols + lane;
  float sum = 0.0f;
  if (col < a.H) {
    const float* p = a.partial + static_cast<int64_t>(which) * a.parts * a.H + col;
#pragma unroll 8
    for (int i = row; i < a.parts; i += kRedLanes) sum += p[static_cast<int64_t>(i) * a.H];
  }
  s[row][lane] = sum;
  __syncthreads();
  if (row == 0 && col < a.H) {
    for (int i = 1; i < kRedLanes; ++i) sum += s[i][lane];
    out[col] = sum;
  }
}

// A B200's SMs.  Not asked of the device: the workspace's size and the order of the sums over
// rows follow from the arguments alone.
constexpr int kSms = 148;

// Threads of a row, their groups, and the CTAs: as many as threads_per_sm gives each SM, which
// is what one group of columns a thread leaves room for.  With two and four groups the
// backward's registers (136 and 128 a thread) let fewer of them run at a time (at 4096 columns one of
// three, 144 us for 8192 rows in bf16), and the rest follow as these end.
NormShape norm_shape(int64_t M, int H, int threads_per_sm, bool vec) {
  const int nvec = (H + 7) / 8;
  NormShape s{};
  s.vpt = nvec <= norm_threads(1) ? 1 : nvec <= 2 * norm_threads(2) ? 2 : 4;
  s.T = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  if (!vec) s.T = s.vpt == 4 ? 512 : s.vpt == 2 || s.T > 256 ? 384 : s.T > 128 ? 256 : s.T > 64 ? 128 : 64;
  const int per_sm = std::min(16, std::max(1, threads_per_sm / s.T));
  s.grid = static_cast<int>(std::min<int64_t>(M, kSms * per_sm));
  return s;
}
constexpr int kForwardThreads = 900, kBackwardThreads = 768;  // per SM

// How a call's rows can be moved: as aligned vectors of 8 columns, as shifted ones, or
// else in units of 16 bytes.
struct Moves {
  bool vec, shift, units;
};

// The shape, and the ring: as many stages (2 to 4) as leave room for the SM's other
// CTAs, but two at least, even where an SM then holds fewer CTAs.  Where two stages do not fit
// (the backward of 8192 columns with fp32 x and y) rows are read by element from memory,
// without a ring: 4096 x 8192 1130 us, with bf16 y and a ring of vectors 284.
Moved plan(NormArgs* a, NormShape* s, const Moves& moves, bool x_f32, bool y_f32, int threads_per_sm) {
  constexpr uint32_t kRoom = 216 * 1024;
  for (const Moved moved : {kVector, kShifted, kElements}) {
    if ((moved == kVector && !moves.vec) || (moved == kShifted && !moves.shift)) continue;
    *s = norm_shape(a->M, a->H, threads_per_sm, moved != kElements);
    for (RowDst* d : {&a->r, &a->n, &a->dx, &a->dy}) d->step = d->row * s->grid;
    const uint32_t columns = s->T * s->vpt * 8;
    uint32_t off = 0;
    auto place = [&](RowSrc* r, bool f32) {
      if (!r->p) return;
      r->row = r->ld * (f32 ? 4 : 2);
      r->step = r->row * s->grid;
      r->off = off;
      // a shifted read reaches up to 32 bytes past its group
      off += moved == kElements ? static_cast<uint32_t>(align_up(static_cast<size_t>(a->H) * (f32 ? 4 : 2), 16) + 16)
                                : columns * (f32 ? 4 : 2) + (moved == kShifted ? 32 : 0);
    };
    place(&a->dr, x_f32);
    place(&a->x, x_f32);
    place(&a->dn, a->n_f32);
    place(&a->y, y_f32);
    place(&a->gate, a->gate_f32);
    a->stage_bytes = off;
    // Shifted outputs: rows with 16 bytes before and 32 behind them.
    uint32_t out = 0;
    auto slot = [&](int i, bool there, bool f32) {
      a->out_slot[i] = out + 16;
      if (there && moved == kShifted) out += columns * (f32 ? 4 : 2) + 48;
    };
    slot(0, a->r.p || a->dx.p, x_f32);
    slot(1, a->n.p || a->dy.p, a->n.p ? a->n_f32 : y_f32);
    slot(2, a->dgate && a->gate.p, a->gate_f32);
    a->out_bytes = out;
    const int ctas = std::min(16, std::max(1, threads_per_sm / s->T));
    const uint32_t each = kRoom / ctas;
    a->stages = static_cast<int>(std::max(2u, std::min(4u, each > 2 * out ? (each - 2 * out) / off : 0u)));
    a->out_off = a->stages * off;
    if ((moved != kElements || moves.units) && a->stages * off + 2 * out <= kRoom) return moved;
  }
  a->stages = 0;
  a->out_bytes = 0;
  return kElements;
}

int64_t size_of(int dtype) { return dtype == E4B_F32 ? 4 : 2; }
const char* const kForwardPath[] = {"block_norm.forward.scalar", "block_norm.forward.shifted", "block_norm.forward"};
const char* const kBackwardPath[] = {"block_norm.backward.scalar", "block_norm.backward.shifted", "block_norm.backward"};

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
  if (!y && !p->w_next && M > 0) return fail(E4B_ERR_INVALID_ARGUMENT, "nothing to compute: neither y nor w_next");
  return E4B_OK;
}

// One tensor of rows: its type, stride and alignment.
e4b_status check_rows(const char* name, const void* p, int dtype, int64_t ld, int64_t H, Moves* moves) {
  if (!p) return E4B_OK;
  if (!is_dtype(dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + "'s type must be F32 or BF16");
  if (ld < H) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + "'s leading dimension must be >= H");
  if (!on_element(p, dtype)) return fail(E4B_ERR_INVALID_ARGUMENT, std::string(name) + " must be aligned to its elements");
  moves->vec = moves->vec && vec_base(p, dtype) && ld % 8 == 0;
  moves->shift = moves->shift && aligned16(p);
  moves->units = moves->units && aligned16(p);
  return E4B_OK;
}

NormArgs norm_args(const e4b_block_norm* p, int64_t M, const void* y, int64_t ldy, const void* gate, e4b_gate_kind kind,
                   e4b_dtype gate_dtype, e4b_dtype n_dtype) {
  NormArgs a{};
  a.y = {y, ldy};
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

// What weights, gate and (backward) its gradient allow.
Moves moves_of(const e4b_block_norm* p, const void* gate, e4b_gate_kind kind, e4b_dtype gate_dtype, const void* dgate) {
  Moves m{};
  m.shift = vec_base(p->w_post, p->w_dtype) && vec_base(p->w_next, p->w_dtype);
  if (kind == E4B_GATE_CHANNEL) m.shift = m.shift && vec_base(gate, gate_dtype);
  m.vec = m.shift && p->H % 8 == 0;
  m.units = true;
  if (kind == E4B_GATE_FULL) {
    m.vec = m.vec && vec_base(gate, gate_dtype) && vec_base(dgate, gate_dtype);
    m.units = aligned16(gate);
    m.shift = m.shift && m.units;
  }
  return m;
}

}  // namespace

cudaError_t launch_block_norm_forward(const NormArgs& a, bool x_f32, bool y_f32, const NormShape& s, Moved moved,
                                      cudaStream_t stream) {
  if (x_f32) return y_f32 ? launch_typed<float, float>(a, s, moved, stream) : launch_typed<float, uint16_t>(a, s, moved, stream);
  return y_f32 ? launch_typed<uint16_t, float>(a, s, moved, stream) : launch_typed<uint16_t, uint16_t>(a, s, moved, stream);
}

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
  a.x = {x, ldx};
  a.r.p = r;
  a.r.row = ldr * size_of(x_dtype);
  a.n.p = n;
  a.n.row = ldn * size_of(n_dtype);
  NormShape s{};
  const bool x_f32 = x_dtype == E4B_F32, y_f32 = y && y_dtype == E4B_F32;
  const Moved moved = plan(&a, &s, moves, x_f32, y_f32, kForwardThreads);
  LaunchScope ls("block_norm.forward", st);
  if (cudaError_t err = launch_block_norm_forward(a, x_f32, y_f32, s, moved, st); err != cudaSuccess)
    return cuda_fail(err, "block norm forward launch");
  set_path(kForwardPath[moved]);
  return E4B_OK;
}

size_t e4b_block_norm_backward_workspace_size(int64_t M, const e4b_block_norm* norm) {
  if (!norm || M < 1 || norm->H < 1 || norm->H > kMaxNormH) return 0;
  // of the two ways to move rows, the one with more CTAs (fewer threads each)
  const int parts = std::max(norm_shape(M, static_cast<int>(norm->H), kBackwardThreads, true).grid,
                             norm_shape(M, static_cast<int>(norm->H), kBackwardThreads, false).grid);
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
  a.dr = {dr, lddr};
  a.dn = {dn, lddn};
  if (norm->w_next) a.x = {r, ldr};
  a.dx.p = dx;
  a.dx.row = lddx * size_of(x_dtype);
  a.dy.p = dy;
  a.dy.row = lddy * size_of(y_dtype);
  a.dgate = dgate;
  a.partial = static_cast<float*>(workspace);
  Moved moved = kElements;
  if (M > 0) {
    NormShape s{};
    const bool x_f32 = x_dtype == E4B_F32, y_f32 = y && y_dtype == E4B_F32;
    // the partial sums' rows are vectors of 32 bytes
    moves.vec = moves.vec && vec_base(workspace, E4B_F32);
    moved = plan(&a, &s, moves, x_f32, y_f32, kBackwardThreads);
    a.parts = s.grid;
    LaunchScope ls("block_norm.backward", st);
    if (cudaError_t err = launch_block_norm_backward(a, x_f32, y_f32, s, moved, st); err != cudaSuccess)
      return cuda_fail(err, "block norm backward launch");
  }
  float* dchannel = gate_kind == E4B_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  if (dw_post || dw_next || dchannel) {
    ReduceArgs ra{a.partial, {dw_post, dw_next, dchannel}, a.parts, a.H};
    LaunchScope ls("block_norm.reduce", st);
    if (cudaError_t err = launch_overlapped(block_norm_reduce_kernel, 3 * ((a.H + kRedCols - 1) / kRedCols), kRedCols * kRedLanes, 0,
                                            1, st, ra);
        err != cudaSuccess)
      return cuda_fail(err, "block norm reduce launch");
  }
  set_path(M == 0 ? "block_norm.backward.empty" : kBackwardPath[moved]);
  return E4B_OK;
}

}  // extern "C"
