// Kernels of the block norms (included by the forward's and the backward's
// translation units).
#pragma once

#include "async.cuh"
#include "common.cuh"
#include "e4b_internal.h"

namespace e4b {

constexpr int kMaxNormThreads = 512;

// A tensor of rows that a kernel reads: leading dimension in elements, place in a
// ring stage.
struct RowSrc {
  const void* p;
  int64_t ld;
  uint32_t off;
  int64_t row, step;  // bytes from a row to the next, and to the same CTA's next
};
// One that it writes.
struct RowDst {
  void* p;
  int64_t row, step;
};

struct NormArgs {
  RowSrc x, y, gate;                 // x: also r of the backward; gate: E4B_GATE_FULL's rows
  RowSrc dr, dn;                     // backward
  const void *vec_gate, *w_post, *w_next;  // vec_gate: channel or token gate
  RowDst r, n;                       // forward
  RowDst dx, dy;                     // backward
  void* dgate;
  float* partial;                    // backward: [3][parts][H] column sums (w_post, w_next, channel gate)
  int64_t M;
  int H, parts;
  int stages;                        // of the ring; 0: rows are read from memory directly
  uint32_t stage_bytes;
  uint32_t out_off, out_bytes;       // shifted rows: where the outputs' rows are put together, twice out_bytes
  uint32_t out_slot[3];
  int gate_kind, gate_f32, sigmoid, w_f32, n_f32;
  float scale, offset, eps, inv_h;
};

// Threads of a CTA and the groups of 8 columns that each takes.
struct NormShape {
  int T, vpt, grid;
};
// Most threads of a CTA, and CTAs an SM should hold, by the groups of a thread.
constexpr int norm_threads(int vpt) { return vpt == 4 ? 512 : 384; }

// How a call's rows are moved.  kVector: 8 columns of every row are aligned vectors.
// kShifted: rows start anywhere within 16 bytes, the tensors do not.  kElements: all else.
enum Moved { kElements = 0, kShifted = 1, kVector = 2 };

cudaError_t launch_block_norm_forward(const NormArgs& a, bool x_f32, bool y_f32, const NormShape& s, Moved moved,
                                      cudaStream_t stream);
cudaError_t launch_block_norm_backward(const NormArgs& a, bool x_f32, bool y_f32, const NormShape& s, Moved moved,
                                       cudaStream_t stream);

// ---- pairs of floats --------------------------------------------------------------
// Elementwise work on two columns per instruction (the packed fp32 forms of sm_100).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float lo(F2 a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
  return x;
}
__device__ __forceinline__ float hi(F2 a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
  return y;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Eight columns.
struct F8 {
  F2 p[4];
};
__device__ __forceinline__ F8 zero8() { return {{f2(0.0f), f2(0.0f), f2(0.0f), f2(0.0f)}}; }
__device__ __forceinline__ F8 fill8(float x) { return {{f2(x), f2(x), f2(x), f2(x)}}; }
__device__ __forceinline__ F8 operator*(const F8& a, const F8& b) {
  return {{a.p[0] * b.p[0], a.p[1] * b.p[1], a.p[2] * b.p[2], a.p[3] * b.p[3]}};
}
__device__ __forceinline__ F8 operator*(const F8& a, F2 b) { return {{a.p[0] * b, a.p[1] * b, a.p[2] * b, a.p[3] * b}}; }
__device__ __forceinline__ F8 operator+(const F8& a, F2 b) { return {{a.p[0] + b, a.p[1] + b, a.p[2] + b, a.p[3] + b}}; }
__device__ __forceinline__ F8 fma8(const F8& a, const F8& b, const F8& c) {
  return {{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]), fma2(a.p[2], b.p[2], c.p[2]), fma2(a.p[3], b.p[3], c.p[3])}};
}
__device__ __forceinline__ F8 fma8(const F8& a, F2 b, const F8& c) {
  return {{fma2(a.p[0], b, c.p[0]), fma2(a.p[1], b, c.p[1]), fma2(a.p[2], b, c.p[2]), fma2(a.p[3], b, c.p[3])}};
}
// s + a . b, column pairs apart
__device__ __forceinline__ F2 dot8(const F8& a, const F8& b, F2 s) {
  return fma2(a.p[3], b.p[3], fma2(a.p[2], b.p[2], fma2(a.p[1], b.p[1], fma2(a.p[0], b.p[0], s))));
}
__device__ __forceinline__ float get8(const F8& a, int j) { return j & 1 ? hi(a.p[j >> 1]) : lo(a.p[j >> 1]); }
__device__ __forceinline__ F8 set8(const float v[8]) { return {{f2(v[0], v[1]), f2(v[2], v[3]), f2(v[4], v[5]), f2(v[6], v[7])}}; }

// ---- memory ---------------------------------------------------------------------------
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = float_to_bf16_bits(v); }

__device__ __forceinline__ F8 unpack8(uint4 q) {
  return {{f2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u)),
           f2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u)),
           f2(__uint_as_float(q.z << 16), __uint_as_float(q.z & 0xffff0000u)),
           f2(__uint_as_float(q.w << 16), __uint_as_float(q.w & 0xffff0000u))}};
}
// A 32-byte load.  Coherent, and kept behind pdl_wait(): the launch ahead may have written the
// vector (a channel gate from a product) after this kernel's CTAs had started.
__device__ __forceinline__ F8 load8(const float* p) {
  float v[8];
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p)
               : "memory");
  return {{f2(v[0], v[1]), f2(v[2], v[3]), f2(v[4], v[5]), f2(v[6], v[7])}};
}
__device__ __forceinline__ F8 load8(const uint16_t* p) { return unpack8(*reinterpret_cast<const uint4*>(p)); }
// One 32-byte store: two of 16 bytes would each write half of every sector.
__device__ __forceinline__ void store8(float* p, const F8& v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(lo(v.p[0])), "f"(hi(v.p[0])),
               "f"(lo(v.p[1])), "f"(hi(v.p[1])), "f"(lo(v.p[2])), "f"(hi(v.p[2])), "f"(lo(v.p[3])), "f"(hi(v.p[3]))
               : "memory");
}
__device__ __forceinline__ void store8(uint16_t* p, const F8& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(lo(v.p[0]), hi(v.p[0])), pack_bf16x2(lo(v.p[1]), hi(v.p[1])),
                                            pack_bf16x2(lo(v.p[2]), hi(v.p[2])), pack_bf16x2(lo(v.p[3]), hi(v.p[3])));
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {  // the rest of the unit becomes zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Through L1: the two halves of a 32-byte sector are asked for by two instructions.
__device__ __forceinline__ void cp16_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

__device__ __forceinline__ float sigmoid_f32(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
__device__ __forceinline__ F8 sigmoid8(const F8& g) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = sigmoid_f32(get8(g, j));
  return set8(f);
}
__device__ __forceinline__ float load1(const void* p, int64_t i, int f32) {
  return f32 ? load1(static_cast<const float*>(p) + i) : load1(static_cast<const uint16_t*>(p) + i);
}
__device__ __forceinline__ void store1(void* p, int64_t i, int f32, float v) {
  if (f32)
    store1(static_cast<float*>(p) + i, v);
  else
    store1(static_cast<uint16_t*>(p) + i, v);
}

// ---- rows moved as vectors --------------------------------------------------------------
// A thread's share of a row: VPT groups of 8 adjacent columns, group v of thread
// t at column 8 (v T + t).  Groups past the row's end stand at column 0: they read
// what is there, are left out of sums over columns, and are not written.
template <int VPT>
struct VecCols {
  int T16;       // bytes of one plane of T 16-byte units
  int col[VPT];  // first column of each group
  bool in[VPT];
  __device__ __forceinline__ VecCols(int T, int t, int H) : T16(T * 16) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int at = (v * T + t) * 8;
      in[v] = at < H;
      col[v] = in[v] ? at : 0;
    }
  }
  static constexpr bool kShared = false;  // a thread reads its own places of the ring only
  __device__ __forceinline__ uint32_t place() const { return threadIdx.x * 16; }
  // Into this thread's places of a ring stage (`dst`: its unit of plane 0) from a
  // row: 8 bf16 are one unit, 8 floats two, in two planes.
  template <class E>
  __device__ __forceinline__ void fetch(uint32_t dst, const unsigned char* row, const RowSrc&, int64_t) const {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const E* src = reinterpret_cast<const E*>(row) + col[v];
      if constexpr (sizeof(E) == 2) {
        cp16(dst + v * T16, src);
      } else {
        cp16_l1(dst + v * T16, src);
        cp16_l1(dst + (VPT + v) * T16, src + 4);
      }
    }
  }
  template <class E>
  __device__ __forceinline__ F8 staged(const unsigned char* stage, const RowSrc& s, int64_t, int v) const {
    const unsigned char* src = stage + s.off;
    const uint4 q = *reinterpret_cast<const uint4*>(src + v * T16);
    if constexpr (sizeof(E) == 2) return unpack8(q);
    const uint4 u = *reinterpret_cast<const uint4*>(src + (VPT + v) * T16);
    return {{f2(__uint_as_float(q.x), __uint_as_float(q.y)), f2(__uint_as_float(q.z), __uint_as_float(q.w)),
             f2(__uint_as_float(u.x), __uint_as_float(u.y)), f2(__uint_as_float(u.z), __uint_as_float(u.w))}};
  }
  // A vector over the columns (a weight, a channel gate): held in L1.
  __device__ __forceinline__ F8 vector(const void* p, int f32, int v) const {
    return f32 ? load8(static_cast<const float*>(p) + col[v]) : load8(static_cast<const uint16_t*>(p) + col[v]);
  }
  template <class E>
  __device__ __forceinline__ void store(unsigned char* row, unsigned char*, int v, const F8& f) const {
    if (in[v]) store8(reinterpret_cast<E*>(row) + col[v], f);
  }
  template <class E>
  __device__ __forceinline__ void sums(E* row, int v, const F8& f) const {
    if (in[v]) store8(row + col[v], f);
  }
};

// ---- rows that start anywhere within 16 bytes ----------------------------------------------
// The 16 bytes that start `by` (even, 0 .. 14) bytes after the 16-byte aligned p.
__device__ __forceinline__ uint4 raw16(const unsigned char* p, uint32_t by) {
  const uint2* q = reinterpret_cast<const uint2*>(p + (by & 8));
  const uint2 a = q[0], b = q[1], c = q[2];
  const bool s = by & 4;
  const uint32_t v0 = s ? a.y : a.x, v1 = s ? b.x : a.y, v2 = s ? b.y : b.x, v3 = s ? c.x : b.y, v4 = s ? c.y : c.x;
  const uint32_t h = (by & 2) * 8;
  return make_uint4(__funnelshift_r(v0, v1, h), __funnelshift_r(v1, v2, h), __funnelshift_r(v2, v3, h), __funnelshift_r(v3, v4, h));
}

// The same groups of 8 columns as VecCols, of rows whose first byte lies anywhere in a
// 16-byte unit.  A row comes into the ring as the units that it touches and is
// read across threads, shifted; an output row is put together in shared memory and
// written in the units of its own place one row later, its first and last
// units by element.  The last group of a row may be a part: its columns past H are zero.
template <int VPT>
struct ShiftCols {
  int T, H;
  int col[VPT], count[VPT];  // first column of each group, its columns (0 .. 8)
  bool in[VPT];
  static constexpr bool kShared = true;
  __device__ __forceinline__ ShiftCols(int T_, int t, int H_) : T(T_), H(H_) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      col[v] = (v * T + t) * 8;
      count[v] = max(0, min(8, H - col[v]));
      in[v] = count[v] > 0;
    }
  }
  __device__ __forceinline__ uint32_t place() const { return 0; }
  static __device__ __forceinline__ uint32_t lead_of(const void* row) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u; }
  __device__ __forceinline__ F8 cut(F8 f, int v) const {
    if (count[v] < 8) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f.p[q] = f2(2 * q < count[v] ? lo(f.p[q]) : 0.0f, 2 * q + 1 < count[v] ? hi(f.p[q]) : 0.0f);
    }
    return f;
  }
  // `last`: rows behind this one.  Nothing past the tensor's end is read.
  template <class E>
  __device__ __forceinline__ void fetch(uint32_t dst, const unsigned char* row, const RowSrc& s, int64_t last) const {
    const uint32_t lead = lead_of(row);
    const int bytes = static_cast<int>(lead) + H * static_cast<int>(sizeof(E));
    const unsigned char* src = row - lead;
    const int64_t left = last * s.row + bytes;  // to the tensor's end
    const int safe = left >= bytes + 15 ? bytes + 15 : static_cast<int>(left);
    for (int u = threadIdx.x * 16; u < bytes; u += T * 16) cp16(dst + u, src + u, min(16, safe - u));
  }
  template <class E>
  __device__ __forceinline__ F8 staged(const unsigned char* stage, const RowSrc& s, int64_t m, int v) const {
    const uint32_t lead = (lead_of(s.p) + static_cast<uint32_t>(m) * static_cast<uint32_t>(s.row)) & 15u;
    const unsigned char* src = stage + s.off + col[v] * static_cast<int>(sizeof(E));
    const uint4 q = raw16(src, lead);
    if constexpr (sizeof(E) == 2) return cut(unpack8(q), v);
    const uint4 u = raw16(src + 16, lead);
    return cut({{f2(__uint_as_float(q.x), __uint_as_float(q.y)), f2(__uint_as_float(q.z), __uint_as_float(q.w)),
                 f2(__uint_as_float(u.x), __uint_as_float(u.y)), f2(__uint_as_float(u.z), __uint_as_float(u.w))}}, v);
  }
  __device__ __forceinline__ F8 vector(const void* p, int f32, int v) const {
    if (count[v] == 8)
      return f32 ? load8(static_cast<const float*>(p) + col[v]) : load8(static_cast<const uint16_t*>(p) + col[v]);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < count[v] ? load1(p, col[v] + j, f32) : 0.0f;
    return set8(f);
  }
  // Into the row being put together at `slot`.
  template <class E>
  __device__ __forceinline__ void store(unsigned char*, unsigned char* slot, int v, const F8& f) const {
    if (!in[v]) return;
    uint4* to = reinterpret_cast<uint4*>(slot + col[v] * static_cast<int>(sizeof(E)));
    if constexpr (sizeof(E) == 2) {
      *to = make_uint4(pack_bf16x2(lo(f.p[0]), hi(f.p[0])), pack_bf16x2(lo(f.p[1]), hi(f.p[1])),
                       pack_bf16x2(lo(f.p[2]), hi(f.p[2])), pack_bf16x2(lo(f.p[3]), hi(f.p[3])));
    } else {
      to[0] = make_uint4(__float_as_uint(lo(f.p[0])), __float_as_uint(hi(f.p[0])), __float_as_uint(lo(f.p[1])), __float_as_uint(hi(f.p[1])));
      to[1] = make_uint4(__float_as_uint(lo(f.p[2])), __float_as_uint(hi(f.p[2])), __float_as_uint(lo(f.p[3])), __float_as_uint(hi(f.p[3])));
    }
  }
  // The row put together at `slot` to its place in memory.
  template <class E>
  __device__ __forceinline__ void flush(unsigned char* row, const unsigned char* slot) const {
    const uint32_t lead = lead_of(row);
    const int bytes = static_cast<int>(lead) + H * static_cast<int>(sizeof(E));
    const uint32_t by = (16u - lead) & 15u;
    for (int u = threadIdx.x * 16; u < bytes; u += T * 16) {
      if (u >= static_cast<int>(lead) && u + 16 <= bytes) {
        *reinterpret_cast<uint4*>(row - lead + u) = raw16(slot + u - (lead ? 16 : 0), by);
      } else {
        for (int b = max(u, static_cast<int>(lead)); b < min(u + 16, bytes); b += sizeof(E))
          *reinterpret_cast<E*>(row - lead + b) = *reinterpret_cast<const E*>(slot + b - lead);
      }
    }
  }
  template <class E>
  __device__ __forceinline__ void sums(E* row, int v, const F8& f) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count[v]) row[col[v] + j] = get8(f, j);
  }
};

// ---- other rows -----------------------------------------------------------------------------
// Columns j T + t, j < 8 VPT, of thread t, so that a warp's accesses are adjacent; a
// group v is its columns j = 8 v .. 8 v + 7.  Columns past H read as zero and
// are not written.  T is known at compile time: an element then costs its
// load and little else (the addresses differ by constants).
template <int VPT, int T>
struct Cols {
  int t, H;
  __device__ __forceinline__ int col(int v, int j) const { return (v * 8 + j) * T + t; }
  // Whether any thread has columns 2 q and 2 q + 1 of group v (uniform).
  __device__ __forceinline__ bool any(int v, int q) const { return (v * 8 + 2 * q) * T < H; }
  template <class E, class At>
  __device__ __forceinline__ F8 gather(int v, At at) const {
    F8 f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x = 0.0f, y = 0.0f;
      if (any(v, q)) {
        if (col(v, 2 * q) < H) x = at((v * 8 + 2 * q) * T);
        if (col(v, 2 * q + 1) < H) y = at((v * 8 + 2 * q + 1) * T);
      }
      f.p[q] = f2(x, y);
    }
    return f;
  }
  template <class E>
  __device__ __forceinline__ F8 load(const E* row, int v) const {
    const E* p = row + t;
    return gather<E>(v, [&](int i) { return load1(p + i); });
  }
  template <class E>
  __device__ __forceinline__ void store(E* row, int v, const F8& f) const {
    E* p = row + t;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!any(v, q)) break;
      if (col(v, 2 * q) < H) store1(p + (v * 8 + 2 * q) * T, lo(f.p[q]));
      if (col(v, 2 * q + 1) < H) store1(p + (v * 8 + 2 * q + 1) * T, hi(f.p[q]));
    }
  }
  // The element type known at run time only (uniform over the launch).
  __device__ __forceinline__ F8 load(const void* row, int f32, int v) const {
    return f32 ? load(static_cast<const float*>(row), v) : load(static_cast<const uint16_t*>(row), v);
  }
  __device__ __forceinline__ void store(void* base, int64_t off, int f32, int v, const F8& f) const {
    if (f32)
      store(static_cast<float*>(base) + off, v, f);
    else
      store(static_cast<uint16_t*>(base) + off, v, f);
  }
  // Row m of `s` into its place in `stage`: the 16-byte units that the row
  // touches.  Its neighbours' ends come along, but nothing past the last row's end.
  template <class E>
  __device__ __forceinline__ void fetch(unsigned char* stage, const RowSrc& s, int64_t m, int64_t M) const {
    const uintptr_t at = reinterpret_cast<uintptr_t>(s.p) + m * s.row, lead = at & 15;
    const int bytes = static_cast<int>(lead) + H * static_cast<int>(sizeof(E));
    const uint32_t dst = smem_addr(stage + s.off);
    const char* src = reinterpret_cast<const char*>(at - lead);
    // the units of other rows end inside the tensor; the last few rows' may not
    const bool inside = at - lead + ((bytes + 15) & ~15) <= reinterpret_cast<uintptr_t>(s.p) + (M - 1) * s.row + H * sizeof(E);
    if (inside) {
      for (int u = t * 16; u < bytes; u += T * 16) cp16(dst + u, src + u);
    } else {
      const int64_t left = static_cast<int64_t>(reinterpret_cast<uintptr_t>(s.p) + (M - 1) * s.row + H * sizeof(E) - (at - lead));
      for (int u = t * 16; u < bytes; u += T * 16) cp16(dst + u, src + u, left - u < 16 ? static_cast<int>(left - u) : 16);
    }
  }
  // Group v of row m, from the stage that fetch() filled.
  template <class E>
  __device__ __forceinline__ F8 staged(const unsigned char* stage, const RowSrc& s, int64_t m, int v) const {
    const uint32_t lead = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s.p)) + static_cast<uint32_t>(m * s.row)) & 15u;
    const E* p = reinterpret_cast<const E*>(stage + s.off + lead) + t;
    return gather<E>(v, [&](int i) { return load1(p + i); });
  }
};

// The rows of a CTA, one after another, from a ring, or from memory where they are too
// long for it or their bases are not 16-byte aligned.
template <class XT, class YT, int VPT, int T, bool BWD>
struct Rows {
  const NormArgs& a;
  const Cols<VPT, T>& c;
  unsigned char* ring;
  unsigned char* cur;
  int put_stage = 0, stage = 0;
  int64_t put_row;

  __device__ __forceinline__ Rows(const NormArgs& a_, const Cols<VPT, T>& c_, unsigned char* ring_)
      : a(a_), c(c_), ring(ring_), cur(ring_), put_row(blockIdx.x) {
    for (int i = 0; i + 1 < a.stages; ++i) put();
  }
  __device__ __forceinline__ void put() {
    if (put_row < a.M) {
      unsigned char* to = ring + put_stage * a.stage_bytes;
      if (!BWD || a.w_next) c.template fetch<XT>(to, a.x, put_row, a.M);
      if (a.y.p) c.template fetch<YT>(to, a.y, put_row, a.M);
      if constexpr (BWD) {
        if (a.dr.p) c.template fetch<XT>(to, a.dr, put_row, a.M);
        if (a.w_next) a.n_f32 ? c.template fetch<float>(to, a.dn, put_row, a.M) : c.template fetch<uint16_t>(to, a.dn, put_row, a.M);
      }
      if (a.gate.p) a.gate_f32 ? c.template fetch<float>(to, a.gate, put_row, a.M) : c.template fetch<uint16_t>(to, a.gate, put_row, a.M);
      put_row += gridDim.x;
    }
    cp_commit();
    put_stage = put_stage + 1 == a.stages ? 0 : put_stage + 1;
  }
  // Makes the next row readable and sets off the row `stages - 1` further on, into
  // the stage of the last row, which all threads have left behind at the barrier.
  __device__ __forceinline__ void next() {
    if (!a.stages) return;
    cp_wait(a.stages);
    __syncthreads();
    put();
    cur = ring + stage * a.stage_bytes;
    stage = stage + 1 == a.stages ? 0 : stage + 1;
  }
  template <class E>
  __device__ __forceinline__ F8 load(const RowSrc& s, int64_t m, int v) const {
    if (a.stages) return c.template staged<E>(cur, s, m, v);
    return c.load(static_cast<const E*>(s.p) + m * s.ld, v);
  }
  __device__ __forceinline__ F8 load(const RowSrc& s, int64_t m, int f32, int v) const {
    return f32 ? load<float>(s, m, v) : load<uint16_t>(s, m, v);
  }
  // The gate of a group of columns (before any sigmoid).
  __device__ __forceinline__ F8 gate(int64_t m, int v) const {
    if (a.gate_kind == E4B_GATE_FULL) return load(a.gate, m, a.gate_f32, v);
    if (a.gate_kind == E4B_GATE_CHANNEL) return c.load(a.vec_gate, a.gate_f32, v);
    return fill8(load1(a.vec_gate, m, a.gate_f32));
  }
};

// Sums of one, two, three or six values over the CTA's T threads (a multiple of 32, at most
// 512), to every thread.  Several values share the shuffles: a warp's halves (or
// quarters, eighths) first exchange the values that each will add up (11 shuffles
// for two, 12 for three and 16 for six instead of 18, 27 and 54).  One barrier above one warp:
// a caller that sums again passes another buffer of 64 floats (128 for six).
__device__ __forceinline__ float add_xor(float v, int o) { return v + __shfl_xor_sync(0xffffffffu, v, o); }

template <int NV>
__device__ __forceinline__ void row_sum(float v[NV], int T, float* red) {
  const int lane = threadIdx.x & 31, warps = T >> 5, warp = threadIdx.x >> 5;
  if constexpr (NV == 1) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[0] = add_xor(v[0], o);
    if (T == 32) return;
    if (lane == 0) red[warp] = v[0];
    __syncthreads();
    v[0] = (lane & 15) < warps ? red[lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v[0] = add_xor(v[0], o);
  } else if constexpr (NV == 2) {
    // lanes 0-15 add up value 0, lanes 16-31 value 1
    const bool up = lane & 16;
    float s = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s = add_xor(s, o);
    if (T > 32) {
      if ((lane & 15) == 0) red[(lane >> 4) * 16 + warp] = s;
      __syncthreads();
      s = (lane & 15) < warps ? red[lane] : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s = add_xor(s, o);
    }
    v[0] = __shfl_sync(0xffffffffu, s, 0);
    v[1] = __shfl_sync(0xffffffffu, s, 16);
  } else if constexpr (NV == 6) {
    // lanes 4 i .. 4 i + 3 add up value 0, 1, 2, none, 3, 4, 5, none
    const bool up = lane & 16, mid = lane & 8, odd = lane & 4;
    float t[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) t[i] = (up ? v[i + 3] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 3], 16);
    const float t0 = (mid ? t[2] : t[0]) + __shfl_xor_sync(0xffffffffu, mid ? t[0] : t[2], 8);
    const float t1 = (mid ? 0.0f : t[1]) + __shfl_xor_sync(0xffffffffu, mid ? t[1] : 0.0f, 8);
    float s = (odd ? t1 : t0) + __shfl_xor_sync(0xffffffffu, odd ? t0 : t1, 4);
    s = add_xor(add_xor(s, 2), 1);
    if (T > 32) {
      const int place = (lane >> 2) * 16;
      if ((lane & 3) == 0) red[place + warp] = s;
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int w = (lane & 3) + 4 * j;
        s += w < warps ? red[place + w] : 0.0f;
      }
      s = add_xor(add_xor(s, 2), 1);
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, s, 4 * (i + i / 3));
  } else {
    // lanes 8 i .. 8 i + 7 add up value i (the fourth is none)
    const bool up = lane & 16, odd = lane & 8;
    const float s0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
    const float s1 = (up ? 0.0f : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : 0.0f, 16);
    float s = (odd ? s1 : s0) + __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s = add_xor(s, o);
    if (T > 32) {
      if ((lane & 7) == 0) red[(lane >> 3) * 16 + warp] = s;
      __syncthreads();
      const int w = lane & 7, i = (lane >> 3) * 16;
      s = (w < warps ? red[i + w] : 0.0f) + (w + 8 < warps ? red[i + w + 8] : 0.0f);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s = add_xor(s, o);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = __shfl_sync(0xffffffffu, s, 8 * i);
  }
}

}  // namespace e4b
