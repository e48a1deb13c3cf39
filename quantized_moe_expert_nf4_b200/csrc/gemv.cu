// Products of a few rows (1 to 16 tokens) with a dense weight matrix [N, K]:
// 4-bit codes with group scales, or bf16.
//
//   y[m, n] = sum over groups g of  s[n, g] * sum_{k in g} x[m, k] * v[n, k]
//   v = codebook[code] (NF4, FP4), code - zero[n, g] (int4), or the bf16 weight (s = 1)
//
// Bound: HBM at large N * K (each weight is read once), launch and memory
// latency at small.  A warp takes 16 weight rows as the rows of an m16n8k16 MMA
// and the tokens as its 8 columns (two column sets above 8 tokens); K is cut
// into chunks of 128 bytes of a row.  The warps of a CTA are KW-way split over
// the chunks and cover 16 * (8 / KW) rows; clusters of CTAs split K further
// where the rows alone cannot fill the GPU.  Each warp streams its 16 x 128-byte
// pieces through its own ring of cp.async stages, so no warp waits for
// another until the partial sums meet; pieces of the next rows are in flight
// while a CTA adds up the last ones.
//
// Within a block of 32 k, lane (g, t) of the MMA takes k = 8 t .. 8 t + 7 of rows g
// and g + 8 (one word of codes each) and of token g: the same permutation of k on
// both operands.  The pieces lie in shared memory with their 16-byte units
// exchanged by row, so that those reads touch every bank once.
//
// Codes become exact bf16 values: int4 by or-ing the code into the mantissa of
// 128 and subtracting 128 + zero, both exact; codebook entries by a table of byte pairs in
// shared memory.  Products and group sums are fp32 in the MMA, the scales
// multiply the group sums in fp32.  A codebook is taken times a factor, and the scales
// over it, at which its entries fall nearer to bf16 values: 6 for FP4 (e2m1 values,
// exact), 1.43672 for NF4 (of all factors the one with the least error over the codes
// of Gaussian weights in blocks of 64: 0.78e-3 of the weights' rms instead of
// 1.36e-3, and 1.7e-3 of an entry at most instead of 3.1e-3).  With bf16 output that
// is all: the rounding stays below the output's.  With fp32 output an NF4 entry is the sum
// of two bf16 values of one sign, times 1.4376 (of all factors the one with the least
// error of such pairs: 2^-18.8 of an entry at most).
//
// Measured on the device (graph replays, three sets of tensors in turn; the last
// call's leave L2 in between, the others' stay):
//   1 x 2048 x 2048 int4, blocks of 32, zero points    3.4 us (0.4 at the copy bandwidth)
//   1 x 2880 x 5760 NF4, SwiGLU                        6.7 us (1.4): the tables' build, then
//                                                      two or three chunks a warp
//   13 x 2880 x 16411 FP4, blocks of 32               19.1 us (4.1)
//   8 x 4096 x 32768 int4, blocks of 128, fp32 out    23.5 us (10.7): 3.0 TB/s
//   1 x 4096 x 14336 int4, blocks of 128              13.2 us (4.6)
//   8 x 4096 x 32768 NF4, blocks of 64, fp32 out      42 us (11.0): two tables
// The large ones wait more than they issue, at four warps a scheduler: the last int4 call of 8
// tokens has its issue slots 52% busy.  Codes and products take 32 (int4) to 59 (table)
// cycles for 16 rows x 32 k and scheduler, 16 more for a second set of tokens: 6 of the FP4 call's 19 us.
// A chunk's tokens (4 KB for 8, 8 KB for 16, beside 2 KB of codes a row tile) are loaded at its
// head and used at once.  A copy of the kernel without 7 of 8 products took 15.5 us for the
// int4 call, one without the copies 22.8.  Measured and not kept for it: x in shared
// memory and 16 to 32 warps (26.6), a warp for the sums alone (39), all of K
// by one warp (31.9: 128-byte pieces of 2 KB rows use DRAM pages badly), x read
// again by every block (35), (chunk, row tile) items in equal runs with all sums
// in shared memory (25.7), rows shared out evenly to the last row tile (24.0).
#include <cooperative_groups.h>

#include <algorithm>

#include "async.cuh"
#include "common.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;

enum Fmt { kFmtCodebook = 0, kFmtInt4 = 1, kFmtBf16 = 2 };

struct Params {
  GemvArgs a;
  int chunks;     // ceil(row bytes / 128)
  int kw;         // warps that share a row tile
  int split;      // CTAs of a cluster that share a row tile
  int tiles;      // CTA tiles of 16 RT * (8 / kw) rows
  float book, over_book;  // the codebook's factor, and what the scales take of it
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int bytes = in ? 16 : 0;  // 0: writes zeros, reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// As mma16816, from zero.
__device__ __forceinline__ void mma16816_first(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// 16-byte unit `u` (0..7) of row `row` of a piece lies at unit u ^ swz(row): eight
// rows give eight places for one unit, and two adjacent rows' four units do not meet.
__device__ __forceinline__ uint32_t swz(int row) { return ((row & 1) << 2) | ((row >> 1) & 3); }

// Eight codebook codes (byte i: element 2i in the high nibble) -> four bf16 pairs in
// element order, one table lookup per byte.  The table holds each byte's pair once
// per lane (entry b of lane l at byte 128 b + 4 l), so lookups never share a
// bank; `lane_table` is the table's shared address + 4 l, its low 15 bits 4 l.
// Two integer instructions and one shared load per pair instead of byte permutes
// over the codebook in registers (21 integer instructions per word, on a pipe of half
// the issue rate): 13 x 2880 x 16411 FP4 21.2 us from 29.7, the scales' earlier
// loads included.
__device__ __forceinline__ void decode_table(uint32_t w, const unsigned char* lane_table, uint32_t v[4]) {
  v[0] = *reinterpret_cast<const uint32_t*>(lane_table + ((w << 7) & 0x7f80u));
  v[1] = *reinterpret_cast<const uint32_t*>(lane_table + ((w >> 1) & 0x7f80u));
  v[2] = *reinterpret_cast<const uint32_t*>(lane_table + ((w >> 9) & 0x7f80u));
  v[3] = *reinterpret_cast<const uint32_t*>(lane_table + ((w >> 17) & 0x7f80u));
}

// Eight int4 codes -> bf16 pairs of elements (1, 5), (0, 4), (3, 7), (2, 6), each
// 128 + code - (128 + zero); `zz` is bf16(128 + zero) in both halves.
struct Int4Bits {
  uint32_t mask, exponent;
};
__device__ __forceinline__ Int4Bits int4_bits() {
  Int4Bits k;
  asm volatile("mov.b32 %0, 0x000f000f;\n\tmov.b32 %1, 0x43004300;" : "=r"(k.mask), "=r"(k.exponent));
  return k;
}
__device__ __forceinline__ void decode_int4(uint32_t w, uint32_t zz, const Int4Bits& k, uint32_t v[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t q;  // (w >> 4 i) & 0x000f000f | 0x43004300: one instruction once the constants sit in registers
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(q) : "r"(w >> (4 * i)), "r"(k.mask), "r"(k.exponent));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(q), "r"(zz));
  }
}

// FMT: weight format; GB: blocks of 32 k in a group; NT: sets of 8 tokens; RT: row
// tiles of 16 per warp; TWO: codebook entries as two bf16 values.
template <int FMT, int GB, int NT, int RT, bool TWO>
struct Cfg {
  static constexpr int kBlocks = FMT == kFmtBf16 ? 2 : 8;   // blocks of 32 k in a chunk
  static constexpr int kChunkK = kBlocks * 32;
  static constexpr int kGroups = FMT == kFmtBf16 ? 1 : kBlocks / GB;  // groups in a chunk
  static constexpr uint32_t kPiece = RT * 16 * 128;
  // Pieces in flight per warp: 64 KB per CTA, 32 beside two tables.
  static constexpr int kStages = TWO ? 2 : 4 / RT;
  static constexpr uint32_t kTable = FMT == kFmtCodebook ? 256 * 128 : 0;
  static constexpr uint32_t kTables = kTable * (TWO ? 2 : 1);
  static constexpr uint32_t kSmem = kTables + kWarps * kStages * kPiece;
  static constexpr uint32_t kSums = 2 * kWarps * RT * NT * 32 * 16;  // `red`
  // launch_gemv() counts on two CTAs an SM (228 KB, of which each CTA costs 1 more).
  static_assert(2 * (kSmem + kSums + 1024) <= 228 * 1024, "two CTAs fit an SM");
};

template <int FMT, int GB, int NT, int RT, bool TWO>
__global__ void __launch_bounds__(kWarps * 32, 2) gemv_kernel(const __grid_constant__ Params p) {
  using C = Cfg<FMT, GB, NT, RT, TWO>;
  constexpr int NB = C::kBlocks, NG = C::kGroups, KS = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float4 red[2][kWarps][RT][NT][32];
  const GemvArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int kw = p.kw, wk = warp % kw, wr = warp / kw;  // this warp's share of K, its row tiles of the CTA's
  const int rank = p.split > 1 ? static_cast<int>(blockIdx.x % p.split) : 0;
  const int cta = p.split > 1 ? static_cast<int>(blockIdx.x / p.split) : static_cast<int>(blockIdx.x);
  const int ctas = static_cast<int>(gridDim.x) / p.split;
  const int first = rank * kw + wk, stride = kw * p.split;  // chunks first, first + stride, ...
  const bool glu = a.epi != kGemvNone;
  const int half = a.N / 2;
  const int rows_out = glu ? 8 : 16;         // output columns of a row tile of 16 weight rows
  const int nout = glu ? half : a.N;
  const int warp_out = rows_out * RT, tile_out = warp_out * (kWarps / kw);
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t ring = base + C::kTables + warp * KS * C::kPiece;
  const unsigned char* ring_p = smem + C::kTables + warp * KS * C::kPiece;

  // Row tile j of a tile: MMA rows 0..15 are weight rows o .. o + 15, or the gate
  // rows o .. o + 7 and the up rows half + o .. half + o + 7 of a gated product.
  // Rows past the end read zeros, and are not written.

  const unsigned char* lane_table = smem + lane * 4;
  const Int4Bits bits = int4_bits();
  if constexpr (FMT == kFmtCodebook) {
    // Entry b: the pair of codes (b / 16, b % 16); thread b writes its 32 copies.
    static_assert(kWarps * 32 == 256, "a thread per entry");
    const float hi = p.book * codebook_entry(a.quant, threadIdx.x >> 4), lo = p.book * codebook_entry(a.quant, threadIdx.x & 15);
    // The first of two values is cut, not rounded: the second then has its sign, and an
    // infinite x keeps its own (inf * first + inf * second).
    const uint32_t pair = TWO ? __byte_perm(__float_as_uint(hi), __float_as_uint(lo), 0x7632u) : pack_bf16x2(hi, lo);
    const uint32_t rest = pack_bf16x2(hi - __uint_as_float(pair << 16), lo - __uint_as_float(pair & 0xffff0000u));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = (i + threadIdx.x) & 7;  // spread over the banks
      reinterpret_cast<uint4*>(smem + threadIdx.x * 128)[q] = make_uint4(pair, pair, pair, pair);
      if constexpr (TWO)
        reinterpret_cast<uint4*>(smem + C::kTable + threadIdx.x * 128)[q] = make_uint4(rest, rest, rest, rest);
    }
    __syncthreads();
  }

  // x alone may come from the launch ahead (after_input), which has seen all before it end.
  if (!a.after_input) {
    pdl_wait();
    pdl_launch_dependents();
  }

  // This warp's pieces, in order: every chunk of its share, tile after tile.
  // Lane l copies the 16-byte unit l % 8 of rows l / 8 + 4 i.
  int put_tile = cta, put_chunk = first, put_stage = 0, put_o = 0;
  const unsigned char* put_p = nullptr;
  const int64_t rb4 = a.row_bytes * 4, rb_up = static_cast<int64_t>(half) * a.row_bytes;
  // Place of this lane's unit in rows lane / 8 and, 2 units over, lane / 8 + 4.
  const uint32_t put_dst = (lane >> 3) * 128 + (((lane & 7) ^ swz(lane >> 3)) << 4);
  bool put_whole = false;  // every row of the tile exists
  auto put_rows = [&]() {
    put_o = put_tile * tile_out + wr * warp_out;
    put_whole = put_o + warp_out <= nout;
    put_o += lane >> 3;
    put_p = static_cast<const unsigned char*>(a.w) + put_o * a.row_bytes + (lane & 7) * 16;
  };
  auto put = [&]() {
    if (put_tile < p.tiles && first < p.chunks) {
      const uint32_t dst = ring + put_stage * C::kPiece;
      const unsigned char* src0 = put_p + static_cast<int64_t>(put_chunk) * 128;
      auto src_of = [&](int i) { return src0 + (glu ? (i >> 2) * 2 + (i & 1) : i) * rb4 + (glu && (i & 2) ? rb_up : 0); };
      auto dst_of = [&](int i) { return dst + (put_dst ^ ((i & 1) << 5)) + i * 512; };
      if (put_whole && (put_chunk + 1) * 128ll <= a.row_bytes) {
#pragma unroll
        for (int i = 0; i < 4 * RT; ++i) cp_async16(dst_of(i), src_of(i));
      } else {
        const bool in_k = put_chunk * 128ll + (lane & 7) * 16 < a.row_bytes;
#pragma unroll
        for (int i = 0; i < 4 * RT; ++i) {
          const bool in = in_k && put_o + (glu ? (i >> 2) * 2 + (i & 1) : i) * 4 < nout;
          cp_async16(dst_of(i), in ? src_of(i) : a.w, in);
        }
      }
      put_chunk += stride;
      if (put_chunk >= p.chunks) {
        put_chunk = first;
        put_tile += ctas;
        put_rows();
      }
    }
    cp_async_commit();
    put_stage = put_stage + 1 == KS ? 0 : put_stage + 1;
  };
  put_rows();
#pragma unroll
  for (int s = 0; s < KS - 1; ++s) put();

  // Scales (and zero points) of a chunk's NG groups, rows g and g + 8: lane t of the
  // row's four keeps SPL of them and hands them over by shuffles, so that a
  // chunk's can be loaded while the one before it is multiplied.
  constexpr int SPL = NG > 4 ? NG / 4 : 1;
  uint32_t ns[RT][2][SPL];  // as loaded: converted by their own chunk, which alone waits for them
  uint32_t nz[RT][2][SPL] = {};
  int64_t s_row[RT][2];
  auto scale_rows = [&](int tile) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = tile * tile_out + wr * warp_out + j * rows_out + g + (glu ? 0 : 8 * h);
        s_row[j][h] = o < nout ? static_cast<int64_t>(glu && h ? half + o : o) * a.groups : 0;
      }
  };
  auto load_scales = [&](int chunk) {
    if constexpr (FMT != kFmtBf16) {
#pragma unroll
      for (int i = 0; i < SPL; ++i) {
        const int grp = chunk * NG + (t % (NG / SPL)) * SPL + i;
        const bool in = grp < a.groups;  // zero past K
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t at = s_row[j][h] + (in ? grp : 0);
            ns[j][h][i] = 0;
            if (in) ns[j][h][i] = a.scale_f32 ? static_cast<const uint32_t*>(a.scales)[at] : static_cast<const uint16_t*>(a.scales)[at];
            if constexpr (FMT == kFmtInt4)
              if (a.zeros) nz[j][h][i] = a.zeros[at];
          }
      }
    }
  };
  scale_rows(cta < p.tiles ? cta : 0);
  load_scales(first);

  uint32_t x[NT][NB][4];
  int x_chunk = -1;
  // Columns past the last token repeat it: their products are not written.
  const uint16_t* x_lane[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) x_lane[n] = a.x + min(n * 8 + g, a.M - 1) * a.ldx + t * 8;
  auto load_x = [&](int chunk) {
    x_chunk = chunk;
    const int k = chunk * C::kChunkK;
    uint4 raw[NT][NB];
    if (k + C::kChunkK <= a.K) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < NB; ++b) raw[n][b] = *reinterpret_cast<const uint4*>(x_lane[n] + k + b * 32);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          raw[n][b] = k + b * 32 + t * 8 < a.K ? *reinterpret_cast<const uint4*>(x_lane[n] + k + b * 32)
                                               : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 q = raw[n][b];
        if constexpr (FMT == kFmtInt4) {
          // the pairs that decode_int4 makes
          x[n][b][0] = __byte_perm(q.x, q.z, 0x7632u);
          x[n][b][1] = __byte_perm(q.x, q.z, 0x5410u);
          x[n][b][2] = __byte_perm(q.y, q.w, 0x7632u);
          x[n][b][3] = __byte_perm(q.y, q.w, 0x5410u);
        } else {
          x[n][b][0] = q.x, x[n][b][1] = q.y, x[n][b][2] = q.z, x[n][b][3] = q.w;
        }
      }
    }
  };
  if (a.after_input) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (first < p.chunks) load_x(first);

  int stage = 0, buf = 0;
  const uint32_t piece_lane = g * 128 + (FMT == kFmtBf16 ? 0 : t * 4);
  for (int tile = cta; tile < p.tiles; tile += ctas, buf ^= 1) {
    float acc[RT][NT][4] = {};
    for (int chunk = first; chunk < p.chunks; chunk += stride) {
      if (chunk != x_chunk) load_x(chunk);
      float sc[RT][2][SPL];
      uint32_t zz[RT][2][SPL];
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < SPL; ++i) {
            sc[j][h][i] = __uint_as_float(a.scale_f32 ? ns[j][h][i] : ns[j][h][i] << 16);
            if constexpr (FMT == kFmtCodebook) sc[j][h][i] *= p.over_book;
            zz[j][h][i] = nz[j][h][i] & 15u;
          }
      if (chunk + stride < p.chunks) {
        load_scales(chunk + stride);
      } else if (tile + ctas < p.tiles) {
        scale_rows(tile + ctas);
        load_scales(first);
      }
      // Of group i of the chunk: row g (h = 0) or g + 8 of row tile j.
      auto scale_of = [&](int j, int h, int i) { return __shfl_sync(0xffffffffu, sc[j][h][i % SPL], i / SPL, 4); };
      auto zero_of = [&](int j, int h, int i) {
        if (!a.zeros) return 0x43084308u;
        return (__shfl_sync(0xffffffffu, zz[j][h][i % SPL], i / SPL, 4) | 0x4300u) * 0x10001u;
      };
      cp_async_wait<KS - 2>();
      __syncwarp();  // every lane's copies are in, and every lane is done with the stage filled next
      put();
      const unsigned char* piece = ring_p + stage * C::kPiece + piece_lane;
      float c[RT][NT][4];
      uint32_t z[RT][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          uint32_t v[2][4];  // rows g and g + 8
          if constexpr (FMT == kFmtInt4)
            if (b % GB == 0)
#pragma unroll
              for (int h = 0; h < 2; ++h) z[j][h] = zero_of(j, h, b / GB);
          uint32_t w[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (FMT == kFmtBf16) {
              const uint4 q = *reinterpret_cast<const uint4*>(piece + j * 2048 + h * 1024 +
                                                              ((static_cast<uint32_t>(b * 4 + t) ^ swz(g)) << 4));
              v[h][0] = q.x, v[h][1] = q.y, v[h][2] = q.z, v[h][3] = q.w;
            } else {
              w[h] = *reinterpret_cast<const uint32_t*>(piece + j * 2048 + h * 1024 +
                                                        ((static_cast<uint32_t>(b) ^ swz(g)) << 4));
              if constexpr (FMT == kFmtInt4)
                decode_int4(w[h], z[j][h], bits, v[h]);
              else
                decode_table(w[h], lane_table, v[h]);
            }
          }
#pragma unroll
          for (int two = 0; two < (TWO ? 2 : 1); ++two) {
            if (two) {
              decode_table(w[0], lane_table + C::kTable, v[0]);
              decode_table(w[1], lane_table + C::kTable, v[1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t m[4] = {v[0][2 * i], v[1][2 * i], v[0][2 * i + 1], v[1][2 * i + 1]};
                if (FMT != kFmtBf16 && b % GB == 0 && two == 0 && i == 0)
                  mma16816_first(c[j][n], m, x[n][b][2 * i], x[n][b][2 * i + 1]);
                else
                  mma16816(FMT == kFmtBf16 ? acc[j][n] : c[j][n], m, x[n][b][2 * i], x[n][b][2 * i + 1]);
              }
          }
          if (FMT != kFmtBf16 && b % GB == GB - 1) {
            const float s0 = scale_of(j, 0, b / GB), s1 = scale_of(j, 1, b / GB);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[j][n][0] = fmaf(s0, c[j][n][0], acc[j][n][0]);
              acc[j][n][1] = fmaf(s0, c[j][n][1], acc[j][n][1]);
              acc[j][n][2] = fmaf(s1, c[j][n][2], acc[j][n][2]);
              acc[j][n][3] = fmaf(s1, c[j][n][3], acc[j][n][3]);
            }
          }
        }
      }
      stage = stage + 1 == KS ? 0 : stage + 1;
    }
    // Partial sums of the warps (and CTAs) that share rows, added in a fixed
    // order.  Two buffers: one barrier per tile.
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        red[buf][warp][j][n][lane] = make_float4(acc[j][n][0], acc[j][n][1], acc[j][n][2], acc[j][n][3]);
    if (p.split > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
    if (rank == 0) {
      // A warp adds up a row tile.  Lane (g, t) has rows g and g + 8, tokens 2 t and 2 t + 1.
      for (int task = warp; task < (kWarps / kw) * RT * NT; task += kWarps) {
        const int n = task % NT, j = task / NT % RT, r = task / NT / RT;
        float c[4] = {};
        for (int q = 0; q < p.split; ++q) {
          const float4* from = &red[buf][r * kw][j][n][lane];
          if (q) from = cg::this_cluster().map_shared_rank(from, cg::this_cluster().block_rank() + q);
#pragma unroll 4
          for (int w = 0; w < kw; ++w) {
            const float4 v = from[w * RT * NT * 32];
            c[0] += v.x, c[1] += v.y, c[2] += v.z, c[3] += v.w;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = n * 8 + 2 * t + (i & 1), col = tile * tile_out + r * warp_out + j * rows_out + g + (i >> 1) * 8;
          if (m >= a.M || (glu && i > 1)) continue;
          const float y = glu ? (a.epi == kGemvSilu ? silu_f32(c[i]) : gelu_tanh_f32(c[i])) * c[i | 2] : c[i];
          if (col >= nout) continue;
          const int64_t at = m * a.ldo + col;
          if (a.out_f32)
            static_cast<float*>(a.out)[at] = y;
          else
            static_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(y);
        }
      }
    }
    if (p.split > 1) cg::this_cluster().sync();  // a CTA's sums stay until they are read
  }
  cp_async_wait<0>();
}

template <int FMT, int GB, int NT, int RT, bool TWO>
cudaError_t launch_one(const Params& p, int grid, cudaStream_t stream) {
  constexpr size_t smem = Cfg<FMT, GB, NT, RT, TWO>::kSmem;
  const void* f = reinterpret_cast<const void*>(gemv_kernel<FMT, GB, NT, RT, TWO>);
  if (cudaError_t err = ensure_smem_limit(f, smem); err != cudaSuccess) return err;
  LaunchScope ls(FMT == kFmtBf16 ? "gemv.bf16" : FMT == kFmtInt4 ? "gemv.int4" : "gemv.codebook", stream);
  return launch_overlapped(gemv_kernel<FMT, GB, NT, RT, TWO>, grid, kWarps * 32, smem, p.split, stream, p);
}

template <int FMT, int GB, bool TWO>
cudaError_t launch_rows(const Params& p, int rt, int grid, cudaStream_t stream) {
  if (p.a.M > 8) return launch_one<FMT, GB, 2, 1, TWO>(p, grid, stream);
  if constexpr (!TWO)  // launch_gemv() asks for no two row tiles there
    if (rt == 2) return launch_one<FMT, GB, 1, 2, TWO>(p, grid, stream);
  return launch_one<FMT, GB, 1, 1, TWO>(p, grid, stream);
}

template <int FMT, bool TWO>
cudaError_t launch_group(const Params& p, int rt, int grid, cudaStream_t stream) {
  if (p.a.group == 32) return launch_rows<FMT, 1, TWO>(p, rt, grid, stream);
  if (p.a.group == 64) return launch_rows<FMT, 2, TWO>(p, rt, grid, stream);
  return launch_rows<FMT, 4, TWO>(p, rt, grid, stream);
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  if (cudaError_t err = device_info(&di); err != cudaSuccess) return err;
  Params p{};
  p.a = a;
  p.chunks = static_cast<int>((a.row_bytes + 127) / 128);
  const bool two = a.fmt == kGemvCodebook && a.out_f32 && a.quant != E4B_QUANT_FP4;  // NF4 entries as two bf16 values
  p.book = a.quant == E4B_QUANT_FP4 ? 6.0f : two ? 1.4376f : 1.43672f;
  p.over_book = 1.0f / p.book;
  const int slots = 2 * di.sm_count;  // two CTAs fit an SM
  const int row_tiles = a.epi == kGemvNone ? (a.N + 15) / 16 : (a.N / 2 + 7) / 8;
  // Two row tiles per warp share the tokens' registers and a chunk's overhead; worth it
  // once every warp of the GPU has several chunks anyway (8 x 4096 x 32768 int4 25 us
  // against 30 with one; smaller products would leave SMs without rows).
  // Not with two tables: their shared memory and two row tiles' leave an SM one CTA
  // (8 x 4096 x 32768 NF4, blocks of 64, fp32 out 41.0 us against 45.9 with two row tiles).
  const int rt = a.M <= 8 && !two && static_cast<int64_t>(row_tiles) * p.chunks >= 4ll * slots * kWarps ? 2 : 1;
  // The split of K over a CTA's warps that needs the fewest steps: chunks of a
  // warp's share, and about two for the sums that end a tile.
  const int units = (row_tiles + rt - 1) / rt;
  int64_t best = -1;
  for (int kw = kWarps; kw >= 1; kw /= 2) {
    const int64_t tiles = (units + kWarps / kw - 1) / (kWarps / kw);
    const int64_t cost = (tiles + slots - 1) / slots * ((p.chunks + kw - 1) / kw * rt + 2);
    if (best < 0 || cost < best) {
      best = cost;
      p.kw = kw;
      p.tiles = static_cast<int>(tiles);
    }
  }
  // Few rows and a long K: a cluster's CTAs take K in turns, while all of them
  // have chunks and fit the GPU at once.
  p.split = 1;
  while (p.kw == kWarps && p.split < 8 && p.tiles * p.split * 2 <= slots && p.chunks >= kWarps * p.split * 2) p.split *= 2;
  const int grid = p.split > 1 ? p.tiles * p.split : std::min(p.tiles, slots);
  if (a.fmt == kGemvBf16) return launch_rows<kFmtBf16, 1, false>(p, rt, grid, stream);
  if (a.fmt == kGemvInt4) return launch_group<kFmtInt4, false>(p, rt, grid, stream);
  return two ? launch_group<kFmtCodebook, true>(p, rt, grid, stream) : launch_group<kFmtCodebook, false>(p, rt, grid, stream);
}

}  // namespace e4b

using namespace e4b;

extern "C" e4b_status e4b_gemv_4bit(const uint16_t* x, int64_t M, int64_t ldx, const e4b_group_weight* w,
                                    e4b_epilogue epi, void* out, e4b_dtype out_dtype, int64_t ldo, e4b_stream stream) {
  begin_call();
  if (!w) return fail(E4B_ERR_INVALID_ARGUMENT, "null group weight");
  if (w->quant_type != E4B_QUANT_NF4 && w->quant_type != E4B_QUANT_FP4 && w->quant_type != E4B_QUANT_INT4)
    return fail(E4B_ERR_INVALID_ARGUMENT, "quant_type must be NF4, FP4 or INT4");
  if (w->group != 32 && w->group != 64 && w->group != 128)
    return fail(E4B_ERR_UNSUPPORTED, "group must be 32, 64 or 128");
  if (w->K < 1 || w->K % w->group != 0 || w->K > INT32_MAX / 2)
    return fail(E4B_ERR_UNSUPPORTED, "K must be a positive multiple of the group, below 2^30");
  if (w->N < 1 || w->N > INT32_MAX / 2) return fail(E4B_ERR_UNSUPPORTED, "N must be in [1, 2^30)");
  if (w->scale_dtype != E4B_F32 && w->scale_dtype != E4B_BF16)
    return fail(E4B_ERR_INVALID_ARGUMENT, "scale_dtype must be F32 or BF16");
  if (w->zeros && w->quant_type != E4B_QUANT_INT4)
    return fail(E4B_ERR_INVALID_ARGUMENT, "only INT4 weights have zero points");
  if (!w->packed || !w->scales) return fail(E4B_ERR_INVALID_ARGUMENT, "null packed or scales");
  if (!aligned16(w->packed) || !aligned16(w->scales) || !aligned16(w->zeros))
    return fail(E4B_ERR_INVALID_ARGUMENT, "packed, scales and zeros must be 16-byte aligned");
  if (epi != E4B_EPI_NONE && epi != E4B_EPI_SWIGLU) return fail(E4B_ERR_INVALID_ARGUMENT, "unknown epilogue");
  if (epi == E4B_EPI_SWIGLU && w->N % 2 != 0) return fail(E4B_ERR_INVALID_ARGUMENT, "N must be even with SwiGLU");
  if (out_dtype != E4B_F32 && out_dtype != E4B_BF16) return fail(E4B_ERR_INVALID_ARGUMENT, "out_dtype must be F32 or BF16");
  if (M < 0 || M > 16) return fail(E4B_ERR_UNSUPPORTED, "M must be in [0, 16]: longer inputs take the grouped GEMM");
  if (M > 0 && (!x || !out)) return fail(E4B_ERR_INVALID_ARGUMENT, "null x or out");
  if (ldx < w->K || ldx % 8 != 0) return fail(E4B_ERR_INVALID_ARGUMENT, "ldx must be >= K and a multiple of 8");
  if (ldo < (epi == E4B_EPI_SWIGLU ? w->N / 2 : w->N))
    return fail(E4B_ERR_INVALID_ARGUMENT, "ldo must be at least the output's columns");
  if (!aligned16(x) || !aligned16(out)) return fail(E4B_ERR_INVALID_ARGUMENT, "x and out must be 16-byte aligned");
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  if (M == 0) {
    set_path("gemv.empty");
    return E4B_OK;
  }
  GemvArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.M = static_cast<int>(M);
  a.w = w->packed;
  a.row_bytes = w->K / 2;
  a.fmt = w->quant_type == E4B_QUANT_INT4 ? kGemvInt4 : kGemvCodebook;
  a.quant = w->quant_type;
  a.scales = w->scales;
  a.scale_f32 = w->scale_dtype == E4B_F32;
  a.zeros = w->zeros;
  a.group = w->group;
  a.groups = static_cast<int>(w->K / w->group);
  a.N = static_cast<int>(w->N);
  a.K = static_cast<int>(w->K);
  a.epi = epi == E4B_EPI_SWIGLU ? kGemvSilu : kGemvNone;
  a.out = out;
  a.out_f32 = out_dtype == E4B_F32;
  a.ldo = ldo;
  if (cudaError_t err = launch_gemv(a, reinterpret_cast<cudaStream_t>(stream)); err != cudaSuccess)
    return cuda_fail(err, "gemv launch");
  set_path(w->quant_type == E4B_QUANT_INT4 ? "gemv.int4" : "gemv.codebook");
  return E4B_OK;
}
