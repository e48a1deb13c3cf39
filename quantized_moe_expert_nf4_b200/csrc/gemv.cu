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
// 128 and subtracting 128 + zero, both exact; codebook entries by byte permutes over their bf16
// bytes.  Products and group sums are fp32 in the MMA, the scales
// multiply the group sums in fp32.  With fp32 output a codebook entry is taken as
// the sum of two bf16 values (error 2^-18 of the entry instead of 2^-9); with bf16
// output the first alone, whose rounding stays below the output's.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "e4b_internal.h"

namespace e4b {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kStages = 4;               // 2 KB pieces in flight per warp
constexpr uint32_t kPiece = 16 * 128;    // 16 rows x 128 bytes

enum Fmt { kFmtCodebook = 0, kFmtInt4 = 1, kFmtBf16 = 2 };

struct Params {
  GemvArgs a;
  int chunks;     // ceil(row bytes / 128)
  int kw;         // warps that share a row tile
  int split;      // CTAs of a cluster that share a row tile
  int tiles;      // CTA tiles of 16 * (8 / kw) rows
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int bytes = in ? 16 : 0;  // 0: writes zeros, reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte unit `u` (0..7) of row `row` of a piece lies at unit u ^ swz(row): eight
// rows give eight places for one unit, and two adjacent rows' four units do not meet.
__device__ __forceinline__ uint32_t swz(int row) { return ((row & 1) << 2) | ((row >> 1) & 3); }

// Codebook bytes: word j / 4 byte j % 4 of lo / hi = low / high byte of bf16(entry j).
struct Book {
  uint32_t lo[4], hi[4];
};

// The entries' bf16 values (residual false), or bf16 of what that rounding left.
__device__ __forceinline__ Book make_book(int quant, bool residual) {
  Book t{};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float v = codebook_entry(quant, j);
    if (residual) v -= bf16_bits_to_float(float_to_bf16_bits(v));
    const uint32_t b = float_to_bf16_bits(v);
    t.lo[j >> 2] |= (b & 0xffu) << (8 * (j & 3));
    t.hi[j >> 2] |= (b >> 8) << (8 * (j & 3));
  }
  return t;
}

// Eight codes (byte i: element 2i in the high nibble) -> four bf16 pairs in
// element order.  A byte permute looks up entries 0-7 or 8-15 of four codes at
// once; `pick` keeps, per code, the half that its top bit names.
__device__ __forceinline__ void decode_book(uint32_t w, const Book& t, uint32_t v[4]) {
  const uint32_t s = w & 0x77777777u, pick = ((w >> 1) & 0x44444444u) | 0x32103210u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sh = s >> (16 * h), ph = pick >> (16 * h);
    const uint32_t lo = __byte_perm(__byte_perm(t.lo[0], t.lo[1], sh), __byte_perm(t.lo[2], t.lo[3], sh), ph);
    const uint32_t hi = __byte_perm(__byte_perm(t.hi[0], t.hi[1], sh), __byte_perm(t.hi[2], t.hi[3], sh), ph);
    v[2 * h] = __byte_perm(lo, hi, 0x4051u);
    v[2 * h + 1] = __byte_perm(lo, hi, 0x6273u);
  }
}

// Eight int4 codes -> bf16 pairs of elements (1, 5), (0, 4), (3, 7), (2, 6), each
// 128 + code - (128 + zero); `zz` is bf16(128 + zero) in both halves.
__device__ __forceinline__ void decode_int4(uint32_t w, uint32_t zz, uint32_t v[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t q = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q), *reinterpret_cast<const __nv_bfloat162*>(&zz));
    v[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

template <int FMT>
struct Traits {
  static constexpr int kBlocks = FMT == kFmtBf16 ? 2 : 8;   // blocks of 32 k in a chunk
  static constexpr int kChunkK = kBlocks * 32;
};

// FMT: weight format; GB: blocks of 32 k in a group; NT: sets of 8 tokens;
// TWO: codebook entries as two bf16 values.
template <int FMT, int GB, int NT, bool TWO>
__global__ void __launch_bounds__(kWarps * 32, 2) gemv_kernel(Params p) {
  using Tr = Traits<FMT>;
  constexpr int NB = Tr::kBlocks;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float red[2][kWarps][NT][4][32];
  const GemvArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int kw = p.kw, wk = warp % kw, wr = warp / kw;  // this warp's share of K, its row tile of the CTA's
  const int rank = p.split > 1 ? static_cast<int>(blockIdx.x % p.split) : 0;
  const int cta = p.split > 1 ? static_cast<int>(blockIdx.x / p.split) : static_cast<int>(blockIdx.x);
  const int ctas = static_cast<int>(gridDim.x) / p.split;
  const int first = rank * kw + wk, stride = kw * p.split;  // chunks first, first + stride, ...
  const bool glu = a.epi != kGemvNone;
  const int half = a.N / 2;
  const int rows_out = glu ? 8 : 16;         // output columns of a warp's row tile
  const int nout = glu ? half : a.N;
  const int tile_out = rows_out * (kWarps / kw);
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * kStages * kPiece;
  const unsigned char* ring_p = smem + warp * kStages * kPiece;

  // Weight row of MMA row r (0..15) of this warp's part of a tile: rows 8..15 are
  // the up rows of a gated product.  Rows past the end read row 0, and are not written.
  auto weight_row = [&](int tile, int r, bool* in) -> int64_t {
    const int o = tile * tile_out + wr * rows_out + (glu ? (r & 7) : r);
    *in = o < nout;
    if (!*in) return 0;
    return glu && r >= 8 ? half + o : o;
  };

  // The pieces of this warp, in order: every chunk of its share, tile after tile.
  int put_tile = cta, put_chunk = first;
  int put_stage = 0;
  auto put = [&]() {
    if (put_tile < p.tiles && first < p.chunks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 4 + (lane >> 3), u = lane & 7;
        bool in;
        const int64_t row = weight_row(put_tile, r, &in);
        const int64_t off = static_cast<int64_t>(put_chunk) * 128 + u * 16;
        in = in && off < a.row_bytes;
        cp_async16(ring + put_stage * kPiece + r * 128 + ((u ^ swz(r)) << 4),
                   static_cast<const unsigned char*>(a.w) + (in ? row * a.row_bytes + off : 0), in);
      }
      put_chunk += stride;
      if (put_chunk >= p.chunks) {
        put_chunk = first;
        put_tile += ctas;
      }
    }
    cp_async_commit();
    put_stage = put_stage + 1 == kStages ? 0 : put_stage + 1;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) put();

  Book book{}, rest{};
  if constexpr (FMT == kFmtCodebook) {
    book = make_book(a.quant, false);
    if constexpr (TWO) rest = make_book(a.quant, true);
  }
  uint32_t x[NT][NB][4];
  int x_chunk = -1;
  int stage = 0, buf = 0;
  for (int tile = cta; tile < p.tiles; tile += ctas, buf ^= 1) {
    float acc[NT][4] = {};
    bool in0, in1;
    const int64_t row0 = weight_row(tile, g, &in0), row1 = weight_row(tile, g + 8, &in1);
    for (int chunk = first; chunk < p.chunks; chunk += stride) {
      if (chunk != x_chunk) {
        x_chunk = chunk;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int k = chunk * Tr::kChunkK + b * 32 + t * 8;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (n * 8 + g < a.M && k < a.K) q = *reinterpret_cast<const uint4*>(a.x + (n * 8 + g) * a.ldx + k);
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
      // scales (and zero points) of the chunk's groups, rows g and g + 8; zero past K
      float s0[NB / GB + 1], s1[NB / GB + 1];
      uint32_t z0[NB / GB + 1], z1[NB / GB + 1];
      if constexpr (FMT != kFmtBf16) {
#pragma unroll
        for (int i = 0; i < NB / GB; ++i) {
          const int grp = chunk * (NB / GB) + i;
          const bool in = grp < a.groups;
          const int64_t o0 = row0 * a.groups + (in ? grp : 0), o1 = row1 * a.groups + (in ? grp : 0);
          if (a.scale_f32) {
            s0[i] = in ? static_cast<const float*>(a.scales)[o0] : 0.0f;
            s1[i] = in ? static_cast<const float*>(a.scales)[o1] : 0.0f;
          } else {
            s0[i] = in ? bf16_bits_to_float(static_cast<const uint16_t*>(a.scales)[o0]) : 0.0f;
            s1[i] = in ? bf16_bits_to_float(static_cast<const uint16_t*>(a.scales)[o1]) : 0.0f;
          }
          if constexpr (FMT == kFmtInt4) {
            const uint32_t q0 = a.zeros ? a.zeros[o0] & 15u : 8u, q1 = a.zeros ? a.zeros[o1] & 15u : 8u;
            z0[i] = (q0 | 0x4300u) * 0x10001u;
            z1[i] = (q1 | 0x4300u) * 0x10001u;
          }
        }
      }
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const unsigned char* piece = ring_p + stage * kPiece;
      float c[NT][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t v0[4], v1[4];  // rows g and g + 8
        if constexpr (FMT == kFmtBf16) {
          const uint32_t u = (static_cast<uint32_t>(b * 4 + t) ^ swz(g)) << 4;
          const uint4 q0 = *reinterpret_cast<const uint4*>(piece + g * 128 + u);
          const uint4 q1 = *reinterpret_cast<const uint4*>(piece + (g + 8) * 128 + u);
          v0[0] = q0.x, v0[1] = q0.y, v0[2] = q0.z, v0[3] = q0.w;
          v1[0] = q1.x, v1[1] = q1.y, v1[2] = q1.z, v1[3] = q1.w;
        } else {
          const uint32_t u = ((static_cast<uint32_t>(b) ^ swz(g)) << 4) + t * 4;
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(piece + g * 128 + u);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(piece + (g + 8) * 128 + u);
          if constexpr (FMT == kFmtInt4) {
            decode_int4(w0, z0[b / GB], v0);
            decode_int4(w1, z1[b / GB], v1);
          } else {
            decode_book(w0, book, v0);
            decode_book(w1, book, v1);
          }
          if constexpr (TWO) {
            uint32_t r0[4], r1[4];
            decode_book(w0, rest, r0);
            decode_book(w1, rest, r1);
            if (b % GB == 0)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[n][i] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t m[4] = {r0[2 * h], r1[2 * h], r0[2 * h + 1], r1[2 * h + 1]};
                mma16816(c[n], m, x[n][b][2 * h], x[n][b][2 * h + 1]);
              }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* d = FMT == kFmtBf16 ? acc[n] : c[n];
          if (FMT != kFmtBf16 && !TWO && b % GB == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[n][i] = 0.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t m[4] = {v0[2 * h], v1[2 * h], v0[2 * h + 1], v1[2 * h + 1]};
            mma16816(d, m, x[n][b][2 * h], x[n][b][2 * h + 1]);
          }
          if (FMT != kFmtBf16 && b % GB == GB - 1) {
            acc[n][0] = fmaf(s0[b / GB], c[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0[b / GB], c[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1[b / GB], c[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1[b / GB], c[n][3], acc[n][3]);
          }
        }
      }
      __syncwarp();  // the stage that is filled next was read by all lanes
      put();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    // Partial sums of the warps (and CTAs) that share rows, added in a fixed
    // order.  Two buffers: one barrier per tile.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[buf][warp][n][i][lane] = acc[n][i];
    if (p.split > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
    if (rank == 0) {
      const int ntok = a.M;
      const int count = tile_out * ntok;
      for (int i = threadIdx.x; i < count; i += kWarps * 32) {
        const int o = i % tile_out, m = i / tile_out;
        const int col = tile * tile_out + o;
        if (col >= nout) continue;
        const int w0 = (o / rows_out) * kw, r = o % rows_out;
        // MMA result i of lane (g, t): row g + 8 (i / 2), token 2 t + i % 2
        auto total = [&](int row) {
          float s = 0.0f;
          for (int q = 0; q < p.split; ++q) {
            const float* base = &red[buf][w0][m >> 3][((row >> 3) << 1) | (m & 1)][((row & 7) << 2) | ((m & 7) >> 1)];
            if (q) base = cg::this_cluster().map_shared_rank(base, cg::this_cluster().block_rank() + q);
            for (int w = 0; w < kw; ++w) s += base[w * NT * 4 * 32];
          }
          return s;
        };
        float y = total(r);
        if (glu) {
          const float up = total(r + 8);
          y = (a.epi == kGemvSilu ? silu_f32(y) : gelu_tanh_f32(y)) * up;
        }
        const int64_t at = m * a.ldo + col;
        if (a.out_f32)
          static_cast<float*>(a.out)[at] = y;
        else
          static_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(y);
      }
    }
    if (p.split > 1) cg::this_cluster().sync();  // a CTA's sums stay until they are read
  }
  cp_async_wait<0>();
}

template <int FMT, int GB, int NT, bool TWO>
cudaError_t launch_one(const Params& p, int grid, cudaStream_t stream) {
  constexpr size_t smem = kWarps * kStages * kPiece;
  const void* f = reinterpret_cast<const void*>(gemv_kernel<FMT, GB, NT, TWO>);
  if (cudaError_t err = ensure_smem_limit(f, smem); err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  LaunchScope ls(FMT == kFmtBf16 ? "gemv.bf16" : FMT == kFmtInt4 ? "gemv.int4" : "gemv.codebook", stream);
  return cudaLaunchKernelEx(&cfg, gemv_kernel<FMT, GB, NT, TWO>, p);
}

template <int FMT, bool TWO>
cudaError_t launch_group(const Params& p, int grid, cudaStream_t stream) {
  const bool two_sets = p.a.M > 8;
  if (p.a.group == 32)
    return two_sets ? launch_one<FMT, 1, 2, TWO>(p, grid, stream) : launch_one<FMT, 1, 1, TWO>(p, grid, stream);
  if (p.a.group == 64)
    return two_sets ? launch_one<FMT, 2, 2, TWO>(p, grid, stream) : launch_one<FMT, 2, 1, TWO>(p, grid, stream);
  return two_sets ? launch_one<FMT, 4, 2, TWO>(p, grid, stream) : launch_one<FMT, 4, 1, TWO>(p, grid, stream);
}

}  // namespace

cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  if (cudaError_t err = device_info(&di); err != cudaSuccess) return err;
  Params p{};
  p.a = a;
  p.chunks = static_cast<int>((a.row_bytes + 127) / 128);
  const int row_tiles = a.epi == kGemvNone ? (a.N + 15) / 16 : (a.N / 2 + 7) / 8;
  // Two CTAs fit an SM.  The split of K over a CTA's warps that needs the fewest
  // chunks in a row per warp, the widest of equals (its sums are ready first).
  const int slots = 2 * di.sm_count;
  int64_t best = -1;
  for (int kw = kWarps; kw >= 1; kw /= 2) {
    const int64_t tiles = (row_tiles + kWarps / kw - 1) / (kWarps / kw);
    const int64_t cost = (tiles + slots - 1) / slots * ((p.chunks + kw - 1) / kw);
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
  if (a.fmt == kGemvBf16)
    return a.M > 8 ? launch_one<kFmtBf16, 1, 2, false>(p, grid, stream) : launch_one<kFmtBf16, 1, 1, false>(p, grid, stream);
  if (a.fmt == kGemvInt4) return launch_group<kFmtInt4, false>(p, grid, stream);
  return a.out_f32 ? launch_group<kFmtCodebook, true>(p, grid, stream) : launch_group<kFmtCodebook, false>(p, grid, stream);
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
