// Dense gated feed-forward block in bf16, forward and backward.
//
//   pre = x . Wgu^T,  h = act(pre[:, :I]) * pre[:, I:],  out = h . Wd^T
//   dh = dout . Wd,   dgate = dh * up * act'(gate),  dup = dh * act(gate)
//   dx = dpre . Wgu,  dWgu = dpre^T . x,  dWd = dout^T . h
//
// Every product is one tcgen05 GEMM kernel (D[rows, cols] = A . B^T, fp32
// accumulators in TMEM) with its operands read as they lie: an operand whose
// rows are contiguous in memory (a weight in dh and dx, both activations in the
// weights' gradients) is loaded and multiplied MN-major, so nothing is
// transposed.  The gate and up projections, the activation and the product are
// one kernel (a tile holds the same columns of both), and so are dh, the
// activation's derivative and both products with it.
//
// Bound: tensor cores from a few hundred rows; below, the weights' bytes.
// Warps: 0 TMA producer, 1 MMA issuer, 2-5 (2-9) epilogue.  A persistent CTA (or pair)
// walks the tiles; two accumulator sets let an epilogue run under the next
// tile's MMAs.  Tiles: 256 x 256 by a CTA pair (each CTA holds half of A's and B's
// rows, so a stage is 32 KB for 2 x 128 x 256 x 64 products), or 128 x 128 and
// 128 x 64 by single CTAs where the large tiles would leave SMs without work.
// An epilogue warp takes its 32 rows 32 columns at a time from TMEM to registers,
// and hands bf16 pieces of 32 x 32 to TMA stores, which clip at the edges.
//
// Up to 16 rows without saved pre-activations the products stream the weights
// through the warp-MMA kernel of the 4-bit products instead.
//
// Measured, H = I = 2880, against cuBLAS's 1652 (burst) and 1388 (sustained) bf16 TFLOP/s
// on the same GPUs: forward of 4096 tokens 175 us back to back, 1.17 PFLOP/s (149 us in a short
// run); forward and backward of 8192 tokens 1105 us in a loop of a second or more, 1.11 PFLOP/s
// (the power cap lowers the clock), 959 us in a short one.  256 tokens, forward and backward,
// 129 us (floor 23: six launches of one tile a CTA).  One token at H = 4096, I = 11008 51 us,
// 5.3 TB/s.  197 x 2048 x 776 takes 17 us (one tile and its epilogue
// a kernel: latency), one token 8.7 us (two launches).  What the steps brought for
// the long ones: loads and pieces as TMA 972 -> 944 us, tiles walked in groups of 8
// rows 1140 -> 1085 sustained, overlapped launches 1.6%.
//
// Roundings: pre-activations, h and the gradients by them are bf16 between the
// kernels, as a training program stores them; all sums are fp32.
#include <cuda.h>

#include <algorithm>
#include <string>

#include "async.cuh"
#include "common.cuh"
#include "e4b_internal.h"
#include "tcgen05.cuh"

namespace e4b {
namespace {

constexpr int kBK = 64;                       // k per stage: one 128-byte swizzle row
constexpr int kTileM = 128;                   // rows per CTA
constexpr int kWarpEpi = 2;
constexpr uint32_t kABytes = kTileM * 128;
constexpr uint32_t kPieceBytes = 32 * 64;     // staged output: 32 rows x 32 bf16, 64-byte swizzle
constexpr uint32_t kSmemMax = 227 * 1024;

enum Epi { kEpiPlain = 0, kEpiGlu = 1, kEpiDglu = 2 };

// How a product follows the launch ahead of it (see launch_overlapped).  kAfterInput: it
// waits for it before its first load; its start-up is hidden.  kAfterNothing: it reads
// what an earlier one wrote, which had ended when the launch ahead allowed this one to
// start, so its tiles fill the SMs that run out of work in the launch ahead; it
// waits for that one's end before its own, so that the stream's order holds for
// what follows.
enum After { kAfterInput = 0, kAfterNothing = 1 };

// CTAs of a tile (1, or a pair) and its columns; where everything lies in shared
// memory, for an operand B that is MN-major or not and an epilogue.
// SPLIT: CTAs of a cluster that share a tile's k blocks.
template <int CG_, int BN_, int SPLIT_ = 1>
struct Shape {
  static constexpr int CG = CG_, BN = BN_, SPLIT = SPLIT_;
  static constexpr int kBRows = BN / CG;      // B rows per CTA
  static constexpr uint32_t kCols = BN <= 64 ? 128 : BN <= 128 ? 256 : 512;  // TMEM columns: two accumulator sets
  static_assert(2 * BN <= 512 && BN % 32 == 0 && (SPLIT == 1 || CG == 1), "tile shape");
};
template <class S, bool BMN, int EPI>
struct Layout {
  // MN-major rows come in blocks of 64; a last block may be used in part
  static constexpr uint32_t kBBytes = BMN ? (S::kBRows + 63) / 64 * 8192 : S::kBRows * 128;
  static constexpr uint32_t kStage = kABytes + kBBytes;
  // The activation's derivative keeps one warp per scheduler busy longer than a
  // tile's MMAs take: with two the kernel of 8192 x 2880 x 2880 takes 151 us, with one 165.
  static constexpr int kEpiWarps = EPI == kEpiDglu ? 8 : 4;
  static constexpr int kThreads = (kWarpEpi + kEpiWarps) * 32;
  // Pieces of an epilogue warp.  Plain: a ring of single ones.  Gated: two sets of h,
  // gate and up, one filled while the other's stores read it.  Derivative: h, and
  // two pairs of gate and up that are loaded, replaced by their gradients and stored.
  static constexpr int kPieces = EPI == kEpiPlain ? 4 : EPI == kEpiGlu ? 6 : 5;
  static constexpr uint32_t kStageOutBytes = kEpiWarps * kPieces * kPieceBytes;
  // Partial sums of the other CTAs for this one's rows (32 rows x BN fp32 per quarter).
  static constexpr uint32_t kRecvBytes = S::SPLIT > 1 ? (S::SPLIT - 1) * (4 / S::SPLIT) * S::BN * 128 : 0;
  static constexpr int kFit = static_cast<int>((kSmemMax - 2048 - kStageOutBytes - kRecvBytes) / kStage);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr uint32_t kOffOut = kStages * kStage;
  static constexpr uint32_t kOffRecv = kOffOut + kStageOutBytes;
  static constexpr uint32_t kOffBar = kOffRecv + kRecvBytes;
  static constexpr uint32_t kSmem = kOffBar + (2 * kStages + 4 + 16) * 8 + 16 + 1024;
  static_assert(kSmem <= kSmemMax && kStages >= 3, "tile fits");
};

struct TileParams {
  int rows, cols, K;       // of D and the contraction; for the gated tile, cols of h
  int m_tiles, n_tiles;
  int group;               // row tiles that are walked together (tile_at)
  int half;                // gated: first up row of B (I)
  int act;
  int write_pre;           // kEpiGlu: also store the pre-activations
  int after;               // how the kernel follows the launch before it (After)
  int* err;
};

__device__ __forceinline__ float sigmoid_of(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// act(g) and its derivative.  GELU (tanh form) is g s, s = sigmoid(2 v), v = k (g + c g^3).
__device__ __forceinline__ float act_value(int act, float g) {
  return act == E4B_ACT_SILU ? g * sigmoid_of(g) : gelu_tanh_f32(g);
}
__device__ __forceinline__ void act_both(int act, float g, float* a, float* da) {
  if (act == E4B_ACT_SILU) {
    const float s = sigmoid_of(g);
    *a = g * s;
    *da = fmaf(*a, 1.0f - s, s);
  } else {
    constexpr float k2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float s = sigmoid_of(k2 * (g + 0.044715f * g * g * g));
    *a = g * s;
    // far out s (1 - s) is 0, and g^2 may not become infinite before it is multiplied by that
    *da = s + g * s * (1.0f - s) * k2 * (1.0f + 0.134145f * fminf(g * g, 1e30f));
  }
}

// One staged piece: 32 columns of this lane's row as four 16-byte units, exchanged
// by the 64-byte swizzle (unit ^ (row / 2) % 4).
__device__ __forceinline__ void stage_row(unsigned char* piece, int lane, const float v[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(piece + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(pack_bf16x2(v[8 * u], v[8 * u + 1]), pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                   pack_bf16x2(v[8 * u + 4], v[8 * u + 5]), pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
}

// The 32 bf16 of this lane's row of a piece that a TMA load laid out like that.
__device__ __forceinline__ void read_row(const unsigned char* piece, int lane, float v[32]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 q = *reinterpret_cast<const uint4*>(piece + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * u + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * u + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Tile t of the walk: `group` row tiles by all column tiles, rows fastest, then the
// next row tiles.  The tiles at work at one time then form a block whose operands
// stay in L2.
__device__ __forceinline__ void tile_at(const TileParams& p, int t, int* m, int* n) {
  const int per = p.group * p.n_tiles, g = t / per, r = t - g * per;
  const int rows = min(p.group, p.m_tiles - g * p.group);
  *n = r / rows;
  *m = g * p.group + r - *n * rows;
}

// AMN, BMN: the operand's rows are contiguous in memory (MN-major).
template <class S, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(Layout<S, BMN, EPI>::kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                    const __grid_constant__ CUtensorMap tm_o0, const __grid_constant__ CUtensorMap tm_o1,
                    const __grid_constant__ CUtensorMap tm_o2, const __grid_constant__ CUtensorMap tm_i0,
                    const __grid_constant__ CUtensorMap tm_i1, const __grid_constant__ TileParams p) {
  using L = Layout<S, BMN, EPI>;
  constexpr int CG = S::CG, BN = S::BN, KS = L::kStages;
  constexpr int kOutCols = EPI == kEpiGlu ? BN / 2 : BN;  // columns of D's tile that reach memory
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* empty = full + KS;
  uint64_t* acc_full = empty + KS;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* in_full = acc_empty + 2;  // [epilogue warp][2]: its pre-activations' pieces
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int SPLIT = S::SPLIT;
  const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;
  const int part = SPLIT > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / (CG * SPLIT), step = static_cast<int>(gridDim.x) / (CG * SPLIT);
  const int tiles = p.m_tiles * p.n_tiles, KB = (p.K + kBK - 1) / kBK;
  // This CTA's k blocks: all of them, or its part (never empty, see launch_gemm).
  const int kb_per = (KB + SPLIT - 1) / SPLIT, kb_first = part * kb_per, kb_end = min(KB, kb_first + kb_per);

  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], L::kEpiWarps * CG);
    }
    for (int s = 0; s < 16; ++s) mbar_init(&in_full[s], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_slot, S::kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, S::kCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (CG == 2 || SPLIT > 1)
    cluster_sync_all();  // the others have started and set up what this CTA writes to
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (p.after == kAfterInput) pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    // The stage's bytes of both CTAs of a pair are counted on rank 0's barrier.
    uint32_t it = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int m_tile, n_tile;
      tile_at(p, t, &m_tile, &n_tile);
      const int m0 = m_tile * (kTileM * CG) + rank * kTileM;
      for (int kb = kb_first; kb < kb_end; ++kb, ++it) {
        const int s = it % KS;
        if (it >= KS && !mbar_wait_warp(&empty[s], ((it / KS) - 1) & 1)) {
          record_error(p.err, kErrWaitEmpty);
          ok = false;
          break;
        }
        if (lane == 0) {
          unsigned char* a = smem + s * L::kStage;
          unsigned char* b = a + kABytes;
          const int k0 = kb * kBK;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * L::kStage);
          const uint32_t bar = CG == 2 ? cluster_addr(&full[s], 0) : 0;
          auto load = [&](unsigned char* dst, const CUtensorMap* map, int x, int y) {
            if constexpr (CG == 2)
              tma_load_2d_pair(dst, map, x, y, bar);
            else
              tma_load_2d(dst, map, x, y, &full[s]);
          };
          if constexpr (AMN) {
            load(a, &tm_a, m0, k0);
            load(a + kABytes / 2, &tm_a, m0 + 64, k0);
          } else {
            load(a, &tm_a, k0, m0);
          }
          if constexpr (EPI == kEpiGlu) {
            // the same columns' gate and up rows: one CTA each of a pair, halves of a single CTA's stage
            const int n0 = n_tile * kOutCols;
            if constexpr (CG == 2) {
              load(b, &tm_b, k0, rank ? p.half + n0 : n0);
            } else {
              load(b, &tm_b, k0, n0);
              load(b + L::kBBytes / 2, &tm_b, k0, p.half + n0);
            }
          } else {
            const int n0 = n_tile * BN + rank * S::kBRows;
            if constexpr (BMN) {
#pragma unroll
              for (int j = 0; j < (S::kBRows + 63) / 64; ++j) load(b + j * 8192, &tm_b, n0 + 64 * j, k0);
            } else {
              load(b, &tm_b, k0, n0);
            }
          }
        }
        __syncwarp();
      }
    }
    // The last stages: consumed (their barriers' last arrivals come from the
    // MMAs), or, after a wait that gave up, at least landed before the CTA ends.
    for (uint32_t j = it < KS ? 0 : it - KS; j < it; ++j) {
      if (ok) ok = mbar_wait_warp(&empty[j % KS], (j / KS) & 1);
      if (!ok && rank == 0) mbar_wait_warp(&full[j % KS], (j / KS) & 1);
    }
    if constexpr (SPLIT > 1) cluster_sync_all();  // with the epilogue's
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32_major(kTileM * CG, BN, AMN, BMN);
      uint32_t it = 0, j = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++j) {
        const uint32_t slot = j & 1;
        if (j >= 2 && !mbar_wait_warp(&acc_empty[slot], ((j >> 1) - 1) & 1)) {
          record_error(p.err, kErrWaitEmpty);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + slot * BN;
        for (int kb = kb_first; kb < kb_end; ++kb, ++it) {
          const int s = it % KS;
          if (!mbar_wait_warp(&full[s], (it / KS) & 1)) {
            record_error(p.err, kErrWaitFull);
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t a = smem_u32(smem + s * L::kStage), b = a + kABytes;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
              const uint64_t ad = AMN ? smem_desc_mn_sw128(a + kk * 2048, 8192) : smem_desc_sw128(a + kk * 32);
              const uint64_t bd = BMN ? smem_desc_mn_sw128(b + kk * 2048, 8192) : smem_desc_sw128(b + kk * 32);
              if constexpr (CG == 2)
                umma_bf16_pair(d, ad, bd, idesc, kb > kb_first || kk ? 1u : 0u);
              else
                umma_bf16(d, ad, bd, idesc, kb > kb_first || kk ? 1u : 0u);
            }
            if constexpr (CG == 2)
              umma_commit_pair(&empty[s]);
            else
              umma_commit(&empty[s]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) {
          if constexpr (CG == 2)
            umma_commit_pair(&acc_full[slot]);
          else
            umma_commit(&acc_full[slot]);
        }
        __syncwarp();
      }
    }
    if constexpr (SPLIT > 1) cluster_sync_all();
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lanes 32 q .. 32 q + 31 = the tile's rows
    unsigned char* pieces = smem + L::kOffOut + (warp - kWarpEpi) * L::kPieces * kPieceBytes;
    uint32_t j = 0, piece_no = 0;
    bool ok = true;
    // kEpiDglu: the saved gate and up pieces of the next 32 columns are loaded while
    // these are worked on, the first ones of a tile while its MMAs run.
    // A pair of warps with the same rows takes the columns' halves.
    constexpr int kCols = kOutCols * 4 / L::kEpiWarps;
    const int c_first = L::kEpiWarps == 8 ? ((warp - kWarpEpi) >> 2) * kCols : 0;
    unsigned char* in_pieces = pieces + kPieceBytes;
    uint64_t* in_bar = in_full + (warp - kWarpEpi) * 2;
    uint32_t in_put = 0, in_get = 0;
    auto put_in = [&](int col, int row0) {
      if (lane == 0) {
        unsigned char* to = in_pieces + (in_put & 1) * 2 * kPieceBytes;
        mbar_arrive_expect_tx(&in_bar[in_put & 1], 2 * kPieceBytes);
        tma_load_2d(to, &tm_i0, col, row0, &in_bar[in_put & 1]);
        tma_load_2d(to + kPieceBytes, &tm_i1, col, row0, &in_bar[in_put & 1]);
      }
      ++in_put;
    };
    for (int t = first; t < tiles && ok; t += step, ++j) {
      const uint32_t slot = j & 1;
      int m_tile, n_tile;
      tile_at(p, t, &m_tile, &n_tile);
      const int row0 = m_tile * (kTileM * CG) + rank * kTileM + q * 32;
      const int col0 = n_tile * kOutCols;
      if constexpr (EPI == kEpiDglu)
        if (row0 < p.rows && col0 + c_first < p.cols && q * SPLIT / 4 == part) {
          if (lane == 0) bulk_wait_group_read<0>();
          put_in(col0 + c_first, row0);
        }
      if (!mbar_wait_warp(&acc_full[slot], (j >> 1) & 1)) {
        record_error(p.err, kErrWaitFull);
        ok = false;
        if constexpr (SPLIT == 1) break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + slot * BN;
      // A split tile: part i of the cluster finishes the rows of quarters [4 i / SPLIT,
      // 4 (i + 1) / SPLIT); the others leave their sums of those rows in its shared memory.
      constexpr int kQuarters = 4 / SPLIT;
      if constexpr (SPLIT > 1) {
        const int owner = q / kQuarters;
        if (owner != part && ok) {
          const int from = part < owner ? part : part - 1;
          const uint32_t to = cluster_addr(smem + L::kOffRecv + (from * kQuarters + q % kQuarters) * BN * 128 + lane * 4, owner);
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            // of a pair of warps with the same rows, each sends half
            if (L::kEpiWarps == 8 && (c >= BN / 2) != (warp - kWarpEpi >= 4)) continue;
            float v[32];
            tmem_ld_32x32b_x32(acc + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) st_cluster_f32(to + (c + i) * 128, v[i]);
          }
        }
        cluster_sync_all();
        if (owner != part || !ok) break;
      }
      // Columns [at, at + 32) of the tile, of this lane's row.
      auto add_parts = [&](int at, float v[32]) {
        if constexpr (SPLIT > 1) {
#pragma unroll
          for (int f = 0; f < SPLIT - 1; ++f) {
            const float* src = reinterpret_cast<const float*>(smem + L::kOffRecv + (f * kQuarters + q % kQuarters) * BN * 128) + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += src[(at + i) * 32];
          }
        }
      };
#pragma unroll 1
      for (int c = c_first; c < c_first + kCols; c += 32) {
        const int col = col0 + c;
        if (row0 >= p.rows || col >= p.cols) break;
        float v[32];
        __syncwarp();  // lane 0 has just set off the last columns' stores
        tmem_ld_32x32b_x32(acc + c, v);
        if constexpr (EPI == kEpiPlain) {
          unsigned char* piece = pieces + (piece_no++ % L::kPieces) * kPieceBytes;
          tmem_ld_wait();
          add_parts(c, v);
          if (lane == 0) bulk_wait_group_read<L::kPieces - 1>();  // the store that last read this piece
          __syncwarp();
          stage_row(piece, lane, v);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_o0, piece, col, row0);
            bulk_commit_group();
          }
        } else if constexpr (EPI == kEpiGlu) {
          float u[32];
          tmem_ld_32x32b_x32(acc + BN / 2 + c, u);
          tmem_ld_wait();
          add_parts(c, v);
          add_parts(BN / 2 + c, u);
          unsigned char* set = pieces + (piece_no++ & 1) * 3 * kPieceBytes;
          if (lane == 0) bulk_wait_group_read<1>();  // the stores that last read this set
          __syncwarp();
          if (p.write_pre) {
            stage_row(set + kPieceBytes, lane, v);
            stage_row(set + 2 * kPieceBytes, lane, u);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = act_value(p.act, v[i]) * u[i];
          stage_row(set, lane, v);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_o0, set, col, row0);
            if (p.write_pre) {
              tma_store_2d(&tm_o1, set + kPieceBytes, col, row0);
              tma_store_2d(&tm_o2, set + 2 * kPieceBytes, col, row0);
            }
            bulk_commit_group();
          }
        } else {
          float g[32], u[32];
          unsigned char* in = in_pieces + (in_get & 1) * 2 * kPieceBytes;
          if (lane == 0) bulk_wait_group_read<0>();  // the last stores, of h and of the other pair
          if (c + 32 < c_first + kCols && col + 32 < p.cols) put_in(col + 32, row0);
          if (!mbar_wait_warp(&in_bar[in_get & 1], (in_get >> 1) & 1)) {
            record_error(p.err, kErrWaitFull);
            ok = false;
            tmem_ld_wait();
            break;
          }
          read_row(in, lane, g);
          read_row(in + kPieceBytes, lane, u);
          ++in_get;
          tmem_ld_wait();
          add_parts(c, v);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float a, da;
            act_both(p.act, g[i], &a, &da);
            const float dh = v[i];
            v[i] = a * u[i];         // h
            g[i] = dh * u[i] * da;   // gate's gradient
            u[i] = dh * a;           // up's gradient
          }
          stage_row(pieces, lane, v);
          stage_row(in, lane, g);
          stage_row(in + kPieceBytes, lane, u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_o0, pieces, col, row0);
            tma_store_2d(&tm_o1, in, col, row0);
            tma_store_2d(&tm_o2, in + kPieceBytes, col, row0);
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(cluster_addr(&acc_empty[slot], 0));
        else
          mbar_arrive(&acc_empty[slot]);
      }
    }
    if constexpr (EPI == kEpiDglu)  // after a wait that gave up: loads in flight land first
      for (; in_get < in_put; ++in_get) mbar_wait_warp(&in_bar[in_get & 1], (in_get >> 1) & 1);
    if (lane == 0) bulk_wait_group_all();
  }
  if (p.after == kAfterNothing) pdl_wait();
  tc_fence_before();
  if constexpr (CG == 2)
    cluster_sync_all();  // the pair's barriers and tiles are used from both sides
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem, S::kCols);
    else
      tmem_dealloc(tmem, S::kCols);
  }
}

// A bf16 matrix in memory: `rows` rows of `cols` elements, ld elements apart.
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
};

bool map_of(CUtensorMap* m, const Mat& a, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw) {
  const uint64_t dims[2] = {static_cast<uint64_t>(a.cols), static_cast<uint64_t>(a.rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(a.ld) * 2};
  const uint32_t box[2] = {box_cols, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.p, dims, strides, box, sw);
}

struct Gemm {
  const char* name;
  Mat a, b;             // as they lie in memory
  Mat out[3];           // o0, and o1, o2 of the gated epilogues (p null: not written)
  Mat in[2];            // kEpiDglu: saved gate and up
  TileParams p;
};

template <class S, bool AMN, bool BMN, int EPI>
cudaError_t launch_shape(const Gemm& g, int sm_count, cudaStream_t stream) {
  using L = Layout<S, BMN, EPI>;
  const void* f = reinterpret_cast<const void*>(ffn_gemm_kernel<S, AMN, BMN, EPI>);
  if (cudaError_t err = ensure_smem_limit(f, L::kSmem); err != cudaSuccess) return err;
  const uint32_t b_rows = EPI == kEpiGlu && S::CG == 1 ? S::kBRows / 2 : S::kBRows;
  CUtensorMap ta, tb, to[3], ti[2];
  if (!(AMN ? map_of(&ta, g.a, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B)
            : map_of(&ta, g.a, kBK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      !(BMN ? map_of(&tb, g.b, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B)
            : map_of(&tb, g.b, kBK, b_rows, CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 3; ++i) {
    if (!g.out[i].p)
      to[i] = to[0];  // never used
    else if (!map_of(&to[i], g.out[i], 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    if (EPI != kEpiDglu)
      ti[i] = to[0];  // never used
    else if (!map_of(&ti[i], g.in[i], 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  TileParams p = g.p;
  p.m_tiles = (p.rows + kTileM * S::CG - 1) / (kTileM * S::CG);
  const int cols = EPI == kEpiGlu ? S::BN / 2 : S::BN;
  p.n_tiles = (p.cols + cols - 1) / cols;
  p.group = 8;  // 4 to 8 measured best: M=8192 H=I=2880 training step 1085 us against 1140 with all rows
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int ctas = S::CG * S::SPLIT;  // of a cluster
  const int64_t clusters = S::SPLIT > 1 ? tiles : std::min<int64_t>(tiles, sm_count / S::CG);
  LaunchScope ls(g.name, stream);
  return launch_overlapped(ffn_gemm_kernel<S, AMN, BMN, EPI>, static_cast<int>(clusters) * ctas, L::kThreads, L::kSmem, ctas,
                           stream, ta, tb, to[0], to[1], to[2], ti[0], ti[1], p);
}

template <bool AMN, bool BMN, int EPI>
cudaError_t launch_gemm(const Gemm& g, int sm_count, cudaStream_t stream) {
  const int glu = EPI == kEpiGlu ? 2 : 1;
  auto tiles = [&](int rows, int cols) {
    return ((g.p.rows + rows - 1) / rows) * static_cast<int64_t>((g.p.cols * glu + cols - 1) / cols);
  };
  // The largest tile that still gives every SM work.  (Narrower pair tiles, 224 or
  // 192 columns, waste less of a last round but measured slower, 8192 x 5760 x 2880
  // 234 us at 192 against 197: a pair tile's loads are 64 bytes a cycle and SM at
  // 256 x 256 already, and grow with every column taken away.)
  if (tiles(256, 256) >= sm_count / 2) return launch_shape<Shape<2, 256>, AMN, BMN, EPI>(g, sm_count, stream);
  if (tiles(128, 128) >= sm_count) return launch_shape<Shape<1, 128>, AMN, BMN, EPI>(g, sm_count, stream);
  // Small tiles; where even those are few, two or four CTAs share the k blocks of one.
  const int64_t small = tiles(128, 64);
  const int KB = (g.p.K + kBK - 1) / kBK;
  if (small * 4 <= sm_count && KB >= 16) return launch_shape<Shape<1, 64, 4>, AMN, BMN, EPI>(g, sm_count, stream);
  if (small * 2 <= sm_count && KB >= 8) return launch_shape<Shape<1, 64, 2>, AMN, BMN, EPI>(g, sm_count, stream);
  return launch_shape<Shape<1, 64>, AMN, BMN, EPI>(g, sm_count, stream);
}

constexpr size_t kErrBytes = 256;
size_t forward_bytes(int64_t M, int64_t I) { return kErrBytes + align_up(static_cast<size_t>(M) * I * 2, 256); }
size_t backward_bytes(int64_t M, int64_t I) { return kErrBytes + 3 * align_up(static_cast<size_t>(M) * I * 2, 256); }

constexpr int64_t kMaxDim = 1 << 20;

e4b_status check_ffn(const e4b_gated_ffn* w, int64_t M, int64_t ldx, const void* x) {
  if (!w) return fail(E4B_ERR_INVALID_ARGUMENT, "null gated ffn");
  if (w->H < 8 || w->H % 8 != 0 || w->H > kMaxDim || w->I < 8 || w->I % 8 != 0 || w->I > kMaxDim)
    return fail(E4B_ERR_UNSUPPORTED, "H and I must be positive multiples of 8, at most 2^20");
  if (w->act != E4B_ACT_SILU && w->act != E4B_ACT_GELU_TANH) return fail(E4B_ERR_INVALID_ARGUMENT, "unknown activation");
  if (!w->gate_up || !w->down) return fail(E4B_ERR_INVALID_ARGUMENT, "null gate_up or down");
  if (!aligned16(w->gate_up) || !aligned16(w->down))
    return fail(E4B_ERR_INVALID_ARGUMENT, "gate_up and down must be 16-byte aligned");
  if (M < 0 || M > (1 << 24)) return fail(E4B_ERR_UNSUPPORTED, "M must be in [0, 2^24]");
  if (ldx < w->H || ldx % 8 != 0) return fail(E4B_ERR_INVALID_ARGUMENT, "ldx must be >= H and a multiple of 8");
  if (M > 0 && !x) return fail(E4B_ERR_INVALID_ARGUMENT, "null x");
  if (!aligned16(x)) return fail(E4B_ERR_INVALID_ARGUMENT, "x must be 16-byte aligned");
  return E4B_OK;
}

}  // namespace
}  // namespace e4b

using namespace e4b;

extern "C" {

size_t e4b_gated_ffn_forward_workspace_size(int64_t M, const e4b_gated_ffn* w) {
  return w && M > 0 && w->I > 0 ? forward_bytes(M, w->I) : 0;
}

size_t e4b_gated_ffn_backward_workspace_size(int64_t M, const e4b_gated_ffn* w) {
  return w && M > 0 && w->I > 0 ? backward_bytes(M, w->I) : 0;
}

e4b_status e4b_gated_ffn_forward(const uint16_t* x, int64_t M, int64_t ldx, const e4b_gated_ffn* w, uint16_t* out,
                                 uint16_t* pre, void* workspace, size_t workspace_bytes, e4b_stream stream) {
  begin_call();
  if (e4b_status s = check_ffn(w, M, ldx, x); s != E4B_OK) return s;
  if (M > 0 && !out) return fail(E4B_ERR_INVALID_ARGUMENT, "null out");
  if (!aligned16(out) || !aligned16(pre)) return fail(E4B_ERR_INVALID_ARGUMENT, "out and pre must be 16-byte aligned");
  if (e4b_status s = check_workspace("gated ffn forward", e4b_gated_ffn_forward_workspace_size(M, w), workspace,
                                     workspace_bytes);
      s != E4B_OK)
    return s;
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  if (M == 0) {
    set_path("ffn.empty");
    return E4B_OK;
  }
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int H = static_cast<int>(w->H), I = static_cast<int>(w->I), rows = static_cast<int>(M);
  uint16_t* h = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + kErrBytes);
  if (M <= 16 && !pre) {
    GemvArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.M = rows;
    a.w = w->gate_up;
    a.row_bytes = w->H * 2;
    a.fmt = kGemvBf16;
    a.N = 2 * I;
    a.K = H;
    a.epi = w->act == E4B_ACT_SILU ? kGemvSilu : kGemvGelu;
    a.out = h;
    a.ldo = I;
    if (cudaError_t err = launch_gemv(a, st); err != cudaSuccess) return cuda_fail(err, "ffn gate_up launch");
    a.after_input = true;
    a.x = h;
    a.ldx = I;
    a.w = w->down;
    a.row_bytes = w->I * 2;
    a.N = H;
    a.K = I;
    a.epi = kGemvNone;
    a.out = out;
    a.ldo = H;
    if (cudaError_t err = launch_gemv(a, st); err != cudaSuccess) return cuda_fail(err, "ffn down launch");
    set_path("ffn.forward.rows");
    return E4B_OK;
  }
  DeviceInfo di;
  if (cudaError_t err = device_info(&di); err != cudaSuccess) return cuda_fail(err, "device query");
  Gemm g{};
  g.name = "ffn.gate_up";
  g.a = {x, M, w->H, ldx};
  g.b = {w->gate_up, 2 * w->I, w->H, w->H};
  g.out[0] = {h, M, w->I, w->I};
  if (pre) {
    g.out[1] = {pre, M, w->I, 2 * w->I};
    g.out[2] = {pre + w->I, M, w->I, 2 * w->I};
  }
  g.p.rows = rows;
  g.p.cols = I;
  g.p.K = H;
  g.p.half = I;
  g.p.act = w->act;
  g.p.write_pre = pre != nullptr;
  g.p.err = static_cast<int*>(workspace);
  if (cudaError_t err = launch_gemm<false, false, kEpiGlu>(g, di.sm_count, st); err != cudaSuccess)
    return cuda_fail(err, "ffn gate_up launch");
  Gemm d{};
  d.name = "ffn.down";
  d.a = {h, M, w->I, w->I};
  d.b = {w->down, w->H, w->I, w->I};
  d.out[0] = {out, M, w->H, w->H};
  d.p.rows = rows;
  d.p.cols = H;
  d.p.K = I;
  d.p.err = g.p.err;
  if (cudaError_t err = launch_gemm<false, false, kEpiPlain>(d, di.sm_count, st); err != cudaSuccess)
    return cuda_fail(err, "ffn down launch");
  set_path("ffn.forward.tc");
  return E4B_OK;
}

e4b_status e4b_gated_ffn_backward(const uint16_t* x, int64_t M, int64_t ldx, const e4b_gated_ffn* w,
                                  const uint16_t* pre, const uint16_t* dout, uint16_t* dx, uint16_t* dgate_up,
                                  uint16_t* ddown, void* workspace, size_t workspace_bytes, e4b_stream stream) {
  begin_call();
  if (e4b_status s = check_ffn(w, M, ldx, x); s != E4B_OK) return s;
  if (M > 0 && (!pre || !dout)) return fail(E4B_ERR_INVALID_ARGUMENT, "null pre or dout");
  if (!aligned16(pre) || !aligned16(dout) || !aligned16(dx) || !aligned16(dgate_up) || !aligned16(ddown))
    return fail(E4B_ERR_INVALID_ARGUMENT, "pre, dout and the gradients must be 16-byte aligned");
  if (e4b_status s = check_workspace("gated ffn backward", e4b_gated_ffn_backward_workspace_size(M, w), workspace,
                                     workspace_bytes);
      s != E4B_OK)
    return s;
  if (e4b_status s = check_sm100(); s != E4B_OK) return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int H = static_cast<int>(w->H), I = static_cast<int>(w->I), rows = static_cast<int>(M);
  if (M == 0) {
    cudaError_t err = cudaSuccess;
    if (dgate_up) err = cudaMemsetAsync(dgate_up, 0, static_cast<size_t>(2 * w->I) * w->H * 2, st);
    if (ddown && err == cudaSuccess) err = cudaMemsetAsync(ddown, 0, static_cast<size_t>(w->I) * w->H * 2, st);
    if (err != cudaSuccess) return cuda_fail(err, "zero of the weights' gradients");
    set_path("ffn.backward.empty");
    return E4B_OK;
  }
  DeviceInfo di;
  if (cudaError_t err = device_info(&di); err != cudaSuccess) return cuda_fail(err, "device query");
  uint16_t* h = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + kErrBytes);
  uint16_t* dpre = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + forward_bytes(M, I));
  Gemm g{};
  g.name = "ffn.dh";
  g.a = {dout, M, w->H, w->H};
  g.b = {w->down, w->H, w->I, w->I};  // rows of B are the columns of Wd [H, I]
  g.out[0] = {h, M, w->I, w->I};
  g.out[1] = {dpre, M, w->I, 2 * w->I};
  g.out[2] = {dpre + I, M, w->I, 2 * w->I};
  g.p.rows = rows;
  g.p.cols = I;
  g.p.K = H;
  g.p.half = I;
  g.p.act = w->act;
  g.in[0] = {pre, M, w->I, 2 * w->I};
  g.in[1] = {pre + I, M, w->I, 2 * w->I};
  g.p.err = static_cast<int*>(workspace);
  if (cudaError_t err = launch_gemm<false, true, kEpiDglu>(g, di.sm_count, st); err != cudaSuccess)
    return cuda_fail(err, "ffn dh launch");
  // The gradients read what dh writes; the first of them waits for it, the others start behind that one.
  int after = kAfterInput;
  if (dx) {
    Gemm d{};
    d.name = "ffn.dx";
    d.p.after = after;
    after = kAfterNothing;
    d.a = {dpre, M, 2 * w->I, 2 * w->I};
    d.b = {w->gate_up, 2 * w->I, w->H, w->H};
    d.out[0] = {dx, M, w->H, w->H};
    d.p.rows = rows;
    d.p.cols = H;
    d.p.K = 2 * I;
    d.p.err = g.p.err;
    if (cudaError_t err = launch_gemm<false, true, kEpiPlain>(d, di.sm_count, st); err != cudaSuccess)
      return cuda_fail(err, "ffn dx launch");
  }
  if (dgate_up) {
    Gemm d{};
    d.name = "ffn.dgate_up";
    d.p.after = after;
    after = kAfterNothing;
    d.a = {dpre, M, 2 * w->I, 2 * w->I};
    d.b = {x, M, w->H, ldx};
    d.out[0] = {dgate_up, 2 * w->I, w->H, w->H};
    d.p.rows = 2 * I;
    d.p.cols = H;
    d.p.K = rows;
    d.p.err = g.p.err;
    if (cudaError_t err = launch_gemm<true, true, kEpiPlain>(d, di.sm_count, st); err != cudaSuccess)
      return cuda_fail(err, "ffn dgate_up launch");
  }
  if (ddown) {
    Gemm d{};
    d.name = "ffn.ddown";
    d.p.after = after;
    d.a = {dout, M, w->H, w->H};
    d.b = {h, M, w->I, w->I};
    d.out[0] = {ddown, w->H, w->I, w->I};
    d.p.rows = H;
    d.p.cols = I;
    d.p.K = rows;
    d.p.err = g.p.err;
    if (cudaError_t err = launch_gemm<true, true, kEpiPlain>(d, di.sm_count, st); err != cudaSuccess)
      return cuda_fail(err, "ffn ddown launch");
  }
  set_path("ffn.backward.tc");
  return E4B_OK;
}

}  // extern "C"
