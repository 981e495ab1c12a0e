// Many rows: W is decoded once into a workspace of MFMA operands, and a dense
// product reads it from there (rows.hip decides from how many rows on).
//
// Workspace layout. A "tile" is 16 output columns of the product, a "kstep" 32
// columns of its contraction; [tile][kstep][lane][8] bf16 holds lane (j, g)'s
// MFMA operand, W at output column 16 tile + j and contraction columns
// 32 kstep + 8 g .. +7, so a wave's operand is 1 KB in a row: it reaches LDS
// by linear copies and is read from there without bank conflicts.
//   forward     output columns = rows of W, contraction = K (gated: the tiles
//               of the gate and of the up matrix alternate)
//   transposed  output columns = columns of W, contraction = N, padded with
//               zeros to whole steps of 64 (two matrices one after the other)
#pragma once

#include "decode.hpp"

namespace trellis {
namespace {

constexpr int kDenseRows = 256;   // rows of a workgroup's tile
constexpr int kDenseStep = 64;    // contraction columns per step
constexpr int kDenseThreads = 512;

// bf16 weight of a window: code * q where the row's scale allows it, else the
// page's chain (see decode.hpp).
__device__ __forceinline__ float window_weight(uint32_t win, float s, float q, float k, bool exact) {
  return exact ? trellis_value(code_of(win)) * s : __builtin_fmaf(code_plus_magic(win), q, k);
}

struct Unpack {
  const uint32_t *codes[2];
  const uint16_t *scales[2];
  uint16_t *w;
  int32_t n, k;
  int32_t ksteps;   // of the whole contraction
  int32_t first, tiles;  // tiles of this launch: first, number (per matrix)
  int32_t matrices;
};

// Forward: one wave per 16 rows of W and 256-weight block, 8 operands.
template <int BITS>
__global__ __launch_bounds__(256) void unpack_rows_kernel(Unpack U) {
  constexpr int wpb = 8 * BITS;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int blocks = U.k >> 8;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int which = blockIdx.y;
  if (id >= (int64_t)U.tiles * blocks) return;
  const int tile = (int)(id / blocks), b = (int)(id - (int64_t)tile * blocks);
  const int n = (U.first + tile) * 16 + j, row = n < U.n ? n : U.n - 1;  // columns past N are not stored
  const uint32_t *bw = U.codes[which] + ((int64_t)row * blocks + b) * wpb;
  const float s = bf16_bits_to_f32(U.scales[which][row]);
  float q, kq;
  alu_row_constants(s, q, kq);
  const bool exact = !__all(alu_scale_ok(s));
  const int base = (248 - 8 * g) * BITS, w0 = base >> 5, off = base & 31;
  uint64_t f[8];
#pragma unroll
  for (int st = 0; st < 8; ++st) {
    const int w = w0 - st * BITS, next = w + 1 == wpb ? 0 : w + 1;
    f[st] = (((uint64_t)bw[next] << 32) | bw[w]) >> off;
  }
  bf16x8 *out = reinterpret_cast<bf16x8 *>(U.w) +
                (((int64_t)tile * U.matrices + which) * U.ksteps + b * 8) * 64 + lane;
#pragma unroll
  for (int st = 0; st < 8; ++st) {
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = (__bf16)window_weight((uint32_t)(f[st] >> ((7 - e) * BITS)) & 0xFFFu, s, q, kq, exact);
    out[st * 64] = v;
  }
}

// Transposed: one wave per kstep (32 rows of W) and 64 columns; lane (j, g)
// decodes columns 4 j .. +3 of rows 8 g .. +7 and so holds, for each of the
// four columns, one lane's whole operand.
template <int BITS>
__global__ __launch_bounds__(256) void unpack_columns_kernel(Unpack U) {
  __shared__ bf16x8 turn[4][4 * 64];
  constexpr int wpb = 8 * BITS;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int per = U.ksteps / U.matrices;  // ksteps of one matrix
  const int groups = U.tiles >> 2;        // of 64 columns
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= (int64_t)groups * per) return;
  const int which = blockIdx.y;
  const int ks = (int)(id / groups), grp = (int)(id - (int64_t)ks * groups);
  const int col = (U.first + 4 * grp) * 16 + 4 * j;  // first of the lane's four columns
  const int pos = (252 - (col & 255)) * BITS, w0 = pos >> 5, sh = pos & 31, w1 = w0 + 1 == wpb ? 0 : w0 + 1;
  const int64_t row_words = (int64_t)(U.k >> 8) * wpb, blk = (int64_t)(col >> 8) * wpb;
  bf16x8 v[4];
  uint32_t f[8];
  float s[8];
  bool in_range = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int n = ks * 32 + 8 * g + e, row = n < U.n ? n : U.n - 1;
    const uint32_t *bw = U.codes[which] + row * row_words + blk;
    f[e] = __builtin_amdgcn_alignbit(bw[w1], bw[w0], sh);
    s[e] = n < U.n ? bf16_bits_to_f32(U.scales[which][row]) : 0.f;
    in_range = in_range && alu_scale_ok(s[e]);
  }
  const bool exact = !__all(in_range);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float q, kq;
    alu_row_constants(s[e], q, kq);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c][e] = (__bf16)window_weight((f[e] >> ((3 - c) * BITS)) & 0xFFFu, s[e], q, kq, exact);
  }
  // Through the wave's own LDS, so that each store writes 1 KB in a row: lane
  // (j, g) holds slots 16 g + 4 (j mod 4) .. +3 of tile j / 4.
  bf16x8 *const mine = turn[threadIdx.x >> 6];
#pragma unroll
  for (int c = 0; c < 4; ++c) mine[(j >> 2) * 64 + g * 16 + 4 * (j & 3) + c] = v[c];
  bf16x8 *out = reinterpret_cast<bf16x8 *>(U.w) + ((int64_t)(4 * grp) * U.ksteps + (int64_t)which * per + ks) * 64 + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[(int64_t)i * U.ksteps * 64] = mine[i * 64 + lane];
}

// Rows padded with zeros to whole contraction steps, four elements a thread.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t *__restrict__ src, int64_t rows, int cols,
                                                       int padded, uint16_t *__restrict__ dst) {
  const int quads = padded >> 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * quads) return;
  const int64_t row = i / quads;
  const int c = (int)(i - row * quads) * 4;
  const uint2 z = {0u, 0u};
  reinterpret_cast<uint2 *>(dst)[i] = c < cols ? *reinterpret_cast<const uint2 *>(src + row * cols + c) : z;
}

struct Dense {
  const uint16_t *p, *p2;  // [m, cols], cols a multiple of 64; p2 from step steps1 on
  const uint16_t *w;       // operands, from tile 0 of this launch on
  uint16_t *out, *gate, *up;
  int32_t m, cols, steps, steps1;
  int32_t width;           // row length of the outputs
  int32_t first;           // first output column of this launch (gated: of one matrix)
  int32_t tiles;           // operand tiles of this launch
  int32_t mtiles, ntiles;  // workgroup tiles
  LowRank low;
};

// Direct copies from memory to LDS, 16 bytes a lane to base + 16 lane. Written
// as inline assembly: the compiler would wait for every copy before each LDS
// read. The copies are waited for explicitly (step_barrier); s_nop 4 gives the
// wait states after a vector write of the scalar operands and of M0.
__device__ __forceinline__ void copy_to_lds(uint32_t lds, uint32_t off, const void *base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One workgroup (8 waves, 4 by rows x 2 by columns): 256 rows by 32 NT
// columns. Wave: 64 rows by 16 NT columns, 4 x NT accumulators. Each step
// stages 64 contraction columns of both operands in one of two LDS buffers
// while the other is multiplied. A row's eight 16-byte vectors are stored
// permuted by (row / 2) mod 8, which spreads the sixteen rows that a wave
// reads together over all banks (the copies can only write in lane order, so
// the permutation is made in the addresses they read from). The operands'
// roles are W then P, so a lane holds four consecutive output columns of one
// row and stores 8 bytes at a time.
template <int NT, bool GATED, bool T>
__global__ __launch_bounds__(kDenseThreads) void dense_kernel(Dense D) {
  constexpr int kA = kDenseRows * kDenseStep * 2, kB = 2 * NT * 2048, kBuffer = kA + kB;
  constexpr int kCopies = kB / 1024;  // of 1 KB
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 3, wn = wave >> 2;
  const int j = lane & 15, g = lane >> 4;
  // Consecutive workgroups go to the eight XCDs in turn: each XCD gets a run
  // of consecutive tiles, row tiles first, whose operands its L2 shares.
  const int total = D.mtiles * D.ntiles, each = total >> 3, rest = total & 7;
  const int xcd = blockIdx.x & 7, seq = blockIdx.x >> 3;
  const int id = xcd * each + (xcd < rest ? xcd : rest) + seq;
  const int tn = id / D.mtiles, tm = id - tn * D.mtiles;
  const int m0 = tm * kDenseRows;
  const int ksteps = 2 * D.steps;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds;

  // P: copy i of a wave (of 4) takes rows 8 (4 wave + i) .. +7.
  uint32_t aoff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (4 * wave + i) + (lane >> 3);
    const int row = m0 + r < D.m ? r : D.m - 1 - m0;  // rows past m feed outputs that are not stored
    aoff[i] = (uint32_t)row * (uint32_t)(D.cols * 2) + (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) * 16);
  }
  const unsigned char *const pa = reinterpret_cast<const unsigned char *>(D.p + (int64_t)m0 * D.cols);
  const unsigned char *const pa2 = reinterpret_cast<const unsigned char *>(D.p2 + (int64_t)m0 * D.cols);
  const unsigned char *const pb = reinterpret_cast<const unsigned char *>(D.w) + (int64_t)tn * 2 * NT * ksteps * 1024;
  const int btiles = D.tiles - tn * 2 * NT;  // of this workgroup, at least 1
  auto stage = [&](int s) {
    const uint32_t at = lds0 + (uint32_t)((s & 1) * kBuffer);
    const unsigned char *a = s < D.steps1 ? pa + (int64_t)s * 128 : pa2 + (int64_t)(s - D.steps1) * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) copy_to_lds(at + (uint32_t)((4 * wave + i) * 1024), aoff[i], a);
#pragma unroll
    for (int i = 0; i < (kCopies + 7) / 8; ++i) {
      const int c = wave + 8 * i;
      if (kCopies % 8 == 0 || c < kCopies) {
        // tiles past the last repeat it (their columns are not stored)
        const int t = (c >> 1) < btiles ? c >> 1 : btiles - 1;
        copy_to_lds(at + kA + (uint32_t)(c * 1024), (uint32_t)lane * 16,
                    pb + ((int64_t)t * ksteps + 2 * s + (c & 1)) * 1024);
      }
    }
  };

  f32x4 acc[4][NT];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t arow = (uint32_t)((64 * wm + j) * 128), sw = (uint32_t)((j >> 1) & 7);
  stage(0);
  step_barrier();
  for (int s = 0; s < D.steps; ++s) {
    if (s + 1 < D.steps) stage(s + 1);
    const unsigned char *const buf = lds + (s & 1) * kBuffer;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8 a[4], b[NT];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = *reinterpret_cast<const bf16x8 *>(buf + arow + i * 2048 + ((uint32_t)(4 * kk + g) ^ sw) * 16);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        b[i] = *reinterpret_cast<const bf16x8 *>(buf + kA + ((wn * NT + i) * 2 + kk) * 1024 + lane * 16);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i], a[r], acc[r][i], 0, 0, 0);
    }
    step_barrier();
  }

  // Lane (j, g), accumulator (r, i): row m0 + 64 wm + 16 r + j, operand tile
  // tn 2 NT + wn NT + i, its columns 4 g .. +3.
  const int tile0 = tn * 2 * NT + wn * NT;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = m0 + 64 * wm + 16 * r + j;
    if constexpr (!GATED) {
      if (D.low.rank > 0) {
        const int rowc = row < D.m ? row : D.m - 1;
        int idx = row < D.m ? D.low.index[row] : -1;
        if (idx >= D.low.count) idx = -1;
        uint64_t left = __ballot(idx >= 0) & 0xFFFFull;
        while (left) {
          const int a = __builtin_amdgcn_readlane(idx, __builtin_ctzll(left));
          left &= ~__ballot(idx == a);
          for (int i = 0; i < NT; ++i) {
            const int col = D.first + (tile0 + i) * 16 + j;
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            for (int r0 = 8 * g; r0 < D.low.rank_p + 8 * g; r0 += 32) {
              const float *tp = D.low.t + (int64_t)rowc * D.low.rank_p + r0;
              bf16x8 hi, lo, f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                hi[e] = (__bf16)tp[e];
                lo[e] = (__bf16)(tp[e] - (float)hi[e]);
                uint16_t v = 0;
                if (col < D.width && r0 + e < D.low.rank)
                  v = T ? D.low.factor[((int64_t)a * D.low.rank + r0 + e) * D.width + col]
                        : D.low.factor[((int64_t)a * D.width + col) * D.low.rank + r0 + e];
                f[e] = __builtin_bit_cast(__bf16, v);
              }
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, hi, d, 0, 0, 0);
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, lo, d, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < NT; ++q)
              if (q == i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][q][e] += idx == a ? d[e] : 0.f;
          }
        }
      }
    }
    if (row >= D.m) continue;
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < NT; i += 2) {
        const int col = D.first + ((tile0 + i) >> 1) * 16 + 4 * g;
        if (col >= D.width) continue;
        const int64_t o = (int64_t)row * D.width + col;
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = silu_mul(acc[r][i][e], acc[r][i + 1][e]);
        store4(D.out + o, h);
        if (D.gate) store4(D.gate + o, acc[r][i]);
        if (D.up) store4(D.up + o, acc[r][i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int col = D.first + (tile0 + i) * 16 + 4 * g;
        if (col < D.width) store4(D.out + (int64_t)row * D.width + col, acc[r][i]);
      }
    }
  }
}

}  // namespace
}  // namespace trellis
