// Many rows: W is decoded once into a workspace of MFMA operands, P's rows are
// copied into the same form, and a dense product reads both from there
// (plan_of in rows.hip decides where).
//
// Workspace layout of either side. A "tile" is 16 rows of P or 16 output
// columns, a "step" 32 columns of the contraction; [step][tile][lane][8] bf16
// holds lane (j, g)'s MFMA operand: row or output column 16 tile + j,
// contraction columns 32 step + 8 g .. +7. What a workgroup
// stages per step is then one run of memory on each side: it spreads evenly
// over the memory channels (rows of P as they come are a multiple of 2 KB
// apart for most widths, and a step's bytes of each lie in a few channels), reaches LDS by linear copies and is read
// from there without bank conflicts.
//   forward     output columns = rows of W, contraction = K (gated: the tiles
//               of the gate and of the up matrix alternate)
//   transposed  output columns = columns of W, contraction = N, padded with
//               zeros to a multiple of 64 (two matrices one after the other)
#pragma once

#include "decode.hpp"

namespace trellis {
namespace {

constexpr int kDenseRows = 256;   // rows of a workgroup's tile
constexpr int kDenseStep = 32;    // contraction columns per step
constexpr int kDenseThreads = 512;

// bf16 weight of a window: code * q, or the page's chain where a row's scale
// lies outside the range in which the two agree (see decode.hpp).
__device__ __forceinline__ float window_weight(uint32_t win, float s, float q, float k, bool chain) {
  return chain ? trellis_value(code_of(win)) * s : __builtin_fmaf(code_plus_magic(win), q, k);
}

struct Unpack {
  const uint32_t *codes[2];
  const uint16_t *scales[2];
  uint16_t *w;
  int32_t n, k;
  int32_t steps;         // of the whole contraction
  int32_t first, tiles;  // tiles of this launch: first, number (per matrix)
  int32_t matrices;
};

// Forward: one wave per 16 rows of W and 256-weight block, 8 operands. Bound by
// its writes: K = 5120, N = 17408, k = 4 in 48 us, 223 MB at 4.6 TB/s (a plain
// copy reaches 5.2).
template <int BITS>
__global__ __launch_bounds__(256) void unpack_rows_kernel(Unpack U) {
  constexpr int wpb = 8 * BITS;
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int blocks = U.k >> 8;
  // (at most 2^18 tiles of 2^10 blocks)
  const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int which = blockIdx.y;
  if (id >= (uint32_t)U.tiles * (uint32_t)blocks) return;
  const int tile = (int)(id / (uint32_t)blocks), b = (int)(id - (uint32_t)tile * (uint32_t)blocks);
  const int n = (U.first + tile) * 16 + j, row = n < U.n ? n : U.n - 1;  // columns past N are not stored
  const uint32_t *bw = U.codes[which] + ((int64_t)row * blocks + b) * wpb;
  const float s = bf16_bits_to_f32(U.scales[which][row]);
  float q, kq;
  alu_row_constants(s, q, kq);
  const bool chain = !__all(alu_scale_ok(s));
  const int base = (248 - 8 * g) * BITS, w0 = base >> 5, off = base & 31;
  uint64_t f[8];
#pragma unroll
  for (int st = 0; st < 8; ++st) {
    const int w = w0 - st * BITS, next = w + 1 == wpb ? 0 : w + 1;
    f[st] = (((uint64_t)bw[next] << 32) | bw[w]) >> off;
  }
  const int64_t stride = (int64_t)U.tiles * U.matrices * 64;  // of a step
  bf16x8 *out = reinterpret_cast<bf16x8 *>(U.w) + 8 * b * stride + ((int64_t)tile * U.matrices + which) * 64 + lane;
  // (two loops: a choice at every weight costs more than the weight)
  auto decode = [&](auto chained) {
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      bf16x8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = (__bf16)window_weight((uint32_t)(f[st] >> ((7 - e) * BITS)) & 0xFFFu, s, q, kq, decltype(chained)::value);
      out[st * stride] = v;
    }
  };
  if (chain) decode(std::true_type{});
  else decode(std::false_type{});
}

// Transposed: one wave per step (32 rows of W) and 256-column block. The rows'
// code words go through the wave's LDS (read from memory lane by lane they cost
// a load per two weights); lane (j, g) then decodes, 64 columns at a time,
// columns 4 j .. +3 of rows 8 g .. +7, which is one lane's whole operand for
// each of the four columns. K = 5120, N = 17408, k = 4 in 51 us, 224 MB at 4.4
// TB/s (64 us with the words read by each lane, 87 us before the operands were
// stored a kilobyte at a time).
template <int BITS>
__global__ __launch_bounds__(256) void unpack_columns_kernel(Unpack U) {
  constexpr int wpb = 8 * BITS, kRow = wpb + 4;  // words of a row's block, and in LDS
  __shared__ __attribute__((aligned(16))) uint32_t words[4][32 * kRow];
  __shared__ bf16x8 turn[4][4 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
  const int per = U.steps / U.matrices;  // steps of one matrix
  const int blocks = U.tiles >> 4;       // of 256 columns
  // (at most 2^10 blocks of 2^17 steps)
  const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + wave);
  if (id >= (uint32_t)blocks * (uint32_t)per) return;
  const int which = blockIdx.y;
  const int ks = (int)(id / (uint32_t)blocks), blk = (int)(id - (uint32_t)ks * (uint32_t)blocks);
  const int64_t row_words = (int64_t)(U.k >> 8) * wpb;
  const uint32_t *const base = U.codes[which] + (int64_t)((U.first >> 4) + blk) * wpb;
  u32x4 v[BITS];
#pragma unroll
  for (int i = 0; i < BITS; ++i) {
    const int at = (64 * i + lane) * 4, n = ks * 32 + at / wpb;
    v[i] = *reinterpret_cast<const u32x4 *>(base + (n < U.n ? n : U.n - 1) * row_words + at % wpb);
  }
  float q[8], kq[8], sc[8];
  bool in_range = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int n = ks * 32 + 8 * g + e;
    sc[e] = n < U.n ? bf16_bits_to_f32(U.scales[which][n]) : 0.f;  // rows past N weigh nothing
    alu_row_constants(sc[e], q[e], kq[e]);
    in_range = in_range && alu_scale_ok(sc[e]);
  }
  const bool chain = !__all(in_range);
#pragma unroll
  for (int i = 0; i < BITS; ++i) {
    const int at = (64 * i + lane) * 4;
    *reinterpret_cast<u32x4 *>(&words[wave][at / wpb * kRow + at % wpb]) = v[i];
  }
  bf16x8 *const mine = turn[wave];
  bf16x8 *out = reinterpret_cast<bf16x8 *>(U.w) + (((int64_t)which * per + ks) * U.tiles + 16 * blk) * 64 + lane;
  auto decode = [&](auto chained) {
#pragma unroll
    for (int part = 0; part < 4; ++part) {
      const int pos = (252 - 64 * part - 4 * j) * BITS, w0 = pos >> 5, sh = pos & 31, w1 = w0 + 1 == wpb ? 0 : w0 + 1;
      bf16x8 w[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t *row = &words[wave][(8 * g + e) * kRow];
        const uint32_t f = __builtin_amdgcn_alignbit(row[w1], row[w0], sh);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c][e] = (__bf16)window_weight(__builtin_amdgcn_ubfe(f, (3 - c) * BITS, 12), sc[e], q[e], kq[e], decltype(chained)::value);
      }
      // Through the wave's LDS again, so that each store writes 1 KB in a row:
      // lane (j, g) holds slots 16 g + 4 (j mod 4) .. +3 of tile j / 4.
#pragma unroll
      for (int c = 0; c < 4; ++c) mine[(j >> 2) * 64 + g * 16 + 4 * (j & 3) + c] = w[c];
#pragma unroll
      for (int i = 0; i < 4; ++i) out[(4 * part + i) * 64] = mine[i * 64 + lane];
    }
  };
  if (chain) decode(std::true_type{});
  else decode(std::false_type{});
}

// Eight columns of a row of P; rows past m and columns past `cols` are zero.
// Rows start at multiples of 8 bytes, of 16 where WIDE (cols a multiple of 8).
template <bool WIDE>
__device__ __forceinline__ u32x4 row_vector(const uint16_t *src, int64_t row, int64_t m, int cols, int c) {
  if constexpr (WIDE) return row < m && c < cols ? *reinterpret_cast<const u32x4 *>(src + row * cols + c) : u32x4{0u, 0u, 0u, 0u};
  u32x2 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v[h] = u32x2{0u, 0u};
    if (row < m && c + 4 * h < cols) v[h] = *reinterpret_cast<const u32x2 *>(src + row * cols + c + 4 * h);
  }
  return u32x4{v[0][0], v[0][1], v[1][0], v[1][1]};
}
// Rows of P as operands: one wave per two steps and 16-row tile. 2048 rows of
// 17408 in 23 us, 143 MB at 6.2 TB/s (part of it in the Infinity Cache).
template <bool WIDE>
__global__ __launch_bounds__(256) void pack_rows_kernel(const uint16_t *__restrict__ src, int m, int cols, int tiles,
                                                        int steps, uint16_t *__restrict__ dst) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int pairs = steps >> 1;
  if (id >= (int64_t)tiles * pairs) return;
  const int tile = (int)(id / pairs), step = 2 * (int)(id - (int64_t)tile * pairs);
  u32x4 *out = reinterpret_cast<u32x4 *>(dst) + ((int64_t)step * tiles + tile) * 64 + lane;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    out[(int64_t)h * tiles * 64] = row_vector<WIDE>(src, (int64_t)tile * 16 + j, m, cols, (step + h) * 32 + 8 * g);
}

// The gated block's elementwise gradients (see gated_grad_kernel) as rows and
// as operands: steps 0 .. steps - 1 hold dgate, the next `steps` dup. The
// operands are the rounded gradients: bf16 is what the matrix cores multiply at
// this rate, the rounded ones are outputs anyway, and two halves of each would
// double the product. dx is then off by 1.4 times what one rounding costs (each
// of its 2 N terms by up to 2^-8, of either sign). 2048 rows of 17408 in 112 us:
// 214 MB read and 285 MB written, 4.5 TB/s.
template <bool WIDE>
__global__ __launch_bounds__(256) void gated_grad_pack_kernel(const uint16_t *__restrict__ dh,
                                                              const uint16_t *__restrict__ gate,
                                                              const uint16_t *__restrict__ up, int m, int cols, int tiles,
                                                              int steps, uint16_t *__restrict__ dgate,
                                                              uint16_t *__restrict__ dup, uint16_t *__restrict__ dst) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int pairs = steps >> 1;
  if (id >= (int64_t)tiles * pairs) return;
  const int tile = (int)(id / pairs), step = 2 * (int)(id - (int64_t)tile * pairs);
  u32x4 *out = reinterpret_cast<u32x4 *>(dst) + ((int64_t)step * tiles + tile) * 64 + lane;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = (int64_t)tile * 16 + j;
    const int c = (step + h) * 32 + 8 * g;
    const u32x4 d = row_vector<WIDE>(dh, row, m, cols, c), gv = row_vector<WIDE>(gate, row, m, cols, c), uv = row_vector<WIDE>(up, row, m, cols, c);
    u32x4 pg, pu;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float og[2], ou[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        gated_gradients(bf16_half(d[e], k), bf16_half(gv[e], k), bf16_half(uv[e], k), og[k], ou[k]);
      pg[e] = (uint32_t)bf16_of(og[0]) | ((uint32_t)bf16_of(og[1]) << 16);
      pu[e] = (uint32_t)bf16_of(ou[0]) | ((uint32_t)bf16_of(ou[1]) << 16);
    }
    out[(int64_t)h * tiles * 64] = pg;
    out[(int64_t)(steps + h) * tiles * 64] = pu;
    if constexpr (WIDE) {
      if (row < m && c < cols) {
        *reinterpret_cast<u32x4 *>(dgate + row * cols + c) = pg;
        *reinterpret_cast<u32x4 *>(dup + row * cols + c) = pu;
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (row < m && c + 4 * k < cols) {
        *reinterpret_cast<u32x2 *>(dgate + row * cols + c + 4 * k) = u32x2{pg[2 * k], pg[2 * k + 1]};
        *reinterpret_cast<u32x2 *>(dup + row * cols + c + 4 * k) = u32x2{pu[2 * k], pu[2 * k + 1]};
      }
  }
}

struct Dense {
  const uint16_t *p, *w;   // operands of the rows, and of the columns of this launch
  uint16_t *out, *gate, *up;
  float *partials;         // [splits][m][16 wtiles], where the contraction is split
  int32_t m, steps;        // steps: an even number
  int32_t splits;          // of the contraction
  int32_t width;           // row length of the outputs
  int32_t first;           // first output column of this launch (gated: of one matrix)
  int32_t ptiles, wtiles;  // operand tiles
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
// Waits until at most N of the wave's copies are on their way and its LDS
// reads are done, then for the workgroup.
template <int N>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// LDS buffers of a step: as many as fit in 160 KB, at most 6.
constexpr int dense_step_bytes(int nt, int rt = 4) { return (4 * rt + 2 * nt) * 1024; }
constexpr int dense_buffers(int nt, int rt = 4) {
  return 160 * 1024 / dense_step_bytes(nt, rt) < 6 ? 160 * 1024 / dense_step_bytes(nt, rt) : 6;
}

// One workgroup (8 waves, 4 by rows x 2 by columns): 256 rows by 32 NT
// columns. Wave: 64 rows by 16 NT columns, 4 x NT accumulators. A step's
// operands (32 contraction columns of both sides) are copied into one of S LDS
// buffers, S steps ahead; a wave reads the operands of step s + 1 into
// registers while it multiplies step s. One barrier a step: it says that step
// s + 1 has landed and that step s has been read, so its buffer takes step
// s + S. The operands' roles are W then P, so a lane holds four consecutive
// output columns of one row and stores 8 bytes at a time.
//
// Bound by the matrix cores with the LDS close behind: per step and CU 1024
// clocks of MFMA against about 770 of LDS reads and 260 of LDS writes by the
// copies. Measured, K = 5120, N = 17408: gated, 4096 rows 1.24-1.31 ms, 1.12 to
// 1.18 PFLOP/s (MFMA 52% busy; without the copies 1.03 ms, without the MFMAs 1.0
// ms); 2048 rows 0.33-0.35 ms, transposed 0.33 ms, 1.1 PFLOP/s. A plain library
// product of these sizes reaches 1.21, 0.88 and 1.26 PFLOP/s on the same card,
// 1.42 on 8192 x 8192 x 8192. Two buffers of 64 columns instead of S of 32: 1.40
// ms. Tried and not kept: four waves of 128 x 128 (2.0 ms), a raised wave
// priority around the MFMAs, the reads before the copies, the other order of
// the accumulators (all within 1%).
// Registers: forward with seven and eight column tiles a wave, the adapters'
// term does not fit beside the accumulators, and its operands go through 104 and
// 180 bytes of scratch memory a lane, in and around the term's loop (once per
// named adapter and 32 rank columns); the steps use none.
// Where a lane's sums lie: lane (j, g), accumulator (r, i): row row0 + 16 r + j,
// operand tile tile0 + i, its columns 4 g .. +3.
struct DenseAt {
  int row0, tile0, split;
};
// between(at): work of the wave's own while the first steps are on their way.
// RT: row tiles of a wave, 4, or 3 for 192 rows a workgroup.
template <int NT, int RT = 4, typename Between>
__device__ __forceinline__ DenseAt dense_sums(const Dense &D, f32x4 (&acc)[RT][NT], Between between) {
  constexpr int kRows = 64 * RT, kA = kRows / 16 * 1024, kBuffer = dense_step_bytes(NT, RT), S = dense_buffers(NT, RT);
  constexpr int kCopies = kBuffer / 1024;  // of 1 KB
  constexpr int kMost = (kCopies + 7) / 8, kFull = kCopies % 8 == 0 ? 8 : kCopies % 8;  // waves 0 .. kFull - 1 copy kMost, the others one less
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 3, wn = wave >> 2;
  // Consecutive workgroups go to the eight XCDs in turn: each XCD gets a run
  // of consecutive tiles, row tiles first, whose operands its L2 shares.
  const int tiles = D.mtiles * D.ntiles, total = tiles * D.splits, each = total >> 3, rest = total & 7;
  const int xcd = blockIdx.x & 7, seq = blockIdx.x >> 3;
  const int id = xcd * each + (xcd < rest ? xcd : rest) + seq;
  const int split = id / tiles, tn = (id - split * tiles) / D.mtiles, tm = id - split * tiles - tn * D.mtiles;
  // this workgroup's steps: an even number from an even one on
  const int begin = 2 * (int)((int64_t)(D.steps >> 1) * split / D.splits);
  const int steps = 2 * (int)((int64_t)(D.steps >> 1) * (split + 1) / D.splits) - begin;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds;

  // Copy c of a step (1 KB): the first kA / 1024 are P's. Tiles past the last
  // repeat it (what they feed is not stored).
  const int atiles = D.ptiles - tm * (kRows / 16), btiles = D.wtiles - tn * 2 * NT;
  const unsigned char *const pa = reinterpret_cast<const unsigned char *>(D.p) + (int64_t)tm * (kRows / 16) * 1024;
  const unsigned char *const pb = reinterpret_cast<const unsigned char *>(D.w) + (int64_t)tn * 2 * NT * 1024;
  const int64_t astride = (int64_t)D.ptiles * 1024, bstride = (int64_t)D.wtiles * 1024;
  // (s counts from `begin`)
  auto stage = [&](int s, uint32_t buffer) {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int c = wave + 8 * i;
      if (kFull == 8 || i < kMost - 1 || wave < kFull) {
        const bool is_a = kA % 8192 == 0 ? i < kA / 8192 : c < kA / 1024;
        const int t = is_a ? c : c - kA / 1024, have = is_a ? atiles : btiles;
        const unsigned char *src = is_a ? pa + (begin + s) * astride : pb + (begin + s) * bstride;
        copy_to_lds(lds0 + buffer + (uint32_t)(c * 1024), (uint32_t)lane * 16, src + (t < have ? t : have - 1) * 1024);
      }
    }
  };
  // All but the last N steps' copies of this wave have landed, workgroup-wide.
  auto landed = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (kFull == 8 || wave < kFull) step_barrier<N * kMost>();
    else step_barrier<N *(kMost - 1)>();
  };

#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const DenseAt at{tm * kRows + 16 * RT * wm, tn * 2 * NT + wn * NT, split};
#pragma unroll
  for (int b = 0; b < S; ++b)
    if (b < steps) stage(b, b * kBuffer);
  between(at);
  struct Operands {
    bf16x8 a[RT], b[NT];
  };
  auto read = [&](Operands &O, uint32_t buffer) {
    const unsigned char *const buf = lds + buffer + lane * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) O.b[i] = *reinterpret_cast<const bf16x8 *>(buf + kA + (wn * NT + i) * 1024);
#pragma unroll
    for (int i = 0; i < RT; ++i) O.a[i] = *reinterpret_cast<const bf16x8 *>(buf + (RT * wm + i) * 1024);
  };
  auto multiply = [&](const Operands &O) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(O.b[i], O.a[r], acc[r][i], 0, 0, 0);
  };
  Operands X, Y;
  uint32_t now = 0;  // buffer of step s
  step_barrier<0>();
  read(X, 0);
  auto step = [&](int s, const Operands &A, Operands &B) {
    if (s + S - 1 < steps) landed(std::integral_constant<int, S - 2>{});
    else step_barrier<0>();
    if (s + S < steps) stage(s + S, now);
    now = now == (S - 1) * kBuffer ? 0 : now + kBuffer;
    read(B, now);  // (past the last step: a buffer's old operands, not used)
    multiply(A);
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, X, Y);
    step(s + 1, Y, X);
  }
  return at;
}

template <int NT, bool GATED, bool T>
__global__ __launch_bounds__(kDenseThreads) void dense_kernel(Dense D) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  f32x4 acc[4][NT];
  const DenseAt at = dense_sums<NT>(D, acc, [&](const DenseAt &at) {
    const int row0 = at.row0, tile0 = at.tile0, split = at.split;
    if constexpr (!GATED) {
      // The adapters' term first, while the first steps are on their way: lane l
      // looks up row row0 + l; for every adapter that the wave's rows name, the
      // products are kept only in the rows that name it (see low_rank_tiles).
      if (D.low.rank > 0 && split == 0) {
        int idx = row0 + lane < D.m ? D.low.index[row0 + lane] : -1;
        if (idx >= D.low.count) idx = -1;
        uint64_t left = __ballot(idx >= 0);
        while (left) {
          const int a = __builtin_amdgcn_readlane(idx, __builtin_ctzll(left));
          const uint64_t rows = __ballot(idx == a);
          left &= ~rows;
          for (int r0 = 8 * g; r0 < D.low.rank_p + 8 * g; r0 += 32) {
            // The factor's operands, each loaded while the one before it is
            // multiplied (the barriers keep the loads in flight to two tiles').
            // Offsets past the adapter's block, and those of rank columns past
            // the rank, read as zero.
            const uint32_t block = (uint32_t)D.low.rank * (uint32_t)D.width * 2;
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint16_t *>(D.low.factor + (int64_t)a * D.low.rank * D.width), (short)0, (int)block, kRawBuffer);
            const uint32_t col0 = (uint32_t)(D.first + tile0 * 16 + j);
            auto fetch = [&](int i) {
              if constexpr (T) {
                bf16x8 f;
                const uint32_t o = ((uint32_t)r0 * (uint32_t)D.width + col0) * 2 + 32u * (uint32_t)i;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  f[e] = __builtin_bit_cast(__bf16, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                                                        rs, o + (uint32_t)e * (uint32_t)D.width * 2, 0, 0));
                return f;
              } else {
                const uint32_t o = ((col0 + 16u * (uint32_t)i) * (uint32_t)D.low.rank + (uint32_t)r0) * 2;
                if ((D.low.rank & 7) == 0)
                  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rs, r0 < D.low.rank ? o : 0x80000000u, 0, 0));
                bf16x8 f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  f[e] = __builtin_bit_cast(__bf16, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                                                        rs, r0 + e < D.low.rank ? o + 2u * (uint32_t)e : 0x80000000u, 0, 0));
                return f;
              }
            };
            // (two row tiles at a time: t's operands for four take too many registers)
#pragma unroll
            for (int rp = 0; rp < 4; rp += 2) {
              bf16x8 hi[2], lo[2];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int row = row0 + 16 * (rp + r) + j;
                const f32x4 *tp = reinterpret_cast<const f32x4 *>(D.low.t + (int64_t)(row < D.m ? row : D.m - 1) * D.low.rank_p + r0);
                const f32x4 t0 = tp[0], t1 = tp[1];
                halves({t0[0], t0[1], t0[2], t0[3], t1[0], t1[1], t1[2], t1[3]}, hi[r], lo[r]);
              }
              bf16x8 next = fetch(0);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const bf16x8 f = next;
                __builtin_amdgcn_sched_barrier(0);
                if (i + 1 < NT) next = fetch(i + 1);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  f32x4 d = {0.f, 0.f, 0.f, 0.f};
                  d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, hi[r], d, 0, 0, 0);
                  d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, lo[r], d, 0, 0, 0);
                  const bool mine = (rows >> (16 * (rp + r) + j)) & 1;
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[rp + r][i][e] += mine ? d[e] : 0.f;
                }
              }
            }
          }
        }
      }
    }
  });
  const int row0 = at.row0, tile0 = at.tile0, split = at.split;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = row0 + 16 * r + j;
    if (row >= D.m) continue;
    if (D.splits > 1) {
      float *const q = D.partials + ((int64_t)split * D.m + row) * (16 * (int64_t)D.wtiles) + tile0 * 16 + 4 * g;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (tile0 + i < D.wtiles) *reinterpret_cast<f32x4 *>(q + 16 * i) = acc[r][i];
      continue;
    }
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

// Sums of the splits (where the tiles alone do not fill the card: 257 rows of
// K = 5120 have 40 to 80), in order, rounded (gated: gate and up first, then the
// product): four output columns a thread.
template <bool GATED>
__global__ __launch_bounds__(256) void join_splits_kernel(Dense D) {
  const int quads = 4 * D.wtiles / (GATED ? 2 : 1);  // per row
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)D.m * quads) return;
  const int64_t row = id / quads;
  const int c = (int)(id - row * quads) * 4;
  if (D.first + c >= D.width) return;
  const float *q = D.partials + row * (16 * (int64_t)D.wtiles) + (GATED ? (c >> 4) * 32 + (c & 15) : c);
  const int64_t plane = (int64_t)D.m * 16 * D.wtiles;
  f32x4 v = {0.f, 0.f, 0.f, 0.f}, u = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < D.splits; ++s) {
    v += *reinterpret_cast<const f32x4 *>(q + s * plane);
    if constexpr (GATED) u += *reinterpret_cast<const f32x4 *>(q + s * plane + 16);
  }
  const int64_t o = row * D.width + D.first + c;
  if constexpr (GATED) {
    f32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = silu_mul(v[e], u[e]);
    store4(D.out + o, h);
    if (D.gate) store4(D.gate + o, v);
    if (D.up) store4(D.up + o, u);
  } else {
    store4(D.out + o, v);
  }
}

}  // namespace
}  // namespace trellis
