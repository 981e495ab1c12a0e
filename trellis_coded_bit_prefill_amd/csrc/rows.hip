// Fine-tuned packed Trellis layers at any number of rows, gfx950: low-rank
// adapters beside the shared projection, the gated block, and the backward
// passes of both.
//
// Every entry point here contains one product of a dense bf16 matrix with a
// packed matrix W[N, K], in one of two directions:
//   forward     out[M, N] = P[M, K] . W^T   (contraction over K)
//   transposed  out[M, K] = P[M, N] . W     (contraction over N)
// and product_kernel computes both: a workgroup owns a tile of rows of P and a
// group of output columns, stages P in LDS one step of the contraction at a
// time, and its waves decode the weights straight into MFMA operand registers,
// once per tile of rows. Where decoding W once for all rows takes less, it goes
// through memory instead (dense.hpp; plan_of chooses).
//
// The low-rank parts are sums of their own: t = x A^T and u = dout B
// (shrink_kernel), added to the product before it is rounded, and the
// gradients of A and B (outer_kernel).
//
// Build flags that matter for exactness: -ffp-contract=off.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <map>
#include <mutex>
#include <new>
#include <thread>
#include <type_traits>
#include <utility>

#include "decode.hpp"
#include "trellis.h"
#include "trellis_testing.h"

namespace trellis {
namespace {

constexpr int kThreads = 512;       // product_kernel: 8 waves
constexpr int kStep = 256;          // contraction columns staged per step
constexpr int kStride = kStep * 2 + 16;  // bytes per staged row (16 B of padding spread the rows over the banks)
constexpr int kRedStride = 128 + 4;  // floats per row of the reduction tile (at most 128 columns at a time)
constexpr int kTableBytes = 4096 * 2;
constexpr int kRawBuffer = 0x00020000;  // gfx9 raw-buffer descriptor word 3
constexpr int kSc1 = 16;                // cache policy: the level that is coherent across the XCDs' L2s
static_assert(2 * 16 * kRedStride * 4 == 2 * 16 * kStride, "the reduction tile reuses the staged rows' space");

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint16_t bf16_of(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// The adapter term's operands. index[m] outside [0, count): the row has no
// adapter. t is float32 [m, rank_p], rank_p = rank rounded up to 32, zero past
// the rank, the gain already in it.
struct LowRank {
  const int32_t *index;
  const uint16_t *factor;  // forward: B[count, N, rank]; transposed: A[count, rank, K]
  const float *t;
  int32_t count, rank, rank_p;
};

struct Product {
  const uint16_t *p, *p2;         // [m, C]; transposed: p2 is the second matrix's rows, or null
  const uint32_t *codes, *codes2;  // codes2: gated (up), or transposed with two matrices
  const uint16_t *scales, *scales2;
  uint16_t *out, *gate, *up;       // gate, up: gated only, null where they are not kept
  float *partials;
  uint32_t *counters;
  int32_t units_q, units_r;  // units (tiles * steps) of a workgroup: units_q, the first units_r one more
  int32_t parts;             // > 0: instead, each tile's steps are split over this many workgroups
  int32_t m, n, k;
  int32_t groups;    // groups of output columns
  int32_t steps;     // contraction steps of a tile (all matrices)
  int32_t steps1;    // those of the first matrix
  LowRank low;
};

// Eight float32 factors of a matrix product, each as the sum of two bf16
// numbers of one sign: the upper half of its bits, and the rest rounded (off by
// at most 2^-16 of v: a half step of the rest, which is below 2^-7). Cut
// instead of rounded, and without a zero or a NaN as the rest of what is not
// zero, so that an infinity on either side of the product gives the infinity
// that v times it gives: of opposite signs the halves' infinities would cancel
// to a NaN. (Below 2^-96 the rest of a v that is one bf16 number already
// vanishes, and an infinity times it gives a NaN.)
__device__ __forceinline__ void halves(const float (&v)[8], bf16x8 &hi, bf16x8 &lo) {
  u32x4 top;
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    top[e / 2] = __builtin_amdgcn_perm(__float_as_uint(v[e + 1]), __float_as_uint(v[e]), 0x07060302u);
  hi = __builtin_bit_cast(bf16x8, top);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u), rest = v[e] - t;
    lo[e] = (__bf16)(fabsf(rest) > 0.f ? rest : t * 0x1p-30f);
  }
}

// The adapters' term of TILES 16-row tiles (every second one from m0 on) and a
// wave's NT column tiles: for every adapter that the rows name, the product of
// t's rows (split in two bf16 numbers) with the factor,
// kept only in the rows that name it, so an adapter's infinities and NaNs stay
// in its own rows. Several adapters' operands are loaded before the first is
// multiplied: one at a time cost about a microsecond each.
// load(a, r0, w): the NT operands for rank columns r0 .. +7.
template <int TILES, int NT, typename Load>
__device__ __forceinline__ void low_rank_tiles(const LowRank &L, int m, int m0, int lane, f32x4 (&sum)[TILES][NT], Load load) {
  constexpr int B = NT == 4 ? 2 : 4;  // adapters at a time
  const int j = lane & 15, g = lane >> 4;
  // lane l: the adapter of row l mod 16 of tile l / 16 (of the wave's)
  const int look = m0 + 32 * (lane >> 4) + j;
  int idx = lane < 16 * TILES && look < m ? L.index[look] : -1;
  if (idx >= L.count) idx = -1;
  const uint64_t named = __ballot(idx >= 0);
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int i = 0; i < NT; ++i) sum[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < L.rank_p; r0 += 32) {
    f32x4 tv[TILES][2];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int row = m0 + 32 * t + j;
      const float *tp = L.t + (int64_t)(row < m ? row : m - 1) * L.rank_p + r0 + 8 * g;
      tv[t][0] = *reinterpret_cast<const f32x4 *>(tp);
      tv[t][1] = *reinterpret_cast<const f32x4 *>(tp + 4);
    }
    for (uint64_t left = named; left;) {
      uint64_t rows[B];
      bf16x8 w[B][NT];
      int a = 0;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        rows[b] = 0;  // none left: the operands again, for no row
        if (left) {
          a = __builtin_amdgcn_readlane(idx, __builtin_ctzll(left));
          rows[b] = __ballot(idx == a);
          left &= ~rows[b];
        }
        load(a, r0 + 8 * g, w[b]);
      }
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        bf16x8 hi, lo;
        halves({tv[t][0][0], tv[t][0][1], tv[t][0][2], tv[t][0][3], tv[t][1][0], tv[t][1][1], tv[t][1][2], tv[t][1][3]}, hi, lo);
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint32_t of = (uint32_t)(rows[b] >> (16 * t)) & 0xFFFFu;
          if (of == 0) continue;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, w[b][i], d, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, w[b][i], d, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[t][i][e] += (of >> (4 * g + e)) & 1 ? d[e] : 0.f;
          }
        }
      }
    }
  }
}

// ---- decoding in the product kernel ------------------------------------------
// Half of the weights go through an LDS table (window -> float16 code, one
// gather and about 3 VALU operations a weight), half through the hash on the
// ALU (about 5.5): gathers and VALU work then run side by side. A wave whose
// rows' scales are not all in the range where code * q is exact takes the
// page's chain for all of them.
__device__ __forceinline__ uint32_t table_code(const unsigned char *table, uint32_t addr) {
  return *reinterpret_cast<const uint16_t *>(table + addr);
}

// Forward lane: weights 8 u .. 8 u + 7 (u = 0 .. 3) of its 32, weight i at
// local bit (31 - i) * BITS of d.
template <int BITS, int U, int... S>
__device__ __forceinline__ void group_addresses(const uint32_t (&d)[BITS + 1], uint32_t (&a)[8],
                                                std::integer_sequence<int, S...>) {
  ((a[S] = win_xa<(31 - 8 * U - S) * BITS, 1>(d)), ...);
}
template <int BITS, int U, int... S>
__device__ __forceinline__ bf16x8 group_hashed(const uint32_t (&d)[BITS + 1], float q, float k, std::integer_sequence<int, S...>) {
  const float f[8] = {__builtin_fmaf(code_plus_magic(win12<(31 - 8 * U - S) * BITS>(d)), q, k)...};
  bf16x8 w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = (__bf16)f[i];
  return w;
}
template <int BITS, int U, int... S>
__device__ __forceinline__ bf16x8 group_chain(const uint32_t (&d)[BITS + 1], float s, std::integer_sequence<int, S...>) {
  const float f[8] = {(trellis_value(code_of(win12<(31 - 8 * U - S) * BITS>(d))) * s)...};
  bf16x8 w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = (__bf16)f[i];
  return w;
}
using Eight = std::make_integer_sequence<int, 8>;

// Codes of group U, gathered from the table. For k = 4 the windows of weights
// i and i + 4 are 16 bits apart and come out of one shifted word.
template <int O, int N>
__device__ __forceinline__ void pair_addresses(const uint32_t (&d)[N], uint32_t mask, uint32_t &low, uint32_t &high) {
  constexpr int sh = O - 1, w = sh < 0 ? 0 : sh >> 5, r = sh & 31;
  uint32_t v;
  if constexpr (sh < 0) v = d[0] << 1;
  else if constexpr (r == 0) v = d[w];
  else v = __builtin_amdgcn_alignbit(d[w + 1], d[w], r);
  low = v & 0x1FFEu;
  high = and_hi16(v, mask);
}
template <int BITS, int U>
__device__ __forceinline__ void gather_codes(const uint32_t (&d)[BITS + 1], const unsigned char *table, uint32_t mask,
                                             uint32_t (&r)[8]) {
  uint32_t a[8];
  if constexpr (BITS == 4) {
    pair_addresses<(31 - 8 * U - 4) * 4>(d, mask, a[4], a[0]);
    pair_addresses<(31 - 8 * U - 5) * 4>(d, mask, a[5], a[1]);
    pair_addresses<(31 - 8 * U - 6) * 4>(d, mask, a[6], a[2]);
    pair_addresses<(31 - 8 * U - 7) * 4>(d, mask, a[7], a[3]);
  } else {
    group_addresses<BITS, U>(d, a, Eight{});
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = table_code(table, a[e]);
}
__device__ __forceinline__ bf16x8 gathered_weights(const uint32_t (&r)[8], float q) {
  bf16x8 w;
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = (__bf16)mix_lo(r[e], q);
  return w;
}
// A workgroup barrier for LDS data: global loads stay in flight across it
// (the compiler's own barrier waits for them).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

enum Kind { kForward = 0, kGated = 1, kTransposed = 2 };

// h = silu(gate) * up in float32, rounded once by the caller.
__device__ __forceinline__ float silu_mul(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// Its gradients: dup = dh silu(gate), dgate = dh up s (1 + gate (1 - s)), s = sigmoid(gate).
__device__ __forceinline__ void gated_gradients(float dh, float gate, float up, float &dgate, float &dup) {
  const float s = 1.0f / (1.0f + expf(-gate));
  dup = dh * gate * s;
  dgate = dh * up * s * (1.0f + gate * (1.0f - s));
}
// The low (k = 0) or high bf16 of a word.
__device__ __forceinline__ float bf16_half(uint32_t v, int k) { return __uint_as_float(k ? v & 0xFFFF0000u : v << 16); }

// Four floats a time, four output columns: rounded and stored (N and K are
// multiples of 4, rows start at multiples of 8 bytes).
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v) {
  typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<u16x4 *>(p) = u16x4{bf16_of(v[0]), bf16_of(v[1]), bf16_of(v[2]), bf16_of(v[3])};
}

}  // namespace
}  // namespace trellis

#include "dense.hpp"

namespace trellis {
namespace {

// One tile: 16 MT rows of P by a group of output columns. 8 waves.
//   forward     group = 64 NT rows of W; wave (wn, wk): rows 16 NT wn .. (NT
//               tiles of 16), half wk of each 256-weight block
//   gated       group = 64 rows of both matrices; wave (wn, wk): rows 16 wn .. +15
//               of the gate (tile 0) and of the up matrix (tile 1)
//   transposed  group = one 256-column block; wave (wn, wk): columns 64 wn .. +63
//               as four 16-column tiles (tile e: columns 4 j + e), rows
//               128 wk .. +127 of each 256-row step
// The units (tile, step) are split evenly over the workgroups, or each tile over
// the same number of them (see shape_of); a tile that several share goes through `partials`, summed in a fixed order by the
// workgroup that arrives last. Code words and P's rows are loaded two steps
// ahead (transposed: code words one 32-row part, P's rows one step ahead).
// OCC: waves per SIMD (4: two workgroups share a CU, so that one decodes while
// the other waits at its barrier).
//
// What bounds it: VALU issue and LDS reads of the decode, about 4.9 VALU
// operations a weight (314 of them, 32 gathers, 8 operand reads and 16 MFMAs
// per step of two tiles, k = 4), once per tile of rows. Measured, K = 5120,
// N = 17408, k = 4 unless said: 27 us at 1 row, 34 us at 24, 50 us for both
// matrices at 19 rows (VALU 44%, LDS 41%, MFMA 8% busy); K = 17408, N = 5120,
// k = 3 at 117 rows 57 us; transposed, k = 3, two matrices, 257 rows in three
// tiles 229 us (VALU 42%, LDS 36%, MFMA 18%). Tried and slower: one column tile
// per wave from four row tiles on (53 against 49 us at 64 rows), two up to two
// (40 against 38.7 at 24), four waves per SIMD from four row tiles on (97
// against 47 at 64: registers spill). Transposed with six row tiles 48 bytes a
// lane go through scratch memory outside the steps.
template <int BITS, int KIND, int MT, int NT, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void product_kernel(Product P) {
  constexpr bool kT = KIND == kTransposed;
  static_assert(kT ? NT == 4 : KIND == kGated ? NT == 2 : NT <= 2, "tiles per wave");
  constexpr int BM = 16 * MT;
  constexpr int BN = kT ? 256 : KIND == kGated ? 64 : 64 * NT;  // output columns of a group
  constexpr int RC = kT ? 128 : 64 * NT;                        // columns reduced per round
  constexpr int wpb = 8 * BITS;
  constexpr int kRounds = kT ? 2 : 1;
  // The table is static LDS, so its reads carry the base in the instruction.
  __shared__ __attribute__((aligned(16))) uint32_t s_table[kTableBytes / 4];
  __shared__ uint32_t arrived[2];
  extern __shared__ __attribute__((aligned(16))) unsigned char xs[];  // two buffers of BM rows
  const unsigned char *const table = reinterpret_cast<const unsigned char *>(s_table);
  // transposed: two buffers of 256 row constants (q, k) and scales, and the
  // buffers' flags of scales outside the exact range, one per wave
  f32x2 *const rowq = reinterpret_cast<f32x2 *>(xs + 2 * BM * kStride);
  float *const rows_s = reinterpret_cast<float *>(rowq + 512);
  uint32_t *const rowf = reinterpret_cast<uint32_t *>(rows_s + 512);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 3, wk = wave >> 2;
  const int j = lane & 15, g = lane >> 4;

  const uint32_t row_bytes = (uint32_t)(P.k >> 8) * wpb * 4;
  const int cols = kT ? P.n : P.k;  // columns of P
  auto start_of = [&](int c) {
    return P.parts ? c / P.parts * P.steps + c % P.parts * P.steps / P.parts
                   : c * P.units_q + (c < P.units_r ? c : P.units_r);
  };
  int unit = start_of(blockIdx.x);
  const int end = start_of(blockIdx.x + 1);
  // The current segment: steps s0 .. s1 - 1 of a tile.
  int tile = unit / P.steps, s0 = unit - tile * P.steps, s1 = end - unit < P.steps - s0 ? s0 + (end - unit) : P.steps;
  int m0 = tile / P.groups * BM, group = tile % P.groups;

  // Staged rows of P: thread t takes 8 columns of row t / 32 + 16 r.
  // (Past the last step it is staged again: straight-line code keeps the rows
  // in registers and the memory waits exact.)
  struct Rows {
    u32x4 x[MT];
    float s;
  };
  const uint32_t row_b = (uint32_t)cols * 2;
  const uint32_t xoff = (uint32_t)(tid >> 5) * row_b + (uint32_t)(tid & 31) * 16;
  auto fetch = [&](int s, Rows &R) {
    const bool second = kT && s >= P.steps1;
    const int at = second ? s - P.steps1 : s;
    const uint32_t valid_b = (uint32_t)(P.m - m0 < BM ? P.m - m0 : BM) * row_b;
    // rows past m lie outside the buffer and read as zero
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>((second ? P.p2 : P.p) + (int64_t)m0 * cols + (int64_t)at * kStep), (short)0,
        (int)(valid_b - (uint32_t)at * (kStep * 2)), kRawBuffer);
    // transposed: so do columns past N (rows start at multiples of 8 bytes)
    const int left = cols - at * kStep - (tid & 31) * 8;
#pragma unroll
    for (int r = 0; r < MT; ++r) {
      const uint32_t o = xoff + (uint32_t)(16 * r) * row_b;
      if constexpr (!kT) {
        R.x[r] = __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0);
      } else {
        const u32x2 a = __builtin_amdgcn_raw_buffer_load_b64(rs, left > 0 ? o : 0x80000000u, 0, 0);
        const u32x2 b = __builtin_amdgcn_raw_buffer_load_b64(rs, left > 4 ? o + 8 : 0x80000000u, 0, 0);
        R.x[r] = u32x4{a[0], a[1], b[0], b[1]};
      }
    }
    if constexpr (kT) {
      const int row = at * kStep + tid;
      R.s = tid < 256 && row < P.n ? bf16_bits_to_f32((second ? P.scales2 : P.scales)[row]) : 0.f;
    }
  };
  auto put = [&](int s, const Rows &R) {
    unsigned char *dst = xs + (s & 1) * BM * kStride;
#pragma unroll
    for (int r = 0; r < MT; ++r)
      *reinterpret_cast<u32x4 *>(dst + (r * 16 + (tid >> 5)) * kStride + (tid & 31) * 16) = R.x[r];
    if constexpr (kT) {
      if (tid < 256) {
        float q, k;
        alu_row_constants(R.s, q, k);
        rowq[(s & 1) * 256 + tid] = f32x2{q, k};
        rows_s[(s & 1) * 256 + tid] = R.s;
        const bool out = !__all(alu_scale_ok(R.s));
        if (lane == 0) rowf[(s & 1) * 4 + wave] = out;
      }
    }
  };
  // Reduction of a finished segment (tile, steps a0 .. a1 - 1), and its store.
  constexpr int kPart = BM * RC * kRounds;  // floats of a tile's partial
  float *const red = reinterpret_cast<float *>(xs);
  // columns of P.out handled per round, and the store of four sums
  auto finish = [&](int am0, int agroup, int row, int c, f32x4 v, f32x4 v2) {
    const int mrow = am0 + row;
    if (mrow >= P.m) return;
    if constexpr (KIND == kGated) {
      const int n = agroup * BN + c;
      if (n >= P.n) return;
      const int64_t o = (int64_t)mrow * P.n + n;
      f32x4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = silu_mul(v[e], v2[e]);
      store4(P.out + o, h);
      if (P.gate) store4(P.gate + o, v);
      if (P.up) store4(P.up + o, v2);
    } else {
      const int width = kT ? P.k : P.n, n = agroup * BN + c;
      if (n >= width) return;
      store4(P.out + (int64_t)mrow * width + n, v);
    }
  };
  f32x4 acc[MT][NT];
  auto reduce = [&](int a0, int a1, int am0, int agroup) {
    // The two wk halves meet in LDS, [wk][row][128 columns]; then each thread
    // takes four columns of a row at a time.
    // (The thread's number goes through an empty asm here, so that nothing of
    // this part is computed ahead and kept in registers through the steps.)
    int et = tid;
    asm volatile("" : "+v"(et));
    const int ej = et & 15, eg = (et >> 4) & 3;
    const bool whole = a0 == 0 && a1 == P.steps;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (a0 == 0 ? 1 : 0);
    for (int round = 0; round < kRounds; ++round) {
      if (round) lds_barrier();
      if (!kT || (wn >> 1) == round) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float *r = red + (wk * BM + mt * 16 + 4 * eg + e) * kRedStride;
            if constexpr (kT) {
              *reinterpret_cast<f32x4 *>(r + 64 * (wn & 1) + 4 * ej) =
                  f32x4{acc[mt][0][e], acc[mt][1][e], acc[mt][2][e], acc[mt][3][e]};
            } else {
#pragma unroll
              for (int i = 0; i < NT; ++i)
                r[KIND == kGated ? 64 * i + 16 * wn + ej : 16 * NT * wn + 16 * i + ej] = acc[mt][i][e];
            }
          }
        // The adapters' term joins the sums of the wave that holds the tile's
        // last step, half of the row tiles in each wk.
        if (KIND != kGated && a1 == P.steps && P.low.rank > 0) {
          // (one row tile: the first wk alone)
          // Transposed: one row tile at a time, as the sums of the second
          // round are still in registers.
          constexpr int TILES = kT ? 1 : (MT + 1) / 2;
          for (int first = wk; first < MT; first += 2 * TILES) {
            f32x4 term[TILES][NT];
            low_rank_tiles<TILES, NT>(P.low, P.m, am0 + 16 * first, et & 63, term, [&](int a, int r0, bf16x8 (&w)[NT]) {
              if constexpr (kT) {
                const int k0 = agroup * BN + 64 * wn + 4 * ej;
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  bf16x4 v = {};
                  if (r0 + e < P.low.rank)
                    v = *reinterpret_cast<const bf16x4 *>(P.low.factor + ((int64_t)a * P.low.rank + r0 + e) * P.k + k0);
#pragma unroll
                  for (int c = 0; c < 4; ++c) w[c][e] = v[c];
                }
              } else {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                  const int n = agroup * BN + 16 * NT * wn + 16 * i + ej;
                  const uint16_t *q = P.low.factor + ((int64_t)a * P.n + n) * P.low.rank + r0;
                  if ((P.low.rank & 7) == 0) {
                    w[i] = bf16x8{};
                    if (n < P.n && r0 < P.low.rank) w[i] = *reinterpret_cast<const bf16x8 *>(q);
                  } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                      w[i][e] = __builtin_bit_cast(__bf16, n < P.n && r0 + e < P.low.rank ? q[e] : (uint16_t)0);
                  }
                }
              }
            });
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float *r = red + (wk * BM + (2 * t + first) * 16 + 4 * eg + e) * kRedStride;
                if constexpr (kT) {
                  f32x4 *v = reinterpret_cast<f32x4 *>(r + 64 * (wn & 1) + 4 * ej);
                  *v += f32x4{term[t][0][e], term[t][1][e], term[t][2][e], term[t][3][e]};
                } else {
#pragma unroll
                  for (int i = 0; i < NT; ++i) r[16 * NT * wn + 16 * i + ej] += term[t][i][e];
                }
              }
          }
        }
      }
      lds_barrier();
      if (whole && KIND == kGated) {
        for (int q = et; q < BM * 16; q += kThreads) {
          const int row = q >> 4, c = (q & 15) * 4;
          const f32x4 *r0 = reinterpret_cast<const f32x4 *>(red + row * kRedStride + c);
          const f32x4 *r1 = reinterpret_cast<const f32x4 *>(red + (BM + row) * kRedStride + c);
          finish(am0, agroup, row, c, r0[0] + r1[0], r0[16] + r1[16]);
        }
      } else {
        const __amdgpu_buffer_rsrc_t ws =
            __builtin_amdgcn_make_buffer_rsrc(P.partials + slot * kPart, (short)0, kPart * 4, kRawBuffer);
        for (int q = et; q < BM * (RC / 4); q += kThreads) {
          const int row = q / (RC / 4), c = (q % (RC / 4)) * 4;
          const f32x4 v = *reinterpret_cast<const f32x4 *>(red + row * kRedStride + c) +
                          *reinterpret_cast<const f32x4 *>(red + (BM + row) * kRedStride + c);
          if (whole) finish(am0, agroup, row, round * RC + c, v, v);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ws,
                                                   (uint32_t)((round * BM + row) * RC + c) * 4, 0, kSc1);
        }
      }
    }
  };
  // Tiles shared with other workgroups: at most a range's first and its last.
  int shared0 = -1, shared1 = -1;
  if constexpr (!kT) {
    float sc[NT];
    uint16_t sb[NT];  // the rows' scales as loaded
    const unsigned char *base[NT];
    uint32_t size[NT];
    const int wb = 2 * BITS * g + BITS * (1 - wk);
    const uint32_t off = (uint32_t)j * row_bytes + 4 * wb, off_next = (uint32_t)j * row_bytes + 4 * ((wb + BITS) % wpb);
    struct Words {
      uint32_t d[NT][BITS + 1];
    };
    auto load = [&](int s, Words &W) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        // rows past N lie outside the buffer and read as zero
        const uint32_t blk = (uint32_t)s * (wpb * 4);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<unsigned char *>(base[i] + blk), (short)0, (int)(size[i] ? size[i] - blk : 0u), kRawBuffer);
        if constexpr (BITS == 4) {
          const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
#pragma unroll
          for (int b = 0; b < 4; ++b) W.d[i][b] = v[b];
        } else if constexpr (BITS == 2) {
          const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
          W.d[i][0] = v[0];
          W.d[i][1] = v[1];
        } else {
#pragma unroll
          for (int b = 0; b < BITS; ++b) W.d[i][b] = __builtin_amdgcn_raw_buffer_load_b32(rs, off + 4 * b, 0, 0);
        }
        W.d[i][BITS] = __builtin_amdgcn_raw_buffer_load_b32(rs, off_next, 0, 0);
      }
    };
    Words A, B;
    // P's rows of the steps that A and B belong to; with eight row tiles there
    // are no registers for two steps, and they are loaded one step ahead.
    constexpr bool kFar = MT <= 6;
    Rows X, Y;
    auto request = [&]() {
      fetch(s0, X);
      if constexpr (kFar) fetch(s0 + 1 < s1 ? s0 + 1 : s0, Y);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int n0 = KIND == kGated ? group * BN + 16 * wn : group * BN + 16 * NT * wn + 16 * i;
        const uint32_t *c = KIND == kGated && i ? P.codes2 : P.codes;
        const uint16_t *sp = KIND == kGated && i ? P.scales2 : P.scales;
        const int rows = P.n - n0 < 0 ? 0 : P.n - n0 < 16 ? P.n - n0 : 16;
        base[i] = reinterpret_cast<const unsigned char *>(c) + (int64_t)n0 * row_bytes;
        size[i] = (uint32_t)rows * row_bytes;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(sp + n0), (short)0, rows * 2, kRawBuffer);
        sb[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (uint32_t)j * 2, 0, 0);
      }
      load(s0, A);
      load(s0 + 1 < s1 ? s0 + 1 : s0, B);
    };
    request();
    // The table, while the first loads are on their way.
  #pragma unroll
    for (int i = 0; i < 2048 / kThreads; ++i) s_table[i * kThreads + tid] = code_entry_pair((uint32_t)(i * kThreads + tid));
      for (;;) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
      float q[NT], kq[NT];
      bool exact = true;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        sc[i] = bf16_bits_to_f32(sb[i]);
        alu_row_constants(sc[i], q[i], kq[i]);
        exact = exact && alu_scale_ok(sc[i]);
      }
      const bool chain = !__all(exact);
      put(s0, X);
      lds_barrier();
      // Rows with scales outside the exact range take a loop of their own.
      auto step = [&](int s, Words &W, Rows &mine, const Rows &next, auto chained) {
        if constexpr (kFar) fetch(s + 2 < s1 ? s + 2 : s1 - 1, mine);  // (its rows are in LDS)
        else fetch(s + 1 < s1 ? s + 1 : s, X);
        const unsigned char *xb = xs + (s & 1) * BM * kStride + j * kStride + (192 - 64 * g + 32 * wk) * 2;
        auto multiply = [&](int u, const bf16x8 (&w)[NT]) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const bf16x8 x = *reinterpret_cast<const bf16x8 *>(xb + mt * 16 * kStride + 16 * u);
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[i], acc[mt][i], 0, 0, 0);
          }
          // bounds the registers that operands read ahead take
          __builtin_amdgcn_sched_barrier(0);
        };
        bf16x8 w[NT];
        if constexpr (decltype(chained)::value) {
#define TRELLIS_CHAIN(U)                                                                                  \
  _Pragma("unroll") for (int i = 0; i < NT; ++i) w[i] = group_chain<BITS, U>(W.d[i], sc[i], Eight{});     \
  multiply(U, w);
          TRELLIS_CHAIN(0) TRELLIS_CHAIN(1) TRELLIS_CHAIN(2) TRELLIS_CHAIN(3)
#undef TRELLIS_CHAIN
          load(s + 2 < s1 ? s + 2 : s1 - 1, W);
        } else {
          // Two phases: the codes of one table group are gathered while one
          // group goes through the ALU.
          const uint32_t mask = 0x1FFEu;
          uint32_t r[NT][8];
#define TRELLIS_PHASE(TABLE, ALU, AFTER)                                                                      \
  _Pragma("unroll") for (int i = 0; i < NT; ++i) gather_codes<BITS, TABLE>(W.d[i], table, mask, r[i]);        \
  _Pragma("unroll") for (int i = 0; i < NT; ++i) w[i] = group_hashed<BITS, ALU>(W.d[i], q[i], kq[i], Eight{}); \
  AFTER;                                                                                                      \
  multiply(ALU, w);                                                                                           \
  _Pragma("unroll") for (int i = 0; i < NT; ++i) w[i] = gathered_weights(r[i], q[i]);                         \
  multiply(TABLE, w);
          TRELLIS_PHASE(0, 2, (void)0)
          TRELLIS_PHASE(1, 3, load(s + 2 < s1 ? s + 2 : s1 - 1, W))
#undef TRELLIS_PHASE
        }
        put(s + 1, kFar ? next : X);
        lds_barrier();
      };
      auto steps = [&](auto chained) {
        for (int s = s0;;) {
          step(s, A, X, Y, chained);
          if (++s == s1) break;
          step(s, B, Y, X, chained);
          if (++s == s1) break;
        }
      };
      if (chain) steps(std::true_type{});
      else steps(std::false_type{});
      // The next segment is requested before this one is reduced.
      const int a0 = s0, a1 = s1, am0 = m0, agroup = group, at = tile;
      unit += s1 - s0;
      const bool more = unit < end;
      if (more) {
        tile = unit / P.steps;
        s0 = unit - tile * P.steps;
        s1 = end - unit < P.steps - s0 ? s0 + (end - unit) : P.steps;
        m0 = tile / P.groups * BM;
        group = tile % P.groups;
        request();
      }
      if (a0 > 0 || a1 < P.steps) {
        if (shared0 < 0) shared0 = at;
        else shared1 = at;
      }
      reduce(a0, a1, am0, agroup);
      if (!more) break;
      lds_barrier();  // the reduction is done with P's space
    }
  } else {
    // Lane (j, g) decodes columns 64 wn + 4 j .. +3 of the block for rows
    // 8 g .. 8 g + 7 of each 32-row MFMA part: the lowest of the four
    // windows starts at stream bit (252 - 64 wn - 4 j) * BITS, the others
    // BITS apart, 3 BITS + 12 <= 24 bits in all.
    const int pos = (252 - 64 * wn - 4 * j) * BITS;
    const uint32_t w0 = (uint32_t)(pos >> 5), sh = (uint32_t)(pos & 31);
    const uint32_t row0 = (uint32_t)(128 * wk + 8 * g) * row_bytes;
    const uint32_t o_lo = row0 + 4 * w0, o_hi = row0 + 4 * ((w0 + 1) % wpb);
    struct Words {
      uint32_t lo[8], hi[8];
    };
    auto load = [&](int part, Words &W) {
      const int parts = 4 * (s1 - s0);
      if (part >= parts) part = parts - 1;
      const int s = s0 + (part >> 2);
      const bool second = s >= P.steps1;
      const int n0 = (second ? s - P.steps1 : s) * kStep;
      const int rows = P.n - n0 < kStep ? P.n - n0 : kStep;
      const unsigned char *base = reinterpret_cast<const unsigned char *>(second ? P.codes2 : P.codes) +
                                  (int64_t)n0 * row_bytes + (int64_t)group * wpb * 4;
      // rows past N lie outside the buffer and read as zero
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<unsigned char *>(base), (short)0, (int)((uint32_t)rows * row_bytes - (uint32_t)group * wpb * 4), kRawBuffer);
      const uint32_t ro = (uint32_t)(32 * (part & 3)) * row_bytes;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        W.lo[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, o_lo + ro + (uint32_t)e * row_bytes, 0, 0);
        W.hi[e] = __builtin_amdgcn_raw_buffer_load_b32(rs, o_hi + ro + (uint32_t)e * row_bytes, 0, 0);
      }
    };
    Words W;
    Rows X;
    auto request = [&]() {
      fetch(s0, X);
      load(0, W);
    };
    request();
    // The table, while the first loads are on their way.
#pragma unroll
    for (int i = 0; i < 2048 / kThreads; ++i) s_table[i * kThreads + tid] = code_entry_pair((uint32_t)(i * kThreads + tid));
      for (;;) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
      put(s0, X);
      lds_barrier();
      auto compute = [&](int part, bool chain) {
        const int s = s0 + (part >> 2), p = part & 3;
        const int at = (s & 1) * 256 + 128 * wk + 32 * p + 8 * g;
        uint32_t fields[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) fields[e] = __builtin_amdgcn_alignbit(W.hi[e], W.lo[e], sh);
        load(part + 1, W);
        bf16x8 w[4];
#pragma unroll
        for (int h = 0; h < 8; h += 4) {  // four rows at a time
          const uint32_t(&f)[4] = *reinterpret_cast<uint32_t(*)[4]>(fields + h);
          if (chain) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float sc = rows_s[at + h + e];
#pragma unroll
              for (int c = 0; c < 4; ++c)
                w[c][h + e] = (__bf16)(trellis_value(code_of(__builtin_amdgcn_ubfe(f[e], (3 - c) * BITS, 12))) * sc);
            }
          } else {
            uint32_t r[2][4];
            f32x2 qk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              r[0][e] = table_code(table, (f[e] >> (3 * BITS - 1)) & 0x1FFEu);
              r[1][e] = table_code(table, (f[e] >> (2 * BITS - 1)) & 0x1FFEu);
              qk[e] = rowq[at + h + e];
            }
#pragma unroll
            for (int c = 2; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[c][h + e] = (__bf16)__builtin_fmaf(code_plus_magic(__builtin_amdgcn_ubfe(f[e], (3 - c) * BITS, 12)), qk[e][0], qk[e][1]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) w[c][h + e] = (__bf16)mix_lo(r[c][e], qk[e][0]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        const unsigned char *xb = xs + (s & 1) * BM * kStride + j * kStride + (128 * wk + 32 * p + 8 * g) * 2;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const bf16x8 x = *reinterpret_cast<const bf16x8 *>(xb + mt * 16 * kStride);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[mt][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[c], acc[mt][c], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      for (int s = s0; s < s1; ++s) {
        const int part = 4 * (s - s0);
        fetch(s + 1 < s1 ? s + 1 : s, X);
        const uint32_t *fl = rowf + (s & 1) * 4;
        const bool chain = __builtin_amdgcn_readfirstlane(fl[0] | fl[1] | fl[2] | fl[3]) != 0;
        for (int p = 0; p < 4; ++p) compute(part + p, chain);
        put(s + 1, X);
        lds_barrier();
      }
      // The next segment is requested before this one is reduced.
      const int a0 = s0, a1 = s1, am0 = m0, agroup = group, at = tile;
      unit += s1 - s0;
      const bool more = unit < end;
      if (more) {
        tile = unit / P.steps;
        s0 = unit - tile * P.steps;
        s1 = end - unit < P.steps - s0 ? s0 + (end - unit) : P.steps;
        m0 = tile / P.groups * BM;
        group = tile % P.groups;
        request();
      }
      if (a0 > 0 || a1 < P.steps) {
        if (shared0 < 0) shared0 = at;
        else shared1 = at;
      }
      reduce(a0, a1, am0, agroup);
      if (!more) break;
      lds_barrier();  // the reduction is done with P's space
    }
  }

  // Shared tiles: once this workgroup's partials are complete at the coherent
  // level its tiles' counters move; the workgroup that arrives last at a tile
  // adds the partials in order and stores the tile.
  if (shared0 < 0) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid < 2) {
    const int t = tid ? shared1 : shared0;
    if (t >= 0) arrived[tid] = __hip_atomic_fetch_add(&P.counters[t], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  // the workgroup that holds unit u
  auto owner = [&](int u) {
    const int cut = P.units_r * (P.units_q + 1);
    return u < cut ? u / (P.units_q + 1) : P.units_r + (u - cut) / P.units_q;
  };
  for (int i = 0; i < 2; ++i) {
    const int t = i ? shared1 : shared0;
    if (t < 0) continue;
    const int c0 = P.parts ? t * P.parts : owner(t * P.steps), c1 = P.parts ? c0 + P.parts - 1 : owner(t * P.steps + P.steps - 1);
    if (arrived[i] != (uint32_t)(c1 - c0)) continue;
    if (tid == 0) __hip_atomic_store(&P.counters[t], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int tm0 = t / P.groups * BM, tgroup = t % P.groups;
    // The tile's first workgroup keeps its partial in its second slot (the
    // tile is where its range ends), the others in their first. Four loads at
    // a time; those past the last lie outside the buffer and give zero.
    const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(
        P.partials + (int64_t)(2 * c0 + 1) * kPart, (short)0, (2 * (c1 - c0) + 1) * kPart * 4, kRawBuffer);
    constexpr int kQuads = KIND == kGated ? BM * 16 : kRounds * BM * (RC / 4);  // of outputs
    constexpr int kSums = KIND == kGated ? 2 : 1;                             // sums behind each output
    constexpr int kBatch = kQuads / kThreads >= 4 && !kT ? 4 : kQuads / kThreads >= 2 ? 2 : 1;  // quads of a thread at a time
    for (int q0 = tid; q0 < kQuads; q0 += kBatch * kThreads) {
      f32x4 v[kBatch][kSums];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int h = 0; h < kSums; ++h) v[b][h] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int c = c0; c <= c1; c += 4) {
        f32x4 part[4][kBatch][kSums];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int h = 0; h < kSums; ++h) {
              const int q = q0 + b * kThreads;
              const uint32_t slot = c + u == c0 ? 0u : (uint32_t)(2 * (c + u - c0) - 1);
              const uint32_t at = KIND == kGated ? (uint32_t)((q >> 4) * RC + 64 * h + (q & 15) * 4) : 4u * (uint32_t)q;
              part[u][b][h] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                            ws, c + u <= c1 ? (slot * kPart + at) * 4 : 0x80000000u, 0, kSc1));
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int h = 0; h < kSums; ++h) v[b][h] += part[u][b][h];
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int q = q0 + b * kThreads;
        if (kQuads % (kBatch * kThreads) != 0 && q >= kQuads) continue;
        if constexpr (KIND == kGated) {
          finish(tm0, tgroup, q >> 4, (q & 15) * 4, v[b][0], v[b][1]);
        } else {
          const int round = q / (BM * (RC / 4)), row = q / (RC / 4) % BM, c = (q % (RC / 4)) * 4;
          finish(tm0, tgroup, row, round * RC + c, v[b][0], f32x4{});
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// t[m, r] = gain[i] * sum_c P[m, c] F(i, r, c), i = index[m]: float32, zero
// past the rank and in rows without an adapter.
//   forward     P = x,    F(i, r, c) = A[i][r][c]   (c < K)
//   transposed  P = dout, F(i, r, c) = B[i][c][r]   (c < N)
// One workgroup: 16 MS rows, 32 rank columns, one span of c. Its waves share
// out the adapters that the rows name and, where there are fewer adapters than
// waves, the columns; an adapter's product is kept in its own rows only. The
// waves' sums meet in LDS, the spans' in `partials`, added in order by the
// workgroup that arrives last.
// Bound by latency on few rows (6 us for 1 row and 8 us for 24 rows with 16
// adapters at K = 5120: a load, a product, and a second round trip to join
// spans) and by reading P on many (2048 rows, K = 5120, rank 32: 15 us, 1.4
// TB/s; with N = 17408 beside it 45 us).
// ---------------------------------------------------------------------------
struct Shrink {
  const uint16_t *p;
  const uint16_t *factor;
  const float *gain;
  const int32_t *index;
  float *t;
  float *partials;
  uint32_t *counters;
  int32_t m, cols, count, rank, rank_p;
  int32_t span, spans;
};
constexpr int kSpanBatch = 16;     // spans that a thread adds: one batch of loads
constexpr int kFactorStride = 40;  // elements per staged row of B: 32 and padding

template <bool T, int MS, int WAVES>
struct ShrinkSpace {
  f32x4 part[WAVES][MS * 2 * 64];
  uint16_t staged[T ? WAVES : 1][T ? 32 * kFactorStride : 8];
  uint32_t arrived;
  float gains[16 * MS];  // of the rows; zero without an adapter
};

// z of zs: the rank columns' tile.
template <bool T, int MS, int WAVES>
__device__ __forceinline__ void shrink(const Shrink &S, int z, int zs, ShrinkSpace<T, MS, WAVES> &space) {
  constexpr int kPart = MS * 2 * 64;  // vectors of four sums: [row tile][rank tile][lane]
  auto &part = space.part;
  auto &staged = space.staged;
  auto &arrived = space.arrived;
  auto &gains = space.gains;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane & 15, g = lane >> 4;
  const int span = blockIdx.y;
  const int64_t m0 = (int64_t)blockIdx.x * (16 * MS);
  // lane l: the adapter of row m0 + l
  int idx = lane < 16 * MS && m0 + lane < S.m ? S.index[m0 + lane] : -1;
  if (idx >= S.count) idx = -1;
  float gain = 0.f;  // (used at the end only: loaded now, it is not waited for there)
  if (wave == 0 && idx >= 0) gain = S.gain[idx];
  const uint64_t named = __ballot(idx >= 0);
  int distinct = 0;
  for (uint64_t left = named; left; ++distinct) left &= ~__ballot(idx == __builtin_amdgcn_readlane(idx, __builtin_ctzll(left)));
  const int rows_left = (int)(S.m - m0 < 16 * MS ? S.m - m0 : 16 * MS);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t *>(S.p + m0 * S.cols), (short)0, (int)((uint32_t)rows_left * (uint32_t)S.cols * 2), kRawBuffer);
  const int c_end = S.cols - span * S.span < S.span ? S.cols : (span + 1) * S.span;
  f32x4 acc[MS][2];
#pragma unroll
  for (int i = 0; i < MS; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Fewer adapters than waves: wave w takes adapter w mod distinct and one of
  // the parts of its columns; else adapters w, w + WAVES, ...
  const int share = distinct < WAVES ? distinct : WAVES;
  const int mine = share > 0 ? wave % share : 0, part_i = share > 0 ? wave / share : 0;
  const int parts = share > 0 ? (WAVES - mine + share - 1) / share : 1;
  int at = 0;
  for (uint64_t left = named; left; ++at) {
    const int a = __builtin_amdgcn_readlane(idx, __builtin_ctzll(left));
    const uint64_t rows = __ballot(idx == a);
    left &= ~rows;
    if (at % share != mine) continue;
    f32x4 d[MS][2];
#pragma unroll
    for (int i = 0; i < MS; ++i) d[i][0] = d[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // U steps of 32 columns are loaded before the first is multiplied. Loads
    // of what does not exist (columns past the span, rows past m, rank columns
    // past the rank) take an offset outside their buffer and give zero.
    constexpr int U = MS == 1 && !T ? 4 : 2;
    constexpr uint32_t kNone = 0x80000000u;
    const bool vectors = T && (S.rank & 7) == 0, wide = !T || (S.cols & 7) == 0;
    const uint32_t block = (uint32_t)S.rank * (uint32_t)S.cols;
    const __amdgpu_buffer_rsrc_t rf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>(S.factor + (int64_t)a * block), (short)0, (int)(block * 2), kRawBuffer);
    for (int c0 = span * S.span + 32 * U * part_i; c0 < c_end; c0 += 32 * U * parts) {
      bf16x8 w[U][2];
      u32x4 b[U][2], x[U][MS];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c0 + 32 * u, c = cu + 8 * g;
        const bool in = cu < c_end;
#pragma unroll
        for (int i = 0; i < MS; ++i) {
          const uint32_t o = ((uint32_t)(16 * i + j) * (uint32_t)S.cols + (uint32_t)c) * 2;
          if (wide) {
            x[u][i] = __builtin_amdgcn_raw_buffer_load_b128(rx, in && c < S.cols ? o : kNone, 0, 0);
          } else {  // rows start at multiples of 8 bytes
            const u32x2 lo = __builtin_amdgcn_raw_buffer_load_b64(rx, in && c < S.cols ? o : kNone, 0, 0);
            const u32x2 hi = __builtin_amdgcn_raw_buffer_load_b64(rx, in && c + 4 < S.cols ? o + 8 : kNone, 0, 0);
            x[u][i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
          }
        }
        if constexpr (!T) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t r = (uint32_t)(32 * z + 16 * h + j);  // past the rank: outside the adapter's block
            w[u][h] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                                                     rf, in ? (r * (uint32_t)S.cols + (uint32_t)c) * 2 : kNone, 0, 0));
          }
        } else if (vectors) {
          // 32 rows of B by 32 rank columns: lane l takes the 16 bytes at
          // column 8 (l mod 4) of rows l / 4 and 16 + l / 4
          const int r = 32 * z + 8 * (lane & 3);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t n = (uint32_t)(cu + 16 * h + (lane >> 2));
            b[u][h] = __builtin_amdgcn_raw_buffer_load_b128(
                rf, in && r < S.rank ? (n * (uint32_t)S.rank + (uint32_t)r) * 2 : kNone, 0, 0);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 32 * z + 16 * h + j;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[u][h][e] = __builtin_bit_cast(
                  __bf16, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                              rf, in && r < S.rank ? ((uint32_t)(c + e) * (uint32_t)S.rank + (uint32_t)r) * 2 : kNone, 0, 0));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (vectors) {  // turned in the wave's own LDS
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<u32x4 *>(&staged[wave][(16 * h + (lane >> 2)) * kFactorStride + 8 * (lane & 3)]) = b[u][h];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[u][h][e] = __builtin_bit_cast(__bf16, staged[wave][(8 * g + e) * kFactorStride + 16 * h + j]);
        }
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            d[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u][i]), w[u][h], d[i][h], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((rows >> (16 * i + 4 * g + e)) & 1) {
          acc[i][0][e] += d[i][0][e];
          acc[i][1][e] += d[i][1][e];
        }
  }
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    part[wave][(2 * i) * 64 + lane] = acc[i][0];
    part[wave][(2 * i + 1) * 64 + lane] = acc[i][1];
  }
  if (wave == 0 && lane < 16 * MS) gains[lane] = gain;
  __syncthreads();
  const int64_t cell = (int64_t)blockIdx.x * zs + z;
  float *const base = S.partials + cell * S.spans * (kPart * 4);
  const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(base, (short)0, S.spans * kPart * 16, kRawBuffer);
  auto sum_waves = [&](int v) {
    f32x4 s = part[0][v];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += part[w][v];
    return s;
  };
  if (S.spans > 1) {
    for (int v = tid; v < kPart; v += 64 * WAVES)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum_waves(v)), ws, (uint32_t)((span * kPart + v) * 16), 0, kSc1);
    // The partial is complete at the coherent level before the counter moves.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) arrived = __hip_atomic_fetch_add(&S.counters[cell], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != (uint32_t)S.spans - 1) return;
    if (tid == 0) __hip_atomic_store(&S.counters[cell], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // SHARES threads add a vector's spans, 16 each (past the last span: outside
  // the buffer, zero), and their sums meet in LDS.
  constexpr int SHARES = 64 * WAVES / kPart > 0 ? 64 * WAVES / kPart : 1;
  if (S.spans > 1) {
    for (int v = tid; v < kPart * SHARES; v += 64 * WAVES) {
      f32x4 p[kSpanBatch], sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kSpanBatch; ++s)
        p[s] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             ws, (uint32_t)(((v / kPart * kSpanBatch + s) * kPart + v % kPart) * 16), 0, kSc1));
#pragma unroll
      for (int s = 0; s < kSpanBatch; ++s) sum += p[s];
      part[v / kPart][v % kPart] = sum;
    }
    __syncthreads();
  }
  for (int v = tid; v < kPart; v += 64 * WAVES) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (S.spans > 1) {
#pragma unroll
      for (int s = 0; s < SHARES; ++s) sum += part[s][v];
    } else {
      sum = sum_waves(v);
    }
    const int l = v & 63, r = 32 * z + 16 * ((v >> 6) & 1) + (l & 15);
    const int row0 = 16 * (v >> 7) + 4 * (l >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      // (past the rank an infinity of P gave a NaN)
      if (m0 + row0 + e < S.m) S.t[(m0 + row0 + e) * S.rank_p + r] = r < S.rank ? sum[e] * gains[row0 + e] : 0.f;
  }
}

template <int MS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void shrink_kernel(Shrink S) {
  __shared__ __attribute__((aligned(16))) ShrinkSpace<false, MS, WAVES> space;
  shrink<false, MS, WAVES>(S, blockIdx.z, gridDim.z, space);
}

// The 32-row chunks that an adapter's rows lie in: range[a] = [first, last + 1).
__device__ __forceinline__ void chunk_range(const int32_t *__restrict__ index, int m, int a, i32x2 *range, int (&ends)[2]) {
  if (threadIdx.x == 0) {
    ends[0] = 0x7fffffff;
    ends[1] = -1;
  }
  __syncthreads();
  int first = 0x7fffffff, last = -1;
  for (int i = threadIdx.x; i < m; i += blockDim.x)
    if (index[i] == a) {
      if (first == 0x7fffffff) first = i;
      last = i;
    }
  if (last >= 0) {
    atomicMin(&ends[0], first);
    atomicMax(&ends[1], last);
  }
  __syncthreads();
  if (threadIdx.x == 0) range[a] = ends[1] < 0 ? i32x2{0, 0} : i32x2{ends[0] >> 5, (ends[1] >> 5) + 1};
}

// What the backward pass needs before its products, in one launch: t, u (z
// below zs: t, below 2 zs: u) and the adapters' chunk ranges (z = 2 zs). Three
// launches of their own took about 10 us more. 23 us at 509 rows (K = 17408,
// N = 5120, rank 8), 45 us at 2048 (K = 5120, N = 17408, rank 32).
struct BackwardSums {
  Shrink t, u;
  i32x2 *range;
};
template <int MS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void backward_sums_kernel(BackwardSums B) {
  __shared__ __attribute__((aligned(16))) union {
    ShrinkSpace<false, MS, WAVES> t;
    ShrinkSpace<true, MS, WAVES> u;
    int ends[2];
  } space;
  const int zs = gridDim.z >> 1, z = blockIdx.z;
  if (z < zs) {
    if ((int64_t)blockIdx.x * (16 * MS) < B.t.m && (int)blockIdx.y < B.t.spans) shrink<false, MS, WAVES>(B.t, z, zs, space.t);
  } else if (z < 2 * zs) {
    if ((int64_t)blockIdx.x * (16 * MS) < B.u.m && (int)blockIdx.y < B.u.spans) shrink<true, MS, WAVES>(B.u, z - zs, zs, space.u);
  } else {
    for (int a = blockIdx.y * gridDim.x + blockIdx.x; a < B.t.count; a += gridDim.x * gridDim.y)
      chunk_range(B.t.index, B.t.m, a, B.range, space.ends);
  }
}

// Gradients of the factors: sum over an adapter's rows of P[m, c] V[m, r].
//   dA[a][r][c]: P = x,    V = u    (c < K)
//   dB[a][c][r]: P = dout, V = t    (c < N)
// One workgroup (4 waves): 64 columns c and 32 rank columns of one adapter;
// wave w takes the 32-row chunks w, w + 4, ... of the adapter's range and the
// waves' sums meet in LDS in order. A chunk of P goes through the wave's own
// LDS, which turns it (contraction is over rows); rows of other adapters enter
// as zeros on both sides (a NaN in them must not count). V as the sum of two
// bf16 numbers (2^-16 relative). The next chunk is loaded ahead. 2048 rows,
// K = 5120, N = 17408, rank 32, two adapters: 46 us, 97 MB read (2.1 TB/s; what
// it waits for is each wave's own chain of chunks). A chunk between an adapter's
// first and last row is read whether or not it holds one of its rows: adapters
// whose rows alternate read all of x and dout each (the whole backward call of
// these sizes: 442 us with eight adapters in runs, 689 alternating; 492 and 1538
// with 32).
struct Outer {
  const uint16_t *x, *dout;
  const float *u, *t;
  const int32_t *index;
  const i32x2 *range;
  uint16_t *da, *db;
  int32_t m, n, k, rank, rank_p;
  int32_t tiles_a;  // 64-column tiles of x; those of dout follow
};
constexpr int kTurnStride = 72;  // elements per staged row: 64 and padding

__global__ __launch_bounds__(256) void outer_kernel(Outer O) {
  __shared__ __attribute__((aligned(16))) uint16_t turn[4][32 * kTurnStride];
  __shared__ f32x4 part[4][8 * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 15, g = lane >> 4;
  const int a = blockIdx.y, r0 = blockIdx.z * 32;
  const bool is_a = (int)blockIdx.x < O.tiles_a;
  const int tile = is_a ? blockIdx.x : blockIdx.x - O.tiles_a;
  const uint16_t *const P = is_a ? O.x : O.dout;
  const float *const V = is_a ? O.u : O.t;
  const int cols = is_a ? O.k : O.n;
  const int c0 = tile * 64;
  const i32x2 range = O.range[a];
  f32x4 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Chunk {
    u32x2 p[8];     // rows 8 i + lane / 8 (i < 4), 8 columns as two halves
    float v[2][8];  // rows 8 g + e, rank columns 16 h + j
    uint32_t rows;  // which of the 32 rows are the adapter's
  };
  const int pc = c0 + 8 * (lane & 7);
  const bool wide = (cols & 7) == 0;
  auto load = [&](int ch, Chunk &C) {
    const int m0 = ch * 32;
    const int mi = m0 + (lane & 31);
    C.rows = (uint32_t)__ballot(mi < O.m && O.index[mi < O.m ? mi : 0] == a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + 8 * i + (lane >> 3);
      const uint16_t *q = P + (int64_t)(m < O.m ? m : O.m - 1) * cols + pc;
      C.p[2 * i] = C.p[2 * i + 1] = u32x2{0u, 0u};
      if (wide) {
        if (pc < cols) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(q);
          C.p[2 * i] = u32x2{v[0], v[1]};
          C.p[2 * i + 1] = u32x2{v[2], v[3]};
        }
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (pc + 4 * h < cols) C.p[2 * i + h] = *reinterpret_cast<const u32x2 *>(q + 4 * h);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int m = m0 + 8 * g + e;
      const float *q = V + (int64_t)(m < O.m ? m : O.m - 1) * O.rank_p + r0 + j;
      C.v[0][e] = q[0];
      C.v[1][e] = q[16];
    }
  };
  auto use = [&](const Chunk &C) {
    uint16_t *const mine = turn[wave];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + (lane >> 3);
      u32x4 v = u32x4{C.p[2 * i][0], C.p[2 * i][1], C.p[2 * i + 1][0], C.p[2 * i + 1][1]};
      if (!((C.rows >> row) & 1)) v = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4 *>(mine + row * kTurnStride + 8 * (lane & 7)) = v;
    }
    bf16x8 hi[2], lo[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (C.rows >> (8 * g + e)) & 1 ? C.v[h][e] : 0.f;
      halves(v, hi[h], lo[h]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x8 p;
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = __builtin_bit_cast(__bf16, mine[(8 * g + e) * kTurnStride + 16 * i + j]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (is_a) {  // rows r, columns c
          acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[h], p, acc[i][h], 0, 0, 0);
          acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[h], p, acc[i][h], 0, 0, 0);
        } else {     // rows c, columns r
          acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, hi[h], acc[i][h], 0, 0, 0);
          acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, lo[h], acc[i][h], 0, 0, 0);
        }
    }
  };
  const int first = range[0] + wave, last = range[1];
  if (first < last) {
    Chunk A, B;
    load(first, A);
    for (int ch = first;;) {
      load(ch + 4 < last ? ch + 4 : ch, B);
      use(A);
      if ((ch += 4) >= last) break;
      load(ch + 4 < last ? ch + 4 : ch, A);
      use(B);
      if ((ch += 4) >= last) break;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    part[wave][(2 * i) * 64 + lane] = acc[i][0];
    part[wave][(2 * i + 1) * 64 + lane] = acc[i][1];
  }
  __syncthreads();
  for (int v = threadIdx.x; v < 8 * 64; v += 256) {
    const f32x4 s = ((part[0][v] + part[1][v]) + part[2][v]) + part[3][v];
    const int l = v & 63, h = (v >> 6) & 1, i = v >> 7;
    const int lj = l & 15, lg = l >> 4;
    if (is_a) {
      const int c = c0 + 16 * i + lj;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * h + 4 * lg + e;
        if (r < O.rank) O.da[((int64_t)a * O.rank + r) * O.k + c] = bf16_of(s[e]);
      }
    } else {
      const int r = r0 + 16 * h + lj;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = c0 + 16 * i + 4 * lg + e;
        if (c < O.n && r < O.rank) O.db[((int64_t)a * O.n + c) * O.rank + r] = bf16_of(s[e]);
      }
    }
  }
}

// The gated block's elementwise gradients as rows, four elements a thread.
__global__ __launch_bounds__(256) void gated_grad_kernel(const uint16_t *__restrict__ dh, const uint16_t *__restrict__ gate,
                                                         const uint16_t *__restrict__ up, int64_t quads,
                                                         uint16_t *__restrict__ dgate, uint16_t *__restrict__ dup) {
  typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  const u16x4 d = reinterpret_cast<const u16x4 *>(dh)[i], gv = reinterpret_cast<const u16x4 *>(gate)[i],
              uv = reinterpret_cast<const u16x4 *>(up)[i];
  f32x4 og, ou;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    gated_gradients(bf16_bits_to_f32(d[e]), bf16_bits_to_f32(gv[e]), bf16_bits_to_f32(uv[e]), a, b);
    og[e] = a;
    ou[e] = b;
  }
  store4(dgate + 4 * i, og);
  store4(dup + 4 * i, ou);
}

__global__ __launch_bounds__(256) void clear_kernel(uint32_t *__restrict__ p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0u;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kMaxDevices = 64;

struct Space {
  unsigned char *bytes = nullptr;
  size_t size = 0;
  uint32_t *counters = nullptr;
  size_t ncounters = 0;
};
struct Key {
  int dev;
  hipStream_t stream;
  std::thread::id thread;  // the per-thread default stream is one handle for many streams
  bool operator<(const Key &o) const {
    if (dev != o.dev) return dev < o.dev;
    if (stream != o.stream) return stream < o.stream;
    return thread < o.thread;
  }
};
std::mutex g_lock;
std::map<Key, Space> g_space;
int g_cus[kMaxDevices];

bool geom_ok(const trellis_geom &g) {
  return g.t == TRELLIS_T && g.l == TRELLIS_L && (g.bits == 2 || g.bits == 3 || g.bits == 4) && g.k >= TRELLIS_T &&
         g.k <= TRELLIS_MAX_K && g.k % TRELLIS_T == 0 && g.n >= 4 && g.n <= TRELLIS_MAX_N && g.n % 4 == 0;
}
bool on(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Whether a runtime call worked. The runtime keeps a call's error until it is
// read, whatever succeeds after it: left there, it would be taken for the next
// launch's, here or in the caller's program.
bool worked(hipError_t e) {
  if (e == hipSuccess) return true;
  (void)hipGetLastError();
  return false;
}

trellis_status device(int &dev, int &cus) {
  if (!worked(hipGetDevice(&dev)) || dev < 0 || dev >= kMaxDevices) return TRELLIS_E_HIP;
  if (g_cus[dev] == 0 && (!worked(hipDeviceGetAttribute(&g_cus[dev], hipDeviceAttributeMultiprocessorCount, dev)) ||
                          g_cus[dev] <= 0))
    return TRELLIS_E_HIP;
  cus = g_cus[dev];
  return TRELLIS_OK;
}

// The stream's workspace: grown on demand and kept (launches still queued and
// captured graphs may hold an outgrown buffer's address, so none is freed).
// Not while the stream is captured: the clearing of new counters would become
// part of the graph, and eager calls before its first replay would find them
// as the allocator left them.
trellis_status space(int dev, hipStream_t stream, size_t size, size_t ncounters, Space *&out) {
  const std::thread::id tid = stream == hipStreamPerThread ? std::this_thread::get_id() : std::thread::id();
  Space *slot = nullptr;
  try {
    slot = &g_space[Key{dev, stream, tid}];
  } catch (const std::bad_alloc &) {
    return TRELLIS_E_HIP;
  }
  Space &w = *slot;
  if (w.size < size || w.ncounters < ncounters) {
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (!worked(hipStreamIsCapturing(stream, &capture)) || capture != hipStreamCaptureStatusNone) return TRELLIS_E_HIP;
  }
  if (w.size < size) {
    // By half as much again at least, so that the outgrown buffers of ever
    // longer calls stay within twice the last one's size.
    const size_t more = w.size + w.size / 2;
    void *p = nullptr;
    if (size < more && worked(hipMalloc(&p, more))) {
      size = more;
    } else if (!worked(hipMalloc(&p, size))) {
      return TRELLIS_E_HIP;
    }
    w.bytes = static_cast<unsigned char *>(p);
    w.size = size;
  }
  if (w.ncounters < ncounters) {
    void *p = nullptr;
    if (!worked(hipMalloc(&p, ncounters * 4))) return TRELLIS_E_HIP;
    (void)hipGetLastError();
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((ncounters + 255) / 256)), dim3(256), 0, stream,
                       static_cast<uint32_t *>(p), (int64_t)ncounters);
    if (hipGetLastError() != hipSuccess) {
      (void)worked(hipFree(p));
      return TRELLIS_E_HIP;
    }
    w.counters = static_cast<uint32_t *>(p);
    w.ncounters = ncounters;
  }
  out = &w;
  return TRELLIS_OK;
}

typedef void (*ProductFn)(Product);
constexpr int kRowTiles[] = {1, 2, 4, 6, 8};
constexpr int kMts = 5;
// Tiles per wave and waves per SIMD for each number of row tiles. Forward up
// to two row tiles: one tile per wave, whose finer units split more evenly.
constexpr int wave_tiles(int kind, int mt) { return kind == kTransposed ? 4 : kind == kGated || mt > 2 ? 2 : 1; }
constexpr int waves_per_simd(int kind, int mt) { return kind != kTransposed && mt <= 2 ? 4 : 2; }
template <int BITS, int KIND, int MT>
constexpr ProductFn product_one() {
  return &product_kernel<BITS, KIND, MT, wave_tiles(KIND, MT), waves_per_simd(KIND, MT)>;
}
template <int BITS, int KIND>
ProductFn product_of(int i) {
  switch (i) {
    case 0: return product_one<BITS, KIND, 1>();
    case 1: return product_one<BITS, KIND, 2>();
    case 2: return product_one<BITS, KIND, 4>();
    case 3: return product_one<BITS, KIND, 6>();
    default: return product_one<BITS, KIND, KIND == kTransposed ? 6 : 8>();
  }
}
template <int KIND>
ProductFn product_of(int bits, int i) {
  return bits == 2 ? product_of<2, KIND>(i) : bits == 3 ? product_of<3, KIND>(i) : product_of<4, KIND>(i);
}
ProductFn product_fn(int kind, int bits, int i) {
  return kind == kForward ? product_of<kForward>(bits, i) : kind == kGated ? product_of<kGated>(bits, i)
                                                                           : product_of<kTransposed>(bits, i);
}

// How a product is laid over the card.
struct Shape {
  int kind, bits, mt;  // mt: index into kRowTiles
  int64_t tiles, units;
  int groups, steps, steps1, grid, parts;
  size_t partial_bytes, lds;
};
Shape shape_of(int kind, trellis_geom g, int32_t m, int matrices, int cus) {
  Shape s{};
  s.kind = kind;
  s.bits = g.bits;
  // at most 128 rows a tile, transposed 96 (its waves hold four column tiles)
  const int most_rows = kind == kTransposed ? 96 : 128;
  const int64_t chunks = ((int64_t)m + most_rows - 1) / most_rows;
  const int need = (int)((((int64_t)m + chunks - 1) / chunks + 15) / 16);
  while (kRowTiles[s.mt] < need) ++s.mt;
  const int bm = 16 * kRowTiles[s.mt];
  const int64_t rows = ((int64_t)m + bm - 1) / bm;
  const int mt = kRowTiles[s.mt];
  const int bn = kind == kTransposed ? 256 : kind == kGated ? 64 : 64 * wave_tiles(kind, mt);
  s.groups = ((kind == kTransposed ? g.k : g.n) + bn - 1) / bn;
  s.steps1 = ((kind == kTransposed ? g.n : g.k) + kStep - 1) / kStep;
  s.steps = kind == kTransposed ? s.steps1 * matrices : s.steps1;
  s.tiles = rows * s.groups;
  s.units = s.tiles * s.steps;
  const int64_t room = (int64_t)cus * waves_per_simd(kind, mt) / 2;  // workgroups the card holds at once
  s.grid = (int)(s.units < room ? s.units : room);
  // Tiles split over the same number of workgroups each, where that leaves at
  // most a tenth of the card idle: no workgroup then reduces two tiles' parts
  // (K = 17408, N = 5120, 117 rows: 40 tiles of 68 steps, 6 workgroups each).
  // Tiles of up to three steps are not split: joining costs more than a step.
  const int64_t each = room / s.tiles;
  if (each >= 1 && (s.steps <= 3 || (each <= s.steps && s.tiles * each * 10 >= room * 9))) {
    s.parts = s.steps <= 3 ? 1 : (int)each;
    s.grid = (int)s.tiles * s.parts;
  }
  s.partial_bytes = (size_t)2 * s.grid * bm * (kind == kGated ? 128 : bn) * 4;
  s.lds = (size_t)2 * bm * kStride + (kind == kTransposed ? 512 * 12 + 8 * 4 : 0);
  return s;
}

trellis_status launch(const Shape &s, Product p, hipStream_t stream) {
  const ProductFn fn = product_fn(s.kind, s.bits, s.mt);
  static bool ready[kMaxDevices][3][3][kMts];
  int dev = 0, cus = 0;
  if (device(dev, cus) != TRELLIS_OK) return TRELLIS_E_HIP;
  bool &done = ready[dev][s.kind][s.bits - 2][s.mt];
  if (!done) {
    if (!worked(hipFuncSetAttribute(reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, (int)s.lds)))
      return TRELLIS_E_HIP;
    done = true;
  }
  p.units_q = (int)(s.units / s.grid);
  p.units_r = (int)(s.units % s.grid);
  p.parts = s.parts;
  p.groups = s.groups;
  p.steps = s.steps;
  p.steps1 = s.steps1;
  (void)hipGetLastError();
  hipLaunchKernelGGL(fn, dim3((unsigned)s.grid), dim3(kThreads), s.lds, stream, p);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

// ---- many rows (dense.hpp) ---------------------------------------------------

// Test hook (trellis_test_force_path).
std::atomic<int> g_path{-1}, g_tiles{0};

// Operand workspace of one launch; larger matrices go in slabs of columns, one
// 256-column block at least (more than this from 2^21 rows of W on, transposed).
constexpr int64_t kOperandBytes = (int64_t)1 << 30;

struct DenseShape {
  int nt;              // accumulator tiles per wave
  int splits;          // of the contraction
  int matrices;        // gated: 2 in the tiles, transposed: in the contraction
  int steps, steps1;
  int64_t tiles, slab;  // operand tiles in all and per launch
  int ptiles;
  double us;           // what the product's rounds are reckoned to take
  size_t operand_bytes, row_bytes, partial_bytes;
};
DenseShape dense_shape(int kind, trellis_geom g, int32_t m, int matrices, int cus) {
  DenseShape s{};
  s.matrices = matrices;
  const bool t = kind == kTransposed;
  s.steps1 = ((t ? g.n : g.k) + 63) / 64 * 2;  // an even number
  s.steps = t ? s.steps1 * matrices : s.steps1;
  const int64_t width = t ? g.k : g.n, one = (width + 15) / 16;
  s.tiles = kind == kGated ? 2 * one : one;
  // The column tile and the split of the contraction whose rounds over the
  // card cost least, in us. A round costs 0.073 a step and accumulator tile,
  // 0.125 a step (staging) and 3.7 to start and store; the partial sums of a
  // split are written and read once more, 0.32 a MB. Fitted to the times of
  // every column tile and split at 448 sizes (all four operators, 200 to 4096
  // rows, K and N from 256 to 17408): the choice is 0.3% slower than the best on
  // average and 9% at most, as fewer than all 256 workgroups cost what they
  // leave idle (gated, K = 4096, N = 1024, 384 rows: 75.6 us in one split, 35.7
  // in seven).
  const int64_t mt = (m + kDenseRows - 1) / kDenseRows;
  const int64_t tile_bytes = (int64_t)s.steps * 1024;
  const bool several = s.tiles > 16 && tile_bytes * s.tiles > kOperandBytes;  // launches
  double best = 0;
  for (int nt = 8; nt >= 4; --nt) {
    if (kind == kGated && nt % 2) continue;
    // Contractions so long that 16 nt operand tiles exceed a launch's operands
    // go in slabs of 16 tiles and multiples of it: of whole workgroup tiles for
    // nt = 4 and 8 alone (the rest of a cut one would be stored over the next
    // slab's columns).
    if (several && nt % 4 && tile_bytes * 16 * nt > kOperandBytes) continue;
    const int64_t wg = mt * ((s.tiles + 2 * nt - 1) / (2 * nt));
    for (int splits = 1; splits == 1 || (splits <= 8 && splits <= s.steps / 16); ++splits) {
      const double rounds = (double)((wg * splits + cus - 1) / cus);
      double cost = rounds * ((double)s.steps / splits * (0.073 * nt + 0.125) + 3.7);
      if (splits > 1) cost += 0.8 + 0.32e-6 * ((double)splits * m * s.tiles * 16 * 4);
      if (s.nt == 0 || cost < best) {
        best = cost;
        s.nt = nt;
        s.splits = splits;
      }
    }
  }
  int64_t slab = kOperandBytes / tile_bytes / (16 * s.nt) * (16 * s.nt);  // whole workgroup tiles, fours and pairs
  const int forced = g_tiles.load(std::memory_order_relaxed);
  if (forced > 0) slab = ((int64_t)forced + 16 * s.nt - 1) / (16 * s.nt) * (16 * s.nt);
  if (slab == 0) slab = kOperandBytes / tile_bytes / 16 * 16;  // long contractions: whole 256-column blocks,
  if (slab == 0) slab = 16;                                    // one at least (512 bytes per row of W)
  if (slab > s.tiles) slab = s.tiles;
  s.slab = slab;
  s.operand_bytes = (size_t)(slab * tile_bytes);
  s.ptiles = (int)(((int64_t)m + 15) / 16);
  s.us = best;
  s.row_bytes = (size_t)s.ptiles * s.steps * 1024;
  s.partial_bytes = s.splits > 1 ? (size_t)s.splits * m * slab * 16 * 4 : 0;
  return s;
}

typedef void (*DenseFn)(Dense);
template <bool T>
DenseFn dense_of(int nt) {
  switch (nt) {
    case 4: return &dense_kernel<4, false, T>;
    case 5: return &dense_kernel<5, false, T>;
    case 6: return &dense_kernel<6, false, T>;
    case 7: return &dense_kernel<7, false, T>;
    default: return &dense_kernel<8, false, T>;
  }
}
DenseFn dense_fn(int kind, int nt) {
  if (kind == kGated) return nt == 4 ? &dense_kernel<4, true, false> : nt == 6 ? &dense_kernel<6, true, false> : &dense_kernel<8, true, false>;
  return kind == kTransposed ? dense_of<true>(nt) : dense_of<false>(nt);
}

// What the elementwise gradients are computed from (transposed with two matrices).
struct GatedGrads {
  const uint16_t *dh, *gate, *up;
  uint16_t *dgate, *dup;
};

trellis_status launch_dense(int kind, const DenseShape &s, trellis_geom g, const Product &p, const GatedGrads *grads,
                            unsigned char *operands, hipStream_t stream) {
  unsigned char *const rows = operands + up256(s.operand_bytes);
  const DenseFn fn = dense_fn(kind, s.nt);
  const size_t lds = (size_t)dense_buffers(s.nt) * dense_step_bytes(s.nt);
  static bool ready[kMaxDevices][3][9];
  int dev = 0, cus = 0;
  if (device(dev, cus) != TRELLIS_OK) return TRELLIS_E_HIP;
  if (!ready[dev][kind][s.nt]) {
    if (!worked(hipFuncSetAttribute(reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds)))
      return TRELLIS_E_HIP;
    ready[dev][kind][s.nt] = true;
  }
  Dense d{};
  d.p = reinterpret_cast<const uint16_t *>(rows);
  d.w = reinterpret_cast<const uint16_t *>(operands);
  d.out = p.out;
  d.gate = p.gate;
  d.up = p.up;
  d.m = p.m;
  d.steps = s.steps;
  d.splits = s.splits;
  d.partials = reinterpret_cast<float *>(rows + up256(s.row_bytes));
  d.ptiles = s.ptiles;
  d.width = kind == kTransposed ? g.k : g.n;
  d.mtiles = (p.m + kDenseRows - 1) / kDenseRows;
  d.low = p.low;
  (void)hipGetLastError();
  const dim3 pack((unsigned)(((int64_t)s.ptiles * (s.steps1 / 2) + 3) / 4));
  uint16_t *const to = reinterpret_cast<uint16_t *>(rows);
  const int width = kind == kTransposed ? g.n : g.k;
  if (grads)
    hipLaunchKernelGGL(width % 8 ? gated_grad_pack_kernel<false> : gated_grad_pack_kernel<true>, pack, dim3(256), 0, stream,
                       grads->dh, grads->gate, grads->up, p.m, width, s.ptiles, s.steps1, grads->dgate, grads->dup, to);
  else
    hipLaunchKernelGGL(width % 8 ? pack_rows_kernel<false> : pack_rows_kernel<true>, pack, dim3(256), 0, stream, p.p, p.m,
                       width, s.ptiles, s.steps1, to);
  if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
  for (int64_t first = 0; first < s.tiles; first += s.slab) {
    const int tiles = (int)(s.tiles - first < s.slab ? s.tiles - first : s.slab);
    Unpack u{{p.codes, p.codes2}, {p.scales, p.scales2}, reinterpret_cast<uint16_t *>(operands), g.n, g.k, s.steps, 0, 0, 1};
    if (kind == kTransposed) {
      u.first = (int)first;
      u.tiles = tiles;
      u.matrices = s.matrices;
      const int64_t waves = (int64_t)(tiles / 16) * s.steps1;
      const dim3 grid((unsigned)((waves + 3) / 4), (unsigned)s.matrices);
      if (g.bits == 2) hipLaunchKernelGGL(unpack_columns_kernel<2>, grid, dim3(256), 0, stream, u);
      else if (g.bits == 3) hipLaunchKernelGGL(unpack_columns_kernel<3>, grid, dim3(256), 0, stream, u);
      else hipLaunchKernelGGL(unpack_columns_kernel<4>, grid, dim3(256), 0, stream, u);
    } else {
      const int mats = kind == kGated ? 2 : 1;
      u.first = (int)(first / mats);
      u.tiles = tiles / mats;
      u.matrices = mats;
      const int64_t waves = (int64_t)u.tiles * (g.k >> 8);
      const dim3 grid((unsigned)((waves + 3) / 4), (unsigned)mats);
      if (g.bits == 2) hipLaunchKernelGGL(unpack_rows_kernel<2>, grid, dim3(256), 0, stream, u);
      else if (g.bits == 3) hipLaunchKernelGGL(unpack_rows_kernel<3>, grid, dim3(256), 0, stream, u);
      else hipLaunchKernelGGL(unpack_rows_kernel<4>, grid, dim3(256), 0, stream, u);
    }
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
    d.first = (int)(first * 16 / (kind == kGated ? 2 : 1));
    d.wtiles = tiles;
    d.ntiles = (tiles + 2 * s.nt - 1) / (2 * s.nt);
    hipLaunchKernelGGL(fn, dim3((unsigned)(d.mtiles * d.ntiles * s.splits)), dim3(kDenseThreads), lds, stream, d);
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
    if (s.splits > 1) {
      const int64_t quads = (int64_t)p.m * 4 * tiles / (kind == kGated ? 2 : 1);
      const dim3 grid((unsigned)((quads + 255) / 256));
      if (kind == kGated) hipLaunchKernelGGL(join_splits_kernel<true>, grid, dim3(256), 0, stream, d);
      else hipLaunchKernelGGL(join_splits_kernel<false>, grid, dim3(256), 0, stream, d);
      if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
    }
  }
  return TRELLIS_OK;
}

// Workspace of a product, and its launch with that workspace.
struct Plan {
  bool dense;
  Shape fused;
  DenseShape many;
  size_t bytes;
  int64_t counters;
};
// What decoding in the product is reckoned to take (us): the longest workgroup's
// steps, by kind and row tiles (three-bit codes straddle words: 0.42 more), the
// reduction of each tile that it has a part of, and the joining of shared tiles
// (their partials through memory, and one tile's through one workgroup).
double fused_us(const Shape &s) {
  static const double step[3][kMts] = {{1.5, 1.5, 1.5, 2.2, 2.8}, {2.1, 2.1, 2.1, 2.5, 2.6}, {2.0, 2.0, 4.1, 5.5, 5.5}};
  const int64_t steps = s.parts ? (s.steps + s.parts - 1) / s.parts : (s.units + s.grid - 1) / s.grid;
  const double part = (double)s.partial_bytes / 2 / s.grid;
  int64_t tiles = 1;
  if (!s.parts) tiles = s.units % s.grid == 0 && steps % s.steps == 0 ? steps / s.steps : (steps - 1) / s.steps + (s.steps > 1 ? 2 : 1);
  double us = steps * (step[s.kind][s.mt] + (s.bits == 3 ? 0.42 : 0)) + tiles * (0.8 + 20e-6 * part);
  if (s.parts != 1) {
    double share = s.parts ? s.parts : (double)s.grid / s.tiles + 1;
    if (share > s.steps) share = s.steps;
    us += part * (0.366e-6 * s.grid + 8.5e-6 * share);
  }
  return us;
}
// Whether W is decoded once into the workspace: where unpacking it, packing the
// rows and the dense product of both are reckoned to take less than decoding it
// in the product for every tile of rows. The figures of both sides are fitted
// to their times at 3776 points (all four operators, 1 to 4096 rows, sixteen
// matrices with K and N from 256 to 17408): the side taken is 0.4% slower than
// the better one on average, at 48 points more than 10% and at most 21%.
// Measured, decoding in the product against this (us), k = 4. K = 5120, N =
// 17408: adapters 130 / 146 at 353 rows, 167 / 149 at 385, 200 / 195 at 576;
// gated 260 / 295 at 449, 337 / 335 at 576, 420 / 339 at 768; adapters_backward
// 148 / 141 at 193, 155 / 172 at 257, 188 / 178 at 353; gated_backward 215 /
// 266 at 257, 279 / 276 at 353, 339 / 292 at 385. K = 17408, N = 5120: adapters
// 196 / 216 at 640, 270 / 242 at 1024; gated 185 / 249 at 353, 334 / 322 at 640
// (at 512 it takes the 263 of 247 / 263); adapters_backward 156 / 172 at 257,
// 194 / 176 at 353; gated_backward 210 / 270 at 257, 336 / 277 at 385. K =
// 1024, N = 4096: adapters 32 / 45 at 1024, 53 / 47 at 2048; gated 20 / 35 at
// 449, 69 / 52 at 2048; adapters_backward 47 / 48 at 97, 66 / 60 at 449;
// gated_backward 44 / 41 at 97, 50 / 45 at 449.
Plan plan_of(int kind, trellis_geom g, int32_t m, int matrices, int cus) {
  Plan p{};
  p.fused = shape_of(kind, g, m, matrices, cus);
  const int forced = g_path.load(std::memory_order_relaxed);
  p.dense = forced == 1 || p.fused.units >= ((int64_t)1 << 30);  // (the product kernel counts them in 32 bits)
  if (p.dense) {
    p.many = dense_shape(kind, g, m, matrices, cus);
  } else if (forced < 0) {
    const double mb = 2e-6 * (kind == kGated ? 2 : matrices) * g.n * g.k;
    const double rows_mb = 4e-6 * m * (kind == kTransposed ? (double)g.n * matrices : g.k);
    const double rest = fused_us(p.fused) - (6.5 + 0.187 * mb + 0.14 * rows_mb);
    if (rest > 0) {  // (the layout of few rows' dense product is not worked out)
      p.many = dense_shape(kind, g, m, matrices, cus);
      p.dense = p.many.us < rest;
    }
  }
  if (p.dense) {
    p.bytes = up256(p.many.operand_bytes) + up256(p.many.row_bytes) + p.many.partial_bytes;
  } else {
    p.bytes = p.fused.partial_bytes;
    p.counters = p.fused.tiles;
  }
  return p;
}
trellis_status run(const Plan &pl, int kind, trellis_geom g, Product p, const GatedGrads *grads, unsigned char *ws,
                   hipStream_t stream) {
  if (pl.dense) return launch_dense(kind, pl.many, g, p, grads, ws, stream);
  if (grads) {
    const int64_t quads = (int64_t)p.m * (g.n / 4);
    (void)hipGetLastError();
    hipLaunchKernelGGL(gated_grad_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, grads->dh,
                       grads->gate, grads->up, quads, grads->dgate, grads->dup);
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
  }
  p.partials = reinterpret_cast<float *>(ws);
  return launch(pl.fused, p, stream);
}

// A shrink product: 64 rows a workgroup where there are enough to fill the
// card that way, else 16; spans of columns until the card is full.
struct ShrinkShape {
  int64_t groups, cells;  // of rows; with the rank's
  int ms, spans, span;
  size_t partial_bytes;
};
ShrinkShape shrink_shape(int m, int cols, int count, int rank, int cus) {
  ShrinkShape s{};
  s.ms = m >= 512 ? 4 : 1;
  s.groups = ((int64_t)m + 16 * s.ms - 1) / (16 * s.ms);
  s.cells = s.groups * ((rank + 31) / 32);
  int64_t spans = ((int64_t)cus + s.cells - 1) / s.cells;
  // A wave takes 128 columns at a time, and the waves that share an adapter as
  // many side by side: a narrower span leaves waves without work, and up to two
  // such spans cost less than what joining spans does (about 3 us).
  const int named = s.ms == 1 && count < 8 ? (count < m ? count : m) : 8;
  const int least = 128 * (8 / named);
  const int64_t most = cols <= 2 * least ? 1 : (cols + least - 1) / least;
  if (spans > most) spans = most;
  const int batches = s.ms == 1 ? 4 : 1;  // SHARES of the kernel
  if (spans > kSpanBatch * batches) spans = kSpanBatch * batches;
  s.span = (int)((cols + spans - 1) / spans + 31) / 32 * 32;
  s.spans = (cols + s.span - 1) / s.span;
  s.partial_bytes = s.spans > 1 ? (size_t)s.cells * s.spans * s.ms * 2 * 1024 : 0;
  return s;
}
trellis_status launch_shrink(const ShrinkShape &h, const Shrink &s, hipStream_t stream) {
  (void)hipGetLastError();
  const dim3 grid((unsigned)h.groups, (unsigned)h.spans, (unsigned)(s.rank_p / 32));
  if (h.ms == 4) hipLaunchKernelGGL((shrink_kernel<4, 4>), grid, dim3(256), 0, stream, s);
  else hipLaunchKernelGGL((shrink_kernel<1, 8>), grid, dim3(512), 0, stream, s);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}
trellis_status launch_backward_sums(const ShrinkShape &ht, const ShrinkShape &hu, const BackwardSums &b, hipStream_t stream) {
  (void)hipGetLastError();
  // Many adapters for few rows: workgroups beside the sums' for their ranges.
  const int64_t ranges = ((b.t.count < 256 ? b.t.count : 256) + ht.groups - 1) / ht.groups;
  int64_t y = ht.spans > hu.spans ? ht.spans : hu.spans;
  if (y < ranges) y = ranges;
  const dim3 grid((unsigned)ht.groups, (unsigned)y, (unsigned)(2 * (b.t.rank_p / 32) + 1));
  if (ht.ms == 4) hipLaunchKernelGGL((backward_sums_kernel<4, 4>), grid, dim3(256), 0, stream, b);
  else hipLaunchKernelGGL((backward_sums_kernel<1, 8>), grid, dim3(512), 0, stream, b);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

}  // namespace
}  // namespace trellis

using namespace trellis;

#define TRELLIS_TRY(e)                      \
  do {                                      \
    const trellis_status rc_ = (e);         \
    if (rc_ != TRELLIS_OK) return rc_;      \
  } while (0)

extern "C" {

int trellis_test_force_path(int path, int tiles) {
  if (path < -1 || path > 1 || tiles < 0) return -2;
  g_path.store(path);
  g_tiles.store(tiles);
  return 0;
}

trellis_status trellis_adapters(const uint16_t *x, int32_t m, const uint32_t *codes, const uint16_t *scales,
                                trellis_geom g, const uint16_t *a, const uint16_t *b, const float *gain,
                                const int32_t *index, int32_t count, int32_t rank, uint16_t *out, void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (count < 1 || count > TRELLIS_MAX_ADAPTERS || rank < 1 || rank > TRELLIS_MAX_RANK) return TRELLIS_E_ADAPTERS;
  if (!x || !codes || !scales || !a || !b || !gain || !index || !out) return TRELLIS_E_NULL;
  if (!on(x, 16) || !on(codes, 16) || !on(scales, 2) || !on(a, 16) || !on(b, 16) || !on(gain, 4) || !on(index, 4) ||
      !on(out, 16))
    return TRELLIS_E_ALIGN;
  hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
  std::lock_guard<std::mutex> lock(g_lock);
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const int rank_p = (rank + 31) / 32 * 32;
  const Plan s = plan_of(kForward, g, m, 1, cus);
  const ShrinkShape h = shrink_shape(m, g.k, count, rank, cus);
  const size_t t_bytes = up256((size_t)m * rank_p * 4), hp = up256(h.partial_bytes);
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, t_bytes + hp + s.bytes, (size_t)(s.counters > h.cells ? s.counters : h.cells), w));
  float *const t = reinterpret_cast<float *>(w->bytes);
  Shrink sh{x, a, gain, index, t, reinterpret_cast<float *>(w->bytes + t_bytes), w->counters, m, g.k, count, rank, rank_p, h.span, h.spans};
  TRELLIS_TRY(launch_shrink(h, sh, stream));
  Product p{};
  p.p = x;
  p.codes = codes;
  p.scales = scales;
  p.out = out;
  p.counters = w->counters;
  p.m = m;
  p.n = g.n;
  p.k = g.k;
  p.low = LowRank{index, b, t, count, rank, rank_p};
  return run(s, kForward, g, p, nullptr, w->bytes + t_bytes + hp, stream);
}

trellis_status trellis_adapters_backward(const uint16_t *dout, const uint16_t *x, int32_t m, const uint32_t *codes,
                                         const uint16_t *scales, trellis_geom g, const uint16_t *a, const uint16_t *b,
                                         const float *gain, const int32_t *index, int32_t count, int32_t rank,
                                         uint16_t *dx, uint16_t *da, uint16_t *db, void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (count < 1 || count > TRELLIS_MAX_ADAPTERS || rank < 1 || rank > TRELLIS_MAX_RANK) return TRELLIS_E_ADAPTERS;
  if (!dout || !x || !codes || !scales || !a || !b || !gain || !index || !dx || !da || !db) return TRELLIS_E_NULL;
  if (!on(dout, 16) || !on(x, 16) || !on(codes, 16) || !on(scales, 2) || !on(a, 16) || !on(b, 16) || !on(gain, 4) ||
      !on(index, 4) || !on(dx, 16) || !on(da, 16) || !on(db, 16))
    return TRELLIS_E_ALIGN;
  hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
  std::lock_guard<std::mutex> lock(g_lock);
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const int rank_p = (rank + 31) / 32 * 32;
  const Plan s = plan_of(kTransposed, g, m, 1, cus);
  const ShrinkShape hx = shrink_shape(m, g.k, count, rank, cus), hd = shrink_shape(m, g.n, count, rank, cus);
  const size_t t_bytes = up256((size_t)m * rank_p * 4), r_bytes = up256((size_t)count * sizeof(i32x2));
  // t's and u's spans are joined at the same time: partials and counters of their own.
  const size_t part_t = up256(hx.partial_bytes), sums = part_t + hd.partial_bytes;
  const int64_t cells = hx.cells + hd.cells;
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, 2 * t_bytes + r_bytes + (sums > s.bytes ? sums : s.bytes),
                    (size_t)(s.counters > cells ? s.counters : cells), w));
  float *const t = reinterpret_cast<float *>(w->bytes), *const u = reinterpret_cast<float *>(w->bytes + t_bytes);
  i32x2 *const range = reinterpret_cast<i32x2 *>(w->bytes + 2 * t_bytes);
  unsigned char *const rest = w->bytes + 2 * t_bytes + r_bytes;
  const BackwardSums b_sums{Shrink{x, a, gain, index, t, reinterpret_cast<float *>(rest), w->counters, m, g.k, count, rank,
                                   rank_p, hx.span, hx.spans},
                            Shrink{dout, b, gain, index, u, reinterpret_cast<float *>(rest + part_t), w->counters + hx.cells, m,
                                   g.n, count, rank, rank_p, hd.span, hd.spans},
                            range};
  TRELLIS_TRY(launch_backward_sums(hx, hd, b_sums, stream));
  Product p{};
  p.p = dout;
  p.codes = codes;
  p.scales = scales;
  p.out = dx;
  p.counters = w->counters;
  p.m = m;
  p.n = g.n;
  p.k = g.k;
  p.low = LowRank{index, a, u, count, rank, rank_p};
  TRELLIS_TRY(run(s, kTransposed, g, p, nullptr, rest, stream));
  Outer o{x, dout, u, t, index, range, da, db, m, g.n, g.k, rank, rank_p, g.k / 64};
  hipLaunchKernelGGL(outer_kernel, dim3((unsigned)(o.tiles_a + (g.n + 63) / 64), (unsigned)count, (unsigned)(rank_p / 32)),
                     dim3(256), 0, stream, o);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

trellis_status trellis_gated(const uint16_t *x, int32_t m, const uint32_t *codes_gate, const uint16_t *scales_gate,
                             const uint32_t *codes_up, const uint16_t *scales_up, trellis_geom g, uint16_t *h,
                             uint16_t *gate, uint16_t *up, void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (!x || !codes_gate || !scales_gate || !codes_up || !scales_up || !h) return TRELLIS_E_NULL;
  if (!on(x, 16) || !on(codes_gate, 16) || !on(scales_gate, 2) || !on(codes_up, 16) || !on(scales_up, 2) || !on(h, 16) ||
      !on(gate, 16) || !on(up, 16))
    return TRELLIS_E_ALIGN;
  hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
  std::lock_guard<std::mutex> lock(g_lock);
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const Plan s = plan_of(kGated, g, m, 1, cus);
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, s.bytes, (size_t)s.counters, w));
  Product p{};
  p.p = x;
  p.codes = codes_gate;
  p.codes2 = codes_up;
  p.scales = scales_gate;
  p.scales2 = scales_up;
  p.out = h;
  p.gate = gate;
  p.up = up;
  p.counters = w->counters;
  p.m = m;
  p.n = g.n;
  p.k = g.k;
  return run(s, kGated, g, p, nullptr, w->bytes, stream);
}

trellis_status trellis_gated_backward(const uint16_t *dh, const uint16_t *gate, const uint16_t *up, int32_t m,
                                      const uint32_t *codes_gate, const uint16_t *scales_gate,
                                      const uint32_t *codes_up, const uint16_t *scales_up, trellis_geom g,
                                      uint16_t *dx, uint16_t *dgate, uint16_t *dup, void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (!dh || !gate || !up || !codes_gate || !scales_gate || !codes_up || !scales_up || !dx || !dgate || !dup)
    return TRELLIS_E_NULL;
  if (!on(dh, 16) || !on(gate, 16) || !on(up, 16) || !on(codes_gate, 16) || !on(scales_gate, 2) || !on(codes_up, 16) ||
      !on(scales_up, 2) || !on(dx, 16) || !on(dgate, 16) || !on(dup, 16))
    return TRELLIS_E_ALIGN;
  hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
  std::lock_guard<std::mutex> lock(g_lock);
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const Plan s = plan_of(kTransposed, g, m, 2, cus);
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, s.bytes, (size_t)s.counters, w));
  const GatedGrads grads{dh, gate, up, dgate, dup};
  Product p{};
  p.p = dgate;
  p.p2 = dup;
  p.codes = codes_gate;
  p.codes2 = codes_up;
  p.scales = scales_gate;
  p.scales2 = scales_up;
  p.out = dx;
  p.counters = w->counters;
  p.m = m;
  p.n = g.n;
  p.k = g.k;
  return run(s, kTransposed, g, p, &grads, w->bytes, stream);
}

}  // extern "C"
