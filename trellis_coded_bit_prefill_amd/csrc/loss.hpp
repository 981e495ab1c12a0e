// Losses over a packed vocabulary matrix W[N, K]: softmax cross entropy against
// one entry a row and against a teacher's listed entries, and the gradient of x.
// Part of rows.hip, whose products, plans and workspaces they use.
//
// With l2 = l log2(e) / T, R a row's largest l2 and S = sum_v 2^(l2_v - R):
//   lse = (R + log2 S) ln 2,  p_v = 2^(l2_v - R) / S,
//   d_v = T (p_v - q_v),      dx = d W  (the gradient with respect to the logits is d).
// The listed entries are taken out of the sum first and added at the end, so
// that a row with one entry has 1 - p = S' / S from the sum S' over the others:
// as the difference of two numbers near 1 it would lose its digits.
//
// Few rows: the logits of a chunk of rows lie in the workspace in float32
// (loss_rows). Many rows: the product's tiles are turned into 2^(l2 - ref) in
// bf16 before they leave the registers, as the second product's operands, with
// each tile's sums beside them (vocabulary_kernel, loss_dense).

namespace trellis {
namespace {

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr int kMaxTop = TRELLIS_MAX_TOP;
constexpr float kLowest = -3.402823466e38f;
constexpr int64_t kLogitBytes = (int64_t)1 << 30;  // of a chunk of rows

// The rows' lists: logits null: one entry of probability 1 (cross entropy).
struct Lists {
  const int32_t *index;
  const float *logits;
  float *listed;     // [m, top]: l2 of the listed entries
  int32_t n, top;
  float temperature, scale2;  // scale2: log2(e) / T
  float *loss, *lse;
};

// The vocabulary entry at a place of the lists, -1 where there is none: an index
// outside, or a teacher's logit of -inf. Such a place must not count, or a row of
// one entry beside it would lose the digits of its 1 - p. (Lists of one place keep
// it whatever its logit: row_single puts it back into the sum.)
__device__ __forceinline__ int list_entry(const Lists &L, int64_t place) {
  const int at = L.index[place];
  if (at < 0 || at >= L.n) return -1;
  return L.top > 1 && L.logits[place] == -__builtin_inff() ? -1 : at;
}

// (largest, sum of 2^(v - largest)) of two parts of a row; a part without finite
// entries has kLowest and 0.
__device__ __forceinline__ f32x2 join_stats(f32x2 a, f32x2 b) {
  const float r = fmaxf(a[0], b[0]);
  return f32x2{r, a[1] * __builtin_amdgcn_exp2f(a[0] - r) + b[1] * __builtin_amdgcn_exp2f(b[0] - r)};
}
__device__ __forceinline__ f32x2 join_stats_wave(f32x2 a) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) a = join_stats(a, f32x2{__shfl_xor(a[0], o), __shfl_xor(a[1], o)});
  return a;
}

constexpr int kStatSpan = 4096;  // logits of a workgroup

// Largest and sum of a span of a row without the listed entries, whose l2 go to
// `listed`: a bit map in LDS says which they are.
__global__ __launch_bounds__(256) void row_stats_kernel(Lists L, const float *__restrict__ logits,
                                                        f32x2 *__restrict__ stats) {
  __shared__ f32x2 part[4];
  __shared__ uint32_t listed[kStatSpan / 32];
  const int64_t row = blockIdx.x;  // (y and z of a grid are limited to 2^16)
  const int tid = threadIdx.x, first = blockIdx.y * kStatSpan;
  const float *const l = logits + row * L.n;
  const float inf = __builtin_inff();
  f32x4 v[kStatSpan / 1024];
#pragma unroll
  for (int i = 0; i < kStatSpan / 1024; ++i) {
    const int c = first + 1024 * i + 4 * tid;
    v[i] = f32x4{-inf, -inf, -inf, -inf};
    if (c < L.n) v[i] = *reinterpret_cast<const f32x4 *>(l + c) * L.scale2;
  }
  if (tid < kStatSpan / 32) listed[tid] = 0u;
  __syncthreads();
  if (tid < L.top) {
    const int at = list_entry(L, row * L.top + tid);
    if (at >= first && at - first < kStatSpan) {
      L.listed[row * L.top + tid] = l[at] * L.scale2;
      atomicOr(&listed[(at - first) >> 5], 1u << (at & 31));
    }
  }
  __syncthreads();
  float r = kLowest;
#pragma unroll
  for (int i = 0; i < kStatSpan / 1024; ++i) {
    const uint32_t out = listed[32 * i + (tid >> 3)] >> (4 * (tid & 7));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((out >> e) & 1) v[i][e] = -inf;
      r = fmaxf(r, v[i][e]);
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kStatSpan / 1024; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(v[i][e] - r);
  const f32x2 a = join_stats_wave(f32x2{r, s});
  if ((tid & 63) == 0) part[tid >> 6] = a;
  __syncthreads();
  if (tid == 0) stats[row * gridDim.y + blockIdx.y] = join_stats(join_stats(part[0], part[1]), join_stats(part[2], part[3]));
}

// What a workgroup of 256 threads works out of a row's list and of its other
// entries' sum; the list in LDS.
struct RowList {
  int at[kMaxTop];       // -1: none
  float q[kMaxTop], qs[kMaxTop];  // of each place; of the entry, all its places together
  float add[kMaxTop];    // d of the entry (its first place in the list), without T
  uint8_t first[kMaxTop];
  float red[2][4];
  f32x2 total;           // R and S of the whole row
  int rest_at[kMaxTop], rests;  // listed_rests()
  float rest[kMaxTop], rest_scale[kMaxTop];
};
__device__ __forceinline__ float sum_256(float v, float *red) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}
__device__ __forceinline__ float max_256(float v, float *red) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}
// -log p of a row's only entry: log(1 + S' / e).
__device__ __forceinline__ float sole_loss(f32x2 rest, float l2) {
  if (l2 == __builtin_inff()) return l2 - l2;
  const float ratio = (rest[0] - l2) * kLn2 + logf(rest[1]);
  return ratio > 0.f ? ratio + log1pf(expf(-ratio)) : log1pf(expf(ratio));
}
// row_list for lists of one: nothing to sum, every thread works it out.
__device__ __forceinline__ bool row_single(const Lists &L, int64_t row, f32x2 rest, bool whole, RowList &S, bool write) {
  int at = L.index[row];
  if (at >= L.n) at = -1;
  const bool valid = at >= 0;
  const float z = valid && L.logits ? L.logits[row] : 0.f;
  const bool alive = valid && z != -__builtin_inff();
  const float q = (z - z) + 1.f;  // softmax of one logit; NaN where it is not a number
  const float l2 = valid ? L.listed[row] : 0.f;
  const float rmax = valid && !whole ? fmaxf(l2, rest[0]) : rest[0];
  const float others = rest[1] * __builtin_amdgcn_exp2f(rest[0] - rmax);
  const float sum = others + (valid && !whole ? __builtin_amdgcn_exp2f(l2 - rmax) : 0.f);
  S.at[threadIdx.x] = threadIdx.x == 0 ? at : -1;
  S.first[threadIdx.x] = threadIdx.x == 0 && valid;
  S.add[threadIdx.x] = q * (-others / sum);
  S.qs[threadIdx.x] = q;
  if (threadIdx.x == 0) {
    S.total = f32x2{rmax, sum};
    if (write) {
      L.loss[row] = alive ? L.temperature * L.temperature * q * sole_loss(rest, l2) : 0.f;
      L.lse[row] = (rmax + __builtin_amdgcn_logf(sum)) * kLn2;
    }
  }
  __syncthreads();
  return alive;
}
// rest: R' and S' of the entries that are not listed, or of all (`whole`; then
// the list has not exactly one entry, else some digits of 1 - p are lost).
// Returns whether the row has entries; loss and lse where `write`.
static_assert(kMaxTop == 256, "one thread an entry");
__device__ bool row_list(const Lists &L, int64_t row, f32x2 rest, bool whole, RowList &S, bool write) {
  const int j = threadIdx.x;
  const float inf = __builtin_inff();
  if (L.top == 1) return row_single(L, row, rest, whole, S, write);
  const int at = j < L.top ? list_entry(L, row * L.top + j) : -1;
  float z = -inf, l2 = -inf;
  if (at >= 0) {
    z = L.logits[row * L.top + j];
    l2 = L.listed[row * L.top + j];
  }
  S.at[j] = at;
  // q: softmax of the list. A NaN among the teacher's logits is a NaN in the sum.
  // The difference first: the lowest finite logit, a mask's, times log2(e) / T
  // would be -inf, which is no entry, and the largest inf.
  const float zmax = fmaxf(max_256(z, S.red[0]), kLowest);
  const float z2 = (z - zmax) * L.scale2, e = at >= 0 ? __builtin_amdgcn_exp2f(z2) : 0.f;
  const float total = sum_256(e, S.red[1]);
  const bool alive = total != 0.f;
  const float q = alive ? e / total : 0.f;
  S.q[j] = q;
  __syncthreads();
  // every entry once: its first place adds to the sum
  bool first = at >= 0;
  float qs = 0.f;
  for (int k = 0; k < L.top; ++k)
    if (S.at[k] == at) {
      qs += S.q[k];
      if (k < j) first = false;
    }
  const float rmax = whole ? rest[0] : fmaxf(max_256(first ? l2 : -inf, S.red[0]), rest[0]);
  const float here = first ? __builtin_amdgcn_exp2f(l2 - rmax) : 0.f;
  const float others = rest[1] * __builtin_amdgcn_exp2f(rest[0] - rmax);
  const float sum = others + (whole ? 0.f : sum_256(here, S.red[1]));
  const float lse2 = rmax + __builtin_amdgcn_logf(sum);
  // one entry alone: 1 - p and the loss from the others' sum
  const bool alone = sum_256(first ? 1.f : 0.f, S.red[0]) == 1.f && !whole;
  if (j == 0) S.total = f32x2{rmax, sum};
  S.first[j] = first;
  S.qs[j] = qs;
  S.add[j] = !first ? 0.f : alone ? qs * (-others / sum) : here / sum - qs;
  float term = q != 0.f ? q * (z2 - __builtin_amdgcn_logf(total)) * kLn2 : 0.f;  // q log q
  if (!alone) {
    if (q != 0.f) term += q * (lse2 - l2) * kLn2;
  } else if (first) {
    term += sole_loss(rest, l2);
  }
  const float loss = sum_256(term, S.red[1]);
  if (write && j == 0) {
    L.loss[row] = alive ? L.temperature * L.temperature * loss : 0.f;
    L.lse[row] = lse2 * kLn2;
  }
  __syncthreads();
  return alive;
}

// What the listed entries' gradients lose as operands: the logits' gradients are
// bf16 in the product with W, because that is what the matrix cores multiply at
// their rate, each off by up to 2^-8 of itself. Over the vocabulary these errors
// have either sign and cancel for the most part. Those of the listed entries, which
// are most of a row's gradient, do not (dx off by 0.0019 to 0.0029 relative, where
// its own last rounding alone is 0.0017). So their rests x - bf16(x) are multiplied
// with their rows of W here, in float32, and `add` [m, k] joins the product's sums:
// 0.0017 then, but where an unlisted entry is most of a gradient. Left out are rests
// of entries so small that, squared, all of them are at most a sixteenth of the
// list's gradients (their error then at most a quarter of what it was).
// It costs cross entropy 1.5 us of 18 at 5 rows and 25 of 5060 at 2048 (N = 131072,
// K = 5120), 3 of 165 at 19 rows with lists of 8, 25 to 60 of 2650 at 2048 with
// lists of 64; at worst, lists of 256 entries of like gradients, as much as a row of
// W decoded for each: 16384 x 4096, 192 rows, 141 to 225.
// value: what the workgroup's thread j has rounded for its entry, 0 where it has
// none; wave w of `waves` takes the 256-column blocks w, w + waves ..
struct Rests {
  const uint32_t *codes;
  const uint16_t *scales;
  float *add;
  int32_t blocks;  // of 256 columns
};
template <int BITS>
__device__ __forceinline__ void listed_rests(const Lists &L, const Rests &F, int64_t row, float value, int wave0, int waves,
                                             RowList &S) {
  constexpr int wpb = 8 * BITS;
  const int j = threadIdx.x, lane = j & 63, wave = __builtin_amdgcn_readfirstlane(j >> 6);
  const float rest = value - bf16_bits_to_f32(bf16_of(value)), part = value != 0.f ? S.add[j] : 0.f;
  const float all = sum_256(part * part, S.red[0]);
  // (an infinity or a NaN is the product's)
  const bool keep = fabsf(rest) > 0.f && fabsf(rest) < __builtin_inff() && !(part * part * (16.f * (float)L.top) < all);
  const uint64_t kept = __ballot(keep);
  const float s = keep ? bf16_bits_to_f32(F.scales[S.at[j]]) : 1.f;
  const bool odd = !__all(alu_scale_ok(s));
  __syncthreads();
  if (lane == 0) {
    S.red[0][wave] = (float)__popcll(kept);
    S.red[1][wave] = odd ? 1.f : 0.f;
  }
  __syncthreads();
  int at = 0;
  for (int w = 0; w < wave; ++w) at += (int)S.red[0][w];
  const int count = __builtin_amdgcn_readfirstlane((int)((S.red[0][0] + S.red[0][1]) + (S.red[0][2] + S.red[0][3])));
  const bool chain = __builtin_amdgcn_readfirstlane((S.red[1][0] + S.red[1][1]) + (S.red[1][2] + S.red[1][3]) != 0.f) != 0;
  if (keep) {
    const int to = at + (int)__popcll(kept & ((1ull << lane) - 1ull));
    S.rest_at[to] = S.at[j];
    S.rest[to] = rest;
    S.rest_scale[to] = s;
  }
  __syncthreads();
  const int pos = (252 - 4 * lane) * BITS, w0 = pos >> 5, w1 = w0 + 1 == wpb ? 0 : w0 + 1, sh = pos & 31;
  auto columns = [&](auto chained) {
    for (int b = __builtin_amdgcn_readfirstlane(wave0); b < F.blocks; b += waves) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      // `some` entries' words on their way at once: one after the other they would cost a memory latency each
      auto take = [&](int i, auto some) {
        constexpr int U = decltype(some)::value;
        uint32_t f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t *const bw = F.codes + ((int64_t)__builtin_amdgcn_readfirstlane(S.rest_at[i + u]) * F.blocks + b) * wpb;
          f[u] = __builtin_amdgcn_alignbit(bw[w1], bw[w0], sh);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float r = S.rest[i + u], sc = S.rest_scale[i + u];
          float q, kq;
          alu_row_constants(sc, q, kq);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = __builtin_fmaf(r, (float)(__bf16)window_weight(__builtin_amdgcn_ubfe(f[u], (3 - c) * BITS, 12), sc, q, kq, decltype(chained)::value), v[c]);
        }
      };
      int i = 0;
      for (; i + 16 <= count; i += 16) take(i, std::integral_constant<int, 16>{});
      for (; i + 4 <= count; i += 4) take(i, std::integral_constant<int, 4>{});
      for (; i < count; ++i) take(i, std::integral_constant<int, 1>{});
      *reinterpret_cast<f32x4 *>(F.add + (row * F.blocks + b) * 256 + 4 * lane) = v;
    }
  };
  if (chain) columns(std::true_type{});
  else columns(std::false_type{});
}

// Loss and lse of a row and, where d is not null, the gradient of its logits in
// a span, and the listed entries' rests in a part of the columns.
template <int BITS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 4))) void row_loss_kernel(Lists L, const float *__restrict__ logits,
                                                       const f32x2 *__restrict__ stats, int spans,
                                                       uint16_t *__restrict__ d, Rests F) {
  __shared__ RowList S;
  const int64_t row = blockIdx.x;
  // every wave joins the spans, in the same order
  f32x2 rest = {kLowest, 0.f};
  for (int i = threadIdx.x & 63; i < spans; i += 64) rest = join_stats(rest, stats[row * spans + i]);
  rest = join_stats_wave(rest);
  const bool alive = row_list(L, row, rest, false, S, blockIdx.y == 0);
  if (!d) return;
  const float r = S.total[0], f = alive ? L.temperature / S.total[1] : 0.f;
  const int c0 = blockIdx.y * kStatSpan;
  const float *const l = logits + row * L.n;
  uint16_t *const o = d + row * L.n;
#pragma unroll
  for (int i = 0; i < kStatSpan / 1024; ++i) {
    const int c = c0 + 1024 * i + 4 * (int)threadIdx.x;
    if (c >= L.n) continue;
    const f32x4 v = *reinterpret_cast<const f32x4 *>(l + c) * L.scale2;
    f32x4 g;
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = alive ? f * __builtin_amdgcn_exp2f(v[e] - r) : 0.f;
    store4(o + c, g);
  }
  __syncthreads();
  const int at = S.at[threadIdx.x];
  const float value = S.first[threadIdx.x] && alive ? L.temperature * S.add[threadIdx.x] : 0.f;
  if (S.first[threadIdx.x] && at >= c0 && at < c0 + kStatSpan && alive) o[at] = bf16_of(value);
  listed_rests<BITS>(L, F, row, value, (int)blockIdx.y * 4 + (int)(threadIdx.x >> 6), 4 * (int)gridDim.y, S);
}

// Rows of up to 16384 logits in one launch instead of three: the row stays in
// registers, 64 logits a thread at most, and a bit map in LDS says which are listed.
constexpr int kWholeRow = 16384;
template <int BITS>
__global__ __launch_bounds__(256) void whole_row_kernel(Lists L, const float *__restrict__ logits,
                                                        uint16_t *__restrict__ d, Rests F) {
  __shared__ RowList S;
  __shared__ uint32_t listed[kWholeRow / 32];
  __shared__ f32x2 part[4];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const float *const l = logits + row * L.n;
  constexpr int kQuads = kWholeRow / 1024;
  const float inf = __builtin_inff();
  f32x4 v[kQuads];
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int c = 1024 * i + 4 * tid;
    v[i] = f32x4{-inf, -inf, -inf, -inf};
    if (c < L.n) v[i] = *reinterpret_cast<const f32x4 *>(l + c);
  }
  const int at = tid < L.top ? list_entry(L, row * L.top + tid) : -1;
  if (tid < L.top) L.listed[row * L.top + tid] = at >= 0 ? l[at] * L.scale2 : 0.f;
  for (int i = tid; i < (L.n + 31) / 32; i += 256) listed[i] = 0u;
  __syncthreads();
  if (at >= 0) atomicOr(&listed[at >> 5], 1u << (at & 31));
  __syncthreads();
  float r = kLowest;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    if (1024 * i < L.n) {
      const int c = 1024 * i + 4 * tid;
      const uint32_t out = c < L.n ? listed[c >> 5] >> (c & 31) : 0u;
      const f32x4 x = v[i] * L.scale2;
      v[i] = f32x4{out & 1 ? -inf : x[0], out & 2 ? -inf : x[1], out & 4 ? -inf : x[2], out & 8 ? -inf : x[3]};
      r = fmaxf(r, fmaxf(fmaxf(v[i][0], v[i][1]), fmaxf(v[i][2], v[i][3])));
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    if (1024 * i < L.n)
      s += (__builtin_amdgcn_exp2f(v[i][0] - r) + __builtin_amdgcn_exp2f(v[i][1] - r)) +
           (__builtin_amdgcn_exp2f(v[i][2] - r) + __builtin_amdgcn_exp2f(v[i][3] - r));
  }
  const f32x2 a = join_stats_wave(f32x2{r, s});
  if ((tid & 63) == 0) part[tid >> 6] = a;
  __syncthreads();
  const f32x2 rest = join_stats(join_stats(part[0], part[1]), join_stats(part[2], part[3]));
  const bool alive = row_list(L, row, rest, false, S, true);
  if (!d) return;
  const float rmax = S.total[0], f = L.temperature / S.total[1];
  uint16_t *const o = d + row * L.n;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int c = 1024 * i + 4 * tid;
    if (c < L.n) {
      f32x4 g;
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = alive ? f * __builtin_amdgcn_exp2f(v[i][e] - rmax) : 0.f;
      store4(o + c, g);
    }
  }
  __syncthreads();
  const float value = S.first[tid] && alive ? L.temperature * S.add[tid] : 0.f;
  if (S.first[tid] && alive) o[S.at[tid]] = bf16_of(value);
  listed_rests<BITS>(L, F, row, value, tid >> 6, 4, S);
}

// dst = dloss[row] * src: a factor a row; dx, rounded once when it was kept, is
// rounded again. (dst may be src: neither is __restrict__.) 2048 rows of 5120: 7 us.
__global__ __launch_bounds__(256) void scale_rows_kernel(const float *__restrict__ f, const uint16_t *src, int64_t vectors,
                                                         int per_row, uint16_t *dst) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vectors; i += (int64_t)gridDim.x * 256) {
    const float s = f[i / per_row];
    const u32x4 v = reinterpret_cast<const u32x4 *>(src)[i];
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = (uint32_t)bf16_of(s * bf16_half(v[e], 0)) | ((uint32_t)bf16_of(s * bf16_half(v[e], 1)) << 16);
    reinterpret_cast<u32x4 *>(dst)[i] = o;
  }
}
constexpr int64_t kScaleGroups = 1 << 22;  // workgroups at most (a launch has fewer than 2^32 threads); beyond, a thread takes several

// ---- many rows ------------------------------------------------------------------

// Logits that are used as they are: a row's tile whose largest l2 lies within
// +-kPlain has 0 in place of its R. The logits of trained models do, and then
// all tiles of a row agree; another tile's reference is its largest l2 rounded
// down, a whole number, so that bringing it to the row's reference later is an
// exact product with a power of two. (2^60 times 2^22 entries and weights up to
// 2^44 stays below float32's and bf16's largest, 2^-60 far above their smallest.)
constexpr float kPlain = 60.f;

struct Vocabulary {
  const int32_t *sole;  // a row's only entry, taken out of its sum, or outside [0, n)
  float *sole_l2;       // its l2
  f32x2 *stats;         // [m][blocks]: reference and sum of a row in a block of columns
  uint16_t *e;          // 2^(l2 - reference) as operands [step][ptiles][lane][8], or null
  float scale2;
  int32_t n, blocks, first_tile, first_block, steps;  // steps: of the operands e
};

// The product's tile in, 2^(l2 - reference) and its sums out. Beside the
// product's steps (see dense_sums) a tile's end costs 4 operations and one
// exponential (a quarter of the rate) for each of its sums. 2048 rows, K = 5120, N
// = 131072: 2.23 to 2.38 ms, 1.16 to 1.23 PFLOP/s (a library product of this size,
// its logits in bf16: 1.21). The exponentials are rounded to bf16 because that is
// what the matrix cores multiply at this rate: each of dx's terms is off by up to
// 2^-8 of itself, of either sign (the sums are of the float32 exponentials).
template <int NT, int RT>
__device__ __forceinline__ void vocabulary_out(const Dense &D, const Vocabulary &V, const DenseAt &at, f32x4 (&acc)[RT][NT]) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int col0 = (V.first_tile + at.tile0) * 16 + 4 * g;  // this lane's first column
  const int block = V.first_block + at.tile0 / NT;
  const float inf = __builtin_inff();
  if (col0 + 16 * NT > V.n) {  // (columns past n: their sums are of whatever the last tile's operands were)
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (col0 + 16 * i >= V.n)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][i] = f32x4{-inf, -inf, -inf, -inf};
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = at.row0 + 16 * r + j;
    const bool in = row < D.m;
    const uint32_t sole = (uint32_t)(in ? V.sole[row] : -1) - (uint32_t)col0;
    if (__any(sole < 16u * NT)) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (sole == 16u * i + e && col0 + 16 * i < V.n) {
            V.sole_l2[row] = acc[r][i][e] * V.scale2;
            acc[r][i][e] = -inf;
          }
    }
    float top = -inf;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, acc[r][i][e]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32)) * V.scale2;
    float ref = 0.f;
    if (!(fabsf(top) <= kPlain)) ref = top == -inf ? kLowest : __builtin_floorf(top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[r][i][e], V.scale2, -ref));
        sum += x[e];
      }
      const int tile = V.first_tile + at.tile0 + i;
      if (V.e && in && (tile >> 1) < V.steps)
        store4(V.e + ((((int64_t)(tile >> 1) * D.ptiles + (row >> 4)) * 64 + j + 16 * (2 * (tile & 1) + (g >> 1))) * 8 + 4 * (g & 1)), x);
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g == 0 && in && block < V.blocks) V.stats[(int64_t)row * V.blocks + block] = f32x2{ref, sum};
  }
}
template <int NT, int RT>
__global__ __launch_bounds__(kDenseThreads) void vocabulary_kernel(Dense D, Vocabulary V) {
  f32x4 acc[RT][NT];
  const DenseAt at = dense_sums<NT, RT>(D, acc, [](const DenseAt &) {});
  vocabulary_out<NT, RT>(D, V, at, acc);
}

// The same with W decoded on the way: few hundred rows, which one or two tiles
// hold (64 RT rows by 128 columns a workgroup, 8 waves, 4 by rows x 2 by columns).
// P's operands reach LDS as in dense_sums, S steps ahead; a 256-weight block's
// code words too, a block ahead, and in every step each wave decodes 16 columns
// of the step after next into one of two LDS tiles. Everything that comes from
// memory is a copy to LDS, so that the waits are the kernel's own: a copy is
// waited for by the number of P's copies issued after it, which the words'
// copies between them only make stricter.
// A step of 384 rows and 128 columns has 768 clocks of MFMA, 640 of LDS reads and
// 256 of writes, and 500 of the decode's VALU work; it takes 1900 (0.78 us; 256
// rows 0.6), as the workgroup's waves meet at every step and the three overlap
// only in part: 0.64 us without the decode, 0.76 without the copies, 0.63 without
// the MFMAs. 333 rows, K = 5120, N = 50004, k = 3 in 241 us; decoded beforehand 139
// and a product of 192-row tiles 246; few rows' kernel, in three tiles, 310.
struct Packed {
  const uint32_t *codes;
  const uint16_t *scales;
  int32_t k;
};
constexpr int kDecodeColumns = 128;
constexpr int decode_lds_fixed(int bits) { return 2 * 8192 + 2 * 4096 * bits; }  // decoded tiles, code words
constexpr int decode_buffers(int bits, int rt) {
  return (160 * 1024 - decode_lds_fixed(bits)) / (4096 * rt) < 6 ? (160 * 1024 - decode_lds_fixed(bits)) / (4096 * rt) : 6;
}
constexpr int decode_lds(int bits, int rt) { return decode_buffers(bits, rt) * 4096 * rt + decode_lds_fixed(bits); }
// Where a row's 16-byte piece c of a block's words lies in LDS: rows lie 128, 96
// or 64 bytes apart, which without this would put 16 or 4 of them in one bank.
template <int BITS>
__device__ __forceinline__ int code_piece(int row, int c) {
  return BITS == 4 ? c ^ (row & 7) : BITS == 2 ? c ^ ((row >> 2) & 3) : c;
}
template <int BITS, int RT>
__global__ __launch_bounds__(kDenseThreads) void vocabulary_decode_kernel(Dense D, Vocabulary V, Packed C) {
  constexpr int NT = 4, kRows = 64 * RT, kA = kRows / 16 * 1024, S = decode_buffers(BITS, RT), kMost = RT / 2;
  constexpr int wpb = 8 * BITS, kCode = 4096 * BITS, kPieces = 2 * BITS;  // words of a row's block; bytes of 128; pieces
  static_assert(RT % 2 == 0 && S >= 3 && S <= 8, "every wave copies as many tiles; words are a block ahead");
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  constexpr uint32_t kB = S * kA, kC = kB + 2 * 8192;
  const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 3, wn = wave >> 2;
  const int total = D.mtiles * D.ntiles, each = total >> 3, rest = total & 7;
  const int xcd = blockIdx.x & 7, seq = blockIdx.x >> 3;
  const int id = xcd * each + (xcd < rest ? xcd : rest) + seq;
  const int tn = id / D.mtiles, tm = id - tn * D.mtiles;
  const int steps = D.steps, blocks = steps >> 3;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)lds;
  const int atiles = D.ptiles - tm * (kRows / 16);
  const unsigned char *const pa = reinterpret_cast<const unsigned char *>(D.p) + (int64_t)tm * (kRows / 16) * 1024;
  const int64_t astride = (int64_t)D.ptiles * 1024;
  auto stage = [&](int s, uint32_t buffer) {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int t = wave + 8 * i;  // (tiles past the last repeat it)
      copy_to_lds(lds0 + buffer + (uint32_t)(t * 1024), (uint32_t)lane * 16, pa + s * astride + (t < atiles ? t : atiles - 1) * 1024);
    }
  };
  // code words: copy c takes pieces 64 c .. +63 of the 128 rows' block
  const int n0 = tn * kDecodeColumns;
  const uint32_t row_bytes = (uint32_t)(C.k >> 8) * wpb * 4;
  const unsigned char *const pc = reinterpret_cast<const unsigned char *>(C.codes) + (int64_t)n0 * row_bytes;
  uint32_t from[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int q = (wave + 8 * i) * 64 + lane, row = q / kPieces, c = code_piece<BITS>(row, q % kPieces);
    from[i] = (uint32_t)(n0 + row < V.n ? row : V.n - 1 - n0) * row_bytes + 16u * (uint32_t)c;
  }
  auto words = [&](int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (wave + 8 * i < kCode / 1024)
        copy_to_lds(lds0 + kC + (uint32_t)((b & 1) * kCode + (wave + 8 * i) * 1024), from[i], pc + (int64_t)b * (wpb * 4));
  };
  // this lane's row of W in the tile that its wave decodes
  const int row = 16 * wave + j, n = n0 + row < V.n ? n0 + row : V.n - 1;
  const float sc = bf16_bits_to_f32(C.scales[n]);
  float q, kq;
  alu_row_constants(sc, q, kq);
  const bool chain = !__all(alu_scale_ok(sc));
  const int base = (248 - 8 * g) * BITS, w0 = base >> 5, off = base & 31;
  // The stream bits of a lane's eight weights of step s, and their weights into
  // the step's tile. (Past the last step: bits and a tile that nobody uses.)
  auto bits = [&](int s) {
    const unsigned char *const mine = lds + kC + ((s >> 3) & 1) * kCode + row * (wpb * 4);
    const int w = w0 - (s & 7) * BITS, next = w + 1 == wpb ? 0 : w + 1;
    const uint32_t lo = *reinterpret_cast<const uint32_t *>(mine + code_piece<BITS>(row, w >> 2) * 16 + (w & 3) * 4);
    const uint32_t hi = *reinterpret_cast<const uint32_t *>(mine + code_piece<BITS>(row, next >> 2) * 16 + (next & 3) * 4);
    return (((uint64_t)hi << 32) | lo) >> off;
  };
  auto decode = [&](int s, uint64_t f, auto chained) {
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = (__bf16)window_weight((uint32_t)(f >> ((7 - e) * BITS)) & 0xFFFu, sc, q, kq, decltype(chained)::value);
    *reinterpret_cast<bf16x8 *>(lds + kB + (s & 1) * 8192 + wave * 1024 + lane * 16) = v;
  };
  f32x4 acc[RT][NT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  words(0);
  if (blocks > 1) words(1);
#pragma unroll
  for (int b = 0; b < S; ++b)
    if (b < steps) stage(b, b * kA);
  step_barrier<0>();
  if (chain) {
    decode(0, bits(0), std::true_type{});
    decode(1, bits(1), std::true_type{});
  } else {
    decode(0, bits(0), std::false_type{});
    decode(1, bits(1), std::false_type{});
  }
  lds_barrier();
  struct Operands {
    bf16x8 a[RT], b[NT];
  };
  auto read = [&](Operands &O, uint32_t buffer, int s) {
    const unsigned char *const bb = lds + kB + (s & 1) * 8192 + lane * 16, *const ba = lds + buffer + lane * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) O.b[i] = *reinterpret_cast<const bf16x8 *>(bb + (wn * NT + i) * 1024);
#pragma unroll
    for (int i = 0; i < RT; ++i) O.a[i] = *reinterpret_cast<const bf16x8 *>(ba + (RT * wm + i) * 1024);
  };
  Operands X, Y;
  uint32_t now = 0;
  read(X, 0, 0);
  uint64_t f = bits(2);
  // Step s: the barrier says that step s + 1 of P has landed, that its decoded
  // tile is written and that step s has been read.
  auto step = [&](int s, const Operands &A, Operands &B, auto chained) {
    if (s + S - 1 < steps) step_barrier<(S - 2) * kMost>();
    else step_barrier<0>();
    if ((s & 7) == 6 && (s >> 3) + 2 < blocks) words((s >> 3) + 2);  // (its place was last read in step s - 2)
    if (s + S < steps) stage(s + S, now);
    now = now == (S - 1) * kA ? 0 : now + kA;
    read(B, now, s + 1);  // (past the last step: old operands, not used)
    const uint64_t next = bits(s + 3);
    decode(s + 2, f, chained);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A.b[i], A.a[r], acc[r][i], 0, 0, 0);
    f = next;
    // The reads and the decode go between the matrix instructions.
#pragma unroll
    for (int i = 0; i < NT * RT; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < RT + NT + 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
  };
  auto loop = [&](auto chained) {
    for (int s = 0; s < steps; s += 2) {
      step(s, X, Y, chained);
      step(s + 1, Y, X, chained);
    }
  };
  if (chain) loop(std::true_type{});
  else loop(std::false_type{});
  const DenseAt at{tm * kRows + 16 * RT * wm, tn * 2 * NT + wn * NT, 0};
  vocabulary_out<NT, RT>(D, V, at, acc);
}

// The second product: float32 sums of every split. 2048 rows, K = 5120, N =
// 131072: 2.24 to 2.30 ms, 1.2 PFLOP/s (a library product: 1.32).
template <int NT, int RT>
__global__ __launch_bounds__(kDenseThreads) void vocabulary_back_kernel(Dense D) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  f32x4 acc[RT][NT];
  const DenseAt at = dense_sums<NT, RT>(D, acc, [](const DenseAt &) {});
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = at.row0 + 16 * r + j;
    if (row >= D.m) continue;
    float *const q = D.partials + ((int64_t)at.split * D.m + row) * (16 * (int64_t)D.wtiles) + at.tile0 * 16 + 4 * g;
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (at.tile0 + i < D.wtiles) *reinterpret_cast<f32x4 *>(q + 16 * i) = acc[r][i];
  }
}

// The only entry of a row's list, or -1: one wave.
__device__ __forceinline__ int sole_entry(const Lists &L, int64_t row, int lane) {
  int one = -1;
  bool several = false;
  for (int j0 = 0; j0 < L.top; j0 += 64) {
    const int at = j0 + lane < L.top ? list_entry(L, row * L.top + j0 + lane) : -1;
    const uint64_t named = __ballot(at >= 0);
    if (!named) continue;
    if (one < 0) one = __builtin_amdgcn_readlane(at, __builtin_ctzll(named));
    several = several || __any(at >= 0 && at != one);
  }
  return several ? -1 : one;
}

// l2 of the listed entries: W's rows decoded where they are named, one wave an
// entry; and each list's only entry. Bound by the decode's VALU work.
template <int BITS>
__global__ __launch_bounds__(256) void listed_kernel(Lists L, int32_t *__restrict__ sole,
                                                     const uint16_t *__restrict__ x, const uint32_t *__restrict__ codes,
                                                     const uint16_t *__restrict__ scales, int blocks) {
  constexpr int wpb = 8 * BITS;
  const int64_t row = blockIdx.x;
  const int j = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (j == 0) {
    const int one = sole_entry(L, row, lane);
    if (lane == 0) sole[row] = one;
  }
  if (j >= L.top) return;
  const int at = __builtin_amdgcn_readfirstlane(list_entry(L, row * L.top + j));
  if (at < 0) return;
  const float s = bf16_bits_to_f32(scales[at]);
  float q, kq;
  alu_row_constants(s, q, kq);
  const bool chain = __builtin_amdgcn_readfirstlane(!alu_scale_ok(s)) != 0;
  const int pos = (252 - 4 * lane) * BITS, w0 = pos >> 5, w1 = w0 + 1 == wpb ? 0 : w0 + 1, sh = pos & 31;
  const uint32_t *const bw = codes + (int64_t)at * blocks * wpb;
  const uint16_t *const xr = x + row * blocks * 256 + 4 * lane;
  float sum = 0.f;
  auto dot = [&](auto chained) {
#pragma unroll 4
    for (int b = 0; b < blocks; ++b) {
      const uint32_t f = __builtin_amdgcn_alignbit(bw[b * wpb + w1], bw[b * wpb + w0], sh);
      const u32x2 v = *reinterpret_cast<const u32x2 *>(xr + 256 * b);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float w = (float)(__bf16)window_weight(__builtin_amdgcn_ubfe(f, (3 - c) * BITS, 12), s, q, kq, decltype(chained)::value);
        sum = __builtin_fmaf(w, bf16_half(v[c >> 1], c & 1), sum);
      }
    }
  };
  if (chain) dot(std::true_type{});
  else dot(std::false_type{});
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) L.listed[row * L.top + j] = sum * L.scale2;
}

// A row's blocks joined: its loss, lse and the factor of its dx (T / S in the
// operands' unit; 0 for a row without entries). Tiles whose reference is not the
// row's are brought to it, and the listed entries' operands become (p - q) S, their
// rests in `add` in the same unit.
template <int BITS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 4))) void row_join_kernel(Lists L, Vocabulary V, int ptiles, int block_columns,
                                                       float *__restrict__ factor, Rests F) {
  __shared__ RowList S;
  const int64_t row = blockIdx.x;
  const f32x2 *const stats = V.stats + row * V.blocks;
  const int sole = V.sole[row];
  const bool whole = !(sole >= 0 && sole < L.n);
  float ref = kLowest;
  for (int b = threadIdx.x; b < V.blocks; b += 256) ref = fmaxf(ref, stats[b][0]);
  ref = max_256(ref, S.red[0]);
  float sum = 0.f, moved = 0.f;
  for (int b = threadIdx.x; b < V.blocks; b += 256) {
    const f32x2 a = stats[b];
    if (a[0] != ref && a[1] != 0.f) moved = 1.f;
    sum += a[1] * __builtin_amdgcn_exp2f(a[0] - ref);
  }
  sum = sum_256(sum, S.red[1]);
  moved = max_256(moved, S.red[0]);
  if (!whole && threadIdx.x == 0) {
    for (int j = 0; j < L.top; ++j) L.listed[row * L.top + j] = V.sole_l2[row];
  }
  __syncthreads();
  const bool alive = row_list(L, row, f32x2{ref, sum}, whole, S, true);
  if (!V.e) return;
  const float rmax = S.total[0], total = S.total[1];
  if (threadIdx.x == 0) factor[row] = alive ? L.temperature * __builtin_amdgcn_exp2f(ref - rmax) / total : 0.f;
  // operand of a column of this row
  auto place = [&](int col) {
    return V.e + (((int64_t)(col >> 5) * ptiles + (row >> 4)) * 64 + (row & 15) + 16 * ((col >> 3) & 3)) * 8 + (col & 7);
  };
  if (moved != 0.f) {
    for (int c = 8 * (int)threadIdx.x; c < V.n; c += 8 * 256) {
      const f32x2 a = stats[c / block_columns];
      if (a[0] == ref) continue;
      const float f = __builtin_amdgcn_exp2f(a[0] - ref);
      u32x4 *const p = reinterpret_cast<u32x4 *>(place(c));
      u32x4 v = *p;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = (uint32_t)bf16_of(f * bf16_half(v[e], 0)) | ((uint32_t)bf16_of(f * bf16_half(v[e], 1)) << 16);
      *p = v;
    }
    __syncthreads();
  }
  float value = 0.f;
  if (S.first[threadIdx.x] && alive) {
    value = whole ? S.add[threadIdx.x] * total : S.qs[threadIdx.x] * -sum;
    *place(S.at[threadIdx.x]) = bf16_of(value);
  }
  listed_rests<BITS>(L, F, row, value, (int)(threadIdx.x >> 6), 4, S);
}

// dx: the splits' sums in order and the rests', times the row's factor (null: 1),
// rounded. Four columns a thread.
__global__ __launch_bounds__(256) void loss_gradient_kernel(const float *__restrict__ partials, int splits, int64_t plane,
                                                            int columns, int width, const float *__restrict__ factor,
                                                            const float *__restrict__ add, int m, uint16_t *__restrict__ dx) {
  const int quads = columns >> 2;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / quads;
  if (row >= m) return;
  const int c = (int)(id - row * quads) * 4;
  const float f = factor ? factor[row] : 1.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (f != 0.f) {
    const f32x4 rests = *reinterpret_cast<const f32x4 *>(add + row * width + c);
    for (int s0 = 0; s0 < splits; s0 += 4) {
      f32x4 part[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)  // (past the last split: its sums again, not added)
        part[s] = *reinterpret_cast<const f32x4 *>(partials + (s0 + s < splits ? s0 + s : splits - 1) * plane + row * columns + c);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s0 + s < splits) v += part[s];
    }
    v = (v + rests) * f;
  }
  store4(dx + row * width + c, v);
}

typedef void (*VocabularyFn)(Dense, Vocabulary);
VocabularyFn vocabulary_fn(int nt, int rt) {
  if (rt == 3) return nt == 4 ? &vocabulary_kernel<4, 3> : nt == 6 ? &vocabulary_kernel<6, 3> : &vocabulary_kernel<8, 3>;
  return nt == 4 ? &vocabulary_kernel<4, 4> : nt == 6 ? &vocabulary_kernel<6, 4> : &vocabulary_kernel<8, 4>;
}
typedef void (*VocabularyDecodeFn)(Dense, Vocabulary, Packed);
template <int BITS>
VocabularyDecodeFn vocabulary_decode_of(int rt) {
  return rt == 4 ? &vocabulary_decode_kernel<BITS, 4> : &vocabulary_decode_kernel<BITS, 6>;
}
VocabularyDecodeFn vocabulary_decode_fn(int bits, int rt) {
  return bits == 2 ? vocabulary_decode_of<2>(rt) : bits == 3 ? vocabulary_decode_of<3>(rt) : vocabulary_decode_of<4>(rt);
}
template <int RT>
DenseFn vocabulary_back_of(int nt) {
  switch (nt) {
    case 4: return &vocabulary_back_kernel<4, RT>;
    case 5: return &vocabulary_back_kernel<5, RT>;
    case 6: return &vocabulary_back_kernel<6, RT>;
    case 7: return &vocabulary_back_kernel<7, RT>;
    default: return &vocabulary_back_kernel<8, RT>;
  }
}
DenseFn vocabulary_back_fn(int nt, int rt) { return rt == 3 ? vocabulary_back_of<3>(nt) : vocabulary_back_of<4>(nt); }

// How the dense products of a loss are laid out: column tile, row tile and (the
// second one: a tile's exponentials need its whole sum) split of the contraction
// whose rounds over the card cost least.
constexpr int64_t kVocabularyBytes = (int64_t)1 << 31;  // decoded weights of a launch
struct VocabularyTile {
  int nt, rt, splits;
  bool decode;  // vocabulary_decode_kernel
  double us;
};
VocabularyTile vocabulary_tile(int64_t m, int64_t tiles, int64_t steps, bool back, int cus) {
  VocabularyTile best{};
  for (int rt = 4; rt >= 3; --rt)
    for (int nt = 8; nt >= 4; nt -= back ? 1 : 2) {
      const int64_t wg = (m + 64 * rt - 1) / (64 * rt) * ((tiles + 2 * nt - 1) / (2 * nt));
      for (int splits = 1; splits == 1 || (back && splits <= 8 && splits <= steps / 16); ++splits) {
        // A last round that leaves workgroups idle costs half of what it leaves:
        // with all of them at work the card's power holds its clock down.
        const double rounds = 0.5 * ((double)((wg * splits + cus - 1) / cus) + (double)(wg * splits) / cus);
        double us = (rounds < 1 ? 1 : rounds) * ((double)steps / splits * (0.0203 * rt * nt + 0.206) + 6);
        if (splits > 1) us += 0.32e-6 * ((double)splits * m * tiles * 16 * 4);
        if (best.nt == 0 || us < best.us) best = VocabularyTile{nt, rt, splits, false, us};
      }
    }
  return best;
}
// The first product's tile, or that of the kernel which decodes on its way.
VocabularyTile vocabulary_first(trellis_geom g, int64_t m, int64_t tiles, int64_t steps, int cus) {
  VocabularyTile best = vocabulary_tile(m, tiles, steps, false, cus);
  best.us += 4 + 0.43e-6 * g.n * (double)g.k;
  if (g_tiles.load(std::memory_order_relaxed) > 0) return best;  // (launches of so many tiles: there are none here)
  for (int rt = 4; rt <= 6; rt += 2) {
    const int64_t wg = (m + 64 * rt - 1) / (64 * rt) * ((tiles + 7) / 8);
    const double us = (double)((wg + cus - 1) / cus) * (steps * (0.09 * rt + 0.23) + 6);  // (power does not bind it)
    if (us < best.us) best = VocabularyTile{4, rt, 1, true, us};
  }
  return best;
}
struct LossShape {
  int32_t rows;       // of a chunk
  VocabularyTile fwd, back;
  int steps, back_steps, ptiles, blocks;
  int64_t tiles, slab, back_tiles, back_slab;  // operand tiles in all and per launch
  size_t operand_bytes, row_bytes, e_bytes, stat_bytes, partial_bytes;
  double us;
};
// The second product of a chunk of rows: its tile, operands and sums.
void loss_back_shape(LossShape &s, trellis_geom g, int64_t rows, int cus) {
  const int forced = g_tiles.load(std::memory_order_relaxed);
  s.back_tiles = g.k / 16;
  s.back_steps = (g.n + 63) / 64 * 2;
  s.ptiles = (int)((rows + 15) / 16);
  s.back = vocabulary_tile(rows, s.back_tiles, s.back_steps, true, cus);
  const int64_t back_bytes = (int64_t)s.back_steps * 1024;
  // Whole workgroup tiles a launch and whole 256-column blocks (a tile takes up to
  // 128 MB: one block at least, whose last workgroup tile may be cut, as may every
  // launch's last).
  s.back_slab = (forced > 0 ? (int64_t)forced : kVocabularyBytes / back_bytes) / 16 * 16;
  if (s.back_slab == 0) s.back_slab = 16;
  if (s.back_slab > s.back_tiles) s.back_slab = s.back_tiles;
  if (s.operand_bytes < (size_t)(s.back_slab * back_bytes)) s.operand_bytes = (size_t)(s.back_slab * back_bytes);
  s.operand_bytes = up256(s.operand_bytes);
  s.e_bytes = up256((size_t)s.ptiles * back_bytes);
  s.partial_bytes = up256((size_t)s.back.splits * rows * s.back_slab * 16 * 4);
}
LossShape loss_shape(trellis_geom g, int32_t m, bool keep, int cus) {
  LossShape s{};
  s.tiles = ((int64_t)g.n + 15) / 16;
  s.steps = (g.k + 63) / 64 * 2;
  const int64_t n_pad = ((int64_t)g.n + 63) / 64 * 64;
  // A chunk's operands of the second product take at most 1 GiB, those of x too,
  // and its statistics (8 bytes a row and 64 columns at the most) 512 MiB; 256
  // rows in any case.
  int64_t rows = keep ? kLogitBytes / (2 * n_pad) : ((int64_t)1 << 29) / (n_pad / 8);
  if (rows > kLogitBytes / (2 * (int64_t)g.k)) rows = kLogitBytes / (2 * (int64_t)g.k);
  rows = rows / 256 * 256;
  if (rows < 256) rows = 256;
  if (rows > m) rows = m;
  s.rows = (int32_t)rows;
  s.fwd = vocabulary_first(g, rows, s.tiles, s.steps, cus);
  s.blocks = (int)((s.tiles + s.fwd.nt - 1) / s.fwd.nt);
  const int64_t tile_bytes = (int64_t)s.steps * 1024;
  const int forced = g_tiles.load(std::memory_order_relaxed);
  // Whole workgroup tiles a launch (a tile takes 8 MB at most).
  const int unit = 2 * s.fwd.nt;
  s.slab = forced > 0 ? ((int64_t)forced + unit - 1) / unit * unit : kVocabularyBytes / tile_bytes / unit * unit;
  if (s.slab > s.tiles || s.fwd.decode) s.slab = s.tiles;
  s.operand_bytes = s.fwd.decode ? 0 : (size_t)(s.slab * tile_bytes);
  s.ptiles = (int)((rows + 15) / 16);
  s.row_bytes = up256((size_t)s.ptiles * tile_bytes);
  s.stat_bytes = up256((size_t)rows * s.blocks * 8);
  s.us = s.fwd.us;
  if (keep) {
    loss_back_shape(s, g, rows, cus);
    s.us += s.back.us + 4 + 0.46e-6 * g.n * (double)g.k;
  }
  s.operand_bytes = up256(s.operand_bytes);
  return s;
}

// A kernel's dynamic LDS; asked for once a device.
bool lds_allowed(bool &done, const void *f, size_t bytes) {
  done = done || worked(hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  return done;
}
size_t lds_of(const VocabularyTile &t) { return (size_t)dense_buffers(t.nt, t.rt) * dense_step_bytes(t.nt, t.rt); }

// dx of a chunk of rows from the logits' gradients as operands e.
struct LossBack {
  const uint32_t *codes;
  const uint16_t *scales, *e;
  uint16_t *operands;
  float *partials;
  const float *factor, *add;  // factor: null for 1
  int32_t m;
  uint16_t *dx;
};
trellis_status loss_back(const LossShape &s, trellis_geom g, const LossBack &b, int dev, hipStream_t stream) {
  static bool ready[kMaxDevices][2][9];
  const DenseFn fn = vocabulary_back_fn(s.back.nt, s.back.rt);
  const size_t lds = lds_of(s.back);
  if (!lds_allowed(ready[dev][s.back.rt - 3][s.back.nt], reinterpret_cast<const void *>(fn), lds)) return TRELLIS_E_HIP;
  Dense d{};
  d.p = b.e;
  d.w = b.operands;
  d.m = b.m;
  d.steps = s.back_steps;
  d.splits = s.back.splits;
  d.ptiles = (b.m + 15) / 16;
  d.mtiles = (b.m + 64 * s.back.rt - 1) / (64 * s.back.rt);
  d.partials = b.partials;
  d.width = g.k;
  (void)hipGetLastError();
  for (int64_t first = 0; first < s.back_tiles; first += s.back_slab) {
    d.wtiles = (int)(s.back_tiles - first < s.back_slab ? s.back_tiles - first : s.back_slab);
    d.ntiles = (d.wtiles + 2 * s.back.nt - 1) / (2 * s.back.nt);
    d.first = (int)first * 16;
    const Unpack u{{b.codes, nullptr}, {b.scales, nullptr}, b.operands, g.n, g.k, s.back_steps, (int)first, d.wtiles, 1};
    TRELLIS_TRY(launch_unpack(true, g.bits, u, stream));
    hipLaunchKernelGGL(fn, dim3((unsigned)(d.mtiles * d.ntiles * d.splits)), dim3(kDenseThreads), lds, stream, d);
    const int columns = 16 * d.wtiles;
    const int64_t threads = (int64_t)b.m * (columns / 4);
    hipLaunchKernelGGL(loss_gradient_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, b.partials,
                       d.splits, (int64_t)b.m * columns, columns, g.k, b.factor, b.add + d.first, b.m, b.dx + d.first);
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
  }
  return TRELLIS_OK;
}

trellis_status loss_dense(const uint16_t *x, int32_t m, const uint32_t *codes, const uint16_t *scales, trellis_geom g,
                          Lists L, uint16_t *dx, hipStream_t stream) {
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const LossShape s = loss_shape(g, m, dx != nullptr, cus);
  const size_t list_bytes = up256((size_t)s.rows * L.top * 4), word_bytes = up256((size_t)s.rows * 4),
               add_bytes = dx ? up256((size_t)s.rows * g.k * 4) : 0;
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream,
                    s.operand_bytes + s.row_bytes + s.e_bytes + s.stat_bytes + s.partial_bytes + add_bytes + list_bytes + 3 * word_bytes, 0, w));
  unsigned char *at = w->bytes;
  auto take = [&](size_t bytes) {
    unsigned char *const p = at;
    at += bytes;
    return p;
  };
  uint16_t *const operands = reinterpret_cast<uint16_t *>(take(s.operand_bytes)),
                 *const packed = reinterpret_cast<uint16_t *>(take(s.row_bytes)),
                 *const e = reinterpret_cast<uint16_t *>(take(s.e_bytes));
  f32x2 *const stats = reinterpret_cast<f32x2 *>(take(s.stat_bytes));
  float *const partials = reinterpret_cast<float *>(take(s.partial_bytes)), *const add = reinterpret_cast<float *>(take(add_bytes));
  L.listed = reinterpret_cast<float *>(take(list_bytes));
  int32_t *const sole = reinterpret_cast<int32_t *>(take(word_bytes));
  float *const sole_l2 = reinterpret_cast<float *>(take(word_bytes)), *const factor = reinterpret_cast<float *>(take(word_bytes));
  static bool ready[kMaxDevices][2][9], decode_ready[kMaxDevices][3][7];
  const VocabularyFn fn = s.fwd.decode ? nullptr : vocabulary_fn(s.fwd.nt, s.fwd.rt);
  const VocabularyDecodeFn decode_fn = s.fwd.decode ? vocabulary_decode_fn(g.bits, s.fwd.rt) : nullptr;
  const size_t lds = s.fwd.decode ? (size_t)decode_lds(g.bits, s.fwd.rt) : lds_of(s.fwd);
  if (!(s.fwd.decode ? lds_allowed(decode_ready[dev][g.bits - 2][s.fwd.rt], reinterpret_cast<const void *>(decode_fn), lds)
                     : lds_allowed(ready[dev][s.fwd.rt - 3][s.fwd.nt], reinterpret_cast<const void *>(fn), lds)))
    return TRELLIS_E_HIP;
  const auto join = g.bits == 2 ? &row_join_kernel<2> : g.bits == 3 ? &row_join_kernel<3> : &row_join_kernel<4>;
  const Lists all = L;
  (void)hipGetLastError();
  for (int32_t m0 = 0; m0 < m; m0 += s.rows) {
    const int32_t mc = m - m0 < s.rows ? m - m0 : s.rows;
    const int ptiles = (mc + 15) / 16;
    L.index = all.index + (int64_t)m0 * L.top;
    L.logits = all.logits ? all.logits + (int64_t)m0 * L.top : nullptr;
    L.loss = all.loss + m0;
    L.lse = all.lse + m0;
    const uint16_t *const xc = x + (int64_t)m0 * g.k;
    if (L.top > 1) {
      const dim3 grid((unsigned)mc, (unsigned)((L.top + 3) / 4));
      const auto listed = g.bits == 2 ? &listed_kernel<2> : g.bits == 3 ? &listed_kernel<3> : &listed_kernel<4>;
      hipLaunchKernelGGL(listed, grid, dim3(256), 0, stream, L, sole, xc, codes, scales, g.k >> 8);
    }
    hipLaunchKernelGGL(pack_rows_kernel<true>, dim3((unsigned)(((int64_t)ptiles * (s.steps / 2) + 3) / 4)), dim3(256), 0,
                       stream, xc, mc, g.k, ptiles, s.steps, packed);
    Dense d{};
    d.p = packed;
    d.w = operands;
    d.m = mc;
    d.steps = s.steps;
    d.splits = 1;
    d.ptiles = ptiles;
    d.mtiles = (mc + 64 * s.fwd.rt - 1) / (64 * s.fwd.rt);
    Vocabulary v{L.top > 1 ? sole : L.index, sole_l2, stats, dx ? e : nullptr, L.scale2, g.n, s.blocks, 0, 0,
                 dx ? s.back_steps : 0};
    for (int64_t first = 0; first < s.tiles; first += s.slab) {
      d.wtiles = (int)(s.tiles - first < s.slab ? s.tiles - first : s.slab);
      d.ntiles = (d.wtiles + 2 * s.fwd.nt - 1) / (2 * s.fwd.nt);
      v.first_tile = (int)first;
      v.first_block = (int)(first / s.fwd.nt);
      if (s.fwd.decode) {  // (one launch)
        hipLaunchKernelGGL(decode_fn, dim3((unsigned)(d.mtiles * d.ntiles)), dim3(kDenseThreads), lds, stream, d, v,
                           Packed{codes, scales, g.k});
        continue;
      }
      const Unpack u{{codes, nullptr}, {scales, nullptr}, operands, g.n, g.k, s.steps, (int)first, d.wtiles, 1};
      TRELLIS_TRY(launch_unpack(false, g.bits, u, stream));
      hipLaunchKernelGGL(fn, dim3((unsigned)(d.mtiles * d.ntiles)), dim3(kDenseThreads), lds, stream, d, v);
    }
    hipLaunchKernelGGL(join, dim3((unsigned)mc), dim3(256), 0, stream, L, v, ptiles, 16 * s.fwd.nt, factor,
                       Rests{codes, scales, add, g.k >> 8});
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
    if (dx)
      TRELLIS_TRY(loss_back(s, g, LossBack{codes, scales, e, operands, partials, factor, add, mc, dx + (int64_t)m0 * g.k},
                            dev, stream));
  }
  return TRELLIS_OK;
}

// The transposed product of few rows' gradients. Up to two row tiles, two
// workgroups share a CU where what that saves (a step takes 1.65 times as long
// for two) is more than the joining of twice as many parts costs: K = 5120, N =
// 65536, 1 row with gradient 140 us against 160; K = 1024, N = 32772 74 against 48.
// With operands it is many rows' second product (loss_back); these in several
// launches lose to decoding in the product (256 rows, K =
// 5120, N = 131072: the whole call 1.51 ms against 1.28).
Plan loss_back_plan(trellis_geom g, int32_t m, int cus) {
  Shape fused = shape_of(kTransposed, g, m, 1, cus, true);
  if (kRowTiles[fused.mt] <= 2) {
    Shape two = shape_of(kTransposed, g, m, 1, cus, true, 2);
    two.crowd = 1.65;
    if (fused_us(two) < fused_us(fused)) fused = two;
  }
  Plan p = plan_of(kTransposed, g, m, 1, cus, &fused);
  if (p.dense && p.many.slab < p.many.tiles && p.fused.units < ((int64_t)1 << 30)) {
    p.dense = false;
    p.bytes = p.fused.partial_bytes;
    p.counters = p.fused.tiles;
  }
  return p;
}
// Whether a loss takes the many rows' way (loss_dense), by what both are reckoned
// to take in us: fitted to 60 points, 96 to 1536 rows of five matrices (N, K: 8192
// 2048 to 131072 5120), where the side taken is 0.2% slower than the faster one on
// average and 10% at most. Measured, few rows' way against this: K = 5120, N =
// 131072, losses 267 / 398 at 128 rows, 440 / 400 at 192, 774 / 530 at 333; with
// gradient 947 / 1019 at 192, 1266 / 1081 at 256, 2521 / 1741 at 509; K = 2048, N =
// 8192, losses 40 / 54 at 509 rows, 61 / 54 at 640.
// Lists of several entries cost this way a row of W decoded for each (3.2 G
// weights a ms), the few rows' way hardly anything, as it has their logits: K =
// 2048, N = 8192, 1024 rows with lists of 16 69 / 69, of 64 73 / 101, of 256 84 /
// 232; K = 5120, N = 131072, 1024 rows of 256 2070 / 1857. On five other matrices,
// lists of 32 and 200 entries among them, the side taken is 0.2% slower than the
// faster one on average and 9% at most.
bool loss_by_operands(trellis_geom g, int32_t m, bool keep, int cus, int top = 1) {
  const int forced = g_path.load(std::memory_order_relaxed);
  if (forced >= 0) return forced == 1;
  const Shape f = shape_of(kForward, g, m, 1, cus, true);
  if (f.units >= ((int64_t)1 << 30)) return true;  // (the product kernel counts them in 32 bits)
  const double mn = 1e-6 * m * (double)g.n, mb = 2e-6 * g.n * (double)g.k;
  double rows = fused_us(f) + (keep ? 20 + 2.8 * mn : 13 + 1.4 * mn);
  if (keep) {
    const Plan b = loss_back_plan(g, m, cus);
    rows += b.dense ? b.many.us + 6.5 + 0.187 * mb + 0.56 * mn : fused_us(b.fused);
  }
  double many = loss_shape(g, m, keep, cus).us + 10;
  if (top > 1) {
    const double entries = (double)m * top;
    many += 3 + entries * (0.16e-3 + 0.24e-6 * g.k);
    // (with gradient each workgroup of row_loss_kernel goes through its row's list)
    rows += entries * (0.055e-3 + (keep && g.n > kWholeRow ? 0.032e-3 * ((g.n + kStatSpan - 1) / kStatSpan) : 0));
  }
  return many < rows;
}

// The logits of a chunk of rows in float32, decoded in the product; then the
// rows' losses; then the transposed product of the logits' gradients.
trellis_status loss_rows(const uint16_t *x, int32_t m, const uint32_t *codes, const uint16_t *scales, trellis_geom g,
                         Lists L, uint16_t *dx, hipStream_t stream) {
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  if (loss_by_operands(g, m, dx != nullptr, cus, L.top)) return loss_dense(x, m, codes, scales, g, L, dx, stream);
  // (64 rows at least: n is at most 2^22; with dx the listed entries' rests too)
  const int64_t most = kLogitBytes / (4 * (int64_t)(dx && g.k > g.n ? g.k : g.n)) / 16 * 16;
  const int32_t rows = m < most ? m : (int32_t)most;
  // Plans of the full chunks and of the last one; the workspace holds either.
  // (Where the transposed product takes operands, it is that of many rows.)
  const int32_t counts[2] = {rows, (m - 1) % rows + 1};
  Shape fwd[2];
  Plan bwd[2] = {};
  LossShape back[2] = {};
  size_t parts = 0;
  int64_t counters = 0;
  for (int i = 0; i < 2; ++i) {
    fwd[i] = shape_of(kForward, g, counts[i], 1, cus, true);
    if (dx) bwd[i] = loss_back_plan(g, counts[i], cus);
    if (bwd[i].dense) {
      loss_back_shape(back[i], g, counts[i], cus);
      bwd[i].bytes = back[i].operand_bytes + back[i].e_bytes + back[i].partial_bytes;
    }
    if (parts < fwd[i].partial_bytes) parts = fwd[i].partial_bytes;
    if (parts < bwd[i].bytes) parts = bwd[i].bytes;
    if (counters < fwd[i].tiles) counters = fwd[i].tiles;
    if (counters < bwd[i].counters) counters = bwd[i].counters;
  }
  const int spans = (g.n + kStatSpan - 1) / kStatSpan;
  const size_t logit_bytes = up256((size_t)rows * g.n * 4), d_bytes = dx ? up256((size_t)rows * g.n * 2) : 0,
               stat_bytes = up256((size_t)rows * spans * 8), listed_bytes = up256((size_t)rows * L.top * 4),
               add_bytes = dx ? up256((size_t)rows * g.k * 4) : 0;
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, logit_bytes + d_bytes + stat_bytes + listed_bytes + add_bytes + parts, (size_t)counters, w));
  float *const logits = reinterpret_cast<float *>(w->bytes);
  uint16_t *const d = reinterpret_cast<uint16_t *>(w->bytes + logit_bytes);
  f32x2 *const stats = reinterpret_cast<f32x2 *>(w->bytes + logit_bytes + d_bytes);
  L.listed = reinterpret_cast<float *>(w->bytes + logit_bytes + d_bytes + stat_bytes);
  float *const add = reinterpret_cast<float *>(w->bytes + logit_bytes + d_bytes + stat_bytes + listed_bytes);
  unsigned char *const rest = w->bytes + logit_bytes + d_bytes + stat_bytes + listed_bytes + add_bytes;
  const auto whole_row = g.bits == 2 ? &whole_row_kernel<2> : g.bits == 3 ? &whole_row_kernel<3> : &whole_row_kernel<4>;
  const auto row_loss = g.bits == 2 ? &row_loss_kernel<2> : g.bits == 3 ? &row_loss_kernel<3> : &row_loss_kernel<4>;
  const Rests rests{codes, scales, add, g.k >> 8};
  const Lists all = L;
  for (int32_t m0 = 0; m0 < m; m0 += rows) {
    const int32_t mc = m - m0 < rows ? m - m0 : rows;
    const int which = m0 + mc == m;
    L.index = all.index + (int64_t)m0 * L.top;
    L.logits = all.logits ? all.logits + (int64_t)m0 * L.top : nullptr;
    L.loss = all.loss + m0;
    L.lse = all.lse + m0;
    Product p{};
    p.p = x + (int64_t)m0 * g.k;
    p.codes = codes;
    p.scales = scales;
    p.logits = logits;
    p.partials = reinterpret_cast<float *>(rest);
    p.counters = w->counters;
    p.m = mc;
    p.n = g.n;
    p.k = g.k;
    TRELLIS_TRY(launch(fwd[which], p, stream));
    if (g.n <= kWholeRow) {
      hipLaunchKernelGGL(whole_row, dim3((unsigned)mc), dim3(256), 0, stream, L, logits, dx ? d : nullptr, rests);
    } else {
      hipLaunchKernelGGL(row_stats_kernel, dim3((unsigned)mc, (unsigned)spans), dim3(256), 0, stream, L, logits, stats);
      hipLaunchKernelGGL(row_loss, dim3((unsigned)mc, dx ? (unsigned)spans : 1u), dim3(256), 0, stream, L, logits,
                         stats, spans, dx ? d : nullptr, rests);
    }
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
    if (!dx) continue;
    if (bwd[which].dense) {
      const LossShape &s = back[which];
      uint16_t *const operands = reinterpret_cast<uint16_t *>(rest), *const e = reinterpret_cast<uint16_t *>(rest + s.operand_bytes);
      float *const partials = reinterpret_cast<float *>(rest + s.operand_bytes + s.e_bytes);
      hipLaunchKernelGGL(g.n % 8 ? pack_rows_kernel<false> : pack_rows_kernel<true>,
                         dim3((unsigned)(((int64_t)s.ptiles * (s.back_steps / 2) + 3) / 4)), dim3(256), 0, stream, d, mc,
                         g.n, s.ptiles, s.back_steps, e);
      if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
      TRELLIS_TRY(loss_back(s, g, LossBack{codes, scales, e, operands, partials, nullptr, add, mc, dx + (int64_t)m0 * g.k},
                            dev, stream));
      continue;
    }
    Product t{};
    t.p = d;
    t.add = add;
    t.codes = codes;
    t.scales = scales;
    t.out = dx + (int64_t)m0 * g.k;
    t.counters = w->counters;
    t.m = mc;
    t.n = g.n;
    t.k = g.k;
    TRELLIS_TRY(run(bwd[which], kTransposed, g, t, nullptr, rest, stream));
  }
  return TRELLIS_OK;
}

}  // namespace
}  // namespace trellis

extern "C" {

trellis_status trellis_cross_entropy(const uint16_t *x, int32_t m, const uint32_t *codes, const uint16_t *scales,
                                     trellis_geom g, const int32_t *target, float *loss, float *lse, uint16_t *dx,
                                     void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (!x || !codes || !scales || !target || !loss || !lse) return TRELLIS_E_NULL;
  if (!on(x, 16) || !on(codes, 16) || !on(scales, 2) || !on(target, 4) || !on(loss, 4) || !on(lse, 4) || !on(dx, 16))
    return TRELLIS_E_ALIGN;
  std::lock_guard<std::mutex> lock(g_lock);
  const Lists l{target, nullptr, nullptr, g.n, 1, 1.f, kLog2E, loss, lse};
  return loss_rows(x, m, codes, scales, g, l, dx, reinterpret_cast<hipStream_t>(hip_stream));
}

trellis_status trellis_distill(const uint16_t *x, int32_t m, const uint32_t *codes, const uint16_t *scales,
                               trellis_geom g, const int32_t *index, const float *logits, int32_t top,
                               float temperature, float *loss, float *lse, uint16_t *dx, void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (top < 1 || top > TRELLIS_MAX_TOP ||
      !(temperature >= TRELLIS_MIN_TEMPERATURE && temperature <= TRELLIS_MAX_TEMPERATURE))
    return TRELLIS_E_RANGE;
  if (!x || !codes || !scales || !index || !logits || !loss || !lse) return TRELLIS_E_NULL;
  if (!on(x, 16) || !on(codes, 16) || !on(scales, 2) || !on(index, 4) || !on(logits, 4) || !on(loss, 4) ||
      !on(lse, 4) || !on(dx, 16))
    return TRELLIS_E_ALIGN;
  std::lock_guard<std::mutex> lock(g_lock);
  const Lists l{index, logits, nullptr, g.n, top, temperature, kLog2E / temperature, loss, lse};
  return loss_rows(x, m, codes, scales, g, l, dx, reinterpret_cast<hipStream_t>(hip_stream));
}

trellis_status trellis_loss_backward(const float *dloss, const uint16_t *dx, int32_t m, int32_t k, uint16_t *out,
                                     void *hip_stream) {
  if (k < TRELLIS_T || k > TRELLIS_MAX_K || k % TRELLIS_T) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (!dloss || !dx || !out) return TRELLIS_E_NULL;
  if (!on(dloss, 4) || !on(dx, 16) || !on(out, 16)) return TRELLIS_E_ALIGN;
  const int64_t vectors = (int64_t)m * (k / 8);
  (void)hipGetLastError();
  const int64_t groups = (vectors + 255) / 256 < kScaleGroups ? (vectors + 255) / 256 : kScaleGroups;
  hipLaunchKernelGGL(scale_rows_kernel, dim3((unsigned)groups), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(hip_stream), dloss, dx, vectors, k / 8, out);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

}  // extern "C"
