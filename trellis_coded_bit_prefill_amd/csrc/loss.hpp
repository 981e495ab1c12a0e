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
// The logits of a chunk of rows lie in the workspace in float32 (loss_rows).

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
  int32_t m, n, top;
  float temperature, scale2;  // scale2: log2(e) / T
  float *loss, *lse;
};

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

// Takes the listed entries out of a row's logits: l2 to `listed`, -infinity in
// their place. One wave a row; all are read before any is replaced, as an entry
// may be listed several times.
__global__ __launch_bounds__(64) void pluck_kernel(Lists L, float *__restrict__ logits) {
  const int64_t row = blockIdx.x;
  float *const l = logits + row * L.n;
  const int32_t *const index = L.index + row * L.top;
  constexpr int kEach = kMaxTop / 64;
  int at[kEach];
  float v[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = threadIdx.x + 64 * i;
    at[i] = j < L.top ? index[j] : -1;
    if (at[i] >= L.n) at[i] = -1;
    v[i] = at[i] >= 0 ? l[at[i]] * L.scale2 : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = threadIdx.x + 64 * i;
    if (j < L.top) L.listed[row * L.top + j] = v[i];
    if (at[i] >= 0) l[at[i]] = -__builtin_inff();
  }
}

constexpr int kStatSpan = 4096;  // logits of a workgroup

// Largest and sum of a span of a row.
__global__ __launch_bounds__(256) void row_stats_kernel(const float *__restrict__ logits, int n, float scale2,
                                                        f32x2 *__restrict__ stats) {
  __shared__ f32x2 part[4];
  const int64_t row = blockIdx.y;
  const int c0 = blockIdx.x * kStatSpan + 4 * (int)threadIdx.x;
  const float *const l = logits + row * n;
  f32x4 v[kStatSpan / 1024];
  float r = kLowest;
#pragma unroll
  for (int i = 0; i < kStatSpan / 1024; ++i) {
    const int c = c0 + 1024 * i;
    v[i] = f32x4{-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
    if (c < n) v[i] = *reinterpret_cast<const f32x4 *>(l + c) * scale2;
#pragma unroll
    for (int e = 0; e < 4; ++e) r = fmaxf(r, v[i][e]);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kStatSpan / 1024; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(v[i][e] - r);
  const f32x2 a = join_stats_wave(f32x2{r, s});
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0)
    stats[row * gridDim.x + blockIdx.x] = join_stats(join_stats(part[0], part[1]), join_stats(part[2], part[3]));
}

// What a workgroup of 256 threads works out of a row's list and of its other
// entries' sum; the list in LDS.
struct RowList {
  int at[kMaxTop];       // -1: none
  float q[kMaxTop], l2[kMaxTop];
  float add[kMaxTop];    // d of the entry (its first place in the list), without T
  uint8_t first[kMaxTop];
  float red[2][4];
  f32x2 total;           // R and S of the whole row
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
// rest: R' and S' of the entries that are not listed. Returns whether the row
// has entries; loss and lse where `write`.
static_assert(kMaxTop == 256, "one thread an entry");
__device__ bool row_list(const Lists &L, int64_t row, f32x2 rest, RowList &S, bool write) {
  const int j = threadIdx.x;
  int at = j < L.top ? L.index[row * L.top + j] : -1;
  if (at >= L.n) at = -1;
  const float inf = __builtin_inff();
  float z = -inf, l2 = -inf;
  if (at >= 0) {
    z = L.logits ? L.logits[row * L.top + j] * L.scale2 : 0.f;
    l2 = L.listed[row * L.top + j];
  }
  S.at[j] = at;
  // q: softmax of the list. A NaN among the teacher's logits is a NaN in the sum.
  const float zmax = fmaxf(max_256(z, S.red[0]), kLowest);
  const float e = at >= 0 ? __builtin_amdgcn_exp2f(z - zmax) : 0.f;
  const float total = sum_256(e, S.red[1]);
  const bool alive = total != 0.f;
  const float q = alive ? e / total : 0.f;
  S.q[j] = q;
  S.l2[j] = l2;
  __syncthreads();
  // every entry once: its first place adds to the sum
  bool first = at >= 0;
  float qs = 0.f;
  for (int k = 0; k < L.top; ++k)
    if (S.at[k] == at) {
      qs += S.q[k];
      if (k < j) first = false;
    }
  const float rmax = fmaxf(max_256(first ? l2 : -inf, S.red[0]), rest[0]);
  const float here = first ? __builtin_amdgcn_exp2f(l2 - rmax) : 0.f;
  const float others = rest[1] * __builtin_amdgcn_exp2f(rest[0] - rmax);
  const float sum = others + sum_256(here, S.red[1]);
  const float lse2 = rmax + __builtin_amdgcn_logf(sum);
  // one entry alone: 1 - p and the loss from the others' sum
  const bool alone = sum_256(first ? 1.f : 0.f, S.red[0]) == 1.f;
  if (j == 0) S.total = f32x2{rmax, sum};
  S.first[j] = first;
  S.add[j] = !first ? 0.f : alone ? -others / sum : here / sum - qs;
  float term = q != 0.f ? q * (z - zmax - __builtin_amdgcn_logf(total)) * kLn2 : 0.f;  // q log q
  if (!alone) {
    if (q != 0.f) term += q * (lse2 - l2) * kLn2;
  } else if (first) {
    const float ratio = (rest[0] - l2) * kLn2 + logf(rest[1]);  // log(S' / e)
    term += ratio > 0.f ? ratio + log1pf(expf(-ratio)) : log1pf(expf(ratio));
    if (l2 == inf) term = l2 - l2;
  }
  const float loss = sum_256(term, S.red[1]);
  if (write && j == 0) {
    L.loss[row] = alive ? L.temperature * L.temperature * loss : 0.f;
    L.lse[row] = lse2 * kLn2;
  }
  __syncthreads();
  return alive;
}

// Loss and lse of a row and, where d is not null, the gradient of its logits in
// a span (bf16, what the matrix cores multiply: each off by 2^-9 of itself, with
// errors of either sign).
__global__ __launch_bounds__(256) void row_loss_kernel(Lists L, const float *__restrict__ logits,
                                                       const f32x2 *__restrict__ stats, int spans,
                                                       uint16_t *__restrict__ d) {
  __shared__ RowList S;
  const int64_t row = blockIdx.y;
  // every wave joins the spans, in the same order
  f32x2 rest = {kLowest, 0.f};
  for (int i = threadIdx.x & 63; i < spans; i += 64) rest = join_stats(rest, stats[row * spans + i]);
  rest = join_stats_wave(rest);
  const bool alive = row_list(L, row, rest, S, blockIdx.x == 0);
  if (!d) return;
  const float r = S.total[0], f = alive ? L.temperature / S.total[1] : 0.f;
  const int c0 = blockIdx.x * kStatSpan;
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
  if (S.first[threadIdx.x] && at >= c0 && at < c0 + kStatSpan && alive)
    o[at] = bf16_of(L.temperature * S.add[threadIdx.x]);
}

// dx = dloss[row] * dx: a factor a row.
__global__ __launch_bounds__(256) void scale_rows_kernel(const float *__restrict__ f, const uint16_t *__restrict__ src,
                                                         int64_t vectors, int per_row, uint16_t *__restrict__ dst) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= vectors) return;
  const float s = f[i / per_row];
  const u32x4 v = reinterpret_cast<const u32x4 *>(src)[i];
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = (uint32_t)bf16_of(s * bf16_half(v[e], 0)) | ((uint32_t)bf16_of(s * bf16_half(v[e], 1)) << 16);
  reinterpret_cast<u32x4 *>(dst)[i] = o;
}

// The logits of a chunk of rows in float32, decoded in the product; then the
// rows' losses; then the transposed product of the logits' gradients.
trellis_status loss_rows(const uint16_t *x, int32_t m, const uint32_t *codes, const uint16_t *scales, trellis_geom g,
                         Lists L, uint16_t *dx, hipStream_t stream) {
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const int64_t most = kLogitBytes / (4 * (int64_t)g.n) / 16 * 16;  // 64 rows at least: n is at most 2^22
  const int32_t rows = m < most ? m : (int32_t)most;
  // Plans of the full chunks and of the last one; the workspace holds either.
  const int32_t counts[2] = {rows, (m - 1) % rows + 1};
  Shape fwd[2];
  Plan bwd[2] = {};
  size_t parts = 0;
  int64_t counters = 0;
  for (int i = 0; i < 2; ++i) {
    fwd[i] = shape_of(kForward, g, counts[i], 1, cus);
    if (dx) bwd[i] = plan_of(kTransposed, g, counts[i], 1, cus);
    if (parts < fwd[i].partial_bytes) parts = fwd[i].partial_bytes;
    if (parts < bwd[i].bytes) parts = bwd[i].bytes;
    if (counters < fwd[i].tiles) counters = fwd[i].tiles;
    if (counters < bwd[i].counters) counters = bwd[i].counters;
  }
  const int spans = (g.n + kStatSpan - 1) / kStatSpan;
  const size_t logit_bytes = up256((size_t)rows * g.n * 4), d_bytes = dx ? up256((size_t)rows * g.n * 2) : 0,
               stat_bytes = up256((size_t)rows * spans * 8), listed_bytes = up256((size_t)rows * L.top * 4);
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, logit_bytes + d_bytes + stat_bytes + listed_bytes + parts, (size_t)counters, w));
  float *const logits = reinterpret_cast<float *>(w->bytes);
  uint16_t *const d = reinterpret_cast<uint16_t *>(w->bytes + logit_bytes);
  f32x2 *const stats = reinterpret_cast<f32x2 *>(w->bytes + logit_bytes + d_bytes);
  L.listed = reinterpret_cast<float *>(w->bytes + logit_bytes + d_bytes + stat_bytes);
  unsigned char *const rest = w->bytes + logit_bytes + d_bytes + stat_bytes + listed_bytes;
  const Lists all = L;
  for (int32_t m0 = 0; m0 < m; m0 += rows) {
    const int32_t mc = m - m0 < rows ? m - m0 : rows;
    const int which = m0 + mc == m;
    L.m = mc;
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
    hipLaunchKernelGGL(pluck_kernel, dim3((unsigned)mc), dim3(64), 0, stream, L, logits);
    hipLaunchKernelGGL(row_stats_kernel, dim3((unsigned)spans, (unsigned)mc), dim3(256), 0, stream, logits, g.n, L.scale2,
                       stats);
    hipLaunchKernelGGL(row_loss_kernel, dim3(dx ? (unsigned)spans : 1u, (unsigned)mc), dim3(256), 0, stream, L, logits, stats,
                       spans, dx ? d : nullptr);
    if (hipGetLastError() != hipSuccess) return TRELLIS_E_HIP;
    if (!dx) continue;
    Product t{};
    t.p = d;
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
  const Lists l{target, nullptr, nullptr, m, g.n, 1, 1.f, kLog2E, loss, lse};
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
  const Lists l{index, logits, nullptr, m, g.n, top, temperature, kLog2E / temperature, loss, lse};
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
  hipLaunchKernelGGL(scale_rows_kernel, dim3((unsigned)((vectors + 255) / 256)), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(hip_stream), dloss, dx, vectors, k / 8, out);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

}  // extern "C"
