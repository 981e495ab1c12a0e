// Embedding from a packed vocabulary matrix with trained rows behind it, and the
// trained rows' gradient from rows sorted by token. Part of rows.hip.

namespace trellis {
namespace {

// One wave a row and 256-column block: lane l decodes columns 4 l .. +3, whose
// windows lie in 24 bits of two words.
template <int BITS>
__global__ __launch_bounds__(256) void embed_kernel(const int32_t *__restrict__ tokens, int64_t waves, int blocks,
                                                    const uint32_t *__restrict__ codes,
                                                    const uint16_t *__restrict__ scales, int n, float scale,
                                                    const uint16_t *__restrict__ extra, int count,
                                                    uint16_t *__restrict__ out) {
  constexpr int wpb = 8 * BITS;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= waves) return;
  const int64_t row = id / blocks;
  const int b = (int)(id - row * blocks), lane = threadIdx.x & 63;
  const int token = tokens[row];
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (token >= 0 && token < n) {
    const uint32_t *const bw = codes + ((int64_t)token * blocks + b) * wpb;
    const float s = bf16_bits_to_f32(scales[token]);
    float q, kq;
    alu_row_constants(s, q, kq);
    const bool chain = !alu_scale_ok(s);
    const int pos = (252 - 4 * lane) * BITS, w0 = pos >> 5, w1 = w0 + 1 == wpb ? 0 : w0 + 1;
    const uint32_t f = __builtin_amdgcn_alignbit(bw[w1], bw[w0], pos & 31);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      v[c] = (float)(__bf16)window_weight(__builtin_amdgcn_ubfe(f, (3 - c) * BITS, 12), s, q, kq, chain) * scale;
  } else if (token >= n && token - n < count) {
    const u32x2 e = *reinterpret_cast<const u32x2 *>(extra + ((int64_t)(token - n) * blocks + b) * 256 + 4 * lane);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = bf16_half(e[c >> 1], c & 1) * scale;
  }
  store4(out + id * 256 + 4 * lane, v);
}

// ---- gradient: rows sorted by token -------------------------------------------
// A stable radix sort of (trained row, row of dout), eight bits a pass, each
// pass: digits counted by 2048 rows, the counts' running sums, the rows placed.
// The first pass leaves out the rows without a trained token.
constexpr int kSortRows = 2048;   // of a workgroup
constexpr int kSortWave = kSortRows / 4;

struct Sort {
  const int32_t *tokens;          // the first pass's input, else null
  const int32_t *key, *row;       // the others': *total pairs
  int32_t *key_out, *row_out;
  uint32_t *counts;               // [256][blocks]
  uint32_t *total;
  int32_t m, first, count, shift, blocks;
};
// Pair i of the input; false where there is none.
__device__ __forceinline__ bool sort_pair(const Sort &S, int i, uint32_t limit, int &key, int &row) {
  if (S.tokens) {
    if (i >= S.m) return false;
    const int token = S.tokens[i];
    if (token < S.first || token - S.first >= S.count) return false;
    key = token - S.first;
    row = i;
    return true;
  }
  if ((uint32_t)i >= limit) return false;
  key = S.key[i];
  row = S.row[i];
  return true;
}

__global__ __launch_bounds__(256) void sort_count_kernel(Sort S) {
  __shared__ uint32_t counts[256];
  counts[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t limit = S.tokens ? 0u : *S.total;
  for (int i = threadIdx.x; i < kSortRows; i += 256) {
    int key, row;
    if (sort_pair(S, (int)blockIdx.x * kSortRows + i, limit, key, row)) atomicAdd(&counts[(key >> S.shift) & 255], 1u);
  }
  __syncthreads();
  S.counts[threadIdx.x * S.blocks + blockIdx.x] = counts[threadIdx.x];
}

// Running sums of the counts, digit by digit: one workgroup.
__global__ __launch_bounds__(1024) void sort_sum_kernel(uint32_t *__restrict__ counts, int n, uint32_t *__restrict__ total) {
  __shared__ uint32_t waves[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t base = 0;
  for (int at = 0; at < n; at += 1024) {
    const int i = at + (int)threadIdx.x;
    const uint32_t v = i < n ? counts[i] : 0u;
    uint32_t s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t up = __shfl_up(s, o);
      if (lane >= o) s += up;
    }
    if (lane == 63) waves[wave] = s;
    __syncthreads();
    uint32_t before = base;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += waves[w];
      base += waves[w];
    }
    if (i < n) counts[i] = before + s - v;
    __syncthreads();
  }
  if (threadIdx.x == 0) *total = base;
}

// Wave w takes the workgroup's pairs 512 w .. +511, 64 at a time in order.
__global__ __launch_bounds__(256) void sort_place_kernel(Sort S, const uint32_t *__restrict__ last_total) {
  __shared__ uint32_t counts[4][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < 4 * 256; i += 256) (&counts[0][0])[i] = 0;
  __syncthreads();
  const uint32_t limit = S.tokens ? 0u : *last_total;
  const int i0 = (int)blockIdx.x * kSortRows + wave * kSortWave;
  for (int i = lane; i < kSortWave; i += 64) {
    int key, row;
    if (sort_pair(S, i0 + i, limit, key, row)) atomicAdd(&counts[wave][(key >> S.shift) & 255], 1u);
  }
  __syncthreads();
  {
    uint32_t at = S.counts[threadIdx.x * S.blocks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t c = counts[w][threadIdx.x];
      counts[w][threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i = lane; i < kSortWave; i += 64) {
    int key = 0, row = 0;
    const bool in = sort_pair(S, i0 + i, limit, key, row);
    const uint32_t digit = (uint32_t)(key >> S.shift) & 255u;
    uint64_t same = __ballot(in);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t set = __ballot((digit >> b) & 1u);
      same &= (digit >> b) & 1u ? set : ~set;
    }
    if (in) {
      const uint32_t before = __popcll(same & ((1ull << lane) - 1ull));
      const uint32_t at = counts[wave][digit] + before;
      S.key_out[at] = key;
      S.row_out[at] = row;
    }
    // (the wave's reads of its counts come before these writes)
    __builtin_amdgcn_wave_barrier();
    if (in && (same >> lane) == 1ull) counts[wave][digit] += (uint32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
}

// Sums of the sorted rows: a wave takes one chunk of pairs and 512 columns (8 a
// lane), and adds up the runs of equal tokens. A run that lies within the chunk
// is finished; what the chunk holds of one that goes on before or behind it goes
// to `parts`, and join_runs_kernel adds those up, chunk by chunk.
struct Sums {
  const uint16_t *dout;
  const int32_t *key, *row;
  const uint32_t *total;
  uint16_t *dextra;
  float *parts;  // [chunks][2][k]: of the chunk's first run, of its last
  int32_t k, chunk, count;
  float scale;
};
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8], float scale) {
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (uint32_t)bf16_of(v[2 * e] * scale) | ((uint32_t)bf16_of(v[2 * e + 1] * scale) << 16);
  *reinterpret_cast<u32x4 *>(p) = o;
}
__global__ __launch_bounds__(64) void sum_runs_kernel(Sums S) {
  const int total = (int)*S.total, c = blockIdx.y * 512 + 8 * (int)threadIdx.x;
  const int begin = blockIdx.x * S.chunk, end = total - begin < S.chunk ? total : begin + S.chunk;
  if (begin >= end || c >= S.k) return;
  float acc[8] = {};
  int run = begin, key = S.key[begin];  // the run's first pair here, and its token
  const bool goes_on_before = begin > 0 && S.key[begin - 1] == key;
  const bool goes_on_behind = end < total && S.key[end] == S.key[end - 1];
  auto flush = [&](int next, bool last) {
    // (a run that fills the chunk and goes on to both sides is its first)
    const bool before = run == begin && goes_on_before, behind = last && goes_on_behind;
    if (before || behind) {
      float *const p = S.parts + ((int64_t)blockIdx.x * 2 + (before ? 0 : 1)) * S.k + c;
#pragma unroll
      for (int e = 0; e < 8; e += 4) *reinterpret_cast<f32x4 *>(p + e) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
    } else {
      store8(S.dextra + (int64_t)key * S.k + c, acc, S.scale);
    }
    run = next;
  };
  constexpr int U = 8;  // rows loaded at a time
  for (int i = begin; i < end; i += U) {
    u32x4 v[U];
    int keys[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = i + u < end ? i + u : end - 1;
      keys[u] = S.key[at];
      v[u] = *reinterpret_cast<const u32x4 *>(S.dout + (int64_t)S.row[at] * S.k + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= end) break;
      if (keys[u] != key) {
        flush(i + u, false);
        key = keys[u];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += bf16_half(v[u][e >> 1], e & 1);
    }
  }
  flush(end, true);
}

// Runs over several chunks: the workgroup of the chunk that a run begins in (and
// does not end in) adds the parts in order.
__global__ __launch_bounds__(64) void join_runs_kernel(Sums S) {
  const int total = (int)*S.total, c = blockIdx.y * 512 + 8 * (int)threadIdx.x;
  const int begin = blockIdx.x * S.chunk, end = begin + S.chunk;
  if (end >= total || c >= S.k) return;  // (the last chunk: nothing goes on behind it)
  const int key = S.key[end - 1];
  if (S.key[end] != key) return;
  if (begin > 0 && S.key[begin - 1] == key && S.key[begin] == key) return;  // begun before this chunk
  float acc[8] = {};
  // its part here is the last run's
  for (int chunk = blockIdx.x, which = 1;; ++chunk, which = 0) {
    const float *const p = S.parts + ((int64_t)chunk * 2 + which) * S.k + c;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += p[e];
    const int stop = (chunk + 1) * S.chunk;
    if (stop >= total || S.key[stop] != key) break;
  }
  store8(S.dextra + (int64_t)key * S.k + c, acc, S.scale);
}

// Zeros in the trained rows that no pair names: a wave a row, which looks its
// token up in the sorted pairs.
__global__ __launch_bounds__(256) void clear_rows_kernel(Sums S) {
  const int e = blockIdx.x * 4 + (int)(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (e >= S.count) return;
  int low = 0, high = (int)*S.total;
  while (low < high) {
    const int mid = (low + high) >> 1;
    if (S.key[mid] < e) low = mid + 1;
    else high = mid;
  }
  if (low < (int)*S.total && S.key[low] == e) return;
  for (int c = 8 * lane; c < S.k; c += 512)
    *reinterpret_cast<u32x4 *>(S.dextra + (int64_t)e * S.k + c) = u32x4{0u, 0u, 0u, 0u};
}

}  // namespace
}  // namespace trellis

extern "C" {

trellis_status trellis_embed(const int32_t *tokens, int32_t m, const uint32_t *codes, const uint16_t *scales,
                             trellis_geom g, float scale, const uint16_t *extra, int32_t count, uint16_t *out,
                             void *hip_stream) {
  if (!geom_ok(g)) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (count < 0 || count > TRELLIS_MAX_TRAINED || !__builtin_isfinite(scale)) return TRELLIS_E_RANGE;
  if (!tokens || !codes || !scales || !out || (count > 0 && !extra)) return TRELLIS_E_NULL;
  if (!on(tokens, 4) || !on(codes, 16) || !on(scales, 2) || !on(extra, 16) || !on(out, 16)) return TRELLIS_E_ALIGN;
  hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
  const int blocks = g.k >> 8;
  const int64_t waves = (int64_t)m * blocks;
  const dim3 grid((unsigned)((waves + 3) / 4));
  (void)hipGetLastError();
  const auto fn = g.bits == 2 ? &embed_kernel<2> : g.bits == 3 ? &embed_kernel<3> : &embed_kernel<4>;
  hipLaunchKernelGGL(fn, grid, dim3(256), 0, stream, tokens, waves, blocks, codes, scales, g.n, scale, extra, count, out);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

trellis_status trellis_embed_backward(const uint16_t *dout, const int32_t *tokens, int32_t m, int32_t k, int32_t first,
                                      int32_t count, float scale, uint16_t *dextra, void *hip_stream) {
  if (k < TRELLIS_T || k > TRELLIS_MAX_K || k % TRELLIS_T) return TRELLIS_E_GEOMETRY;
  if (m < 1 || m > TRELLIS_MAX_ROWS) return TRELLIS_E_M;
  if (count < 1 || count > TRELLIS_MAX_TRAINED || first < 0 || first > TRELLIS_MAX_N || !__builtin_isfinite(scale))
    return TRELLIS_E_RANGE;
  if (!dout || !tokens || !dextra) return TRELLIS_E_NULL;
  if (!on(dout, 16) || !on(tokens, 4) || !on(dextra, 16)) return TRELLIS_E_ALIGN;
  hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
  std::lock_guard<std::mutex> lock(g_lock);
  int dev = 0, cus = 0;
  TRELLIS_TRY(device(dev, cus));
  const int blocks = (m + kSortRows - 1) / kSortRows;
  int chunk = (m + 1023) / 1024;
  if (chunk < 16) chunk = 16;
  const int chunks = (m + chunk - 1) / chunk;
  const size_t pair_bytes = up256((size_t)m * 4), count_bytes = up256((size_t)blocks * 1024),
               part_bytes = (size_t)chunks * 2 * k * 4;
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, 4 * pair_bytes + count_bytes + 256 + part_bytes, 0, w));
  int32_t *const pairs[4] = {reinterpret_cast<int32_t *>(w->bytes), reinterpret_cast<int32_t *>(w->bytes + pair_bytes),
                             reinterpret_cast<int32_t *>(w->bytes + 2 * pair_bytes),
                             reinterpret_cast<int32_t *>(w->bytes + 3 * pair_bytes)};
  uint32_t *const counts = reinterpret_cast<uint32_t *>(w->bytes + 4 * pair_bytes);
  uint32_t *const total = reinterpret_cast<uint32_t *>(w->bytes + 4 * pair_bytes + count_bytes);
  float *const parts = reinterpret_cast<float *>(w->bytes + 4 * pair_bytes + count_bytes + 256);
  (void)hipGetLastError();
  int to = 0;
  for (int shift = 0; shift == 0 || (count - 1) >> shift; shift += 8, to ^= 2) {
    Sort s{shift ? nullptr : tokens, pairs[to ^ 2], pairs[(to ^ 2) + 1], pairs[to], pairs[to + 1], counts, total, m, first,
           count, shift, blocks};
    hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, s);
    hipLaunchKernelGGL(sort_sum_kernel, dim3(1), dim3(1024), 0, stream, counts, 256 * blocks, total);
    hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, s, total);
  }
  to ^= 2;  // the last pass's output
  const Sums s{dout, pairs[to], pairs[to + 1], total, dextra, parts, k, chunk, count, scale};
  const dim3 grid((unsigned)chunks, (unsigned)((k + 511) / 512));
  hipLaunchKernelGGL(clear_rows_kernel, dim3((unsigned)((count + 3) / 4)), dim3(256), 0, stream, s);
  hipLaunchKernelGGL(sum_runs_kernel, grid, dim3(64), 0, stream, s);
  hipLaunchKernelGGL(join_runs_kernel, grid, dim3(64), 0, stream, s);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

}  // extern "C"
